"""The weight gradient from a checkpoint against its definition in 64 bits: a = q*scale, unrounded."""
import pytest
import torch

from tests import _act as A
from tests._gpu import DEV, lz, require_gpu, status_flags, status_word

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _rand(rows, cols, T, seed, std, pad=0, off=0):
    """A rows x cols matrix, in the middle of a buffer of sevens if padded."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = (torch.randn(rows, cols, generator=g, device=DEV) * std).to(T)
    if not pad and not off:
        return v
    flat = torch.full(((rows + 2) * (cols + pad) + off,), 7.0, dtype=T, device=DEV)
    m = flat[off + cols + pad:][:rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return m.copy_(v)


def _values(ck, cols):
    """q*scale of a checkpoint in 64 bits."""
    at, nb = -(-cols // 16) * 16, -(-cols // 128)
    scale = ck[:, at:at + 4 * nb].contiguous().view(torch.float32).double()
    return (ck[:, :cols].double() - 128) * scale.repeat_interleave(128, 1)[:, :cols]


def _call(t, o, i, T, seed, pad=0, off=0, dwpad=0, dwoff=0, acc=False):
    """(dw, the same in 64 bits, the sum of its terms' magnitudes)"""
    dy = _rand(t, o, T, seed, 0.05, pad, off)
    ck = torch.empty(t, lz.ckpt_row_bytes(i), dtype=torch.uint8, device=DEV)
    lz.zero_ckpt_save_q8(t, i, _rand(t, i, T, seed + 1, 1.0), ck)
    dw = _rand(o, i, T, seed + 2, 1.0, dwpad, dwoff)
    before = dw.double() if acc else torch.zeros((), dtype=torch.float64, device=DEV)
    st = status_word()
    n = lz.zero_ckpt_wgrad_q8_workspace(t, o, i)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) if n else None
    lz.zero_ckpt_wgrad_q8(t, o, i, dy, ck, dw, st, workspace=ws, accumulate=acc)
    assert status_flags(st) == 0
    a, d = _values(ck, i), dy.double()
    return dw, d.T @ a + before, d.abs().T @ a.abs() + before.abs()


def _check(name, t, dw, want, mag, T):
    # a enters the product rounded to T (half a step of T per term; q*scale itself is rounded to
    # binary32, half a step more). The tensor cores add binary32 with truncation: a full step
    # (two half steps U) per addition, t additions.
    err = (A.HALF[T] + (2 * (t + 2) + 1) * A.U) * mag
    tol = err + A.HALF[T] * (want.abs() + err) + A.TINY[T]
    off = (dw.double() - want).abs()
    assert bool((off <= tol).all()), (name, float((off / tol).max()))
    # independent rounding errors: those of a, relative to the sum of products of mean zero as to
    # each of them, are at most half a step in the root mean square, those of dw another; 1.25 for
    # the sums' truncation and chance
    rel = float((dw.double() - want).norm() / want.norm())
    assert rel <= 1.25 * 2 ** 0.5 * A.HALF[T], (name, rel)


@pytest.mark.parametrize("T", [F16, BF16])
@pytest.mark.parametrize("t,o,i", [(1, 200, 300), (200, 264, 392), (1024, 768, 768),
                                   (5003, 1537, 1100), (2048, 64, 200)])
def test_weight_gradient_at_unrounded_values(t, o, i, T):
    _check((t, o, i), t, *_call(t, o, i, T, t + o), T)

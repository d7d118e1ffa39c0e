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


# Pairs of CTAs that take several tiles one after the other, at both tile heights.
def _plan(t, o, i):
    """The library's plan: (256-row halves per tile, tiles along the out-features, along the
    in-features, parts of the sum, units), with its measured constants, in binary32."""
    f = torch.tensor
    ti, kb, best = -(-i // 256), -(-t // 64), None
    for m, stage, fixed in ((1, 0.47, 2.5), (2, 0.62, 4.0)):
        to = -(-o // (256 * m))
        for s in range(1, kb + 1):
            if s > 1 and to * ti * s > 148:
                break
            blocks = -(-kb // s)
            parts = -(-kb // blocks)
            units = to * ti * parts
            cost = f(float(-(-units // 74))) * (f(float(blocks)) * f(stage) + f(fixed))
            if parts > 1:
                cost = cost + f(3.0) + f(0.06) * f(float(units * m))
            if best is None or float(cost) < best[0]:
                best = (float(cost), m, to, ti, parts, units)
    return best[1:]


# (tokens, out, in, halves per tile, whether a pair takes a second unit, whether sums are split)
SIZES = [
    (70, 4500, 2500, 1, True, False),      # 180 tiles: both accumulators, ten tiles of in-features
    (200, 4864, 2000, 2, True, False),     # 80 tiles of 512 rows
    (700, 5000, 2304, 2, True, False),     # 90 of 11 stages: the ring of stages turns
    (130, 4871, 2500, 2, True, False),     # dy through its aligned copy
    (16384, 2304, 768, 2, False, True),    # a long sum in four parts
    (16384, 2300, 760, 2, False, True),
    (3000, 1003, 500, 1, False, True),
]


@pytest.mark.parametrize("t,o,i,halves,again,split", SIZES)
def test_sizes_take_the_path_they_are_for(t, o, i, halves, again, split):
    m, to, ti, parts, units = _plan(t, o, i)
    assert (m, units > 74, parts > 1) == (halves, again, split)
    need = to * ti * parts * 256 * m * 256 * 4 if parts > 1 else 0
    if o % 8:
        need += t * (-(-o // 8) * 8) * 2
    assert lz.zero_ckpt_wgrad_q8_workspace(t, o, i) == need


@pytest.mark.parametrize("T", [F16, BF16])
@pytest.mark.parametrize("t,o,i", [c[:3] for c in SIZES])
def test_several_tiles_per_pair(t, o, i, T):
    _check((t, o, i), t, *_call(t, o, i, T, t + o), T)


@pytest.mark.parametrize("t,o,i,pad,off,dwpad,dwoff", [
    (200, 4864, 2000, 1, 0, 0, 0),         # 512-row tiles, dy loaded in place
    (200, 4864, 2000, 0, 4, 0, 0),
    (200, 4864, 2000, 8, 8, 3, 1),         # dw at any alignment
    (130, 4871, 2501, 0, 0, 0, 0),
    (130, 4871, 2501, 2, 3, 5, 3),
    (70, 4500, 2500, 1, 1, 4, 2),          # 256-row tiles
    (16384, 2304, 768, 3, 2, 1, 1)])
@pytest.mark.parametrize("acc", [False, True])
def test_strides(t, o, i, pad, off, dwpad, dwoff, acc):
    dw, want, mag = _call(t, o, i, F16, 7, pad, off, dwpad, dwoff, acc)
    _check((t, o, i, pad, acc), t, dw, want, mag, F16)
    if dwpad or dwoff:
        flat = dw._base.view(-1).clone()
        flat.as_strided(dw.shape, dw.stride(), dw.storage_offset()).fill_(7.0)
        assert bool((flat == 7).all())


@pytest.mark.parametrize("t,o,i", [(16384, 2304, 768), (1024, 768, 768), (5003, 1537, 1100),
                                   (700, 5000, 2304)])
def test_same_bits_every_time(t, o, i):
    dy = _rand(t, o, F16, 1, 0.05)
    ck = torch.empty(t, lz.ckpt_row_bytes(i), dtype=torch.uint8, device=DEV)
    lz.zero_ckpt_save_q8(t, i, _rand(t, i, F16, 2, 1.0), ck)
    st = status_word()
    n = lz.zero_ckpt_wgrad_q8_workspace(t, o, i)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    outs = [torch.empty(o, i, dtype=F16, device=DEV) for _ in range(12)]
    for dw in outs:
        lz.zero_ckpt_wgrad_q8(t, o, i, dy, ck, dw, st, workspace=ws)
    assert all(torch.equal(dw, outs[0]) for dw in outs) and status_flags(st) == 0


@pytest.mark.parametrize("o,stride", [(64, 1 << 41), (64, (1 << 41) + 3), (13, (1 << 40) + 1),
                                      (64, 67)])
def test_one_token_at_any_stride(o, stride):
    """The stride of a single row is used for nothing, however large."""
    i = 136
    dy, a = _rand(1, o, F16, 1, 1.0), _rand(1, i, F16, 2, 1.0)
    ck = torch.empty(1, lz.ckpt_row_bytes(i), dtype=torch.uint8, device=DEV)
    lz.zero_ckpt_save_q8(1, i, a, ck)
    n = lz.zero_ckpt_wgrad_q8_workspace(1, o, i)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    dw, st = torch.empty(o, i, dtype=F16, device=DEV), status_word()
    lz.zero_ckpt_wgrad_q8(1, o, i, (dy.data_ptr(), stride), ck, dw, st, workspace=ws)
    want = dy.double().T @ _values(ck, i)
    _check((o, stride), 1, dw, want, want.abs(), F16)
    assert status_flags(st) == 0

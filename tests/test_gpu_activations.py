"""The activation-side calls on the GPU against plain 64-bit forms: 8-bit checkpoints (byte for
byte), the block boundary and its gradient, and the weight gradient from a checkpoint."""
import itertools

import numpy as np
import pytest
import torch

from tests import _act as A
from tests._gpu import DEV, lz, require_gpu, status_flags, status_word

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def _mat(rows, cols, T, seed, std=1.0, pad=0, off=0):
    """A rows x cols device matrix, in the middle of a wider and longer buffer if padded."""
    v = (torch.randn(rows, cols, generator=_gen(seed)) * std).to(T)
    if not pad and not off:
        return v.to(DEV)
    flat = torch.full(((rows + 2) * (cols + pad) + off + 64,), 7.0, dtype=T, device=DEV)
    m = flat[off + cols + pad:][:rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(v)
    return m


def _ckpt_buf(rows, cols):
    return torch.full((rows, A.row_bytes(cols)), 77, dtype=torch.uint8, device=DEV)


def _ckpt_of(m):
    rec = A.record(m.detach().cpu().float().numpy())
    return torch.from_numpy(rec).to(DEV)


# ---------------------------------------------------------------------------------------------
# checkpoints
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols,pad,off", [
    (1, 1, 0, 0), (3, 2, 0, 0), (1, 127, 0, 0), (2, 128, 0, 0), (5, 129, 0, 0), (7, 16, 3, 1),
    (1, 2048, 0, 0), (33, 1000, 24, 0), (65, 1601, 0, 0), (19, 768, 8, 4), (4, 16640, 0, 0),
    (300, 384, 0, 0), (1027, 640, 0, 0), (3, 8192, 1, 0)])
def test_checkpoint_bytes_and_values(rows, cols, pad, off, T):
    x = _mat(rows, cols, T, rows * 7 + cols, 3.0, pad, off)
    ck = _ckpt_buf(rows + 1, cols)
    lz.zero_ckpt_save_q8(rows, cols, x, ck[:rows])
    want = A.record(x.cpu().float().numpy())
    got = ck.cpu().numpy()
    assert A.same_bytes(got[:rows], want, cols)
    assert (got[rows] == 77).all()
    for T2 in {T, F16, F32}:
        big = torch.full((rows, cols + pad + off), 5.0, dtype=T2, device=DEV)
        out = big[:, off:off + cols]
        lz.zero_ckpt_load_q8(rows, cols, ck[:rows], out)
        ref = torch.from_numpy(A.values(want, cols)).to(T2)
        assert torch.equal(out.cpu(), ref)
        assert (big[:, :off] == 5).all() and (big[:, off + cols:] == 5).all()


@pytest.mark.parametrize("T", [F16, BF16, F32])
def test_checkpoint_special_values(T):
    rows, cols = 12, 300
    x = torch.randn(rows, cols, generator=_gen(5)).to(T)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 299] = float("nan")
    x[3] = torch.finfo(T).tiny * torch.randn(cols, generator=_gen(6)).to(T)   # near subnormal
    x[4, :128] = torch.finfo(T).smallest_normal / 8
    x[5] = torch.finfo(T).max
    x[6] = -torch.finfo(T).max
    x[7, 130:] = 0
    x[8] = float("-inf")
    x[9, ::2] = -0.0
    # half-integer quotients: scale is 2 with amax 254
    x[10] = torch.tensor([254.0] + [2.0 * (k % 100) + 1.0 for k in range(cols - 1)]).to(T)
    if T is F32:
        x[11] = torch.randn(cols, generator=_gen(7)) * 1e-44
    ck = _ckpt_buf(rows, cols)
    lz.zero_ckpt_save_q8(rows, cols, x.to(DEV), ck)
    want = A.record(x.float().numpy())
    assert A.same_bytes(ck.cpu().numpy(), want, cols)
    out = torch.empty(rows, cols, dtype=T, device=DEV)
    lz.zero_ckpt_load_q8(rows, cols, ck, out)
    ref = torch.from_numpy(A.values(want, cols)).to(T)
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(out.cpu()), torch.nan_to_num(ref))
    assert torch.isnan(out[1, :128]).all() and not torch.isnan(out[1, 128:]).any()


@pytest.mark.parametrize("T", [F16, F32])
def test_checkpoint_near_ties(T):
    """Values a few steps around every half-integer quotient keep IEEE division's rounding."""
    rng = np.random.default_rng(3)
    rows, cols = 2000, 128
    amax = rng.uniform(0.5, 2.0, (rows, 1)).astype(np.float32)
    scale = (amax / np.float32(127)).astype(np.float32)
    k = rng.integers(-126, 126, (rows, cols)) + 0.5
    x = (k * scale).astype(np.float32)
    x = np.nextafter(x, x + rng.choice([-1, 1], (rows, cols)).astype(np.float32),
                     dtype=np.float32) if T is F32 else x
    x[:, 0] = amax[:, 0]
    xt = torch.from_numpy(x).to(T)
    ck = _ckpt_buf(rows, cols)
    lz.zero_ckpt_save_q8(rows, cols, xt.to(DEV), ck)
    assert A.same_bytes(ck.cpu().numpy(), A.record(xt.float().numpy()), cols)


def test_checkpoint_rows_are_checkpoints():
    """A range of rows is a checkpoint of its own: two halves saved apart, one read across."""
    x = _mat(10, 777, F16, 1)
    whole, parts = _ckpt_buf(10, 777), _ckpt_buf(10, 777)
    lz.zero_ckpt_save_q8(10, 777, x, whole)
    lz.zero_ckpt_save_q8(4, 777, x[:4], parts[:4])
    lz.zero_ckpt_save_q8(6, 777, x[4:], parts[4:])
    assert torch.equal(whole, parts)
    out = torch.empty(5, 777, dtype=F16, device=DEV)
    lz.zero_ckpt_load_q8(5, 777, whole[3:8], out)
    assert np.array_equal(out.cpu().float().numpy(),
                          torch.from_numpy(A.values(whole.cpu().numpy(), 777)).half()
                          .float().numpy()[3:8])


# ---------------------------------------------------------------------------------------------
# block boundary
# ---------------------------------------------------------------------------------------------
def _boundary(rows, cols, T, post, pre, gate_rows, bias, seed, pad=0, off=0, branch=True):
    """(keyword arguments of the calls, the same in 64 bits, x, h)."""
    def vec(k, mean):
        return (torch.randn(cols, generator=_gen(seed + k)) * 0.2 + mean).to(T).to(DEV)

    d = dict(post_norm=post, pre_norm=pre, post_eps=1e-5, pre_eps=1e-3, residual_scale=0.75,
             branch_scale=1.25)
    if branch and gate_rows:
        d["gate_rows"] = gate_rows
        d["gate"] = _mat(-(-rows // gate_rows), cols, T, seed + 1, 0.5, pad, off)
    if pre != "none":
        d["pre_w"] = vec(2, 1.0)
        if bias:
            d["pre_b"] = vec(3, 0.0)
    if branch and post != "none":
        d["post_w"] = vec(4, 0.5)
        if bias:
            d["post_b"] = vec(5, 0.1)
    ref = {k: A.f64(v) if torch.is_tensor(v) else v for k, v in d.items()}
    x = _mat(rows, cols, T, seed + 6, 1.5, pad, off)
    h = _mat(rows, cols, T, seed + 7, 0.8, pad, off) if branch else None
    if h is not None:
        h += 0.5                          # a mean for LayerNorm to take off
    return d, ref, x, h


SHAPES = [(1, 1), (2, 3), (1, 2048), (5, 129), (3, 768), (70, 64), (33, 1000), (9, 4096),
          (2, 16384), (261, 384), (6, 5000)]
KINDS = ["none", "rms", "layer"]


@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_join_forward(rows, cols, T):
    for i, (post, pre) in enumerate(itertools.product(KINDS, KINDS)):
        gate_rows = [0, 1, max(1, rows // 2), rows][(i + rows) % 4]
        pad, off = [(0, 0), (8, 0), (3, 1)][i % 3]
        d, ref, x, h = _boundary(rows, cols, T, post, pre, gate_rows, i % 2 == 0, 10 * i, pad, off)
        y = _mat(rows, cols, T, 1, 0.0, pad, off)
        u = None if pre == "none" else _mat(rows, cols, T, 1, 0.0, pad, off)
        sy, sh = _ckpt_buf(rows, cols), _ckpt_buf(rows, cols)
        lz.zero_block_join(rows, cols, x=x, h=h, y=y, u=u, save_y=sy, save_h=sh, **d)
        wy, wu, my, mu = A.join(ref, A.f64(x), A.f64(h))
        A.close(f"y {post} {pre}", y, wy, my, T, ROW_FWD)
        if u is not None:
            A.close(f"u {post} {pre}", u, wu, mu, T, A.CHAIN)
        assert A.same_bytes(sh.cpu().numpy(), A.record(h.cpu().float().numpy()), cols)
        assert A.same_bytes(sy.cpu().numpy(), A.record(y.cpu().float().numpy()), cols)


ROW_FWD = A.ROW + 32


def _guard(m):
    """The buffer around a padded matrix from _mat, minus the matrix: all still 7."""
    base = m._base if m._base is not None else m
    flat = base.view(-1).clone()
    keep = torch.ones_like(flat, dtype=torch.bool)
    idx = torch.arange(flat.numel(), device=flat.device)
    keep[torch.as_strided(idx, m.shape, m.stride(), m.storage_offset()).reshape(-1)] = False
    return bool((flat[keep] == 7).all())


@pytest.mark.parametrize("T", [F16, F32])
def test_join_outputs_stay_inside(T):
    rows, cols = 13, 333
    d, ref, x, h = _boundary(rows, cols, T, "rms", "layer", 4, True, 3, 19, 5)
    y, u = (_mat(rows, cols, T, 1, 0.0, 19, 5) for _ in range(2))
    lz.zero_block_join(rows, cols, x=x, h=h, y=y, u=u, **d)
    dx, dh = (_mat(rows, cols, T, 1, 0.0, 19, 5) for _ in range(2))
    dgate = _mat(4, cols, T, 1, 0.0, 19, 5)
    ws = torch.empty(lz.zero_block_join_backward_workspace(rows, cols, 4), dtype=torch.uint8,
                     device=DEV)
    lz.zero_block_join_backward(rows, cols, y=y, h=h, dy=x, du=u, dx=dx, dh=dh, dgate=dgate,
                                workspace=ws, **d)
    for m in (x, h, y, u, dx, dh, dgate):
        assert _guard(m)


def test_join_column_slices_of_one_buffer():
    """x, h, y, u and a gate as column slices of one matrix: they interleave and do not overlap."""
    rows, cols = 6, 96
    big = torch.randn(rows, 5 * cols, generator=_gen(3)).half().to(DEV)
    x, h, y, u, gate = (big[:, i * cols:(i + 1) * cols] for i in range(5))
    d = dict(post_norm="rms", pre_norm="layer", post_eps=1e-5, pre_eps=1e-5, residual_scale=1.0,
             branch_scale=0.5, gate_rows=1, gate=gate)
    ref = dict(d, gate=A.f64(gate))
    lz.zero_block_join(rows, cols, x=x, h=h, y=y, u=u, **d)
    wy, wu, my, mu = A.join(ref, A.f64(x), A.f64(h))
    A.close("y", y, wy, my, F16, ROW_FWD)
    A.close("u", u, wu, mu, F16, A.CHAIN)


@pytest.mark.parametrize("source", ["matrix", "checkpoint"])
def test_norm_of_a_checkpoint(source):
    """Without a branch the call is a norm of x: the recomputation of a block's input."""
    rows, cols = 37, 2048
    d, ref, x, _ = _boundary(rows, cols, F16, "none", "layer", 0, True, 4, branch=False)
    ck = _ckpt_of(x)
    u = torch.empty(rows, cols, dtype=F16, device=DEV)
    src = dict(x=x) if source == "matrix" else dict(x_ckpt=ck)
    lz.zero_block_join(rows, cols, u=u, **src, **d)
    xv = A.f64(x) if source == "matrix" else A.values(ck.cpu().numpy(), cols).astype(np.float64)
    _, wu, _, mu = A.join(ref, xv, None)
    A.close("u", u, wu, mu, F16, A.CHAIN)


def test_join_from_checkpoints():
    rows, cols = 21, 1001
    d, ref, x, h = _boundary(rows, cols, BF16, "rms", "rms", 7, False, 8)
    cx, ch = _ckpt_of(x), _ckpt_of(h)
    y, u = (torch.empty(rows, cols, dtype=BF16, device=DEV) for _ in range(2))
    lz.zero_block_join(rows, cols, x_ckpt=cx, h_ckpt=ch, y=y, u=u, **d)
    xv, hv = (A.values(c.cpu().numpy(), cols).astype(np.float64) for c in (cx, ch))
    wy, wu, my, mu = A.join(ref, xv, hv)
    A.close("y", y, wy, my, BF16, ROW_FWD)
    A.close("u", u, wu, mu, BF16, A.CHAIN)


def test_join_in_place_and_special_rows():
    """y in x's place; a row of zeros, constant rows, an inf and a NaN stay in their rows."""
    rows, cols = 9, 640
    d, ref, x, h = _boundary(rows, cols, F16, "rms", "layer", rows, True, 9)
    x[0], h[0] = 0, 0
    x[1], h[1] = 3.0, 3.0
    x[2, 5] = float("inf")
    h[3, 639] = float("nan")
    keep = x.clone()
    u = torch.empty_like(x)
    sy = _ckpt_buf(rows, cols)
    lz.zero_block_join(rows, cols, x=x, h=h, y=x, u=u, save_y=sy, **d)
    with np.errstate(all="ignore"):
        wy, wu, my, mu = A.join(ref, A.f64(keep), A.f64(h))
    fine = [0, 1, 4, 5, 6, 7, 8]
    A.close("y", x[fine], wy[fine], my[fine], F16, ROW_FWD)
    A.close("u", u[fine], wu[fine], mu[fine], F16, A.CHAIN)
    assert torch.isinf(x[2, 5]) and torch.isfinite(x[2]).sum() == cols - 1
    assert torch.isnan(u[2]).all() and torch.isnan(x[3]).all() and torch.isnan(u[3]).all()
    assert A.same_bytes(sy.cpu().numpy(), A.record(x.cpu().float().numpy()), cols)


def _back(d, rows, cols, T, y, h, dy, du, names, seed=0, accumulate=0, base=None, **kw):
    gates = -(-rows // d["gate_rows"]) if d.get("gate_rows") else 0
    out = {}
    for n in names:
        shape = (rows, cols) if n in ("dx", "dh") else (gates, cols) if n == "dgate" else (cols,)
        out[n] = torch.full(shape, 3.0, dtype=T, device=DEV) if base is None else base[n].clone()
    ws = torch.full((lz.zero_block_join_backward_workspace(rows, cols, d.get("gate_rows", 0)),),
                    0xff, dtype=torch.uint8, device=DEV)
    src = {}
    for k, v in (("y", y), ("h", h)):
        if v is not None:
            src[k + "_ckpt" if v.dtype == torch.uint8 else k] = v
    lz.zero_block_join_backward(rows, cols, dy=dy, du=du, workspace=ws, accumulate=accumulate,
                                **src, **out, **d, **kw)
    return out


@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", SHAPES + [(700, 96), (40, 2048)])
def test_join_backward(rows, cols, T):
    for i, (post, pre) in enumerate(itertools.product(KINDS, KINDS)):
        gate_rows = [0, 1, max(1, rows // 3), rows][(i + cols) % 4]
        pad, off = [(0, 0), (8, 0), (3, 1)][(i + 1) % 3]
        d, ref, y, h = _boundary(rows, cols, T, post, pre, gate_rows, i % 2 == 1, 10 * i, pad, off)
        dy = _mat(rows, cols, T, 100 + i, 0.1, pad, off)
        du = None if pre == "none" else _mat(rows, cols, T, 200 + i, 0.1, pad, off)
        kept = i % 3 != 0
        ys, hs = (_ckpt_of(y), _ckpt_of(h)) if kept else (y, h)
        yv, hv = ((A.values(c.cpu().numpy(), cols).astype(np.float64) for c in (ys, hs)) if kept
                  else (A.f64(y), A.f64(h)))
        names = ["dx", "dh"] + ["dpre_w", "dpre_b"] * (pre != "none") + \
            ["dpost_w", "dpost_b"] * (post != "none") + ["dgate"] * (gate_rows > 0)
        got = _back(d, rows, cols, T, ys, hs, dy, du, names)
        want = A.back(ref, yv, hv, A.f64(dy), A.f64(du))
        for n in names:
            v, m = want[n]
            A.close(f"{n} {post} {pre} gate {gate_rows}", got[n], v, m, T,
                    A.CHAIN if n in ("dx", "dh") else A.CHAIN + rows)


@pytest.mark.parametrize("T,rows,cols", [(F16, 400, 8192), (F16, 330, 16384), (BF16, 350, 5000),
                                         (F32, 300, 4096), (F32, 170, 16384), (F16, 210, 5263)])
@pytest.mark.parametrize("post,pre,gate_rows", [("rms", "rms", 100), ("none", "layer", 0),
                                                ("layer", "layer", 0)])
def test_wide_rows(rows, cols, T, post, pre, gate_rows):
    """Rows that several CTAs share, several rows one after the other per cluster."""
    d, ref, x, h = _boundary(rows, cols, T, post, pre, gate_rows, True, 60)
    y, u = torch.empty_like(x), torch.empty_like(x)
    sy, sh = _ckpt_buf(rows, cols), _ckpt_buf(rows, cols)
    lz.zero_block_join(rows, cols, x=x, h=h, y=y, u=u, save_y=sy, save_h=sh, **d)
    wy, wu, my, mu = A.join(ref, A.f64(x), A.f64(h))
    A.close("y", y, wy, my, T, ROW_FWD)
    A.close("u", u, wu, mu, T, A.CHAIN)
    assert A.same_bytes(sy.cpu().numpy(), A.record(y.cpu().float().numpy()), cols)
    dy, du = _mat(rows, cols, T, 1, 0.1), _mat(rows, cols, T, 2, 0.1)
    names = ["dx", "dh", "dpre_w", "dpre_b"] + ["dpost_w", "dpost_b"] * (post != "none") + \
        ["dgate"] * (gate_rows > 0)
    if T is F32:
        got, yv, hv = _back(d, rows, cols, T, y, h, dy, du, names), A.f64(y), A.f64(h)
    else:
        got = _back(d, rows, cols, T, sy, sh, dy, du, names)
        yv, hv = (A.values(c.cpu().numpy(), cols).astype(np.float64) for c in (sy, sh))
    want = A.back(ref, yv, hv, A.f64(dy), A.f64(du))
    for n in names:
        v, m = want[n]
        A.close(n, got[n], v, m, T, A.CHAIN if n in ("dx", "dh") else A.CHAIN + rows)


def test_join_backward_parts():
    """Any subset of the outputs and gradients: the same bits as from the full call."""
    rows, cols = 50, 384
    d, ref, y, h = _boundary(rows, cols, F16, "layer", "rms", 16, True, 5)
    dy, du = _mat(rows, cols, F16, 1, 0.1), _mat(rows, cols, F16, 2, 0.1)
    names = ["dx", "dh", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b"]
    full = _back(d, rows, cols, F16, y, h, dy, du, names)
    for n in names:
        assert torch.equal(_back(d, rows, cols, F16, y, h, dy, du, [n])[n], full[n]), n
    again = _back(d, rows, cols, F16, y, h, dy, du, names)
    assert all(torch.equal(again[n], full[n]) for n in names)
    # no gradient along the residual, or none of u
    for dyv, duv in ((None, du), (dy, None), (None, None)):
        got = _back(d, rows, cols, F16, y, h, dyv, duv, names)
        zero = np.zeros((rows, cols))
        want = A.back(ref, A.f64(y), A.f64(h), zero if dyv is None else A.f64(dyv),
                      zero if duv is None else A.f64(duv))
        for n in names:
            v, m = want[n]
            A.close(n, got[n], v, m, F16, A.CHAIN + rows)
    # dx in dy's place
    keep = dy.clone()
    out = {n: torch.empty_like(full[n]) for n in names[1:]}
    ws = torch.empty(lz.zero_block_join_backward_workspace(rows, cols, 16), dtype=torch.uint8,
                     device=DEV)
    lz.zero_block_join_backward(rows, cols, y=y, h=h, dy=keep, du=du, dx=keep, workspace=ws,
                                **out, **d)
    assert torch.equal(keep, full["dx"]) and all(torch.equal(out[n], full[n]) for n in out)


@pytest.mark.parametrize("T", [F16, F32])
def test_join_backward_accumulates(T):
    rows, cols = 65, 200
    d, ref, y, h = _boundary(rows, cols, T, "rms", "layer", 32, True, 6)
    dy, du = _mat(rows, cols, T, 1, 0.1), _mat(rows, cols, T, 2, 0.1)
    names = ["dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b"]
    base = {n: _mat(3 if n == "dgate" else 1, cols, T, 30 + i) for i, n in enumerate(names)}
    base = {n: v if n == "dgate" else v[0] for n, v in base.items()}
    want = A.back(ref, A.f64(y), A.f64(h), A.f64(dy), A.f64(du))
    for acc in (0, lz.ZERO_ACC_PARAMS, lz.ZERO_ACC_GATE, 3):
        got = _back(d, rows, cols, T, y, h, dy, du, names, accumulate=acc, base=base)
        for n in names:
            add = acc & (lz.ZERO_ACC_GATE if n == "dgate" else lz.ZERO_ACC_PARAMS)
            v, m = want[n]
            b = A.f64(base[n]) if add else 0.0
            A.close(n, got[n], v + b, m + np.abs(b), T, A.CHAIN + rows)


def test_join_backward_no_rows():
    d, _, _, _ = _boundary(1, 64, F16, "rms", "rms", 0, True, 6)
    vec = {n: torch.full((64,), 3.0, dtype=F16, device=DEV)
           for n in ("dpost_w", "dpost_b", "dpre_w", "dpre_b")}
    ws = torch.empty(max(16, lz.zero_block_join_backward_workspace(0, 64, 0)), dtype=torch.uint8,
                     device=DEV)
    lz.zero_block_join_backward(0, 64, workspace=ws, accumulate=lz.ZERO_ACC_PARAMS, **vec, **d)
    assert all((v == 3).all() for v in vec.values())
    lz.zero_block_join_backward(0, 64, workspace=ws, **vec, **d)
    assert all((v == 0).all() for v in vec.values())


def test_join_backward_against_differences():
    """The gradient of sum(dy*y + du*u) along random directions, by central differences of the
    64-bit forward, against the kernel's fp32 outputs."""
    rows, cols = 6, 40
    d, ref, y, h = _boundary(rows, cols, F32, "layer", "rms", 3, True, 12)
    x = _mat(rows, cols, F32, 40, 1.0)
    dy, du = _mat(rows, cols, F32, 41), _mat(rows, cols, F32, 42)
    y = torch.empty_like(x)
    lz.zero_block_join(rows, cols, x=x, h=h, y=y, **d)
    names = ["dx", "dh", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b"]
    got = _back(d, rows, cols, F32, y, h, dy, du, names)

    def loss(ref_, xv, hv):
        yv, uv, _, _ = A.join(ref_, xv, hv)
        return float((A.f64(dy) * yv).sum() + (A.f64(du) * uv).sum())

    rng = np.random.default_rng(0)
    step = 1e-5
    for n, key in (("dx", None), ("dh", None), ("dgate", "gate"), ("dpost_w", "post_w"),
                   ("dpost_b", "post_b"), ("dpre_w", "pre_w"), ("dpre_b", "pre_b")):
        shape = got[n].shape
        v = rng.standard_normal(tuple(shape))
        ends = []
        for s in (step, -step):
            r2, xv, hv = dict(ref), A.f64(x), A.f64(h)
            if n == "dx":
                xv = xv + s * v
            elif n == "dh":
                hv = hv + s * v
            else:
                r2[key] = ref[key] + s * v
            ends.append(loss(r2, xv, hv))
        slope = (ends[0] - ends[1]) / (2 * step)
        mine = float((A.f64(got[n]) * v).sum())
        # central differences: step^2 * third derivative (order 10 here) ~ 1e-9 relative, and
        # 1e-16/step = 1e-11 of the loss; the kernel's fp32: CHAIN half steps of the sum's terms
        size = float((np.abs(A.f64(got[n]) * v)).sum()) + 1.0
        assert abs(slope - mine) <= 1e-4 * size, (n, slope, mine)


# ---------------------------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------------------------
def _wgrad(t, o, i, T, seed, pad=0, off=0, acc=False, dwpad=0, dwoff=0):
    dy = _mat(t, o, T, seed, 0.05, pad, off)
    a = _mat(t, i, T, seed + 1, 1.0)
    ck = _ckpt_of(a)
    dw = _mat(o, i, T, seed + 2, 1.0, dwpad, dwoff)
    before = A.f64(dw) if acc else 0.0
    st = status_word()
    n = lz.zero_ckpt_wgrad_q8_workspace(t, o, i)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) if n else None
    lz.zero_ckpt_wgrad_q8(t, o, i, dy, ck, dw, st, workspace=ws, accumulate=acc)
    assert status_flags(st) == 0
    av = torch.from_numpy(A.values(ck.cpu().numpy(), i)).to(T).double().numpy()
    dyv = A.f64(dy)
    want = dyv.T @ av + before
    mag = np.abs(dyv).T @ np.abs(av) + np.abs(before)
    # the tensor cores add binary32 with truncation: a full step (2 U) per addition, t additions
    A.close(f"dw {t}x{o}x{i}", dw, want, mag, T, 2 * (t + 2))
    return dw


@pytest.mark.parametrize("T", [F16, BF16])
@pytest.mark.parametrize("t,o,i", [
    (1, 1, 1), (1, 128, 128), (3, 5, 7), (16, 64, 64), (64, 256, 256), (65, 129, 257),
    (100, 300, 1000), (1000, 256, 128), (257, 768, 768), (2048, 64, 200), (33, 2048, 520),
    (129, 1000, 130), (640, 513, 511)])
def test_wgrad(t, o, i, T):
    _wgrad(t, o, i, T, t + o)


@pytest.mark.parametrize("pad,off,dwpad,dwoff", [(8, 0, 0, 0), (1, 0, 0, 0), (0, 1, 0, 1),
                                                 (8, 8, 8, 8), (3, 2, 5, 3), (2, 4, 4, 2)])
@pytest.mark.parametrize("acc", [False, True])
def test_wgrad_strides(pad, off, dwpad, dwoff, acc):
    dw = _wgrad(200, 264, 392, F16, 9, pad, off, acc, dwpad, dwoff)
    if dwpad or dwoff:
        assert _guard(dw)


def test_wgrad_no_tokens_and_accumulate():
    dw = torch.full((30, 50), 3.0, dtype=F16, device=DEV)
    st = status_word()
    lz.zero_ckpt_wgrad_q8(0, 30, 50, None, None, dw, st, accumulate=True)
    assert (dw == 3).all()
    lz.zero_ckpt_wgrad_q8(0, 30, 50, None, None, dw, st)
    assert (dw == 0).all() and status_flags(st) == 0


def test_wgrad_poisoned_block():
    """A block with an inf or NaN makes its 128 columns of the gradient NaN, and no others."""
    t, o, i = 90, 140, 300
    dy = _mat(t, o, F16, 1, 0.1)
    a = _mat(t, i, F16, 2)
    a[17, 130] = float("inf")
    dw = torch.empty(o, i, dtype=F16, device=DEV)
    n = lz.zero_ckpt_wgrad_q8_workspace(t, o, i)
    lz.zero_ckpt_wgrad_q8(t, o, i, dy, _ckpt_of(a), dw, status_word(),
                          workspace=torch.empty(n, dtype=torch.uint8, device=DEV) if n else None)
    assert torch.isnan(dw[:, 128:256]).all()
    assert torch.isfinite(dw[:, :128]).all() and torch.isfinite(dw[:, 256:]).all()


def test_wgrad_same_bits_again():
    a = _wgrad(777, 512, 384, F16, 4)
    b = _wgrad(777, 512, 384, F16, 4)
    assert torch.equal(a, b)

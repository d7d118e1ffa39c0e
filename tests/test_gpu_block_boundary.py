"""The block boundary where its kernels differ: every pair of norms at every alignment, with the saved
rows as matrices and as checkpoints, and with so many rows that each team of warps walks through
several of them."""
import itertools

import numpy as np
import pytest
import torch

from tests import _act as A
from tests._gpu import DEV, lz, require_gpu

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
KINDS = ["none", "rms", "layer"]
PADS = [(0, 0), (8, 0), (3, 1)]          # adjacent rows, strided, strided at any alignment
ROW_FWD = A.ROW + 32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _put(v, T, pad=0, off=0, times=1):
    """`times` copies of a host array's rows as a device matrix of T, in the middle of a wider and
    longer buffer if padded."""
    v = torch.from_numpy(np.ascontiguousarray(v)).to(T).to(DEV).repeat(times, 1)
    if not pad and not off:
        return v
    rows, cols = v.shape
    flat = torch.full(((rows + 2) * (cols + pad) + off,), 7.0, dtype=T, device=DEV)
    m = flat[off + cols + pad:][:rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return m.copy_(v)


def _rounded(v, T):
    return torch.from_numpy(np.ascontiguousarray(v)).to(T).double().numpy()


class Case:
    """A boundary over `times` copies of `rows` different rows (all of them where times is 1), its
    operands on the device and in 64 bits. gate: None, "row" (one gate row per row), "copy" (one per
    copy, all alike) or "one"."""

    def __init__(self, rows, cols, T, post, pre, gate, bias, seed, pad=0, off=0, times=1):
        rng = np.random.default_rng(seed)
        self.rows, self.cols, self.T, self.times = rows, cols, T, times
        self.pad, self.off, self.gate = pad, off, gate

        def mat(n, std, mean=0.0):
            return _rounded(rng.standard_normal((n, cols)) * std + mean, T)

        self.x, self.h = mat(rows, 1.5), mat(rows, 0.8, 0.5)
        self.dy, self.du = mat(rows, 0.1), mat(rows, 0.1)
        self.ref = dict(post_norm=post, pre_norm=pre, post_eps=1e-5, pre_eps=1e-3,
                        residual_scale=0.75, branch_scale=1.25)
        n = {None: 0, "row": rows, "copy": 1, "one": 1}[gate]
        if gate:
            self.ref.update(gate=mat(n, 0.5), gate_rows=1 if gate == "row" else rows)
        for name, there, mean in (("pre_w", pre != "none", 1.0),
                                  ("pre_b", pre != "none" and bias, 0.0),
                                  ("post_w", post != "none", 0.5),
                                  ("post_b", post != "none" and bias, 0.1)):
            if there:
                self.ref[name] = mat(1, 0.2, mean)[0]
        self.kw = dict(self.ref)
        if gate:
            g = self.ref["gate"]
            self.kw["gate"] = self.all(g) if gate in ("row", "copy") else self.put(g)
            self.kw["gate_rows"] = {"row": 1, "copy": rows, "one": rows * times}[gate]
        for name in ("pre_w", "pre_b", "post_w", "post_b"):
            if name in self.ref:
                self.kw[name] = torch.from_numpy(self.ref[name]).to(T).to(DEV)

    def put(self, v):
        return _put(v, self.T, self.pad, self.off)

    def all(self, v):
        return _put(v, self.T, self.pad, self.off, self.times)

    def empty(self):
        return self.all(np.zeros((self.rows, self.cols)))

    def ckpt(self):
        return torch.zeros(self.rows * self.times, A.row_bytes(self.cols), dtype=torch.uint8,
                           device=DEV)

    def first(self, name, m):
        """The first copy of the rows; every other copy has the same bits."""
        c = m.reshape(self.times, self.rows, -1)
        bits = torch.int32 if m.element_size() == 4 else torch.int16 if m.element_size() == 2 \
            else torch.uint8
        same = (c.contiguous().view(bits) == c[:1].contiguous().view(bits)).all(dim=2)
        assert bool(same.all()), (name, same.logical_not().nonzero()[:4].tolist())
        return c[0]

    def forward(self, saves=True, what=""):
        n = self.rows * self.times
        x, h, y = self.all(self.x), self.all(self.h), self.empty()
        u = None if self.ref["pre_norm"] == "none" else self.empty()
        sy, sh = (self.ckpt(), self.ckpt()) if saves else (None, None)
        lz.zero_block_join(n, self.cols, x=x, h=h, y=y, u=u, save_y=sy, save_h=sh, **self.kw)
        wy, wu, my, mu = A.join(self.ref, self.x, self.h)
        A.close("y " + what, self.first("y", y), wy, my, self.T, ROW_FWD)
        if u is not None:
            A.close("u " + what, self.first("u", u), wu, mu, self.T, A.CHAIN)
        if saves:
            for m, ck in ((y, sy), (h, sh)):
                want = A.record(self.first("m", m).cpu().float().numpy())
                assert A.same_bytes(self.first("ckpt", ck).cpu().numpy(), want, self.cols), what

    def backward(self, kept, what="", drop=()):
        """kept: y and h as checkpoints. drop: gradients that are not asked for."""
        n, T = self.rows * self.times, self.T
        pre, post = self.ref["pre_norm"], self.ref["post_norm"]
        yv, hv = self.x, self.h
        src = {}
        for k, v in (("y", yv), ("h", hv)):
            if kept:
                rec = torch.from_numpy(A.record(v.astype(np.float32)))
                src[k + "_ckpt"] = rec.to(DEV).repeat(self.times, 1)
            else:
                src[k] = self.all(v)
        if kept:
            yv, hv = (A.values(A.record(v.astype(np.float32)), self.cols).astype(np.float64)
                      for v in (yv, hv))
        dy = self.all(self.dy)
        du = None if pre == "none" else self.all(self.du)
        out = dict(dx=self.empty(), dh=self.empty())
        for name in ["dpre_w", "dpre_b"] * (pre != "none") + ["dpost_w", "dpost_b"] * (post != "none"):
            out[name] = torch.full((self.cols,), 3.0, dtype=T, device=DEV)
        if self.gate:
            out["dgate"] = torch.full_like(self.kw["gate"], 3.0)
        for name in drop:
            out.pop(name, None)
        ws = torch.full((lz.zero_block_join_backward_workspace(n, self.cols,
                                                               self.kw.get("gate_rows", 0)),),
                        0xff, dtype=torch.uint8, device=DEV)
        lz.zero_block_join_backward(n, self.cols, dy=dy, du=du, workspace=ws, **src, **out,
                                    **self.kw)
        want = A.back(self.ref, yv, hv, self.dy, None if du is None else self.du)
        for name, g in out.items():
            v, m = want[name]
            copies = self.times
            if name in ("dx", "dh") or (name == "dgate" and self.gate == "row"):
                g, copies = self.first(name, g), 1
            elif name == "dgate" and self.gate == "copy":
                c = g.reshape(self.times, -1)
                # (the copies' parts may start at other rows: the same sum in another order)
                for k in range(self.times):
                    A.close(f"dgate {k} {what}", c[k:k + 1], v, m, T, A.CHAIN + self.rows)
                continue
            A.close(f"{name} {what}", g, v * copies, m * copies, T,
                    A.CHAIN if name in ("dx", "dh") else A.CHAIN + n)
        return out


@pytest.mark.parametrize("pad,off", PADS)
@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(9, 264), (160, 1032), (7, 768)])
def test_forward_of_every_kind(rows, cols, T, pad, off):
    for i, (post, pre) in enumerate(itertools.product(KINDS, KINDS)):
        gate = [None, "row", "one", "copy"][(i + i // 4 + rows) % 4]
        Case(rows, cols, T, post, pre, gate, i % 2 == 0, i, pad, off).forward(
            i % 4 != 3, f"{post} {pre} {gate}")


@pytest.mark.parametrize("pad,off", PADS)
@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("gate", [None, "row", "one"])
@pytest.mark.parametrize("rows,cols", [(11, 264), (10, 1000)])
def test_backward_of_every_kind(rows, cols, T, pad, off, kept, gate):
    for i, (post, pre) in enumerate(itertools.product(KINDS, KINDS)):
        c = Case(rows, cols, T, post, pre, gate, i % 2 == 1, i, pad, off)
        c.backward(kept, f"{post} {pre}")
        if gate:                           # a gate whose gradient is not asked for
            c.backward(kept, f"{post} {pre} without dgate", drop=("dgate",))


# Rows enough for four turns and more of every team on 148 SMs: a turn is at most 3 CTAs of 8 warps
# per SM in the forward pass, one of 16 in the gradient, and 256 or 512 columns per warp.
MANY = [(768, 101, 71), (1000, 113, 61), (2048, 101, 41), (5000, 67, 31), (64, 211, 211)]


@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("cols,rows,times", MANY)
def test_many_rows_forward(cols, rows, times, T, pad, off):
    for i, (post, pre, gate) in enumerate([("none", "layer", None), ("rms", "rms", "copy"),
                                           ("layer", "layer", "row"), ("rms", "layer", None)]):
        Case(rows, cols, T, post, pre, gate, True, i, pad, off, times).forward(
            i < 3, f"{post} {pre} {gate}")


@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
@pytest.mark.parametrize("T", [F16, BF16, F32])
@pytest.mark.parametrize("cols,rows,times", MANY)
def test_many_rows_backward(cols, rows, times, T, pad, off):
    for i, (post, pre, gate) in enumerate([("none", "layer", None), ("rms", "rms", "copy"),
                                           ("layer", "layer", "row"), ("none", "rms", "one"),
                                           ("rms", "layer", None)]):
        Case(rows, cols, T, post, pre, gate, True, i, pad, off, times).backward(
            T is not F32 and i % 2 == 0, f"{post} {pre} {gate}")


@pytest.mark.parametrize("cols", [768, 2048, 1001, 8192])
def test_many_rows_from_checkpoints(cols):
    """The recomputation of a block's input, and a boundary of two checkpoints, over many rows."""
    rows, times = 89, -(-70 * 768 // cols)
    c = Case(rows, cols, F16, "rms", "layer", None, True, 3, 0, 0, times)
    rec = [A.record(v.astype(np.float32)) for v in (c.x, c.h)]
    cx, ch = (torch.from_numpy(r).to(DEV).repeat(times, 1) for r in rec)
    xv, hv = (A.values(r, cols).astype(np.float64) for r in rec)
    y, u = c.empty(), c.empty()
    lz.zero_block_join(rows * times, cols, x_ckpt=cx, h_ckpt=ch, y=y, u=u, **c.kw)
    wy, wu, my, mu = A.join(c.ref, xv, hv)
    A.close("y", c.first("y", y), wy, my, F16, ROW_FWD)
    A.close("u", c.first("u", u), wu, mu, F16, A.CHAIN)
    alone = {k: v for k, v in c.ref.items() if not k.startswith("post")}
    alone.update(post_norm="none", residual_scale=1.0)
    kw = {k: v for k, v in c.kw.items() if k.startswith("pre")}
    lz.zero_block_join(rows * times, cols, x_ckpt=cx, u=u, **kw)
    _, wu, _, mu = A.join(alone, xv, None)
    A.close("u alone", c.first("u", u), wu, mu, F16, A.CHAIN)


@pytest.mark.parametrize("T", [F16, F32])
@pytest.mark.parametrize("post,pre", [("layer", "rms"), ("none", "layer"), ("rms", "rms")])
def test_outputs_asked_for(post, pre, T):
    """dx and dh have the same bits whatever else is asked for, and the same call the same bits; the
    column sums of another set of outputs may be rounded otherwise."""
    c = Case(53, 384, T, post, pre, "row", True, 5)
    full = c.backward(False)
    again = c.backward(False)
    assert all(torch.equal(full[n], again[n]) for n in full)
    for keep in full:
        got = c.backward(False, drop=[n for n in full if n != keep])
        if keep in ("dx", "dh"):
            assert torch.equal(got[keep], full[keep]), keep

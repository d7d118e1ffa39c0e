"""The activation-side calls as a training step uses them: together, on side streams, captured in
graphs, with long matrices, and with their gradients going into the buckets of the fused step."""
import numpy as np
import pytest
import torch

import oracle
from tests import _act as A
from tests._gpu import (DEV, HP, ORC_HP, check_f16, check_f32, f16np, f32np, lz, require_gpu,
                        status_flags, status_word)
from zero_partitioned_optimizer_plan_b200 import synth

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def _rand(shape, seed, std=1.0, T=F16):
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(T).to(DEV)


class Block:
    """Buffers of one block's boundary and linear layer (d -> o) over `rows` tokens, and the calls
    of its forward and backward pass."""

    def __init__(self, rows, d, o, seed, dw=None, dvec=None):
        self.rows, self.d, self.o = rows, d, o
        self.x, self.h = _rand((rows, d), seed), _rand((rows, d), seed + 1, 0.5)
        self.kinds = dict(post_norm="rms", pre_norm="layer", residual_scale=0.9, branch_scale=0.8,
                          gate=_rand((2, d), seed + 2, 0.5), gate_rows=-(-rows // 2),
                          post_w=_rand((d,), seed + 3), pre_w=_rand((d,), seed + 4),
                          pre_b=_rand((d,), seed + 5))
        self.y, self.u = (torch.empty(rows, d, dtype=F16, device=DEV) for _ in range(2))
        rb = lz.ckpt_row_bytes(d)
        self.sy, self.sh, self.su = (torch.empty(rows, rb, dtype=torch.uint8, device=DEV)
                                     for _ in range(3))
        self.dout = _rand((rows, o), seed + 6, 0.05)
        self.dy, self.du = _rand((rows, d), seed + 7, 0.05), _rand((rows, d), seed + 8, 0.05)
        self.dx, self.dh = (torch.empty(rows, d, dtype=F16, device=DEV) for _ in range(2))
        self.dw = torch.empty(o, d, dtype=F16, device=DEV) if dw is None else dw
        names = ("dpost_w", "dpre_w", "dpre_b")
        self.vec = dvec or {n: torch.empty(d, dtype=F16, device=DEV) for n in names}
        self.dgate = torch.empty(2, d, dtype=F16, device=DEV)
        self.status = status_word()
        gr = self.kinds["gate_rows"]
        self.ws = torch.empty(max(lz.zero_block_join_backward_workspace(rows, d, gr),
                                  lz.zero_ckpt_wgrad_q8_workspace(rows, o, d), 16),
                              dtype=torch.uint8, device=DEV)

    def forward(self, stream=None):
        lz.zero_block_join(self.rows, self.d, x=self.x, h=self.h, y=self.y, u=self.u,
                           save_y=self.sy, save_h=self.sh, stream=stream, **self.kinds)
        lz.zero_ckpt_save_q8(self.rows, self.d, self.u, self.su, stream=stream)

    def backward(self, stream=None):
        lz.zero_ckpt_wgrad_q8(self.rows, self.o, self.d, self.dout, self.su, self.dw, self.status,
                              workspace=self.ws, stream=stream)
        lz.zero_block_join_backward(self.rows, self.d, y_ckpt=self.sy, h_ckpt=self.sh, dy=self.dy,
                                    du=self.du, dx=self.dx, dh=self.dh, dgate=self.dgate,
                                    workspace=self.ws, stream=stream, **self.vec, **self.kinds)

    def outputs(self):
        return [t.clone() for t in (self.y, self.u, self.sy, self.sh, self.su, self.dw, self.dx,
                                    self.dh, self.dgate, *self.vec.values())]


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_block_against_plain_forms():
    """The whole block: what each call reads is what the one before wrote."""
    b = Block(150, 384, 264, 3)
    b.forward()
    b.backward()
    ref = {k: A.f64(v) if torch.is_tensor(v) else v for k, v in b.kinds.items()}
    ref.update(post_eps=1e-5, pre_eps=1e-5)
    wy, wu, my, mu = A.join(ref, A.f64(b.x), A.f64(b.h))
    A.close("y", b.y, wy, my, F16, A.ROW + 32)
    A.close("u", b.u, wu, mu, F16, A.CHAIN)
    assert A.same_bytes(b.su.cpu().numpy(), A.record(b.u.cpu().float().numpy()), 384)
    a = torch.from_numpy(A.values(b.su.cpu().numpy(), 384)).half().double().numpy()
    dout = A.f64(b.dout)
    A.close("dw", b.dw, dout.T @ a, np.abs(dout).T @ np.abs(a), F16, 2 * (150 + 2))
    yv, hv = (A.values(c.cpu().numpy(), 384).astype(np.float64) for c in (b.sy, b.sh))
    want = A.back(ref, yv, hv, A.f64(b.dy), A.f64(b.du))
    for n, t in [("dx", b.dx), ("dh", b.dh), ("dgate", b.dgate), *b.vec.items()]:
        v, m = want[n]
        A.close(n, t, v, m, F16, A.CHAIN + 150)
    assert status_flags(b.status) == 0


def test_side_streams():
    """Two blocks on two side streams at once give what they give one after the other."""
    blocks = [Block(300, 512, 256, 10), Block(77, 1000, 72, 20)]
    for b in blocks:
        b.forward()
        b.backward()
    torch.cuda.synchronize()
    want = [b.outputs() for b in blocks]
    for t in [t for b in blocks for t in (b.y, b.u, b.dw, b.dx, b.dh, b.dgate)]:
        t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(4):
        for b, s in zip(blocks, streams):
            b.forward(s)
            b.backward(s)
    torch.cuda.synchronize()
    assert all(_same(b.outputs(), w) for b, w in zip(blocks, want))


def test_captured_and_replayed():
    """A captured block, replayed on new inputs, gives what eager calls give; two graphs that
    share one workspace are replayed one after the other."""
    blocks = [Block(260, 640, 320, 30), Block(90, 640, 136, 40)]
    shared = torch.empty(max(b.ws.numel() for b in blocks), dtype=torch.uint8, device=DEV)
    graphs = []
    for b in blocks:
        b.ws = shared
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.forward()
            b.backward()
        graphs.append(g)
    for seed in (1, 2):
        for b in blocks:
            for i, t in enumerate((b.x, b.h, b.dout, b.dy, b.du)):
                t.copy_(_rand(tuple(t.shape), 100 * seed + i))
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [b.outputs() for b in blocks]
        for b in blocks:
            b.forward()
            b.backward()
        torch.cuda.synchronize()
        assert all(_same(b.outputs(), w) for b, w in zip(blocks, got))


def test_many_calls_back_to_back():
    """Calls that follow one another without a wait: each waits for the one before (a chain whose
    every link reads what the last one wrote)."""
    rows, d = 64, 768
    x = _rand((rows, d), 1)
    w = _rand((d,), 2, 0.1) + 1
    bufs = [x.clone() for _ in range(2)]
    ck = torch.empty(rows, lz.ckpt_row_bytes(d), dtype=torch.uint8, device=DEV)
    one = [x.clone() for _ in range(2)]
    for chain, wait in ((bufs, False), (one, True)):
        for i in range(40):
            src, dst = chain[i % 2], chain[1 - i % 2]
            lz.zero_block_join(rows, d, x=src, u=dst, save_y=ck, pre_norm="rms", pre_w=w)
            if wait:
                torch.cuda.synchronize()
            lz.zero_ckpt_load_q8(rows, d, ck, src)
            if wait:
                torch.cuda.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(bufs[0], one[0]) and torch.equal(bufs[1], one[1])


def test_gradients_into_the_fused_step():
    """The block's gradients written straight into each rank's flat fp16 gradient list; the fused
    step over that list gives what the oracle's step gives for the same gradients."""
    nd, rows, d, o = 3, 120, 256, 136
    numels = [o * d, d, d, d]
    plan = lz.zero_plan_create(numels, nd, 2, 0)
    psi, psi_p, _, _ = lz.zero_plan_info(plan)
    off = lz.zero_plan_tensor_offsets(plan)
    grads = [torch.zeros(psi_p, dtype=F16, device=DEV) for _ in range(nd)]
    blocks = []
    for r in range(nd):
        g = grads[r]
        vec = {n: g[off[i]:off[i] + d] for i, n in ((1, "dpost_w"), (2, "dpre_w"), (3, "dpre_b"))}
        b = Block(rows, d, o, 50 + 20 * r, dw=g[off[0]:off[0] + o * d].view(o, d), dvec=vec)
        b.forward()
        b.backward()
        blocks.append(b)
    master, m, v = synth.state_warm(psi_p, seed=9)
    for poison in (False, True):
        if poison:    # an inf activation in one rank: its checkpoint makes the gradient NaN
            blocks[1].h[5, 7] = float("inf")
            blocks[1].forward()
            blocks[1].backward()
        ins = [t.to(DEV) for t in (master, m, v)]
        outs = [torch.empty_like(t) for t in ins]
        params = torch.zeros(psi_p, dtype=F16, device=DEV)
        st = status_word()
        lz.zero_step_fused(psi_p, nd, grads, *ins, *outs, params, HP, 1, st)
        lz.zero_step_commit(psi_p, *ins, *outs, params, st)
        torch.cuda.synchronize()
        g_np = [f16np(g) for g in grads]
        state = [f32np(t).copy() for t in (master, m, v)]
        skipped, *want, p16 = oracle.step(g_np, *state, ORC_HP, 1)
        flags = status_flags(st)
        assert skipped == poison
        if poison:
            assert flags & lz.ZERO_FLAG_OVERFLOW and flags & lz.ZERO_FLAG_SKIPPED
            assert np.array_equal(f32np(outs[0]), f32np(master))
        else:
            assert flags == 0
            for name, g, w in zip(("master", "m", "v"), outs, want):
                check_f32(name, f32np(g), w)
            check_f16("params", f16np(params), p16)


def test_accumulated_micro_batches():
    """Two micro-batches added into one gradient: the second call adds to the first's result."""
    t, o, i = 200, 192, 320
    dy, a = _rand((2 * t, o), 1, 0.05), _rand((2 * t, i), 2)
    ck = torch.empty(2 * t, lz.ckpt_row_bytes(i), dtype=torch.uint8, device=DEV)
    lz.zero_ckpt_save_q8(2 * t, i, a, ck)
    dw = torch.empty(o, i, dtype=F16, device=DEV)
    st = status_word()
    ws = torch.empty(max(16, lz.zero_ckpt_wgrad_q8_workspace(t, o, i)), dtype=torch.uint8,
                     device=DEV)
    first = None
    for k in range(2):
        lz.zero_ckpt_wgrad_q8(t, o, i, dy[k * t:(k + 1) * t], ck[k * t:(k + 1) * t], dw, st,
                              workspace=ws, accumulate=k > 0)
        if k == 0:
            first = A.f64(dw)
    av = torch.from_numpy(A.values(ck.cpu().numpy(), i)).half().double().numpy()[t:]
    d = A.f64(dy)[t:]
    A.close("dw", dw, first + d.T @ av, np.abs(first) + np.abs(d).T @ np.abs(av), F16,
            2 * (t + 2))


def test_offsets_beyond_32_bits():
    """Matrices and checkpoints of more than 4 GiB: the last rows are what a call on them alone
    gives."""
    rows, d, tail = 1_200_000, 2048, 700
    x = torch.zeros(rows, d, dtype=F16, device=DEV)
    x[-tail:] = _rand((tail, d), 1)
    rb = lz.ckpt_row_bytes(d)
    assert x.numel() * 2 > 1 << 32 and rows * rb > 1 << 31
    ck = torch.empty(rows, rb, dtype=torch.uint8, device=DEV)
    lz.zero_ckpt_save_q8(rows, d, x, ck)
    small = torch.empty(tail, rb, dtype=torch.uint8, device=DEV)
    lz.zero_ckpt_save_q8(tail, d, x[-tail:], small)
    assert torch.equal(ck[-tail:], small) and bool((ck[0, :d] == 128).all())
    out = torch.empty_like(x)
    lz.zero_ckpt_load_q8(rows, d, ck, out)
    back = torch.empty(tail, d, dtype=F16, device=DEV)
    lz.zero_ckpt_load_q8(tail, d, small, back)
    assert torch.equal(out[-tail:], back) and not bool(out[:-tail].any())
    w = _rand((d,), 2)
    lz.zero_block_join(rows, d, x=x, u=out, pre_norm="rms", pre_w=w)
    lz.zero_block_join(tail, d, x=x[-tail:], u=back, pre_norm="rms", pre_w=w)
    assert torch.equal(out[-tail:], back)
    dpw, spw = (torch.empty(d, dtype=F16, device=DEV) for _ in range(2))
    dx = torch.empty_like(x)
    ws = torch.empty(lz.zero_block_join_backward_workspace(rows, d, 0), dtype=torch.uint8,
                     device=DEV)
    kw = dict(has_branch=False, pre_norm="rms", pre_w=w, workspace=ws)
    lz.zero_block_join_backward(rows, d, y=x, du=out, dx=dx, dpre_w=dpw, **kw)
    sx = torch.empty(tail, d, dtype=F16, device=DEV)
    lz.zero_block_join_backward(tail, d, y=x[-tail:], du=back, dx=sx, dpre_w=spw, **kw)
    assert torch.equal(dx[-tail:], sx) and not bool(dx[:-tail].any())
    # the sums run in another order: two fp32 sums of tail terms, each rounded to fp16
    u64 = (A.f64(back) * A.f64(x[-tail:]) /
           np.sqrt((A.f64(x[-tail:]) ** 2).mean(1, keepdims=True) + 1e-5))
    A.close("dpre_w", dpw, u64.sum(0), np.abs(u64).sum(0), F16, A.CHAIN + rows)
    A.close("dpre_w", spw, u64.sum(0), np.abs(u64).sum(0), F16, A.CHAIN + tail)


def test_weight_gradient_beyond_32_bits():
    """Only the last stage of tokens is not zero: the long call adds exact zeros to the short one."""
    t, o, i, tail = 64 * 40_000, 1024, 128, 64
    dy = torch.zeros(t, o, dtype=F16, device=DEV)
    dy[-tail:] = _rand((tail, o), 1, 0.1)
    ck = torch.empty(t, lz.ckpt_row_bytes(i), dtype=torch.uint8, device=DEV)
    a = _rand((t // 100, i), 2).repeat(100, 1)
    lz.zero_ckpt_save_q8(t, i, a, ck)
    assert dy.numel() * 2 > 1 << 32
    got, want = (torch.empty(o, i, dtype=F16, device=DEV) for _ in range(2))
    st = status_word()
    for n, out in ((t, got), (tail, want)):
        ws = torch.empty(max(16, lz.zero_ckpt_wgrad_q8_workspace(n, o, i)), dtype=torch.uint8,
                         device=DEV)
        lz.zero_ckpt_wgrad_q8(n, o, i, dy[t - n:], ck[t - n:], out, st, workspace=ws)
    assert torch.equal(got, want) and status_flags(st) == 0

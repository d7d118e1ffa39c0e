"""The activation-side calls inside a zero_overlap_begin/end region: each waits for the region's calls
before it and reads what they wrote; what the calls after it write does not reach it."""
import pytest
import torch

from tests._gpu import DEV, HP, lz, require_gpu, status_flags, status_word
from zero_partitioned_optimizer_plan_b200 import synth

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


class Step:
    """A step over three buckets of rows x d values each. Behind each bucket's call: the parameters it
    wrote are kept in 8 bits, go through a boundary and its gradient, and are the input of a weight
    gradient."""

    def __init__(self, nd, rows, d, o):
        self.nd, self.rows, self.d, self.o, self.n = nd, rows, d, o, rows * d
        n = 3 * self.n
        self.state = [t.to(DEV) for t in synth.state_warm(n, seed=3)]
        self.grads = [synth.grad_f16(n, 1e-3, seed=4, rank=r, step=1).to(DEV) for r in range(nd)]
        self.w = torch.ones(d, dtype=F16, device=DEV)
        self.dout = torch.full((rows, o), 0.25, dtype=F16, device=DEV)
        self.ws = torch.empty(max(lz.zero_ckpt_wgrad_q8_workspace(rows, o, d),
                                  lz.zero_block_join_backward_workspace(rows, d)),
                              dtype=torch.uint8, device=DEV)

    def run(self, region):
        rows, d, n = self.rows, self.d, self.n
        out = [torch.zeros_like(t) for t in self.state]
        params = torch.zeros(3 * n, dtype=F16, device=DEV)
        st = status_word()
        made = []
        torch.cuda.synchronize()
        if region:
            lz.zero_overlap_begin(torch.cuda.current_stream())
        try:
            for k in range(3):
                lo, hi = k * n, (k + 1) * n
                lz.zero_step_fused(n, self.nd, [g[lo:hi] for g in self.grads],
                                   *[t[lo:hi] for t in self.state], *[t[lo:hi] for t in out],
                                   params[lo:hi], HP, 1, st)
                x = params[lo:hi].view(rows, d)
                ck = torch.empty(rows, lz.ckpt_row_bytes(d), dtype=torch.uint8, device=DEV)
                y, u, dx = (torch.empty(rows, d, dtype=F16, device=DEV) for _ in range(3))
                dw = torch.empty(self.o, d, dtype=F16, device=DEV)
                dv = torch.empty(d, dtype=F16, device=DEV)
                lz.zero_block_join(rows, d, x=x, h=x, y=y, u=u, save_y=ck, pre_norm="rms",
                                   pre_w=self.w)
                lz.zero_ckpt_wgrad_q8(rows, self.o, d, self.dout, ck, dw, st, workspace=self.ws)
                lz.zero_block_join_backward(rows, d, y_ckpt=ck, du=u, dx=dx, dpre_w=dv,
                                            pre_norm="rms", pre_w=self.w, workspace=self.ws)
                made += [ck, y, u, dw, dx, dv]
        finally:
            if region:
                lz.zero_overlap_end(torch.cuda.current_stream())
        copies = [t.clone() for t in (*out, params, *made)]     # ordinary work behind the region
        torch.cuda.synchronize()
        assert status_flags(st) == 0
        return copies


@pytest.mark.parametrize("nd,rows,d,o", [(8, 2048, 1024, 264), (2, 1000, 3001, 72)])
def test_inside_a_region(nd, rows, d, o):
    s = Step(nd, rows, d, o)
    want = s.run(False)
    for _ in range(5):
        got = s.run(True)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(got, want))
    assert bool(want[3].any()) and bool(want[-1].any())

"""Refusals of the activation-side calls: every host-detectable argument error returns its status
before anything is launched (no GPU needed: the addresses are never touched)."""
import pytest

from tests import _act as A
from zero_partitioned_optimizer_plan_b200 import build as zbuild

zbuild.build()
from zero_partitioned_optimizer_plan_b200 import libzero as lz  # noqa: E402

BASE = 1 << 40          # fake device addresses, 16 MiB apart
MB = 1 << 24
OK, EINVAL, EALIGN, ENOMEM = lz.ZERO_OK, lz.ZERO_EINVAL, lz.ZERO_EALIGN, lz.ZERO_ENOMEM


def at(k, off=0):
    return BASE + k * MB + off


def code_of(fn, *args, **kw):
    before = lz.zero_kernel_launches()
    try:
        fn(*args, **kw)
        code = OK
    except lz.ZeroError as e:
        code = e.code
    assert lz.zero_kernel_launches() == before
    return code


@pytest.mark.parametrize("cols", [1, 15, 16, 17, 127, 128, 129, 768, 1601, 2048, 16384])
def test_row_bytes(cols):
    assert lz.ckpt_row_bytes(cols) == A.row_bytes(cols)
    assert lz.ckpt_row_bytes(cols) % 32 == 0
    assert lz.ckpt_row_bytes(cols) >= cols + 4 * -(-cols // 128)


@pytest.mark.parametrize("fn", ["save", "load"])
@pytest.mark.parametrize("rows,cols,dtype,m,ck,code", [
    (4, 64, 0, 0, at(1), EINVAL),
    (4, 64, 0, at(0), 0, EINVAL),
    (4, 64, 3, at(0), at(1), EINVAL),
    (4, 64, -1, at(0), at(1), EINVAL),
    (4, 64, 0, (at(0), 63), at(1), EINVAL),
    (4, 1 << 31, 0, (at(0), 1 << 31), at(1), EINVAL),
    (1 << 60, 64, 0, at(0), at(1), EINVAL),
    (4, 64, 0, (at(0), 1 << 62), at(1), EINVAL),
    (4, 64, 0, at(0, 1), at(1), EALIGN),
    (4, 64, 2, at(0, 2), at(1), EALIGN),
    (4, 64, 0, at(0), at(1, 8), EALIGN),
    (4, 64, 0, at(0), at(0, 16), EINVAL),
    (4, 64, 2, (at(0), 512), at(0, 3 * 2048 + 240), EINVAL),
    (0, 64, 0, 0, 0, OK),
    (4, 0, 0, 0, 0, OK),
])
def test_checkpoint_rejects(fn, rows, cols, dtype, m, ck, code):
    if fn == "save":
        got = code_of(lz.zero_ckpt_save_q8, rows, cols, m, ck, dtype=dtype, stream=0)
    else:
        got = code_of(lz.zero_ckpt_load_q8, rows, cols, ck, m, dtype=dtype, stream=0)
    assert got == code


def _wgrad(t=64, o=32, i=48, dy=at(0), ck=at(1), dw=at(2), st=at(3), ws=at(4), wsb=1 << 23,
           dtype=0, acc=False):
    return code_of(lz.zero_ckpt_wgrad_q8, t, o, i, dy, ck, dw, st, workspace=ws,
                   workspace_bytes=wsb, dtype=dtype, accumulate=acc, stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), EINVAL),
    (dict(dtype=7), EINVAL),
    (dict(st=0), EINVAL),
    (dict(dy=0), EINVAL),
    (dict(ck=0), EINVAL),
    (dict(dw=0), EINVAL),
    (dict(dy=(at(0), 31)), EINVAL),
    (dict(dw=(at(2), 47)), EINVAL),
    (dict(t=1 << 31), EINVAL),
    (dict(o=1 << 30, dy=(at(0), 1 << 30)), EINVAL),
    (dict(i=1 << 30, dw=(at(2), 1 << 30)), EINVAL),
    (dict(dy=at(0, 1)), EALIGN),
    (dict(dw=at(2, 1)), EALIGN),
    (dict(ck=at(1, 8)), EALIGN),
    (dict(st=at(3, 2)), EALIGN),
    (dict(dw=at(0, 64)), EINVAL),
    (dict(dw=at(1, 64)), EINVAL),
    (dict(st=at(2, 64)), EINVAL),
    (dict(o=0), OK),
    (dict(i=0), OK),
    (dict(t=0, dy=0, ck=0, acc=True), OK),
])
def test_wgrad_rejects(kw, code):
    assert _wgrad(**kw) == code


def test_wgrad_workspace():
    n = lz.zero_ckpt_wgrad_q8_workspace(1 << 16, 256, 256)
    assert n % 16 == 0
    if n:                                  # a long sum into few outputs is split
        kw = dict(t=1 << 16, o=256, i=256, dy=at(0), ck=at(20), dw=at(40))
        assert _wgrad(**kw, ws=at(60), wsb=n - 1) == ENOMEM
        assert _wgrad(**kw, ws=0, wsb=n) == EINVAL
        assert _wgrad(**kw, ws=at(60, 8), wsb=n) == EALIGN
        assert _wgrad(**kw, ws=at(40, 16), wsb=n) == EINVAL
    with pytest.raises(lz.ZeroError):
        lz.zero_ckpt_wgrad_q8_workspace(1 << 31, 4, 4)


def _join(rows=8, cols=64, dtype=0, **kw):
    args = dict(x=at(0), h=at(1), y=at(2), u=at(3), post_norm="rms", pre_norm="layer",
                post_w=at(4), pre_w=at(5), pre_b=at(6))
    args.update(kw)
    return code_of(lz.zero_block_join, rows, cols, dtype=dtype, stream=0, **args)


BAD_DESC = [
    (dict(dtype=5), EINVAL),
    (dict(post_norm=3), EINVAL),
    (dict(pre_norm=-1), EINVAL),
    (dict(post_eps=-1.0), EINVAL),
    (dict(pre_eps=float("nan")), EINVAL),
    (dict(residual_scale=float("inf")), EINVAL),
    (dict(branch_scale=float("nan")), EINVAL),
    (dict(cols=16385), EINVAL),
    (dict(gate=at(9)), EINVAL),
    (dict(gate_rows=4), EINVAL),
    (dict(gate=(at(9), 63), gate_rows=4), EINVAL),
    (dict(gate=at(9, 1), gate_rows=4), EALIGN),
    (dict(post_norm="none"), EINVAL),
    (dict(pre_b=at(6, 1)), EALIGN),
]


@pytest.mark.parametrize("kw,code", BAD_DESC + [
    (dict(x=0), EINVAL),
    (dict(x_ckpt=at(7)), EINVAL),
    (dict(h_ckpt=at(7)), EINVAL),
    (dict(h=0), EINVAL),
    (dict(h=0, post_norm="none", post_w=0, gate=at(9), gate_rows=8), EINVAL),
    (dict(y=0, u=0), EINVAL),
    (dict(pre_norm="none", pre_w=0, pre_b=0), EINVAL),
    (dict(h=0, h_ckpt=at(7), save_h=at(8)), EINVAL),
    (dict(save_y=at(8, 4)), EALIGN),
    (dict(x=(at(0), 63)), EINVAL),
    (dict(u=(at(3), 1 << 62)), EINVAL),
    (dict(u=at(3, 1)), EALIGN),
    (dict(u=at(2)), EINVAL),
    (dict(u=at(0)), EINVAL),
    (dict(u=at(1)), EINVAL),
    (dict(y=at(0, 2)), EINVAL),
    (dict(y=(at(0), 65)), EINVAL),
    (dict(y=at(1)), EINVAL),
    (dict(save_y=at(2, 16)), EINVAL),
    (dict(y=at(4)), EINVAL),
    (dict(x=(at(0), 256), u=(at(0, 120), 256)), EINVAL),
    (dict(rows=0), OK),
    (dict(cols=0), OK),
])
def test_join_rejects(kw, code):
    assert _join(**kw) == code


def _back(rows=8, cols=64, dtype=0, **kw):
    args = dict(y=at(0), h=at(1), dy=at(2), du=at(3), dx=at(4), dh=at(5), dpost_w=at(6),
                dpre_w=at(7), dpre_b=at(8), post_norm="rms", pre_norm="layer", post_w=at(10),
                pre_w=at(11), pre_b=at(12), workspace=at(13), workspace_bytes=1 << 23)
    args.update(kw)
    return code_of(lz.zero_block_join_backward, rows, cols, dtype=dtype, stream=0, **args)


@pytest.mark.parametrize("kw,code", [c for c in BAD_DESC if "gate" not in c[0]] + [
    (dict(y=0), EINVAL),
    (dict(y_ckpt=at(14)), EINVAL),
    (dict(h=0), EINVAL),
    (dict(h_ckpt=at(14)), EINVAL),
    (dict(has_branch=False), EINVAL),
    (dict(dx=0, dh=0, dpost_w=0, dpre_w=0, dpre_b=0), EINVAL),
    (dict(dgate=at(14)), EINVAL),
    (dict(dpost_b=at(14), post_norm="none", post_w=0, dpost_w=0), EINVAL),
    (dict(pre_norm="none", pre_w=0, pre_b=0, dpre_w=0, dpre_b=0), EINVAL),
    (dict(accumulate=4), EINVAL),
    (dict(workspace=0), EINVAL),
    (dict(workspace_bytes=0), ENOMEM),
    (dict(workspace=at(13, 8)), EALIGN),
    (dict(workspace=at(4)), EINVAL),
    (dict(dx=at(3)), EINVAL),
    (dict(dx=at(0)), EINVAL),
    (dict(dx=(at(2), 80)), EINVAL),
    (dict(dh=at(2)), EINVAL),
    (dict(dh=at(4)), EINVAL),
    (dict(dpre_w=at(11)), EINVAL),
    (dict(dpre_w=at(8)), EINVAL),
    (dict(dpre_w=at(7, 1)), EALIGN),
    (dict(cols=0), OK),
])
def test_join_backward_rejects(kw, code):
    assert _back(**kw) == code


def test_join_backward_workspace_sizes():
    for rows, cols, gate_rows in [(1, 1, 0), (8, 64, 8), (1 << 20, 16384, 1), (1000, 768, 7)]:
        n = lz.zero_block_join_backward_workspace(rows, cols, gate_rows)
        assert n > 0 and n % 16 == 0
        assert n == lz.zero_block_join_backward_workspace(rows, cols, gate_rows)
    with pytest.raises(lz.ZeroError):
        lz.zero_block_join_backward_workspace(8, 16385, 0)


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.float16)
    ck = torch.zeros(4, lz.ckpt_row_bytes(64), dtype=torch.uint8)
    for bad in (lambda: lz.zero_ckpt_save_q8(5, 64, x, ck, stream=0),
                lambda: lz.zero_ckpt_save_q8(4, 64, x.t(), ck, stream=0),
                lambda: lz.zero_ckpt_save_q8(4, 64, x.double(), ck, stream=0),
                lambda: lz.zero_ckpt_save_q8(4, 64, x, ck[:3], stream=0),
                lambda: lz.zero_ckpt_save_q8(4, 64, x, ck.float(), stream=0),
                lambda: lz.zero_ckpt_save_q8(4, 64, at(0), ck, stream=0),
                lambda: lz.zero_ckpt_save_q8(4, 64, x, ck, stream=0),           # host memory
                lambda: lz.zero_ckpt_load_q8(4, 64, ck, at(0), dtype=0, stream=0),
                lambda: lz.zero_block_join(4, 64, x=x, h=x.float(), y=x, stream=0),
                lambda: lz.zero_block_join(4, 64, x=x, u=x.clone(), pre_norm="rms",
                                           pre_w=x[0, :63].clone(), stream=0),
                lambda: lz.zero_block_join_backward(4, 64, dy=x, dx=x.clone(), gate_rows=2,
                                                    gate=x.clone(), stream=0)):
        with pytest.raises(TypeError):
            bad()


HUGE = (1 << 64) - 1


@pytest.mark.parametrize("gate_rows", [9, HUGE, HUGE - 6])
def test_gate_of_more_rows_than_there_are(gate_rows):
    """One gate row for every row, however large gate_rows is: it is checked like any other."""
    kw = dict(gate_rows=gate_rows)
    assert _join(gate=at(9, 1), **kw) == EALIGN
    assert _join(gate=(at(9), 63), **kw) == EINVAL
    assert _join(gate=at(2, 64), **kw) == EINVAL            # inside y
    back = dict(kw, gate=at(15))
    assert _back(dgate=at(14, 1), **back) == EALIGN
    assert _back(dgate=(at(14), 63), **back) == EINVAL
    assert _back(dgate=at(15), **back) == EINVAL            # the gate itself
    assert _back(dgate=at(4, 128), **back) == EINVAL        # inside dx


class OnDevice:
    """What the binding reads of a device tensor. All lie at one address, so that the library refuses
    every call that the binding lets through (its operands overlap)."""

    def __init__(self, shape, dtype, device=1):
        self.shape, self.dtype, self.index = shape, dtype, device
        self.is_cuda = True
        self.nbytes = self.numel() * self.element_size()

    def stride(self):
        return tuple(self.numel(self.shape[i + 1:]) for i in range(len(self.shape)))

    def numel(self, shape=None):
        n = 1
        for s in self.shape if shape is None else shape:
            n *= s
        return n

    def data_ptr(self):
        return at(0)

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index


def test_binding_refuses_workspace_and_status_in_host_memory():
    torch = pytest.importorskip("torch")
    host, word = torch.zeros(64, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    kw = dict(dtype=0, stream=0)
    a = at(0)
    for bad in (lambda: lz.zero_ckpt_wgrad_q8(1 << 16, 256, 256, a, a, a, a, workspace=host, **kw),
                lambda: lz.zero_ckpt_wgrad_q8(64, 256, 256, a, a, a, word, **kw),
                lambda: lz.zero_ckpt_wgrad_q8(64, 256, 256, a, a, a, a, workspace=a, **kw),  # size?
                lambda: lz.zero_block_join_backward(4, 64, dy=a, du=a, y=a, dx=a, dpre_w=a,
                                                    pre_norm="rms", workspace=host, **kw)):
        before = lz.zero_kernel_launches()
        with pytest.raises(TypeError):
            bad()
        assert lz.zero_kernel_launches() == before


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """The calls run on the current device: a tensor of another one is refused, whichever operand it
    is."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(lz, "_several_devices", True)
    monkeypatch.setattr(lz, "_current_device", lambda: 1)
    f16, u8 = torch.float16, torch.uint8
    m, rec = (4, 64), (4, lz.ckpt_row_bytes(64))
    shapes = dict(x=(m, f16), h=(m, f16), y=(m, f16), u=(m, f16), ck=(rec, u8), w=((64,), f16),
                  gate=(m, f16), dw=((64, 64), f16), ws=((1 << 23,), u8),
                  status=((1,), torch.int32))

    def calls(o):
        norms = dict(pre_norm="rms", post_norm="rms", pre_w=o["w"], gate=o["gate"], gate_rows=1,
                     stream=0)
        yield "x ck", lambda: lz.zero_ckpt_save_q8(4, 64, o["x"], o["ck"], stream=0)
        yield "x ck", lambda: lz.zero_ckpt_load_q8(4, 64, o["ck"], o["x"], stream=0)
        yield "x h y u ck w gate", lambda: lz.zero_block_join(
            4, 64, x=o["x"], h=o["h"], y=o["y"], u=o["u"], save_y=o["ck"], **norms)
        yield "x h y u w gate ws", lambda: lz.zero_block_join_backward(
            4, 64, y=o["y"], h=o["h"], dy=o["x"], du=o["u"], dx=at(0), dpre_b=at(0),
            workspace=o["ws"], **norms)
        yield "x ck dw ws status", lambda: lz.zero_ckpt_wgrad_q8(
            4, 64, 64, o["x"], o["ck"], o["dw"], o["status"], workspace=o["ws"], stream=0)

    here = {k: OnDevice(*v) for k, v in shapes.items()}
    for _, call in calls(here):
        with pytest.raises(lz.ZeroError):
            call()
    for other in shapes:
        for names, call in calls(dict(here, **{other: OnDevice(*shapes[other], device=0)})):
            with pytest.raises(TypeError if other in names.split() else lz.ZeroError):
                call()


def test_bf16_gradients_are_not_taken_for_fp16():
    """The steps and buckets read fp16: a bf16 weight gradient is refused (n = 0 launches nothing)."""
    torch = pytest.importorskip("torch")
    g, f = torch.zeros(8, dtype=torch.bfloat16), torch.zeros(8)
    p, st = torch.zeros(8, dtype=torch.float16), torch.zeros(1, dtype=torch.int32)
    args = (f, f, f, f, f, f, p, lz.AdamHP(), 1, st)
    lz.zero_step_fused(0, 1, [p], *args, stream=0)
    lz.zero_step_fused(0, 1, [p.view(torch.int16)], *args, stream=0)
    for bad in (lambda: lz.zero_step_fused(0, 1, [g], *args, stream=0),
                lambda: lz.zero_step_fused(0, 2, [p, g], *args, stream=0),
                lambda: lz.zero_quantize_q8(0, g, torch.zeros(0, dtype=torch.uint8), stream=0)):
        with pytest.raises(TypeError):
            bad()

"""The activation-side operators of libzero as measured cases: 8-bit activation checkpoints, the
block boundary (norm after a block, gate, residual scale, norm before the next one) with its
gradient, and the weight gradient of a linear layer from an 8-bit checkpoint.

Each case is given in two forms over the same prepared inputs: elementary torch operations in 32
bits, and the library's own calls (`own`). `exact` states the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 128                                # columns that share one scale
DEV = "cuda"


def listed():
    return [
        # the residual stream of one token kept and read back: launch latency
        dict(name="ckpt 1x2048 f16", op="ckpt", rows=1, cols=2048, pad=0, type="f16"),
        # a layer's input of the 1.3B list (d = 2048), 8 sequences of 2048 tokens
        dict(name="ckpt 16384x2048 f16", op="ckpt", rows=16384, cols=2048, pad=0, type="f16"),
        # a ragged batch in bf16, taken from the first columns of a wider buffer
        dict(name="ckpt 4099x1601 bf16", op="ckpt", rows=4099, cols=1601, pad=31, type="bf16"),
        # one token through a sandwich-norm boundary with a layer scale: a decoding step
        dict(name="join 1x2048 f16", op="join", rows=1, cols=2048, type="f16", post="rms",
             pre="rms", bias=False, gate_rows=1),
        # GPT-2 small's boundary (x + h, then LayerNorm), 8 sequences of 1024 tokens
        dict(name="join 8192x768 f16", op="join", rows=8192, cols=768, type="f16", post="none",
             pre="layer", bias=True, gate_rows=0),
        # the same of the 1.3B list in training: forward with checkpoints, backward from them
        dict(name="train 16384x2048 f16", op="train", rows=16384, cols=2048, type="f16",
             post="none", pre="layer", bias=True, gate_rows=0, ckpt=True),
        # sandwich RMS norms with one gate per sequence of 1024 tokens, wide rows, bf16
        dict(name="train 8192x4096 bf16", op="train", rows=8192, cols=4096, type="bf16",
             post="rms", pre="rms", bias=False, gate_rows=1024, ckpt=True),
        # 32-bit activations, odd sizes, LayerNorm on both sides, a learned layer scale
        dict(name="train 1531x1001 f32", op="train", rows=1531, cols=1001, type="f32",
             post="layer", pre="layer", bias=True, gate_rows=1531, ckpt=False),
        # GPT-2 small's attention projection over one short micro-batch: few output tiles
        dict(name="wgrad 1024x768x768 f16", op="wgrad", tokens=1024, out=768, inp=768, type="f16"),
        # GPT-2 small's qkv over 16 sequences of 1024 tokens: a long sum into few tiles
        dict(name="wgrad 16384x2304x768 f16", op="wgrad", tokens=16384, out=2304, inp=768,
             type="f16"),
        # the 1.3B list's first MLP matrix over 8 sequences of 2048 tokens: the largest
        dict(name="wgrad 16384x8192x2048 f16", op="wgrad", tokens=16384, out=8192, inp=2048,
             type="f16"),
        # a ragged batch and odd feature counts in bf16
        dict(name="wgrad 5003x1537x1100 bf16", op="wgrad", tokens=5003, out=1537, inp=1100,
             type="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ckpt", "join", "train", "wgrad"])
    if op == "wgrad":
        while True:
            t, o, i = _log(rng, 1, 16384), _log(rng, 8, 8192), _log(rng, 8, 8192)
            if rng.random() < 0.6:                     # most layers are a multiple of 64 wide
                o, i = -(-o // 64) * 64, -(-i // 64) * 64
            if t * o * i <= 16384 * 8192 * 2048:
                return dict(op=op, tokens=t, out=o, inp=i, type=rng.choice(["f16", "bf16"]))
    while True:
        rows, cols = _log(rng, 1, 32768), _log(rng, 64, 16384)
        if rng.random() < 0.6:
            cols = -(-cols // 64) * 64
        if rows * cols <= 16384 * 2048:
            break
    if op == "ckpt":
        return dict(op=op, rows=rows, cols=cols, pad=rng.choice([0, 0, 5, 64]),
                    type=rng.choice(["f16", "f16", "bf16", "f32"]))
    post = rng.choice(["none", "rms", "layer"])
    pre = rng.choice(["rms", "layer"])
    gate = rng.choice([0, rows, _log(rng, 1, rows)])
    kind = rng.choice(["f16", "f16", "bf16", "f32"])
    case = dict(op=op, rows=rows, cols=cols, type=kind, post=post, pre=pre,
                bias=rng.random() < 0.5, gate_rows=gate)
    if op == "train":
        # 32-bit boundaries keep their activations whole: 8 bits are for 16-bit training
        case["ckpt"] = kind != "f32" and rng.random() < 0.8
    return case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _row_bytes(cols):
    """Bytes of one checkpoint row: the codes padded to 16, a scale per block, padded to 32."""
    return -(-(-(-cols // 16) * 16 + 4 * -(-cols // BLOCK)) // 32) * 32


def _randn(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _acts(rows, cols, gen, dtype, pad=0):
    """Activations: unit normal with a few outlier columns, as residual streams have."""
    x = torch.randn((rows, cols + pad), generator=gen, device=DEV)
    hot = torch.randperm(cols, generator=gen, device=DEV)[:max(1, cols // 256)]
    x[:, hot] *= 12.0
    return x.to(dtype)[:, :cols]


def _quant(x):
    """(q, scale per block) of fp32 x [rows, cols]; q as fp32 integers, padded to whole blocks."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    amax = v.abs().amax(2, keepdim=True)
    scale = amax / amax.new_full((1, 1, 1), 127.0)     # a true division, also on the GPU
    bad = ~torch.isfinite(amax)
    q = torch.where((scale == 0) | bad, torch.zeros_like(v), torch.round(v / scale))
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    return q.clamp(-127, 127), scale


def _dequant(q, scale, cols):
    return (q * scale).view(q.shape[0], -1)[:, :cols]


def _pack(x):
    """The checkpoint rows of x, as bytes."""
    rows, cols = x.shape
    q, scale = _quant(x.float())
    c16, nb = -(-cols // 16) * 16, scale.shape[1]
    rec = torch.zeros((rows, _row_bytes(cols)), dtype=torch.uint8, device=x.device)
    rec[:, :c16] = 128
    rec[:, :cols] = (q.view(rows, -1)[:, :cols] + 128).to(torch.uint8)
    rec[:, c16:c16 + 4 * nb] = scale.view(rows, nb).contiguous().view(torch.uint8)
    return rec


def _unpack(rec, cols):
    """fp32 values that checkpoint rows stand for."""
    rows, c16, nb = rec.shape[0], -(-cols // 16) * 16, -(-cols // BLOCK)
    q = rec[:, :cols].float() - 128.0
    scale = rec[:, c16:c16 + 4 * nb].contiguous().view(torch.float32)
    return q * scale.repeat_interleave(BLOCK, 1)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 17)
    T = TYPES[case["type"]]
    s = dict(case=case)
    if case["op"] == "ckpt":
        rows, cols = case["rows"], case["cols"]
        s["x"] = _acts(rows, cols, gen, T, case["pad"])
        s["ckpt"] = torch.empty((rows, _row_bytes(cols)), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty((rows, cols), dtype=T, device=DEV)
        return s
    if case["op"] == "wgrad":
        t, o, i = case["tokens"], case["out"], case["inp"]
        s["dy"] = _randn((t, o), gen, 1e-2, T)
        s["ckpt"] = _pack(_acts(t, i, gen, T))
        s["dw"] = torch.empty((o, i), dtype=T, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    rows, cols, g = case["rows"], case["cols"], case["gate_rows"]
    s["x"], s["h"] = _acts(rows, cols, gen, T), _randn((rows, cols), gen, 0.5, T)
    s["y"], s["u"] = (torch.empty((rows, cols), dtype=T, device=DEV) for _ in range(2))

    def weight(std, mean, there=True):
        return (torch.randn(cols, generator=gen, device=DEV) * std + mean).to(T) if there else None

    s["pre_w"], s["pre_b"] = weight(0.1, 1.0), weight(0.1, 0.0, case["bias"])
    s["post_w"] = weight(0.1, 0.8, case["post"] != "none")
    s["post_b"] = weight(0.1, 0.0, case["post"] != "none" and case["bias"])
    s["gate"] = _randn((-(-rows // g), cols), gen, 0.4, T) if g else None
    s["rs"], s["bs"] = (1.0, 1.0) if case["post"] == "none" else (0.9, 0.7)
    if case["op"] == "train":
        s["dy"], s["du"] = _randn((rows, cols), gen, 1e-2, T), _randn((rows, cols), gen, 1e-2, T)
        if case["ckpt"]:
            for k in ("save_y", "save_h"):
                s[k] = torch.empty((rows, _row_bytes(cols)), dtype=torch.uint8, device=DEV)
        s["dx"], s["dh"] = torch.empty_like(s["dy"]), torch.empty_like(s["dy"])
        for k in ("pre_w", "pre_b", "post_w", "post_b", "gate"):
            s["d" + k] = None if s[k] is None else torch.empty_like(s[k])
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
EPS = 1e-5


def _norm(kind, z, w, b):
    """(normalised, its unit part, 1/deviation) of fp32 rows z."""
    if kind == "none":
        return z, z, None
    c = z - z.mean(1, keepdim=True) if kind == "layer" else z
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    n = c * r
    out = n * w if w is not None else n
    return (out + b if b is not None else out), n, r


def _norm_back(kind, n, r, g):
    """Gradient of the norm's input from the gradient g of its unit part n."""
    if kind == "none":
        return g
    d = g - n * (g * n).mean(1, keepdim=True)
    return r * (d - g.mean(1, keepdim=True) if kind == "layer" else d)


def _plain(s):
    case = s["case"]
    T = TYPES[case["type"]]
    if case["op"] == "ckpt":
        q, scale = _quant(s["x"].float())
        return dict(out=_dequant(q, scale, case["cols"]).to(T))
    if case["op"] == "wgrad":
        return dict(dw=(s["dy"].float().t() @ _unpack(s["ckpt"], case["inp"])).to(T))
    rows, g = case["rows"], case["gate_rows"]
    f = {k: None if s[k] is None else s[k].float()
         for k in ("x", "h", "pre_w", "pre_b", "post_w", "post_b", "gate")}
    gate = f["gate"].repeat_interleave(g, 0)[:rows] if g else 1.0
    hn, _, _ = _norm(case["post"], f["h"], f["post_w"], f["post_b"])
    y = s["rs"] * f["x"] + s["bs"] * gate * hn
    u, _, _ = _norm(case["pre"], y, f["pre_w"], f["pre_b"])
    out = dict(y=y.to(T), u=u.to(T))
    if case["op"] == "join":
        return out
    ys, hs = out["y"].float(), f["h"]
    if case["ckpt"]:
        ys, hs = (_dequant(*_quant(v), case["cols"]) for v in (ys, hs))
    _, yn, yr = _norm(case["pre"], ys, None, None)
    hn, hu, hr = _norm(case["post"], hs, f["post_w"], f["post_b"])
    du = s["du"].float()
    gy = s["dy"].float() + _norm_back(case["pre"], yn, yr, du * f["pre_w"])
    t = s["bs"] * gate * gy
    gt = t * f["post_w"] if f["post_w"] is not None else t
    out["dx"] = (s["rs"] * gy).to(T)
    out["dh"] = _norm_back(case["post"], hu, hr, gt).to(T)
    out["dpre_w"] = (du * yn).sum(0).to(T)
    if f["pre_b"] is not None:
        out["dpre_b"] = du.sum(0).to(T)
    if f["post_w"] is not None:
        out["dpost_w"] = (t * hu).sum(0).to(T)
    if f["post_b"] is not None:
        out["dpost_b"] = t.sum(0).to(T)
    if g:
        group = torch.arange(rows, device=du.device) // g
        dgate = torch.zeros_like(f["gate"])
        out["dgate"] = dgate.index_add_(0, group, s["bs"] * gy * hn).to(T)
    return out


def _own(s):
    from zero_partitioned_optimizer_plan_b200 import libzero as lz
    case = s["case"]
    if case["op"] == "ckpt":
        rows, cols = case["rows"], case["cols"]
        lz.zero_ckpt_save_q8(rows, cols, s["x"], s["ckpt"])
        lz.zero_ckpt_load_q8(rows, cols, s["ckpt"], s["out"])
        return dict(out=s["out"])
    if case["op"] == "wgrad":
        t, o, i = case["tokens"], case["out"], case["inp"]
        if "ws" not in s:
            n = lz.zero_ckpt_wgrad_q8_workspace(t, o, i)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
        lz.zero_ckpt_wgrad_q8(t, o, i, s["dy"], s["ckpt"], s["dw"], s["status"],
                              workspace=s["ws"])
        return dict(dw=s["dw"])
    rows, cols = case["rows"], case["cols"]
    kinds = dict(post_norm=case["post"], pre_norm=case["pre"], post_eps=EPS, pre_eps=EPS,
                 residual_scale=s["rs"], branch_scale=s["bs"], gate=s["gate"],
                 gate_rows=case["gate_rows"], post_w=s["post_w"], pre_w=s["pre_w"],
                 post_b=s["post_b"], pre_b=s["pre_b"])
    train = case["op"] == "train"
    saves = dict(save_y=s["save_y"], save_h=s["save_h"]) if train and case["ckpt"] else {}
    lz.zero_block_join(rows, cols, x=s["x"], h=s["h"], y=s["y"], u=s["u"], **saves, **kinds)
    out = dict(y=s["y"], u=s["u"])
    if not train:
        return out
    grads = {k: s[k] for k in ("dpre_w", "dpre_b", "dpost_w", "dpost_b", "dgate")
             if s[k] is not None}
    saved = dict(y_ckpt=s["save_y"], h_ckpt=s["save_h"]) if case["ckpt"] else \
        dict(y=s["y"], h=s["h"])
    if "ws" not in s:
        n = lz.zero_block_join_backward_workspace(rows, cols, case["gate_rows"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    lz.zero_block_join_backward(rows, cols, dy=s["dy"], du=s["du"], dx=s["dx"], dh=s["dh"],
                                workspace=s["ws"], **saved, **grads, **kinds)
    return dict(out, dx=s["dx"], dh=s["dh"], **grads)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    es = 4 if case["type"] == "f32" else 2
    if case["op"] == "ckpt":         # x in, the checkpoint out and in again, the values out
        n = case["rows"] * case["cols"]
        return dict(bytes=2 * es * n + 2 * case["rows"] * _row_bytes(case["cols"]), flops=4 * n)
    if case["op"] == "wgrad":
        t, o, i = case["tokens"], case["out"], case["inp"]
        return dict(bytes=es * t * o + t * _row_bytes(i) + es * o * i, flops=2 * t * o * i)
    rows, cols, g = case["rows"], case["cols"], case["gate_rows"]
    n = rows * cols
    vecs = 1 + case["bias"] + (case["post"] != "none") * (1 + case["bias"]) + \
        (-(-rows // g) if g else 0)
    b, f = 4 * es * n + vecs * cols * es, 15 * n          # x, h, y, u and the vectors
    if case["op"] == "train":
        # the saved y and h: written by the forward call as checkpoints and read by the
        # backward call, or read whole; dy, du, dx, dh; the vectors and their gradients
        saved = 4 * rows * _row_bytes(cols) if case["ckpt"] else 2 * es * n
        b += saved + 4 * es * n + 2 * vecs * cols * es
        f += 40 * n
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def _values64(x, T):
    """What the checkpoint of x (float64 [rows, cols] of values of T) stands for: per 128 columns
    scale = fl32(max/127), q = the integer nearest fl32(x/scale)."""
    parts = []
    for lo in range(0, x.shape[1], BLOCK):
        v = x[:, lo:lo + BLOCK]
        top = v.abs().max(1, keepdim=True).values
        scale = (top / torch.full_like(top, 127.0)).float().double()
        q = torch.round((v / torch.where(scale > 0, scale, torch.ones_like(scale))).float())
        parts.append(torch.clamp(q.double(), -127, 127) * scale)
    return torch.cat(parts, 1)


def _norm64(kind, z, w, b):
    if kind == "none":
        return z
    if kind == "layer":
        v, m = torch.var_mean(z, dim=1, unbiased=False, keepdim=True)
        z = (z - m) / torch.sqrt(v + EPS)
    else:
        z = z / torch.sqrt(z.square().sum(1, keepdim=True) / z.shape[1] + EPS)
    z = z if w is None else z * w[None]
    return z if b is None else z + b[None]


def exact(case, seed):
    s = prepare(case, seed)
    T = TYPES[case["type"]]
    if case["op"] == "ckpt":
        return dict(out=_values64(s["x"].double(), T))
    if case["op"] == "wgrad":
        rec, i = s["ckpt"], case["inp"]
        codes = rec[:, :i].to(torch.float64) - 128
        at = -(-i // 16) * 16
        scales = rec[:, at:at + 4 * -(-i // BLOCK)].contiguous().view(torch.float32).double()
        a = codes * scales[:, torch.arange(i, device=rec.device) // BLOCK]
        return dict(dw=torch.mm(s["dy"].double().T, a))
    rows, g = case["rows"], case["gate_rows"]
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "h", "gate", "pre_w", "pre_b",
                                                        "post_w", "post_b") if s[k] is not None}
    get = leaf.get

    def boundary(x, h):
        z = s["bs"] * _norm64(case["post"], h, get("post_w"), get("post_b"))
        if g:
            z = z * leaf["gate"][torch.arange(rows, device=z.device) // g]
        return s["rs"] * x + z

    y = boundary(leaf["x"], leaf["h"])
    u = _norm64(case["pre"], y, get("pre_w"), get("pre_b"))
    out = dict(y=y.detach(), u=u.detach())
    if case["op"] == "join":
        return out
    # the backward pass takes y and h as they were kept: y rounded to its type, both in 8 bits
    ys, hs = y.detach().to(T).double(), s["h"].double()
    if case["ckpt"]:
        ys, hs = _values64(ys, T), _values64(hs, T)
    hs = hs.requires_grad_()
    yb = boundary(leaf["x"], hs)
    at = (ys - yb).detach() + yb             # the value kept, with the boundary's derivative
    ub = _norm64(case["pre"], at, get("pre_w"), get("pre_b"))
    total = (at * s["dy"].double()).sum() + (ub * s["du"].double()).sum()
    names = [k for k in ("gate", "pre_w", "pre_b", "post_w", "post_b") if k in leaf]
    got = torch.autograd.grad(total, [leaf["x"], hs] + [leaf[k] for k in names])
    out.update(dx=got[0], dh=got[1], **{"d" + k: v for k, v in zip(names, got[2:])})
    return out

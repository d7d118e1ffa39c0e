"""Plain 64-bit forms of the activation-side operators and their error bounds. Test
infrastructure only: numpy, no code of the library."""
import numpy as np
import torch

U = 2.0 ** -24                       # half a step of binary32
# A row's sum of up to 16384 values runs in chains of at most 128 additions per thread, then a
# tree: at most 160 roundings on any path. A statistic, the two means of a norm's gradient and
# the next norm's three chain at most three such sums after one another; the elementwise
# operations between them add fewer than 30.
ROW = 160
CHAIN = 3 * ROW + 32

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# below the smallest normal a half step is absolute
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}


def f64(x):
    return None if x is None else x.detach().cpu().to(torch.float64).numpy()


def row_bytes(cols):
    return -(-(-(-cols // 16) * 16 + 4 * -(-cols // 128)) // 32) * 32


def quant(x):
    """(q int, scale fp32) of a float32 array, blocks of 128 columns."""
    rows, cols = x.shape
    nb = -(-cols // 128)
    v = np.zeros((rows, nb * 128), np.float32)
    v[:, :cols] = x
    v = v.reshape(rows, nb, 128)
    with np.errstate(all="ignore"):
        amax = np.abs(v).max(2)
        amax[np.isnan(v).any(2)] = np.nan
        scale = (amax / np.float32(127)).astype(np.float32)
        q = np.rint((v / scale[:, :, None]).astype(np.float32))
    bad = ~np.isfinite(amax)
    scale[bad] = np.nan
    q[bad | (scale == 0)] = 0
    return np.clip(q, -127, 127).astype(np.int32).reshape(rows, -1)[:, :cols], scale


def record(x):
    """The checkpoint bytes of a float32 array."""
    rows, cols = x.shape
    q, scale = quant(x)
    c16 = -(-cols // 16) * 16
    rec = np.zeros((rows, row_bytes(cols)), np.uint8)
    rec[:, :c16] = 128
    rec[:, :cols] = (q + 128).astype(np.uint8)
    rec[:, c16:c16 + 4 * scale.shape[1]] = np.ascontiguousarray(scale).view(np.uint8)
    return rec


def same_bytes(got, want, cols):
    """Equal records; a NaN scale may have any payload."""
    c16, nb = -(-cols // 16) * 16, -(-cols // 128)
    gs = np.ascontiguousarray(got[:, c16:c16 + 4 * nb]).view(np.float32)
    ws = np.ascontiguousarray(want[:, c16:c16 + 4 * nb]).view(np.float32)
    nan = np.isnan(ws)
    return (np.array_equal(got[:, :c16], want[:, :c16]) and np.array_equal(np.isnan(gs), nan)
            and np.array_equal(gs[~nan].view(np.uint32), ws[~nan].view(np.uint32))
            and np.array_equal(got[:, c16 + 4 * nb:], want[:, c16 + 4 * nb:]))


def values(rec, cols):
    """fp32 values a record array stands for."""
    rows, c16, nb = rec.shape[0], -(-cols // 16) * 16, -(-cols // 128)
    q = rec[:, :cols].astype(np.float32) - np.float32(128)
    s = np.ascontiguousarray(rec[:, c16:c16 + 4 * nb]).view(np.float32)
    return (q * np.repeat(s, 128, 1)[:, :cols]).astype(np.float32)


def norm(kind, z, eps):
    """(unit rows, 1/deviation, magnitude that the unit rows' rounding errors scale with)."""
    if kind == "none":
        return z, np.ones((z.shape[0], 1)), np.abs(z)
    m = z.mean(1, keepdims=True) if kind == "layer" else np.zeros((z.shape[0], 1))
    c = z - m
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    # the mean's own rounding error is relative to mean|z|
    slack = np.abs(z).mean(1, keepdims=True) * r if kind == "layer" else 0.0
    return c * r, r, np.abs(c * r) + slack


def join(d, x, h):
    """(y, u, magnitudes of both) in 64 bits."""
    rs, bs = d["residual_scale"], d["branch_scale"]
    y, my = rs * x, np.abs(rs * x)
    if h is not None:
        n, _, mn = norm(d["post_norm"], h, d["post_eps"])
        w, b = d.get("post_w"), d.get("post_b")
        w = 1.0 if w is None else w
        b = 0.0 if b is None else b
        g = gate_of(d, x.shape[0])
        y = y + bs * g * (n * w + b)
        my = my + np.abs(bs * g) * (mn * np.abs(w) + np.abs(b))
    if d["pre_norm"] == "none":
        return y, None, my, None
    n, r, mn = norm(d["pre_norm"], y, d["pre_eps"])
    w = 1.0 if d.get("pre_w") is None else d["pre_w"]
    b = 0.0 if d.get("pre_b") is None else d["pre_b"]
    spread = my * r + (my.mean(1, keepdims=True) * r if d["pre_norm"] == "layer" else 0)
    # an error of y also moves the deviation: at most mean(|n| spread) relative
    moved = np.abs(n) * (np.abs(n) * spread).mean(1, keepdims=True)
    return y, n * w + b, my, (mn + spread + moved) * np.abs(w) + np.abs(b)


def gate_of(d, rows):
    if not d.get("gate_rows"):
        return 1.0
    return np.asarray(d["gate"])[np.arange(rows) // d["gate_rows"]]


def back(d, y, h, dy, du, branch=True):
    """{name: (value, magnitude)} of the boundary's gradients in 64 bits at y and h."""
    rows = next(v for v in (y, h, dy, du) if v is not None).shape[0]
    cols = next(v for v in (y, h, dy, du) if v is not None).shape[1]
    out = {}
    gy, mgy = np.zeros((rows, cols)), np.zeros((rows, cols))
    if du is not None:
        n, r, mn = norm(d["pre_norm"], y, d["pre_eps"])
        w = 1.0 if d.get("pre_w") is None else d["pre_w"]
        g = du * w
        m1 = g.mean(1, keepdims=True) if d["pre_norm"] == "layer" else 0.0
        gy = r * (g - m1 - n * (g * n).mean(1, keepdims=True))
        a1 = np.abs(g).mean(1, keepdims=True) if d["pre_norm"] == "layer" else 0.0
        mgy = r * (np.abs(g) + a1 + mn * (np.abs(g) * mn).mean(1, keepdims=True))
        out["dpre_w"] = ((du * n).sum(0), (np.abs(du) * mn).sum(0))
        out["dpre_b"] = (du.sum(0), np.abs(du).sum(0))
    if dy is not None:
        gy, mgy = gy + dy, mgy + np.abs(dy)
    out["dx"] = (d["residual_scale"] * gy, np.abs(d["residual_scale"]) * mgy)
    if not branch:
        return out
    k = d["branch_scale"] * gate_of(d, rows)
    t, mt = k * gy, np.abs(k) * mgy
    if d["post_norm"] == "none":
        out["dh"] = (t, mt)
        hn = mhn = None
        if h is not None:
            hn, mhn = h, np.abs(h)
    else:
        n, r, mn = norm(d["post_norm"], h, d["post_eps"])
        w = 1.0 if d.get("post_w") is None else d["post_w"]
        b = 0.0 if d.get("post_b") is None else d["post_b"]
        g, mg = t * w, mt * np.abs(w)
        layer = d["post_norm"] == "layer"
        m1 = g.mean(1, keepdims=True) if layer else 0.0
        a1 = mg.mean(1, keepdims=True) if layer else 0.0
        out["dh"] = (r * (g - m1 - n * (g * n).mean(1, keepdims=True)),
                     r * (mg + a1 + mn * (mg * mn).mean(1, keepdims=True)))
        out["dpost_w"] = ((t * n).sum(0), (mt * mn).sum(0))
        out["dpost_b"] = (t.sum(0), mt.sum(0))
        hn, mhn = n * w + b, mn * np.abs(w) + np.abs(b)
    if d.get("gate_rows") and hn is not None:
        group = np.arange(rows) // d["gate_rows"]
        size = (rows - 1) // d["gate_rows"] + 1
        v, m = np.zeros((size, cols)), np.zeros((size, cols))
        np.add.at(v, group, d["branch_scale"] * gy * hn)
        np.add.at(m, group, np.abs(d["branch_scale"]) * mgy * mhn)
        out["dgate"] = (v, m)
    return out


def close(name, got, want, mag, T, roundings):
    """|got - want| is at most half a step of T at `want` plus `roundings` half steps of binary32
    at `mag` (the sum of the magnitudes that were added up)."""
    g = got.detach().cpu().to(torch.float64).numpy().reshape(want.shape)
    # the value that is rounded to T is already off by the second term
    err = roundings * U * mag
    tol = err + HALF[T] * (np.abs(want) + err) + TINY[T]
    bad = ~(np.abs(g - want) <= tol)
    both_nan = np.isnan(g) & np.isnan(want)
    bad &= ~both_nan
    same_inf = np.isinf(g) & (g == want)
    bad &= ~same_inf
    assert not bad.any(), (
        f"{name}: {int(bad.sum())} of {bad.size} off, first at "
        f"{tuple(int(i[0]) for i in np.nonzero(bad))}: got {g[bad][0]!r} want {want[bad][0]!r} "
        f"tolerance {tol[bad][0]:.3g}")

"""The layers of include/gm_layers.h in 64 bits, each result with a bound on what fp32 arithmetic may take from it.

The bound of a value is (operations on its way) * 2^-24 * (the same formula with every term's size in place of the
term), which covers each rounding and every cancellation; a result of 16 bits may be off by half a step more.
"""
import math

import numpy as np

EPS32 = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half a step under the normal range


def close(got, ref, size, ops, kind):
    """Whether got is within half a step of ref's type and `ops` fp32 roundings of terms of that size."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    room = HALF[kind] * np.abs(ref) * 1.01 + LEAST[kind] + ops * EPS32 * np.asarray(size, np.float64) * (1 + HALF[kind])
    bad = ~(np.abs(got - ref) <= room)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], ref[bad][:4], room[bad][:4])


def unit(v, size, norm, eps):
    """n(v), sizes of its terms, and 1 / size of each row."""
    mean = 0.0
    if norm == "layer":
        mean = v.mean(1, keepdims=True)
        size = size + size.mean(1, keepdims=True)
    c = v - mean
    r = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    return c * r, size * r, r


def unit_grad(d, d_size, u, u_size, r, norm):
    g = d - u * (d * u).mean(1, keepdims=True)
    size = d_size + u_size * (d_size * u_size).mean(1, keepdims=True)
    if norm == "layer":
        g = g - d.mean(1, keepdims=True)
        size = size + d_size.mean(1, keepdims=True)
    return g * r, size * r


def residual_norm(x, f=None, gx=None, gy=None, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0, before=None,
                  before_bias=None, eps=1e-6):
    """{name: (value, size)} of x', y and, from gx and gy, of the gradients ("dx" and so on). All arrays are float64."""
    out = {}
    x2, s2 = x, np.abs(x)
    if f is not None:
        p, ps = f, np.abs(f)
        if after is not None:
            uf, ufs, rf = unit(f, np.abs(f), norm, eps)
            p, ps = uf * after, ufs * np.abs(after)
            if after_bias is not None:
                p, ps = p + after_bias, ps + np.abs(after_bias)
        k = scale if gate is None else scale * gate
        x2, s2 = x + k * p, s2 + np.abs(k) * ps
    out["x"] = x2, s2
    if before is not None:
        u, us, r = unit(x2, s2, norm, eps)
        y, ys = u * before, us * np.abs(before)
        if before_bias is not None:
            y, ys = y + before_bias, ys + np.abs(before_bias)
        out["y"] = y, ys
    if gx is None and gy is None:
        return out
    dx = np.zeros_like(x) if gx is None else gx
    dxs = np.abs(dx)
    if before is not None:
        g = np.zeros_like(x) if gy is None else gy
        out["dbefore"] = (g * u).sum(0), (np.abs(g) * us).sum(0)
        out["dbefore_bias"] = g.sum(0), np.abs(g).sum(0)
        a, b = unit_grad(g * before, np.abs(g * before), u, us, r, norm)
        dx, dxs = dx + a, dxs + b
    out["dx"] = dx, dxs
    if f is not None:
        dp, dps = k * dx, np.abs(k) * dxs
        if gate is not None:
            dg, dgs = scale * dx * p, abs(scale) * dxs * ps
            out["dgate"] = (dg, dgs) if gate.ndim == 2 else (dg.sum(0), dgs.sum(0))
        if after is not None:
            out["dafter"] = (dp * uf).sum(0), (dps * ufs).sum(0)
            out["dafter_bias"] = dp.sum(0), dps.sum(0)
            out["df"] = unit_grad(dp * after, dps * np.abs(after), uf, ufs, rf, norm)
        else:
            out["df"] = dp, dps
    return out


def norm_ops(dim, rows=0):
    """fp32 operations on the way to a value: sums of a row in a thread (8 columns a turn, long rows in turns of at least
    4096), over a warp and over warps, in up to three means that feed one another, some 24 others; a sum over rows adds its own."""
    chain = 16 + 8 * math.ceil(dim / 4096) + 10
    return 4 * chain + 24 + (math.ceil(rows / 32) + 48 if rows else 0)


def act(z, name):
    """act(z) and its slope."""
    erf = np.vectorize(math.erf, otypes=[np.float64])
    if name in (None, "none"):
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if name == "silu":
        p = 1 / (1 + np.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + erf(z * math.sqrt(0.5)))
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)

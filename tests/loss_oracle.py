"""The losses over a class table (include/gm_losses.h) in 64 bits, from their definitions, and
bounds on how far a computation in 32 bits with 16-bit operands may be from them.

numpy alone; nothing is shared with the package. ``h`` and ``w`` are the operands as they
are stored, widened to float64.
"""
from dataclasses import dataclass

import numpy as np

# unit roundoff (half of eps) of the operands' and gradients' type; f32: three bf16 parts, 24 bits
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


@dataclass
class Teacher:
    """CSR rows: row_ptr, col, val (float64)."""

    row_ptr: np.ndarray
    col: np.ndarray
    val: np.ndarray

    def row(self, i):
        lo, hi = int(self.row_ptr[i]), int(self.row_ptr[i + 1])
        return self.col[lo:hi].astype(np.int64), self.val[lo:hi]


def log_sum_exp(z):
    m = z.max(1, keepdims=True)
    return (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]


def teacher_rows(t, temperature, rows, classes):
    """Dense q (rows x classes) and sum q log q of each row; zeros where a row has nothing to say."""
    q, base = np.zeros((rows, classes)), np.zeros(rows)
    for i in range(rows):
        col, val = t.row(i)
        v = val / temperature
        if v.size == 0 or np.all(v == -np.inf):
            continue
        p = np.exp(v - v.max())
        p /= p.sum()
        q[i, col] = p
        base[i] = np.sum(p[p > 0] * np.log(p[p > 0]))
    return q, base


def forward(h, w, target=None, ignore=-100, teacher=None, temperature=1.0):
    z = h @ w.T
    out = {"z": z}
    n = z.shape[0]
    if target is not None:
        out["lse"] = log_sum_exp(z)
        use = target != ignore
        out["loss"] = np.where(use, out["lse"] - z[np.arange(n), np.where(use, target, 0)], 0.0)
    if teacher is not None:
        q, base = teacher_rows(teacher, temperature, n, w.shape[0])
        out["lse_t"] = log_sum_exp(z / temperature)
        has = q.sum(1) > 0
        out["kl"] = np.where(has, base - (q * z).sum(1) / temperature + out["lse_t"], 0.0)
        out["q"], out["has"] = q, has
    return out


def logit_grads(f, target=None, ignore=-100, g_loss=None, g_lse=None, temperature=1.0, g_kl=None):
    """G = d objective / d z, and the parts its rounding errors scale with: probabilities and one-hot parts."""
    z = f["z"]
    n = z.shape[0]
    soft, hard = np.zeros_like(z), np.zeros_like(z)
    if target is not None:
        use = target != ignore
        gl = np.where(use, g_loss, 0.0)
        a = gl + (0.0 if g_lse is None else g_lse)
        soft += a[:, None] * np.exp(z - f["lse"][:, None])
        hard[np.arange(n), np.where(use, target, 0)] -= gl
    if g_kl is not None:
        b = np.where(f["has"], g_kl / temperature, 0.0)
        soft += b[:, None] * np.exp(z / temperature - f["lse_t"][:, None])
        hard -= b[:, None] * f["q"]
    return soft + hard, np.abs(soft), np.abs(hard)


def logit_error(h, w, steps=None):
    """Bound on the error of a logit: the tensor cores add 16 products at a time and cut each sum to 24 bits,
    so a sum of K products loses at most K / 16 units of the last of 24 bits of the largest partial sum; f32
    operands make six such sums, and leave out products under 2^-24."""
    k = h.shape[1]
    return (6 * (k / 16 + 1) + 8) * 2.0 ** -23 * (np.abs(h) @ np.abs(w).T)


def forward_bounds(f, h, w, temperature=1.0):
    """Elementwise bounds for loss, lse, kl, lse_t. The exponential unit is good to 2^-22 and its argument is rounded
    at a size of at most log2(e) |z - max|; sums of V terms are made of chains of at most 64 and then pairwise."""
    dz = logit_error(h, w).max(1)
    out = {}
    for name, t in (("lse", 1.0), ("lse_t", temperature)):
        if name in f:
            span = np.abs(f["z"]).max(1) / t
            out[name] = dz / t + 2.0 ** -22 * (64 + 4 * span) + 2.0 ** -22 * np.abs(f[name])
    if "loss" in f:
        out["loss"] = out["lse"] + dz + 2.0 ** -22 * (np.abs(f["z"]).max(1) + np.abs(f["lse"]))
    if "kl" in f:
        size = np.abs(f["z"]).max(1) / temperature + np.abs(f["lse_t"]) + np.abs(f["kl"])
        out["kl"] = out["lse_t"] + dz / temperature + 2.0 ** -20 * (8 + size)
    return out


def gradient_bounds(f, grads, h, w, kind, temperature=1.0):
    """Elementwise bounds for dH = G W and dW = G^T H."""
    g, soft, hard = grads
    u = ROUND[kind]
    dz = logit_error(h, w).max(1)
    t = min(1.0, temperature)
    lse = np.zeros(len(dz))
    for name in ("lse", "lse_t"):
        if name in f:
            lse = np.maximum(lse, np.abs(f[name]))
    # the exponent's error: logits and log-sum (as computed and as rounded to 32 bits), argument and unit
    dx = 2 * dz / t + 2.0 ** -22 * (72 + 8 * np.abs(f["z"]).max(1) / t + 4 * lse)
    dg = soft * np.expm1(dx)[:, None] + 2.0 ** -22 * (soft + hard) + u * np.abs(g) * (1 + 2.0 ** -8)
    biggest = (soft + hard).max() if g.size else 0.0
    if kind == "f16":  # G is scaled so that no entry passes 2^15; the smallest half is 2^-24
        dg = dg + 8 * np.abs(hard).max(1).max() * 2.0 ** -37 + biggest * 2.0 ** -36
    out = []
    for a, x, da in ((g, w, dg), (g.T, h, dg.T)):
        k = a.shape[1]
        exact = a @ x
        size = np.abs(a) @ np.abs(x)
        bound = da @ np.abs(x) + (6 * (k / 16 + 1) + 16) * 2.0 ** -23 * size + u * np.abs(exact) * (1 + 2.0 ** -8)
        out.append((exact, bound + (2.0 ** -24 if kind == "f16" else 1e-37)))
    return out

"""What makes the rows that the losses read (include/gm_layers.h): a product with bias, activation and residual in its
epilogue, and the norms around a residual with its gate and scale; forward and backward.

``linear`` and ``residual_norm`` work under torch's autograd. ``linear_forward``, ``linear_backward``,
``residual_norm_forward`` and ``residual_norm_backward`` are the same without it; ``gm_*`` write into the caller's
tensors under the names of the C interface. Matrices are rows of consecutive elements of bfloat16, float16 or float32;
all tensors of a call have one type. Nothing waits for the GPU.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .binding import GmError
from .losses import TYPES, _gradient, _like, _matrix, _On

EXPORTS = ["gm_linear_forward", "gm_linear_backward", "gm_linear_workspace", "gm_norm_forward", "gm_norm_backward", "gm_norm_workspace"]
NORMS = {"rms": 0, "layer": 1}
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


class gm_layer_config(ctypes.Structure):
    _fields_ = [("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class gm_linear(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("n_outs", ctypes.c_int64), ("x", ctypes.c_void_p),
                ("x_ld", ctypes.c_int64), ("w", ctypes.c_void_p), ("w_ld", ctypes.c_int64), ("type", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


class gm_norm(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("type", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("gate_kind", ctypes.c_int32), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("f", ctypes.c_void_p), ("f_ld", ctypes.c_int64),
                ("after", ctypes.c_void_p), ("after_bias", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_ld", ctypes.c_int64), ("before", ctypes.c_void_p), ("before_bias", ctypes.c_void_p)]


class gm_norm_grads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("f", ctypes.c_void_p), ("f_ld", ctypes.c_int64),
                ("gate", ctypes.c_void_p), ("gate_ld", ctypes.c_int64), ("after", ctypes.c_void_p),
                ("after_bias", ctypes.c_void_p), ("before", ctypes.c_void_p), ("before_bias", ctypes.c_void_p)]


_lib = None


def load():
    """The library with the layers' functions typed; raises when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load()
    P, V, I64, I32 = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.gm_linear_forward.argtypes = [P(gm_linear), P(gm_layer_config), V, V, V, I64, V, I64, V, I64]
    lib.gm_linear_backward.argtypes = [P(gm_linear), P(gm_layer_config), V, V, I64, V, I64, V, I64, V, I64, V]
    lib.gm_linear_workspace.argtypes = [P(gm_linear), I32, P(I64)]
    lib.gm_norm_forward.argtypes = [P(gm_norm), V, V, I64, V, I64, V]
    lib.gm_norm_backward.argtypes = [P(gm_norm), P(gm_layer_config), V, V, V, I64, V, I64, P(gm_norm_grads)]
    lib.gm_norm_workspace.argtypes = [P(gm_norm), P(I64)]
    for name in EXPORTS:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _row(name, t, n, like):
    """A contiguous vector of n elements as x's, or None: its address."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.shape != (n,) or t.dtype != like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements of {like.dtype} on {like.device}")
    return t.data_ptr()


def _rows(name, t, like, shape=None):
    return (None, 0) if t is None else _matrix(name, t, like, shape)


def _check(rc, where):
    if rc:
        raise GmError(rc, where)


def _own(t):
    """A matrix that was made for a result, as arguments."""
    return (None, 0) if t is None else (t.data_ptr() or None, t.shape[1])


# ---- product with bias, activation and residual ---------------------------------------------
def _linear(x, w, activation):
    xp, x_ld = _matrix("x", x)
    wp, w_ld = _matrix("w", w, x)
    n, dim = x.shape
    if w.shape[1] != dim or dim < 1 or w.shape[0] < 1:
        raise ValueError(f"x has rows of {dim} elements, w is {w.shape[0]} x {w.shape[1]}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(map(str, ACTIVATIONS))}, not {activation!r}")
    return gm_linear(n, dim, w.shape[0], xp, x_ld, wp, w_ld, TYPES[x.dtype], ACTIVATIONS[activation])


def _linear_run(name, backward, a, device, s, *args):
    lib, need = load(), ctypes.c_int64()
    _check(lib.gm_linear_workspace(a, backward, need), name)
    work = torch.empty(need.value, dtype=torch.uint8, device=device)
    _check(getattr(lib, name)(a, gm_layer_config(work.data_ptr() or None, need.value), s, *args), name)


def gm_linear_forward(x, w, bias, residual, y, z=None, *, activation=None, stream=None):
    a = _linear(x, w, activation)
    shape = (a.n_rows, a.n_outs)
    args = (_row("bias", bias, a.n_outs, x), *_rows("residual", residual, x, shape), *_rows("y", y, x, shape), *_rows("z", z, x, shape))
    with _On(x.device, stream) as s:
        _linear_run("gm_linear_forward", 0, a, x.device, s, *args)


def linear_forward(x, w, bias=None, *, activation=None, residual=None, keep=False, stream=None):
    """(y, z): y = residual + act(z), z = x w^T + bias (x: rows x dim, w: outs x dim). z is None unless ``keep`` and an
    activation, whose gradient reads it. ``activation``: relu, gelu, gelu_tanh, silu, or None."""
    a = _linear(x, w, activation)
    shape = (a.n_rows, a.n_outs)
    args = _row("bias", bias, a.n_outs, x), *_rows("residual", residual, x, shape)
    with _On(x.device, stream) as s:
        y = torch.empty(shape, dtype=x.dtype, device=x.device)
        z = torch.empty_like(y) if keep and a.activation else None
        _linear_run("gm_linear_forward", 0, a, x.device, s, *args, *_own(y), *_own(z))
    return y, z


def gm_linear_backward(x, w, grad, z, dx, dw, dbias, *, activation=None, stream=None):
    a = _linear(x, w, activation)
    shape = (a.n_rows, a.n_outs)
    args = (*_matrix("grad", grad, x, shape), *_rows("z", z, x, shape), *_gradient("dx", dx, x), *_gradient("dw", dw, w),
            _row("dbias", dbias, a.n_outs, x))
    with _On(x.device, stream) as s:
        _linear_run("gm_linear_backward", 1, a, x.device, s, *args)


def linear_backward(x, w, grad, *, activation=None, z=None, need_x=True, need_w=True, need_bias=False, stream=None):
    """(dx, dw, dbias) for the gradient by y; the residual's is that gradient itself. ``z``: linear_forward's, with an activation."""
    a = _linear(x, w, activation)
    shape = (a.n_rows, a.n_outs)
    args = *_matrix("grad", grad, x, shape), *_rows("z", z, x, shape)
    with _On(x.device, stream) as s:
        dx, dw = _like(x, need_x), _like(w, need_w)
        db = torch.empty(a.n_outs, dtype=x.dtype, device=x.device) if need_bias else None
        if need_x or need_w or need_bias:
            _linear_run("gm_linear_backward", 1, a, x.device, s, *args, *_own(dx), *_own(dw), None if db is None else db.data_ptr())
    return dx, dw, db


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, activation):
        ctx.activation = activation
        y, z = linear_forward(x, w, bias, activation=activation, residual=residual, keep=any(ctx.needs_input_grad[:3]))
        ctx.save_for_backward(x, w, z)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, w, z = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = linear_backward(x, w, _dense(g), activation=ctx.activation, z=z, need_x=need[0], need_w=need[1],
                                     need_bias=need[2])
        return dx, dw, db, g if need[3] else None, None


def linear(x, w, bias=None, *, activation=None, residual=None):
    """residual + act(x w^T + bias), differentiable by every tensor given."""
    return _Linear.apply(x, w, bias, residual, activation)


def _dense(g):
    """A gradient whose rows are consecutive elements (an expanded one is not)."""
    return g if g is None or (g.dim() == 2 and g.stride(1) == 1 and g.stride(0) >= g.shape[1]) else g.contiguous()


# ---- norms around a residual ------------------------------------------------------------------
class Normed(NamedTuple):
    """x + scale * gate * n(f), the norm of that (None without ``before``), and what the backward pass reads of each row."""

    x: torch.Tensor
    y: torch.Tensor | None
    stats: torch.Tensor


class NormGrads(NamedTuple):
    """Gradients by the inputs of those names; None for those that were not given or not asked for."""

    x: torch.Tensor | None
    f: torch.Tensor | None
    gate: torch.Tensor | None
    after: torch.Tensor | None
    after_bias: torch.Tensor | None
    before: torch.Tensor | None
    before_bias: torch.Tensor | None


def _norm(x, f, norm, after, after_bias, gate, scale, before, before_bias, eps):
    xp, x_ld = _matrix("x", x)
    n, dim = x.shape
    if dim < 1:
        raise ValueError("x must have rows of an element at least")
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {', '.join(NORMS)}, not {norm!r}")
    if f is None and (after is not None or after_bias is not None or gate is not None):
        raise ValueError("after, after_bias and gate belong to f, which is None")
    if (after is None and after_bias is not None) or (before is None and before_bias is not None):
        raise ValueError("a bias needs its norm's weight")
    fp, f_ld = _rows("f", f, x, x.shape)
    kind, gp, g_ld = 0, None, 0
    if gate is not None:
        if gate.dim() == 1:
            kind, gp = 1, _row("gate", gate, dim, x)
        else:
            kind, (gp, g_ld) = 2, _matrix("gate", gate, x, x.shape)
    return gm_norm(n, dim, TYPES[x.dtype], NORMS[norm], kind, scale, eps, xp, x_ld, fp, f_ld,
                   _row("after", after, dim, x), _row("after_bias", after_bias, dim, x), gp, g_ld,
                   _row("before", before, dim, x), _row("before_bias", before_bias, dim, x))


def _stats(t, x):
    if t is None:
        return None
    if t.shape != (x.shape[0], 4) or t.dtype != torch.float32 or t.device != x.device or not t.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 tensor of {x.shape[0]} x 4 on {x.device}")
    return t.data_ptr() or None


def gm_norm_forward(x, f, x_out, y, stats=None, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0,
                    before=None, before_bias=None, eps=1e-6, stream=None):
    a = _norm(x, f, norm, after, after_bias, gate, scale, before, before_bias, eps)
    with _On(x.device, stream) as s:
        _check(load().gm_norm_forward(a, s, *_rows("x_out", x_out, x, x.shape), *_rows("y", y, x, x.shape),
                                      _stats(stats, x)), "gm_norm_forward")


def residual_norm_forward(x, f=None, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0, before=None,
                          before_bias=None, eps=1e-6, stream=None) -> Normed:
    """x' = x + scale * gate * (n(f) * after + after_bias) and y = n(x') * before + before_bias, a row at a time; n divides
    by the root mean square (``norm="rms"``) or takes the mean off first (``"layer"``). Without ``after``, f is taken as it
    is; without ``f``, x' is x; without ``before``, y is None. ``gate``: a vector, a matrix like x, or None."""
    if f is None and before is None:
        raise ValueError("there is nothing to compute without f and before")
    a = _norm(x, f, norm, after, after_bias, gate, scale, before, before_bias, eps)
    with _On(x.device, stream) as s:
        x2, y = _like(x, f is not None), _like(x, before is not None)
        stats = torch.empty((x.shape[0], 4), dtype=torch.float32, device=x.device)
        _check(load().gm_norm_forward(a, s, *_own(x2), *_own(y), stats.data_ptr() or None), "gm_norm_forward")
    return Normed(x if x2 is None else x2, y, stats)


def gm_norm_backward(x, f, stats, grad_x, grad_y, grads: NormGrads, *, norm="rms", after=None, after_bias=None, gate=None,
                     scale=1.0, before=None, before_bias=None, eps=1e-6, stream=None):
    a = _norm(x, f, norm, after, after_bias, gate, scale, before, before_bias, eps)
    n = x.shape[1]
    g = _gradient("grads.gate", grads.gate, x) if a.gate_kind == 2 else (_row("grads.gate", grads.gate, n, x), 0)
    o = gm_norm_grads(*_gradient("grads.x", grads.x, x), *_gradient("grads.f", grads.f, x), *g,
                      *(_row("grads." + k, getattr(grads, k), n, x) for k in ("after", "after_bias", "before", "before_bias")))
    _norm_backward(a, x, stats, grad_x, grad_y, o, stream)


def _norm_backward(a, x, stats, grad_x, grad_y, o, stream):
    lib, need = load(), ctypes.c_int64()
    gx, gy = _rows("grad_x", grad_x, x, x.shape), _rows("grad_y", grad_y, x, x.shape)
    with _On(x.device, stream) as s:
        _check(lib.gm_norm_workspace(a, need), "gm_norm_backward")
        work = torch.empty(need.value, dtype=torch.uint8, device=x.device)
        cfg = gm_layer_config(work.data_ptr() or None, need.value)
        _check(lib.gm_norm_backward(a, cfg, s, _stats(stats, x), *gx, *gy, o), "gm_norm_backward")


def residual_norm_backward(x, f, grad_x, grad_y, stats, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0,
                           before=None, before_bias=None, eps=1e-6, need=None, stream=None) -> NormGrads:
    """Gradients by the inputs, from those by x' and by y (either may be None: zeros). ``need``: names of the inputs whose
    gradients are wanted (None: of all that are given)."""
    a = _norm(x, f, norm, after, after_bias, gate, scale, before, before_bias, eps)
    given = dict(x=x, f=f, gate=gate, after=after, after_bias=after_bias, before=before, before_bias=before_bias)
    if need is not None and not set(need) <= set(given):
        raise ValueError(f"need may hold {', '.join(given)}, not {', '.join(sorted(set(need) - set(given)))}")
    with _On(x.device, stream):
        out = {k: torch.empty(t.shape, dtype=t.dtype, device=t.device) if t is not None and (need is None or k in need)
               else None for k, t in given.items()}
        if any(t is not None for t in out.values()):
            v = {k: None if t is None else t.data_ptr() or None for k, t in out.items()}
            d = x.shape[1]
            _norm_backward(a, x, stats, grad_x, grad_y,
                           gm_norm_grads(v["x"], d, v["f"], d, v["gate"], d, v["after"], v["after_bias"], v["before"],
                                         v["before_bias"]), stream)
    return NormGrads(**out)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, f, after, after_bias, gate, before, before_bias, norm, scale, eps):
        ctx.rule = dict(norm=norm, scale=scale, eps=eps)
        out = residual_norm_forward(x, f, after=after, after_bias=after_bias, gate=gate, before=before,
                                    before_bias=before_bias, **ctx.rule)
        ctx.save_for_backward(x, f, after, after_bias, gate, before, before_bias, out.stats)
        ctx.set_materialize_grads(False)
        return (out.x if f is not None else None), out.y

    @staticmethod
    @once_differentiable
    def backward(ctx, g_x, g_y):
        x, f, after, after_bias, gate, before, before_bias, stats = ctx.saved_tensors
        names = ("x", "f", "after", "after_bias", "gate", "before", "before_bias")
        need = [k for k, wanted in zip(names, ctx.needs_input_grad) if wanted]
        if g_x is None and g_y is None:
            return (None,) * 10
        d = residual_norm_backward(x, f, _dense(g_x), _dense(g_y), stats, after=after, after_bias=after_bias, gate=gate,
                                   before=before, before_bias=before_bias, need=need, **ctx.rule)
        return *(getattr(d, k) for k in names), None, None, None


def residual_norm(x, f=None, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0, before=None,
                  before_bias=None, eps=1e-6):
    """(x', y) of ``residual_norm_forward``, differentiable by every tensor given."""
    x2, y = _ResidualNorm.apply(x, f, after, after_bias, gate, before, before_bias, norm, float(scale), float(eps))
    return (x if f is None else x2), y

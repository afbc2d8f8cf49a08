"""What makes the rows that the losses read (include/gm_layers.h): a product with bias, activation and residual in its
epilogue, and the norms around a residual with its gate and scale; forward and backward.

``linear`` and ``residual_norm`` work under torch's autograd. ``linear_forward``, ``linear_backward``,
``residual_norm_forward`` and ``residual_norm_backward`` are the same without it; ``gm_*`` write into the caller's
tensors under the names of the C interface. Matrices are rows of consecutive elements of bfloat16, float16 or float32;
all tensors of a call have one type. Nothing waits for the GPU. Arguments are checked, results made and the C interface called
by a compiled extension (csrc/gm_marshal.cpp).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .binding import GmError
from .marshal import call, extension

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


def _run(name, stream, x, *args):
    """A function of the extension, on `stream` where one is given: what it returned after its status."""
    f = getattr(extension(), name)
    rc, *out = f(x, *args) if stream is None else call(f, stream, x, *args)
    if rc:
        raise GmError(rc, "gm_" + name)
    return out


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {', '.join(map(str, ACTIVATIONS))}, not {name!r}")
    return ACTIVATIONS[name]


def _norm(name):
    if name not in NORMS:
        raise ValueError(f"norm must be one of {', '.join(NORMS)}, not {name!r}")
    return NORMS[name]


# ---- product with bias, activation and residual ---------------------------------------------
def gm_linear_forward(x, w, bias, residual, y, z=None, *, activation=None, stream=None):
    _run("linear_forward", stream, x, w, bias, _activation(activation), residual, False, y, z, False)


def linear_forward(x, w, bias=None, *, activation=None, residual=None, keep=False, stream=None):
    """(y, z): y = residual + act(z), z = x w^T + bias (x: rows x dim, w: outs x dim). z is None unless ``keep`` and an
    activation, whose gradient reads it. ``activation``: relu, gelu, gelu_tanh, silu, or None."""
    return tuple(_run("linear_forward", stream, x, w, bias, _activation(activation), residual, keep, None, None, True))


def gm_linear_backward(x, w, grad, z, dx, dw, dbias, *, activation=None, stream=None):
    _run("linear_backward", stream, x, w, grad, _activation(activation), z, dx, dw, dbias, False, False, False)


def linear_backward(x, w, grad, *, activation=None, z=None, need_x=True, need_w=True, need_bias=False, stream=None):
    """(dx, dw, dbias) for the gradient by y; the residual's is that gradient itself. ``z``: linear_forward's, with an activation."""
    if not (need_x or need_w or need_bias):
        return None, None, None
    return tuple(_run("linear_backward", stream, x, w, grad, _activation(activation), z, None, None, None, need_x, need_w, need_bias))


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


def gm_norm_forward(x, f, x_out, y, stats=None, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0,
                    before=None, before_bias=None, eps=1e-6, stream=None):
    _run("norm_forward", stream, x, f, _norm(norm), after, after_bias, gate, scale, before, before_bias, eps, x_out, y, stats, False)


def residual_norm_forward(x, f=None, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0, before=None,
                          before_bias=None, eps=1e-6, stream=None) -> Normed:
    """x' = x + scale * gate * (n(f) * after + after_bias) and y = n(x') * before + before_bias, a row at a time; n divides
    by the root mean square (``norm="rms"``) or takes the mean off first (``"layer"``). Without ``after``, f is taken as it
    is; without ``f``, x' is x; without ``before``, y is None. ``gate``: a vector, a matrix like x, or None."""
    x2, y, stats = _run("norm_forward", stream, x, f, _norm(norm), after, after_bias, gate, scale, before, before_bias, eps,
                        None, None, None, True)
    return Normed(x if x2 is None else x2, y, stats)


def gm_norm_backward(x, f, stats, grad_x, grad_y, grads: NormGrads, *, norm="rms", after=None, after_bias=None, gate=None,
                     scale=1.0, before=None, before_bias=None, eps=1e-6, stream=None):
    _run("norm_backward", stream, x, f, stats, grad_x, grad_y, _norm(norm), after, after_bias, gate, scale, before, before_bias,
         eps, list(grads), False, 0)


_ALL = (1 << len(NormGrads._fields)) - 1


def residual_norm_backward(x, f, grad_x, grad_y, stats, *, norm="rms", after=None, after_bias=None, gate=None, scale=1.0,
                           before=None, before_bias=None, eps=1e-6, need=None, stream=None) -> NormGrads:
    """Gradients by the inputs, from those by x' and by y (either may be None: zeros). ``need``: names of the inputs whose
    gradients are wanted (None: of all that are given)."""
    bits = _ALL
    if need is not None:
        if not set(need) <= set(NormGrads._fields):
            raise ValueError(f"need may hold {', '.join(NormGrads._fields)}, not {', '.join(sorted(set(need) - set(NormGrads._fields)))}")
        bits = sum(1 << NormGrads._fields.index(k) for k in set(need))
    (out,) = _run("norm_backward", stream, x, f, stats, grad_x, grad_y, _norm(norm), after, after_bias, gate, scale, before,
                  before_bias, eps, [], True, bits)
    return NormGrads(*out)


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

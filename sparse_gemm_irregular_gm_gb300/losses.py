"""Losses over a large class table (include/gm_losses.h): softmax cross entropy and
distillation from a teacher's top entries, forward and backward.

The logits are Z = H W^T (``h``: rows x dim, ``w``: classes x dim; bfloat16, float16 or
float32) and are never stored. The teacher is a ``binding.DeviceCSR`` of rows x classes,
columns ascending in a row: what ``binding.spgemm`` returns can be one.

``gm_*`` marshal tensors into the C ABI under its own names. ``xent_forward`` and the
other functions of that kind also allocate the results; ``cross_entropy`` and
``distillation`` are the same under torch's autograd. Nothing waits for the GPU unless
``check=True``, which raises ``binding.GmError`` for a bad target or teacher row of that call;
``gm_loss_status`` raises for those of the calls without it.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import binding
from .binding import DeviceCSR, GmError, gm_csr

GM_LOSS_F32, GM_LOSS_BF16, GM_LOSS_F16 = 0, 1, 2
GM_LOSS_CHECK = 1
EXPORTS = ["gm_xent_forward", "gm_xent_backward", "gm_distill_forward", "gm_distill_backward", "gm_loss_workspace",
           "gm_loss_status"]
TYPES = {torch.float32: GM_LOSS_F32, torch.bfloat16: GM_LOSS_BF16, torch.float16: GM_LOSS_F16}
_ROW_PTR = {torch.int64: 0, torch.int32: binding.GM_INDEX_ROWPTR32}
_COL = {torch.int32: 0, torch.int64: binding.GM_INDEX_COL64}
_VAL = {torch.float64: binding.GM_VALUE_F64, torch.float32: binding.GM_VALUE_F32}


class gm_logits(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_classes", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("h_ld", ctypes.c_int64), ("w", ctypes.c_void_p), ("w_ld", ctypes.c_int64),
                ("type", ctypes.c_int32)]


class gm_labels(ctypes.Structure):
    _fields_ = [("target", ctypes.c_void_p), ("ignore_index", ctypes.c_int64), ("target32", ctypes.c_int32)]


class gm_loss_config(ctypes.Structure):
    _fields_ = [("workspace_cap_bytes", ctypes.c_int64), ("flags", ctypes.c_int32), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64)]


_lib = None


def load():
    """The library with the losses' functions typed; raises when it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    lib = binding.load()
    P, V, I64, I32 = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    head = [P(gm_logits)]
    teacher = [P(gm_csr), I32, I32, ctypes.c_float]
    tail = [P(gm_labels), P(gm_loss_config), V]
    out = [V, I64, V, I64]
    lib.gm_xent_forward.argtypes = head + tail + [V, V]
    lib.gm_xent_backward.argtypes = head + tail + [V, V, V] + out
    lib.gm_distill_forward.argtypes = head + teacher + tail + [V, V, V, V]
    lib.gm_distill_backward.argtypes = head + teacher + tail + [V, V, V, V, V] + out
    lib.gm_loss_workspace.argtypes = head + [I64, I32, P(gm_loss_config), P(I64)]
    lib.gm_loss_status.argtypes = [V]
    for name in EXPORTS:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _matrix(name, t, like=None, shape=None):
    """A CUDA matrix whose rows are consecutive elements: (pointer, elements between rows)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.dtype not in TYPES:
        raise ValueError(f"{name} must be a 2-d CUDA tensor of float32, bfloat16 or float16")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, not {t.dtype} on {t.device}")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, not {(rows, cols)}")
    ld, step = t.stride()
    if (step != 1 and cols > 1) or (ld < cols and rows > 1):
        raise ValueError(f"{name}'s rows must be consecutive elements that do not overlap (strides {t.stride()})")
    return t.data_ptr() or None, (ld if rows > 1 else cols or 1)


_F32 = (torch.float32,)
_INT = (torch.int64, torch.int32)


def _vector(name, t, n, device, dtypes=_F32):
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != (n,) or not t.is_contiguous()
            or t.device != device):
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements of {' or '.join(map(str, dtypes))} on {device}")
    return t.data_ptr() or None


def _same_device(stream, device):
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return stream


class _Call:
    """One call's checked arguments; ``with`` makes its device and stream current, so that what torch
    allocates inside belongs to that stream."""

    def __init__(self, h, w, target, ignore_index, teacher, check, workspace_cap_bytes, stream):
        hp, h_ld = _matrix("h", h)
        wp, w_ld = _matrix("w", w, h)
        self.n, dim = h.shape
        if dim != w.shape[1]:
            raise ValueError(f"h has rows of {dim} elements, w of {w.shape[1]}")
        self.h, self.w, self.device = h, w, h.device
        self.z = gm_logits(self.n, w.shape[0], dim, hp, h_ld, wp, w_ld, TYPES[h.dtype])
        self.labels = None
        if target is not None:
            p = _vector("target", target, self.n, self.device, _INT)
            self.labels = gm_labels(p, ignore_index, target.dtype == torch.int32)
        self.cfg = gm_loss_config(workspace_cap_bytes, GM_LOSS_CHECK if check else 0, None, 0)
        self.teacher = self._teacher(teacher) if teacher is not None else None
        self.given = stream
        self.on = None

    def _teacher(self, t):
        for name, x, kinds in (("row_ptr", t.row_ptr, _ROW_PTR), ("col", t.col, _COL), ("val", t.val, _VAL)):
            if not isinstance(x, torch.Tensor) or x.device != self.device or x.dtype not in kinds or not x.is_contiguous():
                raise ValueError(f"the teacher's {name} must be a contiguous tensor of {' or '.join(map(str, kinds))} "
                                 f"on {self.device}")
        if t.row_ptr.numel() != self.n + 1 or t.col.numel() != t.val.numel():
            raise ValueError(f"the teacher has {t.row_ptr.numel()} row pointers for {self.n} rows, {t.col.numel()} "
                             f"columns and {t.val.numel()} values")
        return t.desc(), _VAL[t.val.dtype], _ROW_PTR[t.row_ptr.dtype] | _COL[t.col.dtype]

    def __enter__(self):
        if self.given is not None:
            self.on = torch.cuda.stream(_same_device(self.given, self.device))  # also makes its device current
        elif torch.cuda.current_device() != self.device.index:
            self.on = torch.cuda.device(self.device)
        if self.on is not None:
            self.on.__enter__()
        return self

    def __exit__(self, *a):
        if self.on is not None:
            self.on.__exit__(*a)

    def vectors(self, k):
        """k uninitialised results, a float a row."""
        return [torch.empty(self.n, dtype=torch.float32, device=self.device) for _ in range(k)]

    def run(self, name, backward, *args):
        lib = load()
        z, cfg, need = self.z, self.cfg, ctypes.c_int64()
        rc = lib.gm_loss_workspace(z, -1 if self.teacher is None else self.teacher[0].nnz, backward, cfg, need)
        if rc:
            raise GmError(rc, name)
        size = need.value
        work = torch.empty(size, dtype=torch.uint8, device=self.device)
        cfg.workspace = work.data_ptr() or None
        cfg.workspace_bytes = size
        stream = (self.given if self.given is not None else torch.cuda.current_stream(self.device.index)).cuda_stream
        if self.teacher is None:
            rc = getattr(lib, name)(z, self.labels, cfg, stream, *args)
        else:
            rc = getattr(lib, name)(z, *self.teacher, self.temperature, self.labels, cfg, stream, *args)
        if rc:
            raise GmError(rc, name)


def gm_loss_status(stream=None):
    """Waits for the stream; raises GmError for what the losses' calls met since the last call."""
    binding._check(load().gm_loss_status(binding._stream_handle(stream)), "gm_loss_status")


# ---- cross entropy -----------------------------------------------------------------------
def gm_xent_forward(h, w, target, loss, lse, *, ignore_index=-100, check=False, stream=None):
    c = _Call(h, w, target, ignore_index, None, check, 0, stream)
    with c:
        c.run("gm_xent_forward", 0, _vector("loss", loss, c.n, c.device), _vector("lse", lse, c.n, c.device))


def gm_xent_backward(h, w, target, lse, grad_loss, grad_lse, dh, dw, *, ignore_index=-100, workspace_cap_bytes=0,
                     check=False, stream=None):
    c = _Call(h, w, target, ignore_index, None, check, workspace_cap_bytes, stream)
    with c:
        _xent_backward(c, lse, grad_loss, grad_lse, _gradient("dh", dh, h), _gradient("dw", dw, w))


def _xent_backward(c, lse, grad_loss, grad_lse, dh, dw):
    n, dev = c.n, c.device
    c.run("gm_xent_backward", 1, _vector("lse", lse, n, dev), _vector("grad_loss", grad_loss, n, dev),
          _vector("grad_lse", grad_lse, n, dev), *dh, *dw)


def _gradient(name, t, of):
    return (None, 0) if t is None else _matrix(name, t, of, of.shape)


def _like(x, need):
    return torch.empty(x.shape, dtype=x.dtype, device=x.device) if need else None


def _own(t):
    """A gradient that _like made, as arguments."""
    return (None, 0) if t is None else (t.data_ptr() or None, max(t.shape[1], 1))


def xent_forward(h, w, target, *, ignore_index=-100, check=False, stream=None):
    """(loss, lse) of each row: lse_i - z_i,target(i), and lse_i = log sum_j exp(z_ij), float32."""
    c = _Call(h, w, target, ignore_index, None, check, 0, stream)
    with c:
        loss, lse = c.vectors(2)
        c.run("gm_xent_forward", 0, loss.data_ptr() or None, lse.data_ptr() or None)
    return loss, lse


def xent_backward(h, w, target, lse, grad_loss, grad_lse=None, *, ignore_index=-100, need_h=True, need_w=True,
                  workspace_cap_bytes=0, check=False, stream=None):
    """(dh, dw) for the derivatives of an objective by loss and (optional) by lse."""
    c = _Call(h, w, target, ignore_index, None, check, workspace_cap_bytes, stream)
    with c:
        dh, dw = _like(h, need_h), _like(w, need_w)
        _xent_backward(c, lse, grad_loss, grad_lse, _own(dh), _own(dw))
    return dh, dw


# ---- distillation --------------------------------------------------------------------------
class Distilled(NamedTuple):
    """Per row: divergence from the teacher, log sum_j exp(z_ij / T); with labels, cross entropy and lse."""

    kl: torch.Tensor
    lse_t: torch.Tensor
    loss: torch.Tensor | None
    lse: torch.Tensor | None


def _distill_call(h, w, teacher, temperature, target, ignore_index, check, workspace_cap_bytes, stream):
    c = _Call(h, w, target, ignore_index, teacher, check, workspace_cap_bytes, stream)
    c.temperature = temperature
    return c


def gm_distill_forward(h, w, teacher, temperature, kl, lse_t, target=None, loss=None, lse=None, *, ignore_index=-100,
                       check=False, stream=None):
    c = _distill_call(h, w, teacher, temperature, target, ignore_index, check, 0, stream)
    with c:
        c.run("gm_distill_forward", 0, *(_vector(k, t, c.n, c.device) for k, t in
                                         (("kl", kl), ("lse_t", lse_t), ("loss", loss), ("lse", lse))))


def gm_distill_backward(h, w, teacher, temperature, lse_t, grad_kl, dh, dw, target=None, lse=None, grad_loss=None,
                        grad_lse=None, *, ignore_index=-100, workspace_cap_bytes=0, check=False, stream=None):
    c = _distill_call(h, w, teacher, temperature, target, ignore_index, check, workspace_cap_bytes, stream)
    with c:
        _distill_backward(c, lse_t, grad_kl, lse, grad_loss, grad_lse, _gradient("dh", dh, h), _gradient("dw", dw, w))


def _distill_backward(c, lse_t, grad_kl, lse, grad_loss, grad_lse, dh, dw):
    n, dev = c.n, c.device
    c.run("gm_distill_backward", 1, _vector("lse_t", lse_t, n, dev), _vector("grad_kl", grad_kl, n, dev),
          _vector("lse", lse, n, dev), _vector("grad_loss", grad_loss, n, dev), _vector("grad_lse", grad_lse, n, dev),
          *dh, *dw)


def distill_forward(h, w, teacher: DeviceCSR, temperature=1.0, *, target=None, ignore_index=-100, check=False,
                    stream=None) -> Distilled:
    """Divergence of softmax(z / T) from the softmax of the teacher's stored values / T, a row; with ``target``
    also the rows' cross entropy at temperature 1, from the same pass."""
    c = _distill_call(h, w, teacher, temperature, target, ignore_index, check, 0, stream)
    with c:
        out = c.vectors(2 if target is None else 4)
        p = [t.data_ptr() or None for t in out]
        c.run("gm_distill_forward", 0, *p, *[None] * (4 - len(p)))
    return Distilled(*out, *[None] * (4 - len(out)))


def distill_backward(h, w, teacher: DeviceCSR, lse_t, grad_kl, temperature=1.0, *, target=None, lse=None,
                     grad_loss=None, grad_lse=None, ignore_index=-100, need_h=True, need_w=True,
                     workspace_cap_bytes=0, check=False, stream=None):
    """(dh, dw) for the derivatives of an objective by kl and, with ``target``, by loss and (optional) lse."""
    c = _distill_call(h, w, teacher, temperature, target, ignore_index, check, workspace_cap_bytes, stream)
    with c:
        dh, dw = _like(h, need_h), _like(w, need_w)
        _distill_backward(c, lse_t, grad_kl, lse, grad_loss, grad_lse, _own(dh), _own(dw))
    return dh, dw


# ---- under autograd --------------------------------------------------------------------------
def _contiguous(g, like):
    return torch.zeros_like(like) if g is None else g.float().contiguous()


class _Xent(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, target, ignore_index):
        loss, lse = xent_forward(h, w, target, ignore_index=ignore_index)
        ctx.save_for_backward(h, w, target, lse)
        ctx.ignore_index = ignore_index
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, g_loss, g_lse):
        h, w, target, lse = ctx.saved_tensors
        dh, dw = xent_backward(h, w, target, lse, _contiguous(g_loss, lse),
                               None if g_lse is None else g_lse.float().contiguous(), ignore_index=ctx.ignore_index,
                               need_h=ctx.needs_input_grad[0], need_w=ctx.needs_input_grad[1])
        return dh, dw, None, None


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, row_ptr, col, val, target, temperature, ignore_index):
        teacher = DeviceCSR(h.shape[0], w.shape[0], row_ptr, col, val)
        f = distill_forward(h, w, teacher, temperature, target=target, ignore_index=ignore_index)
        ctx.save_for_backward(h, w, row_ptr, col, val, target, f.lse_t, f.lse)
        ctx.temperature, ctx.ignore_index = temperature, ignore_index
        ctx.mark_non_differentiable(f.lse_t)
        ctx.set_materialize_grads(False)
        return tuple(f)

    @staticmethod
    @once_differentiable
    def backward(ctx, g_kl, _, g_loss, g_lse):
        h, w, row_ptr, col, val, target, lse_t, lse = ctx.saved_tensors
        teacher = DeviceCSR(h.shape[0], w.shape[0], row_ptr, col, val)
        dh, dw = distill_backward(h, w, teacher, lse_t, _contiguous(g_kl, lse_t), ctx.temperature, target=target,
                                  lse=lse, grad_loss=None if target is None else _contiguous(g_loss, lse),
                                  grad_lse=None if g_lse is None else g_lse.float().contiguous(),
                                  ignore_index=ctx.ignore_index, need_h=ctx.needs_input_grad[0],
                                  need_w=ctx.needs_input_grad[1])
        return dh, dw, None, None, None, None, None, None


def cross_entropy(h, w, target, *, ignore_index=-100):
    """(loss, lse) a row, differentiable by h and w through both."""
    return _Xent.apply(h, w, target, ignore_index)


def distillation(h, w, teacher: DeviceCSR, temperature=1.0, *, target=None, ignore_index=-100) -> Distilled:
    """``distill_forward`` differentiable by h and w through kl, loss and lse (not lse_t). The teacher is a constant:
    values that want a gradient are refused (detach them)."""
    if teacher.n_rows != h.shape[0] or teacher.n_cols != w.shape[0]:
        raise GmError(2, f"the teacher is {teacher.n_rows} x {teacher.n_cols}, the logits {h.shape[0]} x {w.shape[0]}")
    if torch.is_grad_enabled() and teacher.val.requires_grad:
        raise ValueError("the teacher's values require a gradient, which distillation does not have; detach them")
    return Distilled(*_Distill.apply(h, w, teacher.row_ptr, teacher.col, teacher.val, target, float(temperature),
                                     ignore_index))

"""Losses over a large class table (include/gm_losses.h): softmax cross entropy and
distillation from a teacher's top entries, forward and backward.

The logits are Z = H W^T (``h``: rows x dim, ``w``: classes x dim; bfloat16, float16 or
float32) and are never stored. The teacher is a ``binding.DeviceCSR`` of rows x classes,
columns ascending in a row: what ``binding.spgemm`` returns can be one.

``gm_*`` marshal tensors into the C ABI under its own names. ``xent_forward`` and the
other functions of that kind also allocate the results; ``cross_entropy`` and
``distillation`` are the same under torch's autograd. Nothing waits for the GPU unless
``check=True``, which raises ``binding.GmError`` for a bad target or teacher row.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import DeviceCSR, GmError, gm_csr

GM_LOSS_F32, GM_LOSS_BF16, GM_LOSS_F16 = 0, 1, 2
GM_LOSS_CHECK = 1
EXPORTS = ["gm_xent_forward", "gm_xent_backward", "gm_distill_forward", "gm_distill_backward", "gm_loss_status"]
TYPES = {torch.float32: GM_LOSS_F32, torch.bfloat16: GM_LOSS_BF16, torch.float16: GM_LOSS_F16}


class gm_logits(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_classes", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("h", ctypes.c_void_p), ("h_ld", ctypes.c_int64), ("w", ctypes.c_void_p), ("w_ld", ctypes.c_int64),
                ("type", ctypes.c_int32)]


class gm_labels(ctypes.Structure):
    _fields_ = [("target", ctypes.c_void_p), ("ignore_index", ctypes.c_int64), ("target32", ctypes.c_int32)]


class gm_loss_config(ctypes.Structure):
    _fields_ = [("workspace_cap_bytes", ctypes.c_int64), ("flags", ctypes.c_int32)]


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
    lib.gm_loss_status.argtypes = [V]
    for name in EXPORTS:
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def _matrix(name, t, device=None, dtype=None, shape=None):
    """A CUDA matrix whose rows are consecutive elements: (pointer, elements between rows)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2 or t.dtype not in TYPES:
        raise ValueError(f"{name} must be a 2-d CUDA tensor of float32, bfloat16 or float16")
    if (device is not None and t.device != device) or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be {dtype} on {device}, not {t.dtype} on {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, not {tuple(t.shape)}")
    rows, cols = t.shape
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        raise ValueError(f"{name}'s rows must be consecutive elements that do not overlap (strides {t.stride()})")
    return (t.data_ptr() if t.numel() else None), (t.stride(0) if rows > 1 else max(cols, 1))


def _vector(name, t, n, device, dtypes=(torch.float32,)):
    if t is None:
        return None
    if (not isinstance(t, torch.Tensor) or t.device != device or t.dtype not in dtypes or t.dim() != 1
            or t.numel() != n or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous tensor of {n} elements of {' or '.join(map(str, dtypes))} on {device}")
    return t.data_ptr() if n else None


def _logits(h, w):
    hp, h_ld = _matrix("h", h)
    wp, w_ld = _matrix("w", w, h.device, h.dtype)
    if h.shape[1] != w.shape[1]:
        raise ValueError(f"h has rows of {h.shape[1]} elements, w of {w.shape[1]}")
    return gm_logits(h.shape[0], w.shape[0], h.shape[1], hp, h_ld, wp, w_ld, TYPES[h.dtype])


def _labels(h, target, ignore_index):
    if target is None:
        return None
    p = _vector("target", target, h.shape[0], h.device, (torch.int64, torch.int32))
    return gm_labels(p, int(ignore_index), int(target.dtype == torch.int32))


def _teacher(h, w, t: DeviceCSR):
    """(descriptor, value type, index type) of a teacher of rows x classes."""
    n, dev = h.shape[0], h.device
    rp = {torch.int64: 0, torch.int32: binding.GM_INDEX_ROWPTR32}
    col = {torch.int32: 0, torch.int64: binding.GM_INDEX_COL64}
    val = {torch.float64: binding.GM_VALUE_F64, torch.float32: binding.GM_VALUE_F32}
    for name, x, kinds in (("row_ptr", t.row_ptr, rp), ("col", t.col, col), ("val", t.val, val)):
        if not isinstance(x, torch.Tensor) or x.device != dev or x.dtype not in kinds or not x.is_contiguous():
            raise ValueError(f"the teacher's {name} must be a contiguous tensor of {' or '.join(map(str, kinds))} on {dev}")
    if t.row_ptr.numel() != n + 1 or t.col.numel() != t.val.numel():
        raise ValueError(f"the teacher has {t.row_ptr.numel()} row pointers for {n} rows, {t.col.numel()} columns and "
                         f"{t.val.numel()} values")
    return t.desc(), val[t.val.dtype], rp[t.row_ptr.dtype] | col[t.col.dtype]


def _config(check, workspace_cap_bytes):
    if not check and not workspace_cap_bytes:
        return None
    return gm_loss_config(int(workspace_cap_bytes), GM_LOSS_CHECK if check else 0)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


class _On:
    """The tensors' device, and the stream that work and results belong to."""

    def __init__(self, device, stream):
        self.stream = stream if stream is not None else torch.cuda.current_stream(device)
        if self.stream.device != device:
            raise ValueError(f"the stream is on {self.stream.device}, the tensors are on {device}")
        self.on = torch.cuda.stream(self.stream)  # also makes the stream's device current

    def __enter__(self):
        self.on.__enter__()
        return ctypes.c_void_p(self.stream.cuda_stream)

    def __exit__(self, *a):
        return self.on.__exit__(*a)


def gm_loss_status(stream=None):
    """Waits for the stream; raises GmError for what the losses' calls met since the last call."""
    binding._check(load().gm_loss_status(binding._stream_handle(stream)), "gm_loss_status")


# ---- cross entropy -----------------------------------------------------------------------
def gm_xent_forward(h, w, target, loss, lse, *, ignore_index=-100, check=False, stream=None):
    z, lab = _logits(h, w), _labels(h, target, ignore_index)
    n, dev = h.shape[0], h.device
    with _On(dev, stream) as s:
        binding._check(load().gm_xent_forward(_ref(z), _ref(lab), _ref(_config(check, 0)), s,
                                              _vector("loss", loss, n, dev), _vector("lse", lse, n, dev)),
                       "gm_xent_forward")


def gm_xent_backward(h, w, target, lse, grad_loss, grad_lse, dh, dw, *, ignore_index=-100, workspace_cap_bytes=0,
                     check=False, stream=None):
    z, lab = _logits(h, w), _labels(h, target, ignore_index)
    n, dev = h.shape[0], h.device
    dhp, dh_ld = _matrix("dh", dh, dev, h.dtype, h.shape) if dh is not None else (None, 0)
    dwp, dw_ld = _matrix("dw", dw, dev, h.dtype, w.shape) if dw is not None else (None, 0)
    with _On(dev, stream) as s:
        binding._check(load().gm_xent_backward(
            _ref(z), _ref(lab), _ref(_config(check, workspace_cap_bytes)), s, _vector("lse", lse, n, dev),
            _vector("grad_loss", grad_loss, n, dev), _vector("grad_lse", grad_lse, n, dev), dhp, dh_ld, dwp, dw_ld),
            "gm_xent_backward")


def xent_forward(h, w, target, *, ignore_index=-100, check=False, stream=None):
    """(loss, lse) of each row: lse_i - z_i,target(i), and lse_i = log sum_j exp(z_ij), float32."""
    _logits(h, w)
    with _On(h.device, stream):
        loss, lse = (torch.empty(h.shape[0], dtype=torch.float32, device=h.device) for _ in range(2))
    gm_xent_forward(h, w, target, loss, lse, ignore_index=ignore_index, check=check, stream=stream)
    return loss, lse


def _grad_buffers(h, w, need_h, need_w, stream):
    _logits(h, w)
    with _On(h.device, stream):
        return (torch.empty(h.shape, dtype=h.dtype, device=h.device) if need_h else None,
                torch.empty(w.shape, dtype=w.dtype, device=w.device) if need_w else None)


def xent_backward(h, w, target, lse, grad_loss, grad_lse=None, *, ignore_index=-100, need_h=True, need_w=True,
                  workspace_cap_bytes=0, check=False, stream=None):
    """(dh, dw) for the derivatives of an objective by loss and (optional) by lse."""
    dh, dw = _grad_buffers(h, w, need_h, need_w, stream)
    gm_xent_backward(h, w, target, lse, grad_loss, grad_lse, dh, dw, ignore_index=ignore_index,
                     workspace_cap_bytes=workspace_cap_bytes, check=check, stream=stream)
    return dh, dw


# ---- distillation --------------------------------------------------------------------------
class Distilled(NamedTuple):
    """Per row: divergence from the teacher, log sum_j exp(z_ij / T); with labels, cross entropy and lse."""

    kl: torch.Tensor
    lse_t: torch.Tensor
    loss: torch.Tensor | None
    lse: torch.Tensor | None


def gm_distill_forward(h, w, teacher, temperature, kl, lse_t, target=None, loss=None, lse=None, *, ignore_index=-100,
                       check=False, stream=None):
    z, lab = _logits(h, w), _labels(h, target, ignore_index)
    desc, vt, it = _teacher(h, w, teacher)
    n, dev = h.shape[0], h.device
    with _On(dev, stream) as s:
        binding._check(load().gm_distill_forward(
            _ref(z), _ref(desc), vt, it, float(temperature), _ref(lab), _ref(_config(check, 0)), s,
            _vector("kl", kl, n, dev), _vector("lse_t", lse_t, n, dev), _vector("loss", loss, n, dev),
            _vector("lse", lse, n, dev)), "gm_distill_forward")


def gm_distill_backward(h, w, teacher, temperature, lse_t, grad_kl, dh, dw, target=None, lse=None, grad_loss=None,
                        grad_lse=None, *, ignore_index=-100, workspace_cap_bytes=0, check=False, stream=None):
    z, lab = _logits(h, w), _labels(h, target, ignore_index)
    desc, vt, it = _teacher(h, w, teacher)
    n, dev = h.shape[0], h.device
    dhp, dh_ld = _matrix("dh", dh, dev, h.dtype, h.shape) if dh is not None else (None, 0)
    dwp, dw_ld = _matrix("dw", dw, dev, h.dtype, w.shape) if dw is not None else (None, 0)
    with _On(dev, stream) as s:
        binding._check(load().gm_distill_backward(
            _ref(z), _ref(desc), vt, it, float(temperature), _ref(lab), _ref(_config(check, workspace_cap_bytes)), s,
            _vector("lse_t", lse_t, n, dev), _vector("grad_kl", grad_kl, n, dev), _vector("lse", lse, n, dev),
            _vector("grad_loss", grad_loss, n, dev), _vector("grad_lse", grad_lse, n, dev), dhp, dh_ld, dwp, dw_ld),
            "gm_distill_backward")


def distill_forward(h, w, teacher: DeviceCSR, temperature=1.0, *, target=None, ignore_index=-100, check=False,
                    stream=None) -> Distilled:
    """Divergence of softmax(z / T) from the softmax of the teacher's stored values / T, a row; with ``target``
    also the rows' cross entropy at temperature 1, from the same pass."""
    _logits(h, w)
    with _On(h.device, stream):
        out = [torch.empty(h.shape[0], dtype=torch.float32, device=h.device) for _ in range(2 if target is None else 4)]
    out += [None] * (4 - len(out))
    gm_distill_forward(h, w, teacher, temperature, out[0], out[1], target, out[2], out[3], ignore_index=ignore_index,
                       check=check, stream=stream)
    return Distilled(*out)


def distill_backward(h, w, teacher: DeviceCSR, lse_t, grad_kl, temperature=1.0, *, target=None, lse=None,
                     grad_loss=None, grad_lse=None, ignore_index=-100, need_h=True, need_w=True,
                     workspace_cap_bytes=0, check=False, stream=None):
    """(dh, dw) for the derivatives of an objective by kl and, with ``target``, by loss and (optional) lse."""
    dh, dw = _grad_buffers(h, w, need_h, need_w, stream)
    gm_distill_backward(h, w, teacher, temperature, lse_t, grad_kl, dh, dw, target, lse, grad_loss, grad_lse,
                        ignore_index=ignore_index, workspace_cap_bytes=workspace_cap_bytes, check=check, stream=stream)
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
    """``distill_forward`` differentiable by h and w through kl, loss and lse (not lse_t)."""
    if teacher.n_rows != h.shape[0] or teacher.n_cols != w.shape[0]:
        raise GmError(2, f"the teacher is {teacher.n_rows} x {teacher.n_cols}, the logits {h.shape[0]} x {w.shape[0]}")
    return Distilled(*_Distill.apply(h, w, teacher.row_ptr, teacher.col, teacher.val, target, float(temperature),
                                     ignore_index))

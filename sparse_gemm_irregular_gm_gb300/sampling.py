"""A class drawn from each row of logits over a class table (include/gm_sampling.h), by a temperature, top-k, top-p and
min-p, from given random numbers.

``draw`` allocates the results; ``gm_draw`` writes into the caller's tensors under the C interface's name. Nothing waits
for the GPU. A row that cannot be drawn from has index -1, logprob NaN, kept 0.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import GmError
from .losses import TYPES, _matrix, _On, _vector

EXPORTS = ["gm_draw"]


class gm_draw_rule(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("all_temperature", ctypes.c_float), ("all_top_k", ctypes.c_int32),
                ("all_top_p", ctypes.c_float), ("all_min_p", ctypes.c_float)]


_lib = None


def load():
    """The library with the draw's functions typed; raises when it has not been built."""
    global _lib
    if _lib is None:
        lib = binding.load()
        V, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        lib.gm_draw.argtypes = [V, I64, I64, I64, I32, ctypes.POINTER(gm_draw_rule), V, V, V, V, V]
        lib.gm_draw.restype = ctypes.c_int
        _lib = lib
    return _lib


class Drawn(NamedTuple):
    """Per row: the class (int64), the log of its share of what was kept (float32), classes kept (int32)."""

    index: torch.Tensor
    logprob: torch.Tensor
    kept: torch.Tensor


_I32 = (torch.int32,)
_F32 = (torch.float32,)


def gm_draw(logits, u, index, logprob, kept, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    p, ld = _matrix("logits", logits)
    n, device = logits.shape[0], logits.device
    if logits.shape[1] < 1:
        raise ValueError("logits must have a class at least")
    rule = gm_draw_rule(None, None, None, None, 1.0, 0, 1.0, 0.0)
    for name, value, dtypes in (("temperature", temperature, _F32), ("top_k", top_k, _I32), ("top_p", top_p, _F32),
                                ("min_p", min_p, _F32)):
        if isinstance(value, torch.Tensor):
            setattr(rule, name, _vector(name, value, n, device, dtypes))
        else:
            setattr(rule, "all_" + name, value)
    if not isinstance(top_k, torch.Tensor) and rule.all_top_k != top_k:
        raise ValueError(f"top_k must be a whole number of 32 bits, not {top_k}")
    args = [_vector(name, t, n, device, dtypes) for name, t, dtypes in
            (("u", u, _F32), ("index", index, (torch.int64,)), ("logprob", logprob, _F32), ("kept", kept, _I32))]
    with _On(device, stream) as s:
        rc = load().gm_draw(p, n, logits.shape[1], ld, TYPES[logits.dtype], rule, args[0], s, *args[1:])
    if rc:
        raise GmError(rc, "gm_draw")


def draw(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None) -> Drawn:
    """A class a row of ``logits`` (rows x classes; bfloat16, float16 or float32) by the random numbers ``u`` (float32, one
    a row, in [0, 1)). ``temperature`` (0: the largest logit), ``top_k`` (0: off), ``top_p`` (1: off) and ``min_p`` (0: off)
    are numbers, or tensors of one value a row (float32; top_k int32)."""
    _matrix("logits", logits)
    n, device = logits.shape[0], logits.device
    with _On(device, stream):
        out = Drawn(torch.empty(n, dtype=torch.int64, device=device), torch.empty(n, dtype=torch.float32, device=device),
                    torch.empty(n, dtype=torch.int32, device=device))
        gm_draw(logits, u, *out, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, stream=stream)
    return out

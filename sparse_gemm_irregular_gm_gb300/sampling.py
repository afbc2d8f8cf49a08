"""A class drawn from each row of logits over a class table (include/gm_sampling.h), by a temperature, top-k, top-p and
min-p, from given random numbers.

``draw`` allocates the results; ``gm_draw`` writes into the caller's tensors under the C interface's name. Nothing waits
for the GPU. A row that cannot be drawn from has index -1, logprob NaN, kept 0. Arguments are checked and the C interface called
by a compiled extension (csrc/gm_marshal.cpp).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import binding
from .binding import GmError
from .marshal import call, extension

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


def _draw(stream, logits, u, rule, out, make):
    f = extension().draw
    rc, *out = f(logits, u, *rule, *out, make) if stream is None else call(f, stream, logits, u, *rule, *out, make)
    if rc:
        raise GmError(rc, "gm_draw")
    return out


def gm_draw(logits, u, index, logprob, kept, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    _draw(stream, logits, u, (temperature, top_k, top_p, min_p), (index, logprob, kept), False)


def draw(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None) -> Drawn:
    """A class a row of ``logits`` (rows x classes; bfloat16, float16 or float32) by the random numbers ``u`` (float32, one
    a row, in [0, 1)). ``temperature`` (0: the largest logit), ``top_k`` (0: off), ``top_p`` (1: off) and ``min_p`` (0: off)
    are numbers, or tensors of one value a row (float32; top_k int32)."""
    return Drawn(*_draw(stream, logits, u, (temperature, top_k, top_p, min_p), (None, None, None), True))

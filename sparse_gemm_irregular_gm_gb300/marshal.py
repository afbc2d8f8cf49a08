"""The compiled extension that checks tensors, makes results and calls the C interface for the layers and the draw
(csrc/gm_marshal.cpp). There is no fallback: ``extension()`` raises when it has not been built."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import torch

from . import binding
from .losses import _same_device

PATH = os.path.join(binding.HERE, "gm_marshal.so")
FUNCTIONS = ["gm_linear_forward", "gm_linear_backward", "gm_linear_workspace", "gm_norm_forward", "gm_norm_backward",
             "gm_norm_workspace", "gm_draw"]
_ext = None


def extension():
    global _ext
    if _ext is None:
        if not os.path.exists(PATH):
            raise RuntimeError(f"Python extension {PATH} is missing: run __graft_entry__.build() first")
        loader = importlib.machinery.ExtensionFileLoader("gm_marshal", PATH)
        ext = importlib.util.module_from_spec(importlib.util.spec_from_loader("gm_marshal", loader))
        loader.exec_module(ext)
        lib = binding.load()
        ext.init([ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in FUNCTIONS])
        _ext = ext
    return _ext


def call(f, stream, x, *args):
    """f(x, *args) on `stream`, or on the current stream of x's device."""
    if stream is None:
        return f(x, *args)
    if isinstance(x, torch.Tensor):
        _same_device(stream, x.device)
    with torch.cuda.stream(stream):
        return f(x, *args)

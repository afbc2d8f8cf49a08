"""Builds libgm_spgemm.so (CUDA, sm_103a) in-tree with nvcc.

Each translation unit compiles in its own nvcc process (in parallel), then one
nvcc call links the shared library. Objects go to ``_build/`` next to this file. gm_marshal.so, the Python extension of the
layers and the draw, is compiled beside it where torch is installed; the library needs nvcc alone, and is
built whether or not the extension can be.
``build(checked=True)`` builds libgm_spgemm_checked.so instead, with
GM_BOUNDS_CHECK defined: every write of C and of the chunk elements checks its
index first and reports an index out of range as GM_ERR_INTERNAL (objects in
``_build_checked/``). The binding loads it when GM_SPGEMM_CHECKED=1.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgm_spgemm.so")
LIB_CHECKED = os.path.join(HERE, "libgm_spgemm_checked.so")
MARSHAL = os.path.join(HERE, "gm_marshal.so")
MARSHAL_FOR = os.path.join(BUILD, "gm_marshal.for")  # which Python and torch it was compiled for
SOURCES = ["gm_api.cu", "gm_analyze.cu", "gm_scan.cu", "gm_expand.cu", "gm_multisplit.cu", "gm_accum.cu", "gm_rowbitmap.cu",
           "gm_stream.cu", "gm_noalloc.cu", "gm_loss.cu", "gm_loss_prod.cu",
           "gm_loss_skinny.cu", "gm_linear.cu", "gm_norm.cu", "gm_draw.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _newer(path: str, extension: bool) -> bool:
    """Whether path is there and newer than what the library, or the extension, is made from."""
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if (f == "gm_marshal.cpp") == extension]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(f) for f in files)


def made_for() -> str | None:
    """The Python and torch that the extension is compiled for; None without torch, where there is none."""
    if importlib.util.find_spec("torch") is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        import torch
        version = torch.__version__
    return f"python {sys.version}, torch {version}"


def _marshal_is_current(target: str) -> bool:
    if not _newer(MARSHAL, True) or not os.path.exists(MARSHAL_FOR):
        return False
    with open(MARSHAL_FOR) as f:
        return f.read() == target


def build_marshal() -> str:
    """Compile gm_marshal.so, the Python extension that checks tensors and calls the library; needs no CUDA compiler."""
    import sysconfig

    import torch
    at = os.path.dirname(torch.__file__)
    inc = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in inc), os.path.join(CSRC, "gm_marshal.cpp"), "-o", tmp, "-L" + os.path.join(at, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on gm_marshal.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    os.makedirs(os.path.dirname(MARSHAL_FOR), exist_ok=True)
    with open(MARSHAL_FOR, "w") as f:
        f.write(made_for())
    return MARSHAL


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compile (if stale) and return the path of libgm_spgemm.so (or, with checked,
    of libgm_spgemm_checked.so)."""
    lib = LIB_CHECKED if checked else LIB
    bdir = BUILD + "_checked" if checked else BUILD
    target = made_for()
    want_marshal = target is not None and (force or not _marshal_is_current(target))
    with ThreadPoolExecutor(max_workers=1) as ex:
        marshal = ex.submit(build_marshal) if want_marshal else None
        if force or not _newer(lib, False):
            _build_library(lib, bdir, verbose, checked)
        if marshal:
            marshal.result()  # after the library, which needs neither torch nor g++
    return lib


def _build_library(lib: str, bdir: str, verbose: bool, checked: bool) -> None:
    os.makedirs(bdir, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}"]
    if checked:
        flags.append("-DGM_BOUNDS_CHECK")

    def compile_one(src: str) -> str:
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        cmd = [cc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs, "-ldl",  # NVTX loads a profiler's hooks
           "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force=True, verbose=True))

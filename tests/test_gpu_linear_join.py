"""The kernel that joins a product's parts, compiled by itself: where a block of the product gave up, its results are NaN."""
import ctypes
import os
import subprocess

import pytest
import torch

from sparse_gemm_irregular_gm_gb300 import binding, build

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def join(tmp_path_factory):
    binding.load()
    out = str(tmp_path_factory.mktemp("join") / "libjoin.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O1", "-std=c++17", "-shared", "-cudart", "shared", "-Xcompiler", "-fPIC", f"-I{build.INCLUDE}",
                    f"-I{build.CSRC}", os.path.join(HERE, "join_driver.cu"), "-o", out, f"-L{build.HERE}", "-l:libgm_spgemm.so",
                    "-Xlinker", f"-rpath={build.HERE}"], check=True)
    f = ctypes.CDLL(out).join_parts
    V, I64, I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    f.argtypes = [V, I, I64, I64, I64, I, V, V, V, V]
    return f


@pytest.mark.parametrize("rows,outs,splits", [(3, 40, 2), (100, 77, 3), (700, 260, 4)])
@pytest.mark.parametrize("lost_at", [None, 0, 63, 255])
def test_lost_parts_are_no_numbers(join, rows, outs, splits, lost_at):
    ld = (outs + 31) // 32 * 32
    g = torch.Generator(device="cuda").manual_seed(rows)
    acc = torch.randn(splits, rows, ld, device="cuda", generator=g)
    res = torch.randn(rows, outs, device="cuda", generator=g)
    y, z = torch.zeros(rows, outs, device="cuda"), torch.zeros(rows, outs, device="cuda")
    lost = torch.zeros(256, device="cuda", dtype=torch.uint8)
    if lost_at is not None:
        lost[lost_at] = 1
    torch.cuda.synchronize()
    assert join(acc.data_ptr(), splits, rows, outs, ld, 1, res.data_ptr(), y.data_ptr(), z.data_ptr(), lost.data_ptr()) == 0
    if lost_at is None:
        ref = acc.double().sum(0)[:, :outs]
        size = acc.double().abs().sum(0)[:, :outs]
        assert ((z - ref).abs() <= splits * 2.0 ** -24 * size).all()
        assert ((y - (ref.clamp(min=0) + res)).abs() <= (splits + 1) * 2.0 ** -24 * (size + res.abs())).all()
    else:
        assert y.isnan().all() and z.isnan().all()

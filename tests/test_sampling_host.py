"""The draw's C ABI and its binding, without a GPU: exports, layouts, refusals on the host."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from sparse_gemm_irregular_gm_gb300 import sampling

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, OVERFLOW = 0, 1, 3
P = 1 << 20  # refusals come before any array is read, so any address will do


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return sampling.load()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "gm_sampling.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*gm_status\s+(gm_[a-z_]+)\s*\(", src, flags=re.M))
    assert sorted(sampling.EXPORTS) == sorted(names)


def test_struct_is_laid_out_as_in_c(tmp_path):
    c = tmp_path / "sizes.c"
    c.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gm_sampling.h"\nint main(void) { printf("%zu %zu %zu", sizeof(gm_draw_rule), '
                 'offsetof(gm_draw_rule, min_p), offsetof(gm_draw_rule, all_min_p)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    r = sampling.gm_draw_rule
    assert got == [ctypes.sizeof(r), r.min_p.offset, r.all_min_p.offset]


def call(lib, *, rule=(), null_rule=False, **k):
    a = dict(logits=P, n_rows=4, n_classes=10, ld=10, type=1, u=P, index=P, logprob=P, kept=P)
    a.update(k)
    r = dict(temperature=None, top_k=None, top_p=None, min_p=None, all_temperature=1.0, all_top_k=0, all_top_p=1.0, all_min_p=0.0)
    r.update(rule)
    return lib.gm_draw(a["logits"], a["n_rows"], a["n_classes"], a["ld"], a["type"],
                       None if null_rule else sampling.gm_draw_rule(*r.values()), a["u"], None, a["index"], a["logprob"], a["kept"])


@pytest.mark.parametrize("change,status", [
    ({"n_rows": -1}, INVALID), ({"n_classes": 0}, INVALID), ({"ld": 9}, INVALID), ({"type": 3}, INVALID), ({"type": -1}, INVALID),
    ({"logits": None}, INVALID), ({"logits": P + 1}, INVALID), ({"type": 0, "logits": P + 2}, INVALID), ({"u": None}, INVALID),
    ({"u": P + 2}, INVALID), ({"index": None}, INVALID), ({"index": P + 4}, INVALID), ({"logprob": None}, INVALID),
    ({"logprob": P + 1}, INVALID), ({"kept": None}, INVALID), ({"kept": P + 2}, INVALID), ({"null_rule": True}, INVALID),
    ({"n_rows": 1 << 31}, OVERFLOW), ({"n_classes": (1 << 24) + 1, "ld": 1 << 25}, OVERFLOW), ({"ld": 1 << 40}, OVERFLOW)])
def test_bad_arguments(lib, change, status):
    assert call(lib, **change) == status


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("rule", [{"all_temperature": v} for v in (-1.0, NAN, INF, 1e-39)] + [{"all_top_k": -1}] +
                         [{"all_top_p": v} for v in (-0.1, 1.1, NAN)] + [{"all_min_p": v} for v in (-0.1, 1.1, NAN)] +
                         [{"temperature": P + 1}, {"top_k": P + 2}, {"top_p": P + 3}, {"min_p": P + 1}])
def test_bad_rules(lib, rule):
    assert call(lib, rule=rule) == INVALID


@pytest.mark.parametrize("rule", [{"all_temperature": 0.0}, {"all_top_k": 1 << 30}, {"all_top_p": 0.0, "all_min_p": 1.0},
                                  {"all_temperature": -1.0, "temperature": P, "all_top_k": -1, "top_k": P, "all_top_p": 2.0, "top_p": P,
                                   "all_min_p": NAN, "min_p": P}])
def test_no_rows_is_no_work(lib, rule):
    assert call(lib, rule=rule, n_rows=0, logits=None, u=None, index=None, logprob=None, kept=None) == OK


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        sampling.draw(torch.zeros(2, 3), torch.zeros(2))


def test_blocks_of_a_cluster_wait_until_all_have_started():
    """Another block's shared memory may be used only once that block is known to run: the kernel arrives at a barrier of the
    cluster and waits there before its first use. Read from the source: a run cannot show it."""
    src = open(os.path.join(ROOT, "sparse_gemm_irregular_gm_gb300", "csrc", "gm_draw.cu")).read()
    kernel = src[src.index("k_draw(const __grid_constant__"):src.index("// ---- host")]
    kernel = re.sub(r"//[^\n]*", "", kernel)
    uses = [kernel.find(f + "(") for f in ("put_remote_u64", "add_remote_u32", "remote_u32", "remote_u64", "map_to_rank", "cluster_sync_all")]
    first = min(i for i in uses if i >= 0)
    arrive, wait = kernel.find("cluster_arrive()"), kernel.find("cluster_wait()")
    assert 0 <= arrive < wait < first


@pytest.mark.parametrize("missing", [(0,), (1,), (2,), (0, 1), (0, 2), (1, 2), (0, 1, 2)])
def test_binding_refuses_results_that_are_missing(lib, missing):
    out = [torch.zeros(2, dtype=t) for t in (torch.int64, torch.float32, torch.int32)]
    for i in missing:
        out[i] = None
    with pytest.raises(ValueError, match="index, logprob and kept"):
        sampling.gm_draw(torch.zeros(2, 3), torch.zeros(2), *out)

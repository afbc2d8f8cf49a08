"""The losses' C ABI and its binding, without a GPU: exports, layouts, refusals on the host."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from sparse_gemm_irregular_gm_gb300 import binding, losses

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, DIM, OVERFLOW = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return losses.load()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "gm_losses.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*gm_status\s+(gm_[a-z_]+)\s*\(", src, flags=re.M))
    assert sorted(losses.EXPORTS) == sorted(names)
    for n in names:
        assert hasattr(lib, n), n


def test_structs_are_laid_out_as_in_c(tmp_path):
    c = tmp_path / "sizes.c"
    c.write_text('#include <stdio.h>\n#include "gm_losses.h"\nint main(void) { printf("%zu %zu %zu %zu %zu", '
                 'sizeof(gm_logits), sizeof(gm_labels), sizeof(gm_loss_config), offsetof(gm_logits, type), '
                 'offsetof(gm_loss_config, workspace_bytes)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(losses.gm_logits), ctypes.sizeof(losses.gm_labels), ctypes.sizeof(losses.gm_loss_config),
                   losses.gm_logits.type.offset, losses.gm_loss_config.workspace_bytes.offset]


# Refusals come before any array is read, so any address will do.
P = 1 << 20


def logits(**k):
    a = dict(n_rows=4, n_classes=10, dim=8, h=P, h_ld=8, w=P, w_ld=8, type=losses.GM_LOSS_BF16)
    a.update(k)
    return losses.gm_logits(*a.values())


def labels(**k):
    a = dict(target=P, ignore_index=-100, target32=0)
    a.update(k)
    return losses.gm_labels(*a.values())


def config(**k):
    a = dict(workspace_cap_bytes=0, flags=0, workspace=None, workspace_bytes=0)
    a.update(k)
    return losses.gm_loss_config(*a.values())


def csr(**k):
    a = dict(n_rows=4, n_cols=10, nnz=5, row_ptr=P, col_idx=P, vals=P)
    a.update(k)
    return binding.gm_csr(*a.values())


BAD_LOGITS = [({"n_rows": -1}, INVALID), ({"n_classes": 0}, INVALID), ({"dim": 0}, INVALID), ({"type": 3}, INVALID),
              ({"h": None}, INVALID), ({"w": None}, INVALID), ({"h": P + 1}, INVALID), ({"w_ld": 7}, INVALID),
              ({"h_ld": 7}, INVALID), ({"type": losses.GM_LOSS_F32, "w": P + 2}, INVALID),
              ({"n_rows": 1 << 31}, OVERFLOW), ({"n_classes": 1 << 31}, OVERFLOW),
              ({"dim": 1 << 25, "h_ld": 1 << 25, "w_ld": 1 << 25}, OVERFLOW)]


@pytest.mark.parametrize("change,status", BAD_LOGITS)
def test_bad_logits(lib, change, status):
    z = logits(**change)
    assert lib.gm_xent_forward(z, labels(), None, None, P, P) == status
    assert lib.gm_xent_backward(z, labels(), None, None, P, P, None, P, 1 << 26, P, 1 << 26) == status
    assert lib.gm_distill_forward(z, csr(), 1, 0, 1.0, None, None, None, P, P, None, None) == status
    assert lib.gm_loss_workspace(z, -1, 0, None, ctypes.c_int64()) == status


@pytest.mark.parametrize("change", [{"workspace_cap_bytes": -1}, {"flags": 2}, {"workspace": P + 128, "workspace_bytes": 1 << 20},
                                    {"workspace": P, "workspace_bytes": -1}])
def test_bad_config(lib, change):
    assert lib.gm_xent_forward(logits(), labels(), config(**change), None, P, P) == INVALID


@pytest.mark.parametrize("change", [{"target": None}, {"target": P + 4}, {"target32": 2}])
def test_bad_labels(lib, change):
    assert lib.gm_xent_forward(logits(), labels(**change), None, None, P, P) == INVALID


def test_missing_results_and_gradients(lib):
    z, t = logits(), labels()
    assert lib.gm_xent_forward(None, t, None, None, P, P) == INVALID
    assert lib.gm_xent_forward(z, None, None, None, P, P) == INVALID
    assert lib.gm_xent_forward(z, t, None, None, None, P) == INVALID
    assert lib.gm_xent_forward(z, t, None, None, P, None) == INVALID
    assert lib.gm_xent_forward(z, t, None, None, P + 2, P) == INVALID
    back = lambda lse=P, g=P, dh=P, dh_ld=8, dw=P, dw_ld=8: lib.gm_xent_backward(  # noqa: E731
        z, t, None, None, lse, g, None, dh, dh_ld, dw, dw_ld)
    assert back(lse=None) == back(g=None) == back(dh=None, dw=None) == back(dh_ld=7) == back(dw_ld=7) == INVALID
    assert back(dh=P + 1) == back(dw=P + 1) == back(lse=P + 2) == INVALID
    assert lib.gm_distill_forward(z, csr(), 1, 0, 1.0, None, None, None, P, P, P, P) == INVALID  # loss without labels
    assert lib.gm_distill_forward(z, csr(), 1, 0, 1.0, t, None, None, P, P, None, P) == INVALID
    assert lib.gm_loss_workspace(z, -1, 2, None, ctypes.c_int64()) == INVALID
    assert lib.gm_loss_workspace(z, -1, 0, None, None) == INVALID


@pytest.mark.parametrize("change,status", [({"n_rows": 5}, DIM), ({"n_cols": 9}, DIM), ({"nnz": -1}, INVALID),
                                           ({"row_ptr": None}, INVALID), ({"col_idx": None}, INVALID),
                                           ({"vals": None}, INVALID), ({"row_ptr": P + 4}, INVALID), ({"col_idx": P + 2}, INVALID)])
def test_bad_teacher(lib, change, status):
    assert lib.gm_distill_forward(logits(), csr(**change), 1, 0, 1.0, None, None, None, P, P, None, None) == status


@pytest.mark.parametrize("value_type,index_type,temperature", [(2, 0, 1.0), (1, 4, 1.0), (1, 0, 0.0), (1, 0, -1.0), (1, 0, float("nan")),
                                                               (1, 0, float("inf")), (1, 0, 1e-45)])
def test_bad_teacher_types_and_temperature(lib, value_type, index_type, temperature):
    assert lib.gm_distill_forward(logits(), csr(), value_type, index_type, temperature, None, None, None, P, P, None, None) == INVALID


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    h, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        losses.xent_forward(h, w, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        losses.distill_forward(h.float(), w.float(), None)


def test_distillation_checks_the_teachers_sizes():
    t = binding.DeviceCSR(3, 5, None, None, None)
    with pytest.raises(binding.GmError):
        losses.distillation(torch.zeros(2, 8), torch.zeros(5, 8), t)


def test_distillation_refuses_a_teacher_that_wants_a_gradient():
    val = torch.zeros(2, requires_grad=True)
    t = binding.DeviceCSR(2, 5, torch.tensor([0, 1, 2]), torch.tensor([0, 1], dtype=torch.int32), val)
    h, w = torch.zeros(2, 8), torch.zeros(5, 8)
    with pytest.raises(ValueError, match="detach"):
        losses.distillation(h, w, t)
    for call in (lambda: losses.distillation(h, w, binding.DeviceCSR(2, 5, t.row_ptr, t.col, val.detach())),
                 lambda: torch.no_grad()(losses.distillation)(h, w, t)):
        with pytest.raises(ValueError, match="CUDA tensor"):  # what tensors here are refused for
            call()


def test_temperatures_whose_reciprocal_is_finite_but_not_its_exponent(lib):
    for t in (3.5e-39, 4.2e-39):
        assert lib.gm_distill_forward(logits(), csr(), 1, 0, t, None, None, None, P, P, None, None) == INVALID

"""The layers' C ABI and its binding, without a GPU: exports, layouts, refusals on the host; the oracle against differences."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import layer_oracle
from sparse_gemm_irregular_gm_gb300 import layers

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, OVERFLOW = 0, 1, 3
P = 1 << 20  # refusals come before any array is read, so any address will do
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return layers.load()


def test_exports_every_declared_symbol(lib):
    src = open(os.path.join(ROOT, "include", "gm_layers.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*gm_status\s+(gm_[a-z_]+)\s*\(", src, flags=re.M))
    assert sorted(layers.EXPORTS) == sorted(names)


def test_structs_are_laid_out_as_in_c(tmp_path):
    c = tmp_path / "sizes.c"
    structs = [n for n in ("gm_layer_config", "gm_norm", "gm_norm_grads", "gm_linear") if hasattr(layers, n)]
    fields = [(n, getattr(layers, n)._fields_[-1][0]) for n in structs]
    args = ", ".join(f"sizeof({n}), offsetof({n}, {f})" for n, f in fields)
    c.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gm_layers.h"\nint main(void) { size_t v[] = {%s}; '
                 'for (size_t i = 0; i < sizeof v / sizeof v[0]; ++i) printf("%%zu ", v[i]); return 0; }\n' % args)
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(c), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [v for n, f in fields for v in (ctypes.sizeof(getattr(layers, n)), getattr(getattr(layers, n), f).offset)]


def norm(**k):
    a = dict(n_rows=4, dim=8, type=1, norm=0, gate_kind=1, scale=1.0, eps=1e-6, x=P, x_ld=8, f=P, f_ld=8, after=P, after_bias=P,
             gate=P, gate_ld=0, before=P, before_bias=P)
    a.update(k)
    return layers.gm_norm(*a.values())


def grads(**k):
    a = dict(x=P, x_ld=8, f=P, f_ld=8, gate=P, gate_ld=8, after=P, after_bias=P, before=P, before_bias=P)
    a.update(k)
    return layers.gm_norm_grads(*a.values())


@pytest.mark.parametrize("change,status", [
    ({"n_rows": -1}, INVALID), ({"dim": 0}, INVALID), ({"type": 3}, INVALID), ({"norm": 2}, INVALID), ({"gate_kind": 3}, INVALID),
    ({"gate_kind": -1}, INVALID), ({"scale": NAN}, INVALID), ({"scale": INF}, INVALID), ({"eps": -1e-9}, INVALID), ({"eps": NAN}, INVALID),
    ({"x": None}, INVALID), ({"x": P + 1}, INVALID), ({"x_ld": 7}, INVALID), ({"f": None}, INVALID), ({"f_ld": 7}, INVALID),
    ({"f": P + 1}, INVALID), ({"after": None}, INVALID), ({"before": None}, INVALID), ({"gate": None}, INVALID), ({"gate": P + 1}, INVALID),
    ({"gate_kind": 2, "gate_ld": 7}, INVALID), ({"after": P + 1}, INVALID), ({"before_bias": P + 1}, INVALID), ({"type": 0, "x": P + 2}, INVALID),
    ({"n_rows": 1 << 31}, OVERFLOW), ({"dim": 1 << 25, "x_ld": 1 << 25, "f_ld": 1 << 25}, OVERFLOW), ({"x_ld": 1 << 40}, OVERFLOW),
    ({"f_ld": 1 << 40}, OVERFLOW)])
def test_bad_norms(lib, change, status):
    n = norm(**change)
    assert lib.gm_norm_forward(n, None, P, 1 << 26, P, 1 << 26, P) == status
    assert lib.gm_norm_backward(n, None, None, P, P, 1 << 26, P, 1 << 26, grads(x_ld=1 << 26, f_ld=1 << 26)) == status
    assert lib.gm_norm_workspace(n, ctypes.c_int64()) == status


def test_bad_norm_results(lib):
    f = lib.gm_norm_forward
    assert f(None, None, P, 8, P, 8, P) == INVALID
    assert f(norm(), None, None, 0, P, 8, P) == INVALID  # f is added to something
    assert f(norm(), None, P, 8, None, 0, P) == INVALID
    assert f(norm(before=None, before_bias=None), None, P, 8, P, 8, P) == INVALID
    assert f(norm(), None, P, 7, P, 8, P) == INVALID
    assert f(norm(), None, P, 8, P, 7, P) == INVALID
    assert f(norm(), None, P, 16, P, 8, P) == INVALID  # x itself, at another stride
    assert f(norm(), None, P + 1, 8, P, 8, P) == INVALID
    assert f(norm(), None, P, 8, P, 8, P + 4) == INVALID
    assert f(norm(), None, P, 1 << 40, P, 8, P) == OVERFLOW
    assert lib.gm_norm_workspace(norm(), None) == INVALID
    none = dict(x=None, f=None, gate=None, after=None, after_bias=None, before=None, before_bias=None)
    b = lambda n, g, **k: lib.gm_norm_backward(n, k.get("cfg"), None, k.get("stats", P), P, 8, k.get("gy", P), 8, g)  # noqa: E731
    assert b(norm(), None) == INVALID
    assert b(norm(), grads(**none)) == INVALID
    assert b(norm(), grads(), stats=None) == INVALID
    assert b(norm(), grads(), stats=P + 8) == INVALID
    assert b(norm(), grads(x_ld=7)) == INVALID
    assert b(norm(gate_kind=2, gate_ld=8), grads(gate_ld=7)) == INVALID
    assert b(norm(gate_kind=0), grads()) == INVALID
    assert b(norm(after_bias=None), grads()) == INVALID
    assert b(norm(before_bias=None), grads()) == INVALID
    assert b(norm(before=None, before_bias=None), grads(before=None, before_bias=None)) == INVALID  # a gradient by y
    assert b(norm(), grads(after=P + 1)) == INVALID
    assert b(norm(), grads(), cfg=layers.gm_layer_config(P + 128, 1 << 20)) == INVALID
    assert b(norm(), grads(), cfg=layers.gm_layer_config(P, -1)) == INVALID


def test_no_rows_need_no_workspace(lib):
    need = ctypes.c_int64(7)
    assert lib.gm_norm_workspace(norm(n_rows=0, x=None, f=None), need) == OK and need.value == 0
    assert lib.gm_norm_forward(norm(n_rows=0, x=None, f=None), None, None, 8, None, 8, None) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        layers.residual_norm(x, x, before=torch.ones(8))


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("gate", ["vector", "matrix"])
def test_oracle_of_the_norms_against_differences(norm, gate):
    r = np.random.default_rng(1)
    a = dict(x=r.normal(size=(4, 6)), f=r.normal(size=(4, 6)), after=r.normal(size=6), after_bias=r.normal(size=6),
             gate=r.normal(size=6 if gate == "vector" else (4, 6)), before=r.normal(size=6), before_bias=r.normal(size=6))
    gx, gy = r.normal(size=(4, 6)), r.normal(size=(4, 6))
    ref = layer_oracle.residual_norm(**a, gx=gx, gy=gy, norm=norm, scale=0.6)

    def total(b):
        o = layer_oracle.residual_norm(**b, norm=norm, scale=0.6)
        return (o["x"][0] * gx).sum() + (o["y"][0] * gy).sum()

    for name, t in a.items():
        slope = np.zeros_like(t)
        for i in np.ndindex(*t.shape):
            up, down = dict(a, **{name: t.copy()}), dict(a, **{name: t.copy()})
            up[name][i] += 1e-6
            down[name][i] -= 1e-6
            slope[i] = (total(up) - total(down)) / 2e-6
        assert np.allclose(slope, ref["d" + name][0], rtol=1e-5, atol=1e-7), name


def linear(**k):
    a = dict(n_rows=4, dim=8, n_outs=6, x=P, x_ld=8, w=P, w_ld=8, type=1, activation=2)
    a.update(k)
    return layers.gm_linear(*a.values())


@pytest.mark.parametrize("change,status", [
    ({"n_rows": -1}, INVALID), ({"dim": 0}, INVALID), ({"n_outs": 0}, INVALID), ({"type": 3}, INVALID), ({"activation": 5}, INVALID),
    ({"activation": -1}, INVALID), ({"x": None}, INVALID), ({"w": None}, INVALID), ({"x": P + 1}, INVALID), ({"w": P + 1}, INVALID),
    ({"x_ld": 7}, INVALID), ({"w_ld": 7}, INVALID), ({"type": 0, "w": P + 2}, INVALID), ({"n_rows": 1 << 31}, OVERFLOW),
    ({"dim": 1 << 25, "x_ld": 1 << 25, "w_ld": 1 << 25}, OVERFLOW), ({"n_outs": 1 << 25}, OVERFLOW), ({"x_ld": 1 << 40}, OVERFLOW)])
def test_bad_products(lib, change, status):
    p = linear(**change)
    assert lib.gm_linear_forward(p, None, None, P, P, 1 << 26, P, 1 << 26, None, 0) == status
    assert lib.gm_linear_backward(p, None, None, P, 1 << 26, P, 1 << 26, P, 1 << 26, P, 1 << 26, P) == status
    assert lib.gm_linear_workspace(p, 0, ctypes.c_int64()) == status


def test_bad_product_arrays(lib):
    f = lambda bias=P, r=P, r_ld=6, y=P + 4096, y_ld=6, z=None, z_ld=0, cfg=None: lib.gm_linear_forward(  # noqa: E731
        linear(), cfg, None, bias, r, r_ld, y, y_ld, z, z_ld)
    for bad in (dict(bias=P + 1), dict(r=P + 1), dict(r_ld=5), dict(y=None), dict(y=P + 1), dict(y_ld=5), dict(z=P + 1, z_ld=6),
                dict(z=P, z_ld=5), dict(y=P, y_ld=7), dict(cfg=layers.gm_layer_config(P + 128, 1 << 20)), dict(cfg=layers.gm_layer_config(P, -1))):
        assert f(**bad) == INVALID, bad
    assert f(y_ld=1 << 40) == OVERFLOW
    b = lambda g=P, g_ld=6, z=P, z_ld=6, dx=P, dx_ld=8, dw=P, dw_ld=8, db=P: lib.gm_linear_backward(  # noqa: E731
        linear(), None, None, g, g_ld, z, z_ld, dx, dx_ld, dw, dw_ld, db)
    for bad in (dict(g=None), dict(g=P + 1), dict(g_ld=5), dict(z=None), dict(z_ld=5), dict(dx=P + 1), dict(dx_ld=7), dict(dw_ld=7),
                dict(db=P + 1), dict(dx=None, dw=None, db=None)):
        assert b(**bad) == INVALID, bad
    assert lib.gm_linear_workspace(linear(), 2, ctypes.c_int64()) == INVALID
    assert lib.gm_linear_workspace(linear(), 0, None) == INVALID
    need = ctypes.c_int64(7)
    assert lib.gm_linear_workspace(linear(n_rows=0, x=None), 1, need) == OK and need.value == 0
    assert lib.gm_linear_forward(linear(n_rows=0, x=None), None, None, None, None, 0, None, 6, None, 0) == OK


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_oracle_of_the_activations_against_differences(act):
    z = np.linspace(-6, 6, 481) + 0.003
    a, s = layer_oracle.act(z, act)
    up, down = layer_oracle.act(z + 1e-6, act)[0], layer_oracle.act(z - 1e-6, act)[0]
    assert np.allclose((up - down) / 2e-6, s, atol=1e-8)


def test_every_struct_of_the_header_is_bound():
    src = open(os.path.join(ROOT, "include", "gm_layers.h")).read()
    names = re.findall(r"^typedef struct (gm_\w+) \{", src, flags=re.M)
    assert len(names) == 4
    for n in names:
        assert issubclass(getattr(layers, n), ctypes.Structure)

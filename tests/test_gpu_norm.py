"""The norms around a residual on the GPU, every element against 64 bits within derived bounds."""
import itertools

import numpy as np
import pytest
import torch

from layer_oracle import close, norm_ops, residual_norm
from sparse_gemm_irregular_gm_gb300 import layers
from sparse_gemm_irregular_gm_gb300.binding import GmError

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def make(rows, dim, kind, *, after=True, after_bias=True, gate="vector", before=True, before_bias=True, f=True, seed=0, wide=0, offset=0):
    """Inputs on the GPU; wide: columns between rows that belong to none, offset: elements before the first."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7)

    def matrix(std=1.0, mean=0.0):
        big = torch.full((rows * (dim + wide) + offset,), float("nan"), device="cuda", dtype=TYPES[kind])
        m = big[offset:].view(rows, dim + wide)[:, :dim]
        m.copy_(torch.randn(rows, dim, generator=g, device="cuda") * std + mean)
        return m

    def vector(std, mean=0.0):
        big = torch.empty(dim + offset, device="cuda", dtype=TYPES[kind])
        big[offset:] = torch.randn(dim, generator=g, device="cuda") * std + mean
        return big[offset:]

    x = matrix(3.0, 0.5)
    rule = {}
    if f:
        if after:
            rule["after"] = vector(0.2, 1.0)
            if after_bias:
                rule["after_bias"] = vector(0.3)
        if gate:
            rule["gate"] = vector(0.2, 0.5) if gate == "vector" else matrix(0.3, 0.5)
    if before:
        rule["before"] = vector(0.2, 1.0)
        if before_bias:
            rule["before_bias"] = vector(0.3)
    return x, matrix(0.7) if f else None, matrix(0.1), matrix(0.1) if before else None, rule


def wide_of(t):
    return None if t is None else t.double().cpu().numpy()


def check(x, f, gx, gy, rule, kind, got):
    ref = residual_norm(wide_of(x), wide_of(f), wide_of(gx), wide_of(gy),
                        **{k: wide_of(v) if isinstance(v, torch.Tensor) else v for k, v in rule.items()})
    rows, dim = x.shape
    for name, t in got.items():
        value, size = ref[name]
        assert t.shape == value.shape and t.dtype == x.dtype
        close(wide_of(t), value, size, norm_ops(dim, rows if value.ndim == 1 else 0), kind)


def both(x, f, gx, gy, rule, kind, **k):
    o = layers.residual_norm_forward(x, f, **rule)
    got = {} if f is None else {"x": o.x}
    if o.y is not None:
        got["y"] = o.y
    d = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule, **k)
    got.update({"d" + n: t for n, t in d._asdict().items() if t is not None})
    check(x, f, gx, gy, rule, kind, got)
    return got


SHAPES = [(1, 1), (3, 7), (1, 4096), (5, 8), (2, 31), (33, 64), (130, 256), (17, 257), (700, 512), (600, 1032), (40, 1030),
          (9, 2048), (520, 2056), (3, 4095), (5, 4097), (6, 8192), (35, 8193), (2, 20001)]


@pytest.mark.parametrize("rows,dim", SHAPES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_sizes(rows, dim, kind, norm):
    x, f, gx, gy, rule = make(rows, dim, kind, gate="vector" if dim % 2 else "matrix", seed=rows + dim)
    both(x, f, gx, gy, dict(rule, norm=norm, scale=0.7), kind)


PARTS = [p for p in itertools.product([False, True], [None, "vector", "matrix"], [False, True], [False, True]) if True]


@pytest.mark.parametrize("after,gate,before,bias", PARTS)
@pytest.mark.parametrize("dim", [96, 4100])
def test_parts(after, gate, before, bias, dim):
    x, f, gx, gy, rule = make(37, dim, "bf16", after=after, after_bias=bias, gate=gate, before=before, before_bias=bias)
    got = both(x, f, gx, gy, dict(rule, norm="layer", scale=-1.5), "bf16")
    assert set(got) == {"x", "dx", "df"} | ({"y"} if before else set()) | {"d" + k for k in rule}


@pytest.mark.parametrize("rows,dim", [(1, 512), (700, 520), (33, 1024), (305, 1032), (9, 2056), (310, 4096), (5, 4104), (6, 8192), (3, 8184)])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("after,gate,before", [(True, "vector", True), (True, None, True), (False, "vector", True), (True, "vector", False), (False, None, True)])
def test_root_mean_squares_without_biases(rows, dim, kind, after, gate, before):
    x, f, gx, gy, rule = make(rows, dim, kind, after=after, after_bias=False, gate=gate, before=before, before_bias=False, seed=dim)
    both(x, f, gx, gy, dict(rule, scale=0.6), kind)
    if before:
        o = layers.residual_norm_forward(x, f, scale=0.6, **rule)
        d = layers.residual_norm_backward(x, f, None, gy, o.stats, scale=0.6, **rule)  # no gradient by x' but through y
        check(x, f, None, gy, dict(rule, scale=0.6), kind, {"d" + n: t for n, t in d._asdict().items() if t is not None})


@pytest.mark.parametrize("dim", [512, 4096])
def test_wide_strides_without_biases(dim):
    x, f, gx, gy, rule = make(19, dim, "bf16", after_bias=False, before_bias=False, wide=24, offset=8)
    both(x, f, gx, gy, rule, "bf16")


def test_offsets_past_32_bits():
    rows, dim = 540000, 4096  # 2.2e9 elements
    x, f = (torch.zeros(rows, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sx, sf, sgx, sgy, rule = make(3, dim, "bf16", after_bias=False, before_bias=False)
    x[-3:], f[-3:] = sx, sf
    o = layers.residual_norm_forward(x, f, **rule)
    ref = layers.residual_norm_forward(sx, sf, **rule)
    assert torch.equal(o.x[-3:], ref.x) and torch.equal(o.y[-3:], ref.y) and (o.x[:-3] == 0).all()
    gx, gy = (torch.zeros(rows, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gx[-3:], gy[-3:] = sgx, sgy
    d = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule)
    e = layers.residual_norm_backward(sx, sf, sgx, sgy, ref.stats, **rule)
    assert torch.equal(d.x[-3:], e.x) and torch.equal(d.f[-3:], e.f) and (d.x[:-3] == 0).all()
    check(sx, sf, sgx, sgy, rule, "bf16", {"dafter": d.after, "dbefore": d.before, "dgate": d.gate})


@pytest.mark.parametrize("dim", [40, 5000])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_norm_alone(dim, norm):
    x, _, gx, gy, rule = make(21, dim, "f32", f=False)
    both(x, None, gx, gy, dict(rule, norm=norm), "f32")
    o = layers.residual_norm_forward(x, **rule)
    assert o.x is x
    d = layers.residual_norm_backward(x, None, None, gy, o.stats, **rule)  # no gradient by x' but through y
    check(x, None, None, gy, rule, "f32", {"dx": d.x, "dbefore": d.before, "dbefore_bias": d.before_bias})


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("wide,offset", [(8, 0), (3, 0), (0, 1), (5, 2)])
@pytest.mark.parametrize("dim", [64, 77, 4104])
def test_strides(kind, wide, offset, dim):
    x, f, gx, gy, rule = make(19, dim, kind, gate="matrix", wide=wide, offset=offset)
    both(x, f, gx, gy, dict(rule, norm="layer"), kind)


@pytest.mark.parametrize("dim", [136, 4104])
@pytest.mark.parametrize("wide,offset", [(0, 0), (5, 0), (8, 8)])
def test_results_into_the_callers_rows(dim, wide, offset):
    rows = 11
    x, f, gx, gy, rule = make(rows, dim, "bf16", gate="matrix")

    def room():
        big = torch.full((rows * (dim + wide) + offset + 32,), 7.0, device="cuda", dtype=torch.bfloat16)
        return big, big[offset:offset + rows * (dim + wide)].view(rows, dim + wide)[:, :dim]

    bigs, mats = zip(*[room() for _ in range(5)])
    stats = torch.empty(rows, 4, device="cuda")
    layers.gm_norm_forward(x, f, mats[0], mats[1], stats, **rule)
    vec = [torch.empty(dim, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    layers.gm_norm_backward(x, f, stats, gx, gy, layers.NormGrads(mats[2], mats[3], mats[4], *vec), **rule)
    check(x, f, gx, gy, rule, "bf16", dict(zip(["x", "y", "dx", "df", "dgate", "dafter", "dafter_bias", "dbefore", "dbefore_bias"],
                                               [*mats, *vec])))
    for big, m in zip(bigs, mats):  # nothing else was written
        m.fill_(7.0)
        assert (big == 7.0).all()


@pytest.mark.parametrize("dim", [512, 6000])
def test_in_place_residual(dim):
    x, f, gx, gy, rule = make(50, dim, "bf16")
    o = layers.residual_norm_forward(x, f, **rule)
    x2, y = x.clone(), torch.empty_like(x)
    layers.gm_norm_forward(x2, f, x2, y, **rule)
    assert torch.equal(x2, o.x) and torch.equal(y, o.y)


def test_one_gradient_at_a_time_and_runs_repeat():
    x, f, gx, gy, rule = make(300, 520, "bf16")
    o = layers.residual_norm_forward(x, f, **rule)
    whole = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule)
    again = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule)
    for name, t in whole._asdict().items():
        assert torch.equal(t, getattr(again, name)), name
        one = layers.residual_norm_backward(x, f, gx, gy, o.stats, need=[name], **rule)
        assert [k for k, v in one._asdict().items() if v is not None] == [name]
        assert torch.equal(t, getattr(one, name)), name


@pytest.mark.parametrize("dim", [24, 4200])
def test_rows_that_are_all_zero_or_not_finite_stay_alone(dim):
    x, f, gx, gy, rule = make(6, dim, "f32", after_bias=False, before_bias=False)
    clean = layers.residual_norm_forward(x, f, norm="layer", **rule)
    x[1], f[1] = 0, 0
    x[3, dim // 2] = float("inf")
    f[4, 0] = float("nan")
    o = layers.residual_norm_forward(x, f, norm="layer", **rule)
    assert (o.x[1] == 0).all() and (o.y[1] == 0).all()  # 0 / sqrt(eps)
    assert o.y[3].isnan().any() and o.y[4].isnan().all()
    for r in (0, 2, 5):
        assert torch.equal(o.x[r], clean.x[r]) and torch.equal(o.y[r], clean.y[r])
    d = layers.residual_norm_backward(x, f, gx, gy, o.stats, norm="layer", **rule)
    assert d.x[[0, 1, 2, 5]].isfinite().all() and d.f[[0, 1, 2, 5]].isfinite().all()


def test_no_rows():
    x, f, gx, gy, rule = make(0, 48, "bf16")
    o = layers.residual_norm_forward(x, f, **rule)
    assert o.x.shape == o.y.shape == (0, 48)
    d = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule)
    assert d.x.shape == (0, 48) and (d.after == 0).all() and (d.gate == 0).all() and (d.before_bias == 0).all()


@pytest.mark.parametrize("norm,gate", [("rms", "vector"), ("layer", "matrix")])
def test_autograd_against_differences(norm, gate):
    x, f, gx, gy, rule = make(5, 12, "f32", gate=gate, seed=3)
    leaves = {"x": x, "f": f, **rule}
    leaves = {k: v.clone().requires_grad_() for k, v in leaves.items()}

    def total(**v):
        ref = residual_norm(v.pop("x"), v.pop("f"), norm=norm, scale=0.9, **v)
        return (ref["x"][0] * wide_of(gx)).sum() + (ref["y"][0] * wide_of(gy)).sum()

    xo, yo = layers.residual_norm(leaves["x"], leaves["f"], norm=norm, scale=0.9, **{k: leaves[k] for k in rule})
    ((xo * gx).sum() + (yo * gy).sum()).backward()
    step = 1e-6
    for name, t in leaves.items():
        base = {k: wide_of(v.detach()) for k, v in leaves.items()}
        slope = np.zeros(t.shape)
        for i in np.ndindex(*t.shape):
            up, down = ({k: v.copy() for k, v in base.items()} for _ in range(2))
            up[name][i] += step
            down[name][i] -= step
            slope[i] = (total(**up) - total(**down)) / (2 * step)
        # differences of a smooth function: about step^2 off, and the 64-bit sums' rounding over the step
        assert np.allclose(t.grad.double().cpu().numpy(), slope, rtol=1e-4, atol=1e-5 * np.abs(slope).max()), name


def test_autograd_asks_only_for_what_is_wanted():
    x, f, gx, gy, rule = make(8, 64, "bf16")
    f.requires_grad_()
    xo, yo = layers.residual_norm(x, f, **rule)
    yo.sum().backward()  # an expanded gradient; none by x'
    ref = layers.residual_norm_backward(x, f.detach(), None, torch.ones_like(x), layers.residual_norm_forward(x, f.detach(), **rule).stats,
                                        need=["f"], **rule)
    assert torch.equal(f.grad, ref.f)
    y = layers.residual_norm(x.clone().requires_grad_(), before=rule["before"])
    assert y[0].shape == y[1].shape and y[1].grad_fn is not None
    leaf = x.clone().requires_grad_()
    xo, none = layers.residual_norm(leaf, f.detach(), gate=rule["gate"])  # no norm before the next block
    xo.backward(gx)
    assert none is None and torch.equal(leaf.grad, gx)


def test_other_stream_and_graph():
    x, f, gx, gy, rule = make(64, 1024, "bf16")
    o = layers.residual_norm_forward(x, f, **rule)
    d = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p = layers.residual_norm_forward(x, f, stream=s, **rule)
    e = layers.residual_norm_backward(x, f, gx, gy, p.stats, stream=s, **rule)
    s.synchronize()
    assert torch.equal(o.y, p.y) and all(torch.equal(a, b) for a, b in zip(d, e))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = layers.residual_norm_forward(x, f, **rule)
        h = layers.residual_norm_backward(x, f, gx, gy, q.stats, **rule)
    x2, f2, gx2, gy2, _ = make(64, 1024, "bf16", seed=5)
    for a, b in ((x, x2), (f, f2), (gx, gx2), (gy, gy2)):
        a.copy_(b)
    g.replay()
    o = layers.residual_norm_forward(x, f, **rule)
    d = layers.residual_norm_backward(x, f, gx, gy, o.stats, **rule)
    assert torch.equal(o.y, q.y) and all(torch.equal(a, b) for a, b in zip(d, h))


def test_refusals_of_the_device_side_arguments():
    x, f, gx, gy, rule = make(4, 16, "bf16")
    with pytest.raises(ValueError):
        layers.residual_norm_forward(x, f.float(), **rule)
    with pytest.raises(ValueError):
        layers.residual_norm_forward(x, f[:, :8], **rule)
    with pytest.raises(ValueError):
        layers.residual_norm_forward(x.t(), **rule)
    with pytest.raises(ValueError):
        layers.residual_norm_forward(x, norm="rms")
    with pytest.raises(ValueError):
        layers.residual_norm_forward(x, None, gate=rule["gate"], before=rule["before"])
    with pytest.raises(GmError):
        layers.residual_norm_forward(x, f, scale=float("nan"), **rule)
    with pytest.raises(GmError):
        layers.residual_norm_forward(x, f, eps=-1.0, **rule)


# Rows of more than 8192 are walked; the forms between 4096 and 8192 hold 16 columns a thread.
@pytest.mark.parametrize("dim", [8200, 8201])
def test_walked_rows_as_the_others(dim):
    for norm in ("rms", "layer"):
        test_norm_alone(dim, norm)
    test_in_place_residual(dim)
    test_rows_that_are_all_zero_or_not_finite_stay_alone(dim)
    test_results_into_the_callers_rows(dim, 5, 0)
    test_results_into_the_callers_rows(dim, 8, 8)
    for after, gate, before, bias in PARTS:
        test_parts(after, gate, before, bias, dim)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,dim", [(1, 4097), (309, 4100), (6, 5000), (4, 6001), (7, 8191), (3, 8192), (5, 8193)])
@pytest.mark.parametrize("norm,gate", [("layer", "vector"), ("rms", "matrix"), ("layer", None)])
def test_long_rows_in_every_form(rows, dim, kind, norm, gate):
    x, f, gx, gy, rule = make(rows, dim, kind, gate=gate, seed=dim)
    both(x, f, gx, gy, dict(rule, norm=norm, scale=0.7), kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("wide,offset", [(8, 0), (3, 0), (0, 1), (5, 2)])
@pytest.mark.parametrize("dim", [8190, 8200])
def test_strides_of_long_rows(kind, wide, offset, dim):
    test_strides(kind, wide, offset, dim)


def test_an_eps_that_32_bits_take_to_zero_is_refused():
    x, before = torch.zeros(2, 16, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(ValueError, match="eps"):
        layers.residual_norm_forward(x, before=before, eps=1e-46)
    assert (layers.residual_norm_forward(x, before=before, eps=2e-45).y == 0).all()

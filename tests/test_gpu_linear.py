"""The product with bias, activation and residual on the GPU, every element against 64 bits within derived bounds."""
import math

import numpy as np
import pytest
import torch

import layer_oracle
from layer_oracle import EPS32, HALF, LEAST
from sparse_gemm_irregular_gm_gb300 import layers
from sparse_gemm_irregular_gm_gb300.binding import GmError

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
# Steepest slope of an activation and of a slope: |act'| <= 1.13, |act''| <= 0.8 (relu: none; it is taken at the kept z's sign).
SLOPE, BEND = 1.13, 0.8
# fp32 sums on the tensor cores are cut, not rounded, to 24 bits: a whole unit, not half, an addition; additions of a stage's
# 64 elements go 16 at a time. An activation in short form is within 2^-21 of its argument's size.
ACT_ROOM = 2.0 ** -21


def wide_of(t):
    return None if t is None else t.double().cpu().numpy()


def sum_room(length, size):
    return 2.0 ** -23 * (length / 16 + 24) * size


def check(got, ref, room, kind):
    got = wide_of(got)
    assert got.shape == ref.shape
    room = room * (1 + HALF[kind]) + HALF[kind] * np.abs(ref) * 1.01 + LEAST[kind]
    bad = ~(np.abs(got - ref) <= room)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], got[bad][:4], ref[bad][:4], room[bad][:4])


def make(rows, dim, outs, kind, *, bias=True, residual=True, wide=0, offset=0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 3)

    def matrix(n, m, std):
        big = torch.full((n * (m + wide) + offset,), float("nan"), device="cuda", dtype=TYPES[kind])
        v = big[offset:].view(n, m + wide)[:, :m]
        v.copy_(torch.randn(n, m, generator=g, device="cuda") * std)
        return v

    b = torch.empty(outs + offset, device="cuda", dtype=TYPES[kind])
    b.copy_(torch.randn(outs + offset, generator=g, device="cuda") * 0.5)
    return (matrix(rows, dim, 1.0), matrix(outs, dim, 1 / math.sqrt(dim)), b[offset:] if bias else None,
            matrix(rows, outs, 2.0) if residual else None, matrix(rows, outs, 0.25))


def both(x, w, b, r, grad, act, kind, got=None):
    if got is None:
        y, z = layers.linear_forward(x, w, b, activation=act, residual=r, keep=True)
        dx, dw, db = layers.linear_backward(x, w, grad, activation=act, z=z, need_bias=True)
    else:
        y, z, dx, dw, db = got
    assert (z is None) == (act == "none") or got is not None
    rows, dim = x.shape
    X, W, B, R, G = (wide_of(t) for t in (x, w, b, r, grad))
    z64, zs = X @ W.T, np.abs(X) @ np.abs(W).T
    if B is not None:
        z64, zs = z64 + B, zs + np.abs(B)
    zroom = sum_room(dim, zs)
    if z is not None:
        check(z, z64, zroom, kind)
    a, _ = layer_oracle.act(z64, act)
    y64 = a if R is None else a + R
    check(y, y64, SLOPE * zroom + ACT_ROOM * np.abs(z64) + 4 * EPS32 * (np.abs(y64) + (0 if R is None else np.abs(R))), kind)
    # gradients: the slope at z as it was kept
    kept = z64 if z is None else wide_of(z)
    s = layer_oracle.act(kept, act)[1]
    dz = G * s
    short = 0 if kind == "f32" or (act != "none" and rows <= 128) or act == "none" else HALF[kind]  # dz's own rounding
    dz_room = np.abs(G) * (2.0 ** -21 * (1 + np.abs(kept)) if act not in ("none", "relu") else 4 * EPS32) + short * np.abs(dz) + 2 * LEAST[kind]
    if rows <= 128 and act != "none" and kind != "f32":
        dz_room = dz_room + HALF[kind] ** 2 * np.abs(dz)
    check(dx, dz @ W, dz_room @ np.abs(W) + sum_room(w.shape[0], np.abs(dz) @ np.abs(W)), kind)
    check(dw, dz.T @ X, dz_room.T @ np.abs(X) + sum_room(rows, np.abs(dz).T @ np.abs(X)), kind)
    check(db, dz.sum(0), (dz_room - short * np.abs(dz)).sum(0) + EPS32 * (rows / 8 + 600) * np.abs(dz).sum(0), kind)
    return y, z, dx, dw, db


SHAPES = [(1, 1, 1), (1, 64, 64), (3, 7, 5), (16, 256, 1000), (33, 40, 200), (128, 128, 128), (129, 65, 257), (333, 129, 517),
          (256, 1024, 512), (130, 2080, 72), (1000, 96, 24), (520, 520, 520), (2050, 136, 264), (5, 5000, 48), (300, 8, 2000)]


@pytest.mark.parametrize("rows,dim,outs", SHAPES)
@pytest.mark.parametrize("kind", TYPES)
def test_sizes(rows, dim, outs, kind):
    act = ACTS[(rows + dim) % 5]
    both(*make(rows, dim, outs, kind, seed=rows), act, kind)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("bias,residual", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows", [40, 200])
def test_parts(act, kind, bias, residual, rows):
    both(*make(rows, 136, 152, kind, bias=bias, residual=residual), act, kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("wide,offset", [(8, 0), (3, 0), (0, 1), (5, 2), (4, 4)])
@pytest.mark.parametrize("rows,dim,outs", [(70, 72, 96), (150, 33, 47), (9, 1032, 200)])
def test_strides(kind, wide, offset, rows, dim, outs):
    both(*make(rows, dim, outs, kind, wide=wide, offset=offset), "gelu", kind)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("wide,offset", [(0, 0), (5, 0), (8, 8), (8, 1)])
@pytest.mark.parametrize("rows,dim,outs", [(150, 200, 136), (20, 40, 33), (5, 6000, 64)])
def test_results_into_the_callers_rows(kind, wide, offset, rows, dim, outs):
    x, w, b, r, grad = make(rows, dim, outs, kind)

    def room(n, m):
        big = torch.full((n * (m + wide) + offset + 32,), 7.0, device="cuda", dtype=TYPES[kind])
        return big, big[offset:offset + n * (m + wide)].view(n, m + wide)[:, :m]

    (by, y), (bz, z), (bx, dx), (bw, dw) = room(rows, outs), room(rows, outs), room(rows, dim), room(outs, dim)
    db = torch.empty(outs, device="cuda", dtype=TYPES[kind])
    layers.gm_linear_forward(x, w, b, r, y, z, activation="silu")
    layers.gm_linear_backward(x, w, grad, z, dx, dw, db, activation="silu")
    both(x, w, b, r, grad, "silu", kind, (y, z, dx, dw, db))
    for big, m in ((by, y), (bz, z), (bx, dx), (bw, dw)):  # nothing else was written
        m.fill_(7.0)
        assert (big == 7.0).all()


@pytest.mark.parametrize("rows,dim,outs", [(200, 64, 320), (4, 5000, 64)])
def test_result_over_the_residual(rows, dim, outs):
    x, w, b, r, _ = make(rows, dim, outs, "bf16")
    y, _ = layers.linear_forward(x, w, b, activation="gelu", residual=r)
    layers.gm_linear_forward(x, w, b, r, r, activation="gelu")
    assert torch.equal(y, r)


@pytest.mark.parametrize("rows", [100, 400])
def test_one_gradient_at_a_time_and_runs_repeat(rows):
    x, w, b, r, grad = make(rows, 300, 520, "bf16")
    _, z = layers.linear_forward(x, w, b, activation="gelu", keep=True)
    k = dict(activation="gelu", z=z)
    whole = layers.linear_backward(x, w, grad, need_bias=True, **k)
    again = layers.linear_backward(x, w, grad, need_bias=True, **k)
    for i in range(3):
        assert torch.equal(whole[i], again[i])
        one = layers.linear_backward(x, w, grad, need_x=i == 0, need_w=i == 1, need_bias=i == 2, **k)
        assert [t is not None for t in one] == [i == 0, i == 1, i == 2]
        assert torch.equal(whole[i], one[i])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", ACTS)
def test_far_and_special_arguments(kind, act):
    """Where an activation's pieces would overflow, it has its limit; infinities and NaN stay in their rows and columns."""
    big = 60000.0 if kind == "f16" else 1e30
    x = torch.tensor([[1.0], [-1.0], [0.0], [1e-4]], device="cuda", dtype=TYPES[kind])
    w = torch.tensor([[big], [30.0], [10.0], [1.0]], device="cuda", dtype=TYPES[kind])
    y, z = layers.linear_forward(x, w, activation=act, keep=True)
    ref, s = layer_oracle.act(wide_of(x) @ wide_of(w).T, act)
    assert y.isfinite().all()
    check(y, ref, 2.0 ** -20 * np.abs(wide_of(x) @ wide_of(w).T) * (np.abs(wide_of(x) @ wide_of(w).T) < 100), kind)
    dx, _, db = layers.linear_backward(x, w, torch.ones_like(y), activation=act, z=z, need_bias=True)
    assert db.isfinite().all()
    x[1, 0] = float("nan")
    x[3, 0] = float("inf")
    y2, _ = layers.linear_forward(x, w, activation=act)
    assert y2[1].isnan().all() and torch.equal(y2[[0, 2]], y[[0, 2]])
    assert (y2[3] == float("inf")).all()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 4, 5])
@pytest.mark.parametrize("dim,outs", [(8, 3), (200, 515), (512, 1030), (1024, 700), (2056, 129), (4096, 300), (1031, 77)])
def test_few_rows(kind, rows, dim, outs):
    x, w, b, r, grad = make(rows, dim, outs, kind, seed=dim)
    both(x, w, b, r, grad, "gelu_tanh", kind)


def test_offsets_past_32_bits():
    outs, dim = 540000, 4096  # 2.2e9 weights; and as many results
    x, w, b, _, _ = make(2, dim, 8, "bf16", residual=False)
    big = torch.zeros(outs, dim, device="cuda", dtype=torch.bfloat16)
    big[-8:] = w
    bias = torch.zeros(outs, device="cuda", dtype=torch.bfloat16)
    bias[-8:] = b
    for rows in (1, 2):
        y, _ = layers.linear_forward(x[:rows], big, bias, activation="silu")
        ref, _ = layers.linear_forward(x[:rows], w, b, activation="silu")
        assert torch.equal(y[:, -8:], ref) and (y[:, :-8] == 0).all()
    del big
    rows, outs = 70000, 32768
    x, w, b, _, _ = make(rows, 64, outs, "bf16", residual=False)
    y, _ = layers.linear_forward(x, w, b)
    ref, _ = layers.linear_forward(x[-300:].clone(), w, b)
    assert torch.equal(y[-300:], ref)
    odd = torch.empty(rows * (outs + 1), device="cuda", dtype=torch.bfloat16).view(rows, outs + 1)[:, :outs]  # rows off 16 bytes
    layers.gm_linear_forward(x, w, b, None, odd)
    assert torch.equal(odd[-300:], ref)


def test_calls_at_once_on_two_streams():
    x, w, b, r, grad = make(300, 520, 264, "bf16")

    def run(stream=None):
        y, z = layers.linear_forward(x, w, b, activation="gelu", residual=r, keep=True, stream=stream)
        return [y, z, *layers.linear_backward(x, w, grad, activation="gelu", z=z, need_bias=True, stream=stream)]

    ref = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [run(streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for o in out for p, q in zip(o, ref))


def test_no_rows():
    x, w, b, r, grad = make(0, 48, 72, "bf16")
    y, _ = layers.linear_forward(x, w, b, residual=r)
    assert y.shape == (0, 72)
    dx, dw, db = layers.linear_backward(x, w, grad, need_bias=True)
    assert dx.shape == (0, 48) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("act", ACTS)
def test_autograd_against_differences(act):
    x, w, b, r, grad = make(5, 9, 7, "f32", seed=1)
    leaves = [t.clone().requires_grad_() for t in (x, w, b, r)]
    (layers.linear(*leaves[:3], activation=act, residual=leaves[3]) * grad).sum().backward()
    base = [wide_of(t.detach()) for t in leaves]
    G = wide_of(grad)

    def total(x, w, b, r):
        return ((layer_oracle.act(x @ w.T + b, act)[0] + r) * G).sum()

    for k, t in enumerate(leaves):
        slope = np.zeros(t.shape)
        for i in np.ndindex(*t.shape):
            up, down = ([v.copy() for v in base] for _ in range(2))
            up[k][i] += 1e-6
            down[k][i] -= 1e-6
            slope[i] = (total(*up) - total(*down)) / 2e-6
        assert np.allclose(wide_of(t.grad), slope, rtol=1e-4, atol=1e-5 * np.abs(slope).max()), k


def test_autograd_asks_only_for_what_is_wanted():
    x, w, b, r, _ = make(40, 24, 32, "bf16")
    r.requires_grad_()
    y = layers.linear(x, w, b, activation="relu", residual=r)
    y.sum().backward()  # an expanded gradient
    assert (r.grad == 1).all()
    w.requires_grad_()
    layers.linear(x, w).sum().backward()
    assert torch.equal(w.grad, layers.linear_backward(x, w.detach(), torch.ones_like(y), need_x=False)[1])


@pytest.mark.parametrize("rows,dim,outs", [(64, 512, 256), (3, 8192, 128), (300, 100, 60)])
def test_other_stream_and_graph(rows, dim, outs):
    x, w, b, r, grad = make(rows, dim, outs, "bf16")

    def run(stream=None):
        y, z = layers.linear_forward(x, w, b, activation="silu", residual=r, keep=True, stream=stream)
        return [y, z, *layers.linear_backward(x, w, grad, activation="silu", z=z, need_bias=True, stream=stream)]

    here = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    there = run(s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(here, there))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = run()
    for t, u in zip((x, w, b, r, grad), make(rows, dim, outs, "bf16", seed=9)):
        t.copy_(u)
    g.replay()
    assert all(torch.equal(p, q) for p, q in zip(held, run()))


def test_refusals():
    x, w, b, r, grad = make(4, 16, 24, "bf16")
    for bad in (lambda: layers.linear_forward(x, w.float()), lambda: layers.linear_forward(x, w[:, :8]),
                lambda: layers.linear_forward(x.t(), w), lambda: layers.linear_forward(x, w, b[:5]),
                lambda: layers.linear_forward(x, w, residual=r[:2]), lambda: layers.linear_forward(x, w, activation="tanh"),
                lambda: layers.linear_forward(x.cpu(), w), lambda: layers.linear_backward(x, w, grad[:, :4])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(GmError):
        layers.linear_backward(x, w, grad, activation="gelu")  # without z


# Few rows of long ones: the parts are joined by a kernel of their own, four columns a thread where all rows allow it.
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("wide,offset", [(0, 0), (4, 4), (2, 2), (1, 0), (0, 1)])
@pytest.mark.parametrize("rows,dim,outs", [(24, 4104, 256), (24, 4100, 255), (5, 4096, 70), (130, 4096, 260)])
def test_joined_parts(kind, wide, offset, rows, dim, outs):
    both(*make(rows, dim, outs, kind, wide=wide, offset=offset), ACTS[(outs + wide) % 5], kind)
    both(*make(rows, dim, outs, kind, bias=False, wide=wide, offset=offset), "none", kind)


# more tiles than SMs, in every width of tile that the rule takes for such sizes
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,dim,outs", [(2600, 700, 1500), (700, 1536, 2600), (1500, 96, 5200)])
def test_blocks_that_walk_several_tiles(kind, rows, dim, outs):
    both(*make(rows, dim, outs, kind, seed=9), "silu", kind)


@pytest.mark.parametrize("act", ACTS[1:])
@pytest.mark.parametrize("rows", [4, 200])
def test_arguments_past_the_range_in_which_they_are_kept(act, rows):
    """Finite x and W of f16 whose z is past its range: kept as an infinity, at which the slopes are 0 and 1."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.rand(rows, 8, device="cuda", generator=g).add_(0.5).half()
    w = torch.randn(16, 8, device="cuda", generator=g).half()
    w[3], w[7] = -30000.0, 30000.0  # z from -360000 to -120000, and the same above 0
    grad = torch.randn(rows, 16, device="cuda", generator=g).half()
    y, z = layers.linear_forward(x, w, activation=act, keep=True)
    assert (z[:, 3] == -torch.inf).all() and (z[:, 7] == torch.inf).all() and z[:, :3].isfinite().all()
    assert (y[:, 3] == 0).all() and (y[:, 7] == torch.inf).all()
    got = layers.linear_backward(x, w, grad, activation=act, z=z, need_bias=True)
    X, W, G, kept = (wide_of(t) for t in (x, w, grad, z.clamp(-1000, 1000)))  # slopes are 0 or 1 from there on
    s = layer_oracle.act(kept, act)[1]
    assert (s[:, 3] == 0).all() and (s[:, 7] == 1).all()
    dz = G * s
    dz_room = np.abs(G) * 2.0 ** -21 * (1 + np.abs(kept)) * (s != 0) * (s != 1) + HALF["f16"] * np.abs(dz) + 2 * LEAST["f16"]
    # f16 ends at 65504, its steps there are 32: what is 65520 or more, within the room, is rightly an infinity
    ref, room = dz @ W, dz_room @ np.abs(W) + sum_room(16, np.abs(dz) @ np.abs(W))
    past = np.isinf(wide_of(got[0])) & (np.sign(wide_of(got[0])) * ref + room >= 65520)
    check(torch.where(torch.tensor(past, device="cuda"), 0, got[0]), np.where(past, 0, ref), room, "f16")
    check(got[1], dz.T @ X, dz_room.T @ np.abs(X) + sum_room(rows, np.abs(dz).T @ np.abs(X)), "f16")
    check(got[2], dz.sum(0), dz_room.sum(0) + EPS32 * (rows / 8 + 600) * np.abs(dz).sum(0), "f16")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_at_infinity_and_no_number(kind, act):
    x, w, _, _, _ = make(3, 24, 8, kind)
    z = torch.tensor([[torch.inf, -torch.inf] * 4, [1.0, -1.0] * 4, [torch.nan] * 8], device="cuda", dtype=TYPES[kind])
    _, _, db = layers.linear_backward(x[:2], w, torch.ones_like(z[:2]), activation=act, z=z[:2], need_bias=True)
    ref = layer_oracle.act(np.array([1.0, -1.0] * 4), act)[1] + np.array([1.0, 0.0] * 4)
    check(db, ref, 2.0 ** -20, kind)
    dx, _, _ = layers.linear_backward(x, w, torch.ones_like(z), activation=act, z=z, need_w=False)
    assert dx[:2].isfinite().all()
    assert dx[2].isnan().all() or act == "relu"


def small_gradients(x, w, grad, act, z, inside=slice(None), columns=slice(None)):
    """f16: dz is kept in steps of at most half of 2^-25 / 2^13 of the largest finite gradient, or rounded once; slopes to 2^-21."""
    rows = x.shape[0]
    got = layers.linear_backward(x, w, grad, activation=act, z=z, need_bias=True)
    X, W, G, kept = (wide_of(t) for t in (x, w, grad, z))
    most = np.abs(G[np.isfinite(G)]).max()
    G = np.where(np.isfinite(G), G, 0)
    dz = G * layer_oracle.act(kept, act)[1]
    own = np.abs(G) * 2.0 ** -21  # of the slope alone: db is summed before dz is rounded
    dz_room = own + (HALF["f16"] ** 2 if rows <= 128 else HALF["f16"]) * np.abs(dz) + 2.0 ** -38 * most
    k = W.shape[0]
    check(got[0][inside], (dz @ W)[inside], (dz_room @ np.abs(W) + sum_room(k, np.abs(dz) @ np.abs(W)))[inside], "f16")
    check(got[1][columns], (dz.T @ X)[columns], (dz_room.T @ np.abs(X) + sum_room(rows, np.abs(dz).T @ np.abs(X)))[columns], "f16")
    check(got[2][columns], dz.sum(0)[columns], (own.sum(0) + EPS32 * (rows / 8 + 600) * np.abs(dz).sum(0))[columns], "f16")
    return got


@pytest.mark.parametrize("size", [1e-5, 1e-4, 1.0])
@pytest.mark.parametrize("rows,dim,outs,wide", [(1000, 72, 136, 0), (100, 72, 136, 0), (333, 40, 77, 3), (1, 64, 520, 0)])
@pytest.mark.parametrize("act,far", [("gelu", 4.0), ("gelu_tanh", 4.0), ("silu", 10.0)])
def test_small_gradients_of_f16_keep_their_digits(act, far, rows, dim, outs, wide, size):
    x, w, _, _, grad = make(rows, dim, outs, "f16", wide=wide, seed=5)
    w.mul_(0.1)
    b = -torch.linspace(0, far, outs, device="cuda").half()  # slopes from a half to 5e-4
    _, z = layers.linear_forward(x, w, b, activation=act, keep=True)
    grad.mul_(4 * size)
    small_gradients(x, w, grad, act, z)


@pytest.mark.parametrize("rows", [60, 300])
def test_large_gradients_of_f16_stay_finite_past_a_steep_slope(rows):
    x, w, _, _, grad = make(rows, 64, 96, "f16", seed=6)
    w.mul_(2.0 ** -10)
    x.mul_(2.0 ** -10)
    z = torch.full((rows, 96), 1.5, device="cuda").half()  # gelu's slope is 1.128 there
    grad[:, 5] = 65504.0
    dx, dw, _ = small_gradients(x, w, grad, "gelu", z, columns=[i for i in range(96) if i != 5])  # db[5] is past f16
    assert dx.isfinite().all() and dw.isfinite().all()


@pytest.mark.parametrize("rows", [60, 300])
def test_an_infinite_gradient_does_not_cost_the_others_digits(rows):
    x, w, b, _, grad = make(rows, 64, 96, "f16", seed=7)
    _, z = layers.linear_forward(x, w, b, activation="silu", keep=True)
    grad.mul_(1e-4)
    grad[2, 9] = torch.inf
    small_gradients(x, w, grad, "silu", z, inside=[i for i in range(rows) if i != 2], columns=[i for i in range(96) if i != 9])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows", [3, 100, 200])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_an_infinite_gradient_gives_infinities(kind, rows, act):
    x, w, b, _, grad = make(rows, 48, 56, kind, seed=8)
    _, z = layers.linear_forward(x, w, b, activation=act, keep=True)
    if z is not None:
        z[1, 4] = 2.0  # slope over 0
    grad[1, 4] = -torch.inf
    w[4, 3] = x[1, 3] = 1.0
    dx, dw, db = layers.linear_backward(x, w, grad, activation=act, z=z, need_bias=True)
    assert torch.equal(dx[1], -torch.inf * w[4].sign()) and torch.equal(dw[4], -torch.inf * x[1].sign()) and db[4] == -torch.inf
    for t, i in ((dx, 1), (dw, 4), (db, 4)):
        t[i] = 0
        assert t.isfinite().all()


# Sums of 16-bit operands: up to 1024 elements are added 16 at a time, each addition cut to 24 bits, off by 2^-23 of the sum
# so far at most, two such additions where dz has two planes; the parts are added in fp32.
def long_sum_room(length, size, planes=1):
    return (planes * 64 * 2.0 ** -23 + (length / 1024 + 17) * 2.0 ** -24) * size


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rows,dim,outs", [(4096, 16384, 2560), (300, 65536, 520), (24, 262144, 64), (2, 1 << 20, 40)])
def test_long_rows_of_one_sign(kind, rows, dim, outs):
    """The residual takes z away but for its last digits, so that y shows the sum's own error, not its rounding."""
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.rand(rows, dim, device="cuda", generator=g).add_(0.5).to(TYPES[kind])
    w = torch.rand(outs, dim, device="cuda", generator=g).add_(0.5).div_(dim).to(TYPES[kind])
    z = torch.cat([x[i:i + 256].double() @ w.double().T for i in range(0, rows, 256)])
    r = -z.to(TYPES[kind])
    y, _ = layers.linear_forward(x, w, residual=r)
    check(y, wide_of(z + r), long_sum_room(dim, wide_of(z)), kind)


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("rows,dim,outs", [(4096, 2560, 65536), (128, 20480, 65536)])
def test_long_sums_of_gradients_by_x(rows, dim, outs, act):
    """The second half takes away what the first one gave: what is left is the sum's own error."""
    g = torch.Generator(device="cuda").manual_seed(1)
    half = outs // 2
    w = torch.rand(half, dim, device="cuda", generator=g).half().repeat(2, 1)
    grad = torch.rand(rows, half, device="cuda", generator=g).half()
    grad = torch.cat([grad, -grad], 1)
    x = torch.zeros(rows, dim, device="cuda").half()
    z = None if act == "none" else torch.full_like(grad, 1.0)
    dx, _, _ = layers.linear_backward(x, w, grad, activation=act, z=z, need_w=False)
    size = 1.09 * grad.float().abs() @ w.float()  # gelu's slope at 1 is 1.083
    planes = 2 if rows <= 128 and act != "none" else 1
    check(dx, np.zeros((rows, dim)), long_sum_room(outs, wide_of(size), planes), "f16")


def test_long_sums_of_gradients_by_w():
    rows, dim, outs = 65536, 2560, 4096
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.rand(rows // 2, dim, device="cuda", generator=g).half().repeat(2, 1)
    grad = torch.rand(rows // 2, outs, device="cuda", generator=g).half()
    grad = torch.cat([grad, -grad])
    w = torch.zeros(outs, dim, device="cuda").half()
    _, dw, _ = layers.linear_backward(x, w, grad, need_x=False)
    check(dw, np.zeros((outs, dim)), long_sum_room(rows, wide_of(grad.float().abs().T @ x.float())), "f16")


@pytest.mark.parametrize("kind,least", [("bf16", 2.0 ** -120), ("f16", 2.0 ** -24)])
@pytest.mark.parametrize("act,far", [("gelu", 12.5), ("gelu_tanh", 9.5), ("silu", 80.0)])
@pytest.mark.parametrize("rows", [1, 150])
def test_tails_of_activations_are_rounded_once(kind, least, act, far, rows):
    """An activation is within 2^-15 of itself before it is rounded (its form, and roundings of an exponent up to 2^7)."""
    z = -torch.linspace(0.05, far, 5000, device="cuda").to(TYPES[kind])
    x = torch.ones(rows, 1, device="cuda").to(TYPES[kind])
    y, _ = layers.linear_forward(x, z[:, None].contiguous(), activation=act)  # z as it is: one term
    v = wide_of(z)
    if act == "gelu":
        ref = np.array([t * 0.5 * math.erfc(-t / math.sqrt(2)) for t in v])
    elif act == "silu":
        ref = v / (1 + np.exp(-v))
    else:
        ref = v / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    got = wide_of(y)
    room = np.abs(ref) * (HALF[kind] * 1.01 + 2.0 ** -15) + least / 2
    bad = ~(np.abs(got - ref) <= room)
    assert not bad.any(), (int(bad.sum()), v[np.argwhere(bad)[:5, 1]], got[bad][:5], ref[np.argwhere(bad)[:5, 1]])


# Sums longer than 1024 elements on every tile that the rule takes for them, in one part and in several; a, b: rows and columns
# of a result, n: the length of its sums.
@pytest.mark.parametrize("act,kind", [("none", "bf16"), ("silu", "f16")])
@pytest.mark.parametrize("role", ["y", "dx", "dw"])
@pytest.mark.parametrize("a,n,b", [(24, 1100, 64), (24, 5000, 4100), (24, 1100, 20000), (300, 1100, 4100), (520, 1100, 4100), (1024, 5000, 264),
                                   (200, 5000, 1100)])
def test_sums_in_parts_on_every_tile(act, kind, role, a, n, b):
    rows, dim, outs = {"y": (a, n, b), "dx": (a, b, n), "dw": (n, b, a)}[role]
    both(*make(rows, dim, outs, kind, seed=n), act, kind)

"""The losses over a class table on the GPU against the 64-bit oracle (loss_oracle): elementwise bounds derived from
the kernels' roundings, every type, odd sizes, strides, empty rows, refusals."""
import ctypes

import numpy as np
import pytest
import torch

import loss_oracle as lo
from sparse_gemm_irregular_gm_gb300 import binding, inputs, losses

pytestmark = pytest.mark.gpu
KIND = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def wide(t):
    return t.double().cpu().numpy()


def make(kind, n, d, v, seed=0, spread=2.0, pad=0, shift=0, ignored=0.2, t32=False):
    """h, w (with pad elements between rows, starting shift elements into their memory), targets."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for rows, scale in ((n, 1.0), (v, spread / d ** 0.5)):
        x = (torch.randn(rows, d, generator=g) * scale).to(KIND[kind])
        memory = torch.full((shift + rows * (d + pad) + 8,), float("nan"), dtype=KIND[kind], device="cuda")
        m = memory[shift:shift + rows * (d + pad)].view(rows, d + pad)[:, :d]
        m.copy_(x)
        out.append(m)
    target = torch.randint(0, v, (n,), generator=g)
    target[torch.rand(n, generator=g) < ignored] = -100
    if n > 2:
        target[0], target[-1] = 0, v - 1
    return out[0], out[1], target.to(torch.int32 if t32 else torch.int64).cuda()


def make_teacher(n, v, seed=0, longest=40, val=torch.float32, row_ptr=torch.int64, col=torch.int32, empty=0.2):
    rng = np.random.default_rng(seed)
    lens = rng.integers(1, min(longest, v) + 1, size=n)
    lens[rng.random(n) < empty] = 0
    if n > 3:
        lens[1], lens[2], lens[3] = 0, min(longest, v), 1
    rp = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    cols = np.concatenate([np.sort(rng.choice(v, k, replace=False)) for k in lens] + [np.zeros(0)]).astype(np.int64)
    vals = rng.normal(size=rp[-1]) * 2 + 3
    vals[rng.random(vals.size) < 0.05] = -np.inf
    vals = torch.from_numpy(vals).to(val)
    dev = binding.DeviceCSR(n, v, torch.from_numpy(rp).to(row_ptr).cuda(), torch.from_numpy(cols).to(col).cuda(), vals.cuda())
    return dev, lo.Teacher(rp, cols, vals.double().numpy())


def weights(n, k, seed, scale=1.0):
    rng = np.random.default_rng(seed + 77)
    g = (rng.random((k, n)) + 0.5).astype(np.float32) * np.float32(scale / max(n, 1))
    return [torch.from_numpy(x).cuda() for x in g], list(g.astype(np.float64))


def near(got, want, bound, what):
    got = wide(got)
    assert got.shape == want.shape and np.all(np.isfinite(got)), what
    over = np.abs(got - want) - bound
    assert np.all(over <= 0), f"{what}: off by {np.max(np.abs(got - want)):.3g}, at most {np.max(over):.3g} over the bound"


def check_forward(f, h, w, temperature, **got):
    bounds = lo.forward_bounds(f, wide(h), wide(w), temperature)
    for name, t in got.items():
        near(t, f[name], bounds[name], name)


def check_grads(f, grads, h, w, kind, temperature, dh, dw):
    (eh, bh), (ew, bw) = lo.gradient_bounds(f, grads, wide(h), wide(w), kind, temperature)
    if dh is not None:
        near(dh, eh, bh, "dh")
    if dw is not None:
        near(dw, ew, bw, "dw")


SIZES = [(1, 1, 1), (1, 8, 2), (2, 7, 255), (3, 64, 256), (31, 65, 257), (128, 63, 300), (129, 128, 513), (130, 129, 1000),
         (257, 72, 64), (300, 264, 777), (40, 1100, 520), (140, 1100, 300), (5, 2056, 129)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,v", SIZES)
def test_xent(kind, n, d, v):
    h, w, target = make(kind, n, d, v, seed=n + d)
    loss, lse = losses.xent_forward(h, w, target, check=True)
    tn = target.cpu().numpy()
    f = lo.forward(wide(h), wide(w), tn)
    check_forward(f, h, w, 1.0, loss=loss, lse=lse)
    (gl, gs), (gl_n, gs_n) = weights(n, 2, v, scale=64.0 if kind == "f16" else 1.0)
    dh, dw = losses.xent_backward(h, w, target, lse, gl, gs, check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n, gs_n), h, w, kind, 1.0, dh, dw)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("labels", [False, True])
@pytest.mark.parametrize("n,d,v,temperature", [(1, 8, 2, 1.0), (4, 64, 300, 2.0), (131, 72, 700, 0.5), (260, 130, 257, 4.0),
                                               (60, 1100, 520, 2.0), (300, 1100, 130, 1.0)])
def test_distill(kind, labels, n, d, v, temperature):
    h, w, target = make(kind, n, d, v, seed=n + d + v)
    dev, host = make_teacher(n, v, seed=n)
    t, tn = (target, target.cpu().numpy()) if labels else (None, None)
    o = losses.distill_forward(h, w, dev, temperature, target=t, check=True)
    f = lo.forward(wide(h), wide(w), tn, -100, host, temperature)
    check_forward(f, h, w, temperature, kl=o.kl, lse_t=o.lse_t, **({"loss": o.loss, "lse": o.lse} if labels else {}))
    (gk, gl, gs), (gk_n, gl_n, gs_n) = weights(n, 3, v, scale=64.0 if kind == "f16" else 1.0)
    more = dict(target=t, lse=o.lse, grad_loss=gl, grad_lse=gs) if labels else {}
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, temperature, check=True, **more)
    grads = lo.logit_grads(f, tn, -100, gl_n, gs_n, temperature, gk_n)
    check_grads(f, grads, h, w, kind, temperature, dh, dw)


@pytest.mark.parametrize("val", [torch.float32, torch.float64])
@pytest.mark.parametrize("row_ptr", [torch.int32, torch.int64])
@pytest.mark.parametrize("col", [torch.int32, torch.int64])
def test_teacher_types(val, row_ptr, col):
    h, w, _ = make("bf16", 50, 40, 200)
    dev, host = make_teacher(50, 200, val=val, row_ptr=row_ptr, col=col)
    o = losses.distill_forward(h, w, dev, 1.5, check=True)
    f = lo.forward(wide(h), wide(w), None, -100, host, 1.5)
    check_forward(f, h, w, 1.5, kl=o.kl, lse_t=o.lse_t)


def test_long_and_full_teacher_rows():
    """Rows of every class, of more entries than a warp takes, and none."""
    n, v = 70, 3000
    h, w, _ = make("f32", n, 24, v)
    dev, host = make_teacher(n, v, longest=v, empty=0.3)
    o = losses.distill_forward(h, w, dev, 2.0, check=True)
    f = lo.forward(wide(h), wide(w), None, -100, host, 2.0)
    check_forward(f, h, w, 2.0, kl=o.kl, lse_t=o.lse_t)
    (gk,), (gk_n,) = weights(n, 1, 1)
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, check=True)
    check_grads(f, lo.logit_grads(f, temperature=2.0, g_kl=gk_n), h, w, "f32", 2.0, dh, dw)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,pad,shift", [(64, 8, 0), (64, 8, 8), (64, 1, 0), (64, 0, 1), (200, 3, 5), (33, 7, 0), (96, 4, 4), (129, 7, 0)])
def test_strides_and_alignment(kind, d, pad, shift):
    """Rows apart, starting anywhere: read right, and written nowhere else."""
    n, v = 150, 333
    h, w, target = make(kind, n, d, v, pad=pad, shift=shift, t32=True)
    loss, lse = losses.xent_forward(h, w, target, check=True)
    tn = target.cpu().numpy()
    f = lo.forward(wide(h), wide(w), tn)
    check_forward(f, h, w, 1.0, loss=loss, lse=lse)
    (gl,), (gl_n,) = weights(n, 1, d)
    outs = []
    for like in (h, w):
        rows = like.shape[0]
        memory = torch.full((shift + rows * (d + pad) + 8,), 7.0, dtype=KIND[kind], device="cuda")
        outs.append((memory, memory[shift:shift + rows * (d + pad)].view(rows, d + pad)[:, :d]))
    losses.gm_xent_backward(h, w, target, lse, gl, None, outs[0][1], outs[1][1], check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n), h, w, kind, 1.0, outs[0][1], outs[1][1])
    for memory, view in outs:
        view.fill_(7.0)
        assert torch.all(memory == 7.0)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,v,pad,shift,cap", [(100, 65, 700, 0, 0, 0), (100, 65, 700, 1, 1, 1), (9, 130, 513, 0, 2, 0),
                                                 (128, 1029, 300, 0, 1, 1), (64, 1026, 257, 3, 0, 0), (17, 34, 900, 1, 3, 0),
                                                 (12, 257, 1111, 0, 0, 1), (100, 300, 64, 7, 5, 0), (33, 1, 2000, 0, 1, 0)])
def test_class_table_off_16_byte_boundaries_with_few_rows(kind, n, d, v, pad, shift, cap):
    """NaN lies between and around its rows; pieces of 256 classes too."""
    h, w, target = make(kind, n, d, v, pad=pad, shift=shift)
    dev, host = make_teacher(n, v)
    o = losses.distill_forward(h, w, dev, 2.0, target=target, check=True)
    tn = target.cpu().numpy()
    f = lo.forward(wide(h), wide(w), tn, -100, host, 2.0)
    check_forward(f, h, w, 2.0, kl=o.kl, lse_t=o.lse_t, loss=o.loss, lse=o.lse)
    (gk, gl), (gk_n, gl_n) = weights(n, 2, d, scale=64.0 if kind == "f16" else 1.0)
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, target=target, lse=o.lse, grad_loss=gl,
                                     workspace_cap_bytes=cap, check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n, None, 2.0, gk_n), h, w, kind, 2.0, dh, dw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_pieces_change_nothing_but_roundings(kind):
    """A small bound on G cuts the classes into pieces of 256, the last one partial."""
    n, d, v = 200, 136, 1111
    h, w, target = make(kind, n, d, v)
    dev, host = make_teacher(n, v)
    o = losses.distill_forward(h, w, dev, 2.0, target=target, check=True)
    tn = target.cpu().numpy()
    f = lo.forward(wide(h), wide(w), tn, -100, host, 2.0)
    (gk, gl), (gk_n, gl_n) = weights(n, 2, 3)
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, target=target, lse=o.lse, grad_loss=gl,
                                     workspace_cap_bytes=1, check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n, None, 2.0, gk_n), h, w, kind, 2.0, dh, dw)


def test_one_gradient_alone_is_the_same():
    h, w, target = make("bf16", 150, 72, 600)
    _, lse = losses.xent_forward(h, w, target)
    (gl,), _ = weights(150, 1, 0)
    dh, dw = losses.xent_backward(h, w, target, lse, gl)
    only_h, none = losses.xent_backward(h, w, target, lse, gl, need_w=False)
    assert none is None and torch.equal(only_h, dh)
    none, only_w = losses.xent_backward(h, w, target, lse, gl, need_h=False)
    assert none is None and torch.equal(only_w, dw)
    with pytest.raises(binding.GmError):
        losses.xent_backward(h, w, target, lse, gl, need_h=False, need_w=False)


def test_runs_repeat_bit_by_bit():
    h, w, target = make("bf16", 300, 200, 3000)
    dev, _ = make_teacher(300, 3000)
    (gk, gl), _ = weights(300, 2, 0)
    runs = []
    for _ in range(3):
        o = losses.distill_forward(h, w, dev, 2.0, target=target)
        runs.append([*o, *losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, target=target, lse=o.lse, grad_loss=gl)])
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_no_rows():
    h, w, target = make("bf16", 0, 40, 100)
    loss, lse = losses.xent_forward(h, w, target, check=True)
    assert loss.shape == lse.shape == (0,)
    dh, dw = losses.xent_backward(h, w, target, lse, loss, check=True)
    assert dh.shape == (0, 40) and torch.all(dw == 0) and dw.shape == (100, 40)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_every_row_ignored(kind):
    h, w, target = make(kind, 140, 72, 300)
    target.fill_(5)
    h[3] = float("nan")
    loss, lse = losses.xent_forward(h, w, target, ignore_index=5, check=True)
    assert torch.all(loss == 0) and torch.isnan(lse[3]) and torch.isfinite(lse[4:]).all()
    h[3] = 0
    (gl,), _ = weights(140, 1, 0)
    dh, dw = losses.xent_backward(h, w, target, lse, gl, ignore_index=5, check=True)
    assert torch.all(dh == 0) and torch.all(dw == 0)


def test_an_ignored_rows_nan_stays_in_it():
    h, w, target = make("bf16", 200, 72, 300)
    target[7] = -100
    clean = h.clone()
    h[7] = float("nan")
    _, lse = losses.xent_forward(h, w, target)
    _, lse0 = losses.xent_forward(clean, w, target)
    (gl,), _ = weights(200, 1, 0)
    dh, _ = losses.xent_backward(h, w, target, lse, gl, need_w=False)
    dh0, _ = losses.xent_backward(clean, w, target, lse0, gl, need_w=False)
    assert torch.all(dh[7] == 0) and torch.equal(dh, dh0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_values_that_are_not_finite_spoil_their_row_alone(kind, value):
    h, w, target = make(kind, 200, 72, 300, ignored=0.0)
    loss0, _ = losses.xent_forward(h, w, target)
    h[9, 5] = value
    loss, lse = losses.xent_forward(h, w, target, check=True)
    assert not torch.isfinite(lse[9])
    keep = torch.arange(200) != 9
    assert torch.equal(loss[keep.cuda()], loss0[keep.cuda()])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_large_logits(kind):
    """Logits of several hundred: one class has all of the mass."""
    n, d, v = 140, 64, 500
    h, w, target = make(kind, n, d, v, spread=60.0)
    tn = target.cpu().numpy()
    loss, lse = losses.xent_forward(h, w, target, check=True)
    f = lo.forward(wide(h), wide(w), tn)
    check_forward(f, h, w, 1.0, loss=loss, lse=lse)
    (gl,), (gl_n,) = weights(n, 1, 0)
    dh, dw = losses.xent_backward(h, w, target, lse, gl, check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n), h, w, kind, 1.0, dh, dw)


def test_small_weights_in_half_precision():
    """Weights whose products with probabilities lie far under f16's range still reach dH, which does not."""
    n, d, v = 140, 64, 5000
    h, w, target = make("f16", n, d, v, ignored=0.0)
    h *= 0.5
    w *= 16.0  # dH = G W stays in range while G is about 1e-9
    tn = target.cpu().numpy()
    _, lse = losses.xent_forward(h, w, target)
    f = lo.forward(wide(h), wide(w), tn)
    gl = torch.full((n,), 2.0 ** -8, device="cuda")
    dh, dw = losses.xent_backward(h, w, target, lse, gl, check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, np.full(n, 2.0 ** -8)), h, w, "f16", 1.0, dh, dw)


@pytest.mark.parametrize("bad", [-1, 300, 1 << 40, -(1 << 40)])
def test_targets_out_of_range(bad):
    h, w, target = make("bf16", 200, 72, 300, ignored=0.0)
    (gl,), _ = weights(200, 1, 0)
    _, lse0 = losses.xent_forward(h, w, target)
    clean = target.clone()
    clean[11] = -100
    dh0, dw0 = losses.xent_backward(h, w, clean, lse0, gl)
    target[11] = bad
    loss, lse = losses.xent_forward(h, w, target)
    with pytest.raises(binding.GmError) as e:
        losses.gm_loss_status()
    assert e.value.status == 9  # GM_ERR_BAD_INDEX
    losses.gm_loss_status()  # read once
    assert torch.isnan(loss[11]) and torch.isfinite(loss[:11]).all() and torch.equal(lse, lse0)
    dh, dw = losses.xent_backward(h, w, target, lse, gl)
    with pytest.raises(binding.GmError):
        losses.gm_loss_status()
    assert torch.equal(dh, dh0) and torch.equal(dw, dw0)
    with pytest.raises(binding.GmError):
        losses.xent_forward(h, w, target, check=True)


@pytest.mark.parametrize("fault", ["column over", "column under", "order", "repeat", "rows fall", "rows pass the end", "first under"])
def test_malformed_teacher_rows(fault):
    n, v = 60, 200
    h, w, _ = make("bf16", n, 40, v)
    dev, host = make_teacher(n, v, empty=0.0)
    rp = host.row_ptr
    rows = [i for i in range(4, n) if rp[i + 1] - rp[i] >= 3]
    r = rows[len(rows) // 2]
    o0 = losses.distill_forward(h, w, dev, 1.0, check=True)
    at = int(rp[r])
    spoilt = {r}
    if fault == "column over":
        dev.col[at + 2] = v
    elif fault == "column under":
        dev.col[at] = -1
    elif fault == "order":
        dev.col[at], dev.col[at + 1] = int(host.col[at + 1]), int(host.col[at])
    elif fault == "repeat":
        dev.col[at + 1] = int(host.col[at])
    elif fault == "rows fall":
        dev.row_ptr[r + 1] = at - 1
        spoilt = {r, r + 1}
    elif fault == "rows pass the end":
        dev.row_ptr[n] = int(rp[n]) + 5
        spoilt = {n - 1}
    else:
        dev.row_ptr[0] = -3
        spoilt = {0}
    o = losses.distill_forward(h, w, dev, 1.0)
    with pytest.raises(binding.GmError) as e:
        losses.gm_loss_status()
    assert e.value.status == 9
    nan = set(torch.nonzero(torch.isnan(o.kl)).flatten().tolist())
    assert r in nan or nan == spoilt
    assert nan <= spoilt
    good = torch.tensor([i not in spoilt for i in range(n)]).cuda()
    assert torch.equal(o.kl[good], o0.kl[good]) and torch.equal(o.lse_t, o0.lse_t)
    (gk,), _ = weights(n, 1, 0)
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, 1.0)
    with pytest.raises(binding.GmError):
        losses.gm_loss_status()
    for i in nan:
        assert torch.all(dh[i] == 0)
    assert torch.isfinite(dw).all()


def test_teacher_value_that_is_nan_or_infinite():
    n, v = 40, 100
    h, w, _ = make("bf16", n, 40, v)
    dev, host = make_teacher(n, v, empty=0.0)
    for r, x in ((5, float("nan")), (9, float("inf"))):
        dev.val[int(host.row_ptr[r])] = x
    o = losses.distill_forward(h, w, dev, 1.0, check=True)
    assert set(torch.nonzero(torch.isnan(o.kl)).flatten().tolist()) == {5, 9}


def test_gradient_against_differences_of_the_forward_pass():
    """Along random directions, in 32 bits: central differences of the kernel's own loss. A step of 2^-6 leaves a third
    derivative's part under 2^-12 of the weights' sum, and 2^-18 of rounding in each value over the step."""
    n, d, v = 33, 40, 150
    h, w, target = make("f32", n, d, v)
    dev, _ = make_teacher(n, v)
    (gk, gl, gs), _ = weights(n, 3, 0)

    def objective(h, w):
        o = losses.distill_forward(h, w, dev, 2.0, target=target)
        return float((o.kl.double() @ gk.double()) + (o.loss.double() @ gl.double()) + (o.lse.double() @ gs.double()))

    o = losses.distill_forward(h, w, dev, 2.0, target=target)
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, target=target, lse=o.lse, grad_loss=gl, grad_lse=gs)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x, grad in ((h, dh), (w, dw)):
        for _ in range(4):
            step = torch.randn(x.shape, generator=g, device="cuda") * 0.25
            e = 2.0 ** -6
            up = objective(h + e * step, w) if x is h else objective(h, w + e * step)
            down = objective(h - e * step, w) if x is h else objective(h, w - e * step)
            want = float((grad.double() * step.double()).sum())
            assert abs((up - down) / (2 * e) - want) < 2.0 ** -9 * (1 + abs(want))


def test_autograd():
    h, w, target = make("f32", 50, 40, 150)
    dev, _ = make_teacher(50, 150)
    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
    o = losses.distillation(a, b, dev, 2.0, target=target)
    (0.3 * o.loss.mean() + 0.7 * 4.0 * o.kl.mean() + 1e-3 * o.lse.square().mean()).backward()
    x, y = h.double().requires_grad_(), w.double().requires_grad_()
    z = x @ y.T
    rp = dev.row_ptr.tolist()
    kl = torch.zeros(50, dtype=torch.float64, device="cuda")
    logp = torch.log_softmax(z / 2.0, 1)
    for i in range(50):
        if rp[i + 1] > rp[i] and torch.isfinite(dev.val[rp[i]:rp[i + 1]]).any():
            q = torch.softmax(dev.val[rp[i]:rp[i + 1]].double() / 2.0, 0)
            kl[i] = (torch.special.xlogy(q, q) - q * logp[i, dev.col[rp[i]:rp[i + 1]].long()]).sum()
    ce = torch.nn.functional.cross_entropy(z, target, reduction="none", ignore_index=-100)
    (0.3 * ce.mean() + 0.7 * 4.0 * kl.mean() + 1e-3 * torch.logsumexp(z, 1).square().mean()).backward()
    # sums of at most 150 terms of 24 bits; a part in 2^16 of the largest is 2^5 times what they lose
    for got, want in ((a.grad, x.grad), (b.grad, y.grad)):
        assert (got.double() - want).abs().max() <= 2.0 ** -16 * want.abs().max()
    loss, lse = losses.cross_entropy(a, b.detach(), target)
    a.grad = None
    (loss.sum() + lse.sum()).backward()
    assert a.grad is not None and torch.isfinite(a.grad).all()


def test_other_stream_and_callers_workspace():
    h, w, target = make("bf16", 200, 264, 3000)
    loss0, lse0 = losses.xent_forward(h, w, target)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    loss, lse = losses.xent_forward(h, w, target, stream=s)
    s.synchronize()
    assert torch.equal(loss, loss0) and torch.equal(lse, lse0)
    lib = losses.load()
    z = losses.gm_logits(200, 3000, 264, h.data_ptr(), 264, w.data_ptr(), 264, losses.GM_LOSS_BF16)
    lab = losses.gm_labels(target.data_ptr(), -100, 0)
    need = ctypes.c_int64()
    assert lib.gm_loss_workspace(z, -1, 0, None, need) == 0
    work = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    cfg = losses.gm_loss_config(0, 0, work.data_ptr(), need.value - 1)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.gm_xent_forward(z, lab, cfg, stream, loss.data_ptr(), lse.data_ptr()) == 5  # GM_ERR_WORKSPACE
    loss.zero_()
    cfg.workspace = None  # the library's hooks
    assert lib.gm_xent_forward(z, lab, cfg, stream, loss.data_ptr(), lse.data_ptr()) == 0
    torch.cuda.synchronize()
    assert torch.equal(loss, loss0)


def test_graph_capture():
    h, w, target = make("bf16", 200, 264, 3000)
    (gl,), _ = weights(200, 1, 0)

    def step():
        loss, lse = losses.xent_forward(h, w, target)
        return (loss, *losses.xent_backward(h, w, target, lse, gl))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    h.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_class_table_past_32_bit_offsets():
    """2.4e9 elements in W and dW: rows at the far end are read and written there."""
    n, d, v = 3, 2048, 1170000
    w = torch.zeros(v, d, dtype=torch.bfloat16, device="cuda")
    far = [0, 1048575, 1048576, 1048577, v - 2, v - 1]
    g = torch.Generator(device="cuda").manual_seed(0)
    w[far] = torch.randn(len(far), d, generator=g, device="cuda").bfloat16()
    h = (torch.randn(n, d, generator=g, device="cuda") * 0.1).bfloat16()
    target = torch.tensor([v - 1, 1048576, 0], device="cuda")
    loss, lse = losses.xent_forward(h, w, target, check=True)
    z = h.double() @ w[far].double().T
    want = torch.log(torch.exp(z).sum(1) + (v - len(far)))
    # a logit's error is that of 2048 products of size 0.1 and 1, summed 1024 at a time
    assert (lse.double() - want).abs().max() < 1e-4
    at = torch.tensor([far.index(int(t)) for t in target], device="cuda")
    assert (loss.double() - (want - z[torch.arange(n, device="cuda"), at])).abs().max() < 2e-4
    gl = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    dh, dw = losses.xent_backward(h, w, target, lse, gl, check=True)
    p = torch.exp(z - want[:, None]) * gl.double()[:, None]
    p[torch.arange(n, device="cuda"), at] -= gl.double()
    want_w = p.T @ h.double()
    assert (dw[far].double() - want_w).abs().max() <= 2.0 ** -7 * want_w.abs().max()
    want_h = p @ w[far].double()
    assert (dh.double() - want_h).abs().max() <= 2.0 ** -7 * want_h.abs().max()
    # a class nobody has: its gradient is its probability's part alone
    rest = (gl.double() / torch.exp(want)) @ h.double()
    assert (dw[1000000].double() - rest).abs().max() <= 2.0 ** -7 * rest.abs().max()


def test_binding_refuses():
    h, w, target = make("bf16", 20, 40, 100)
    dev, _ = make_teacher(20, 100)
    bad = [(h.float(), w, target), (h, w[:, :39], target), (h.t(), w, target), (h[None], w, target), (h, w, target.float()),
           (h, w, target[:19]), (h, w, target.cpu()), (h, w.cpu(), target), (h[:, ::2], w[:, ::2], target),
           (h[:1].expand(20, 40), w, target), (h.double(), w.double(), target)]
    for args in bad:
        with pytest.raises(ValueError):
            losses.xent_forward(*args)
    _, lse = losses.xent_forward(h, w, target)
    for kw in ({"lse": lse[:5]}, {"grad_loss": lse.half()}, {"grad_loss": lse[::2]}):
        a = dict(lse=lse, grad_loss=lse)
        a.update(kw)
        with pytest.raises(ValueError):
            losses.xent_backward(h, w, target, **a)
    short = binding.DeviceCSR(20, 100, dev.row_ptr[:-1], dev.col, dev.val)
    half = binding.DeviceCSR(20, 100, dev.row_ptr, dev.col, dev.val.half())
    for t in (short, half):
        with pytest.raises(ValueError):
            losses.distill_forward(h, w, t)
    with pytest.raises(binding.GmError):
        losses.distill_forward(h, w, binding.DeviceCSR(20, 101, dev.row_ptr, dev.col, dev.val))
    with pytest.raises(binding.GmError):
        losses.distill_forward(h, w, dev, 0.0)


def test_rows_of_a_sparse_product_teach():
    """C = A A of an R-MAT graph: its rows, as spgemm returns them, are the teacher."""
    A = inputs.rmat(8, 8, seed=2)
    dA = binding.to_device(A)
    C = binding.spgemm(dA, dA)
    n = A.n_rows
    h, w, _ = make("f32", n, 32, n)
    o = losses.distill_forward(h, w, C, 1.0, check=True)
    host = lo.Teacher(C.row_ptr.cpu().numpy(), C.col.cpu().numpy(), C.val.cpu().numpy())
    f = lo.forward(wide(h), wide(w), None, -100, host, 1.0)
    check_forward(f, h, w, 1.0, kl=o.kl, lse_t=o.lse_t)


def test_vertex_embedding_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "vertex_embedding.py")
    spec = importlib.util.spec_from_file_location("vertex_embedding", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    means = example.train(scale=9, edge_factor=8, dim=32, batch=256, steps=60)
    assert torch.isfinite(means).all()
    assert means[-4:].mean() < 0.8 * means[:4].mean()  # chance is the logarithm of 512 vertices


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,v,cap", [(1, 33, 300, 0), (6, 130, 1000, 0), (100, 65, 513, 0), (300, 264, 1111, 0), (150, 129, 700, 1)])
def test_workspace_is_as_large_as_said(kind, n, d, v, cap):
    """The caller's workspace has gm_loss_workspace's bytes, and the memory around it is left alone."""
    h, w, target = make(kind, n, d, v)
    dev, _ = make_teacher(n, v)
    (gk, gl), _ = weights(n, 2, 0)
    want = losses.distill_forward(h, w, dev, 2.0, target=target)
    want_g = losses.distill_backward(h, w, dev, want.lse_t, gk, 2.0, target=target, lse=want.lse, grad_loss=gl,
                                     workspace_cap_bytes=cap)
    lib = losses.load()
    z = losses.gm_logits(n, v, d, h.data_ptr(), h.stride(0), w.data_ptr(), w.stride(0), losses.TYPES[h.dtype])
    lab = losses.gm_labels(target.data_ptr(), -100, 0)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    out = [torch.empty_like(t) for t in want]
    dh, dw = torch.empty(n, d, dtype=h.dtype, device="cuda"), torch.empty(v, d, dtype=h.dtype, device="cuda")
    for backward in (0, 1):
        cfg = losses.gm_loss_config(cap, 0, None, 0)
        need = ctypes.c_int64()
        assert lib.gm_loss_workspace(z, dev.nnz, backward, cfg, need) == 0
        memory = torch.full((need.value + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
        cfg.workspace, cfg.workspace_bytes = memory.data_ptr() + 4096, need.value
        if backward:
            rc = lib.gm_distill_backward(z, dev.desc(), 1, 0, 2.0, lab, cfg, stream, want.lse_t.data_ptr(), gk.data_ptr(),
                                         want.lse.data_ptr(), gl.data_ptr(), None, dh.data_ptr(), d, dw.data_ptr(), d)
        else:
            rc = lib.gm_distill_forward(z, dev.desc(), 1, 0, 2.0, lab, cfg, stream, *(t.data_ptr() for t in out))
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.all(memory[:4096] == 0xa5) and torch.all(memory[4096 + need.value:] == 0xa5)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert torch.equal(dh, want_g[0]) and torch.equal(dw, want_g[1])


def test_streams_at_once():
    """Calls on several streams, other tensor-core work between them: the same results bit by bit."""
    problems = []
    for kind, n, d, v in (("bf16", 300, 264, 3000), ("f32", 200, 64, 5000), ("f16", 50, 129, 4000), ("bf16", 1, 512, 9000)):
        h, w, target = make(kind, n, d, v, ignored=0.0)
        dev, _ = make_teacher(n, v)
        (gk, gl), _ = weights(n, 2, 0)
        problems.append((h, w, target, dev, gk, gl))

    def step(h, w, target, dev, gk, gl):
        o = losses.distill_forward(h, w, dev, 2.0, target=target)
        return (*o, *losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, target=target, lse=o.lse, grad_loss=gl))

    want = [step(*p) for p in problems]
    a = torch.randn(1024, 1024, device="cuda").bfloat16()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for turn in range(12):
        for k, p in enumerate(problems):
            with torch.cuda.stream(streams[(turn + k) % 3]):
                got.append((k, step(*p)))
                a @ a
    torch.cuda.synchronize()
    for k, o in got:
        assert all(torch.equal(x, y) for x, y in zip(o, want[k]))

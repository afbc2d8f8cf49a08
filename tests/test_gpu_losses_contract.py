"""What the losses promise where inputs, callers or memory are out of the ordinary: reports that belong to one call,
masked classes, weights far apart, teachers with large values, malformed row pointers, bounded workspace."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import loss_oracle as lo
from sparse_gemm_irregular_gm_gb300 import binding, losses
from test_gpu_losses import check_forward, check_grads, make, make_teacher, near, weights, wide

pytestmark = pytest.mark.gpu


def test_host_threads_with_rows_of_different_lengths():
    """The few-row kernels' shared memory goes with the row length: calls of several threads do not meet."""
    lib = losses.load()
    held, calls = [], []
    for d in (64, 4096, 64, 4096):
        h, w, target = make("f32", 8, d, 700, ignored=0.0)
        want = losses.xent_forward(h, w, target)
        z = losses.gm_logits(8, 700, d, h.data_ptr(), d, w.data_ptr(), d, losses.GM_LOSS_F32)
        lab = losses.gm_labels(target.data_ptr(), -100, 0)
        need = ctypes.c_int64()
        assert lib.gm_loss_workspace(z, -1, 0, None, need) == 0
        work = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        cfg = losses.gm_loss_config(0, 0, work.data_ptr(), need.value)
        got = [torch.empty_like(t) for t in want]
        stream = torch.cuda.Stream()
        held.append((h, w, target, work, stream, want, got))
        calls.append((z, lab, cfg, ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(got[0].data_ptr()),
                      ctypes.c_void_p(got[1].data_ptr())))
    torch.cuda.synchronize()
    statuses = [set() for _ in calls]

    def turn(k):
        for _ in range(4000):
            statuses[k].add(lib.gm_xent_forward(*calls[k]))

    threads = [threading.Thread(target=turn, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert statuses == [{0}] * len(calls)
    for *_, want, got in held:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_a_checked_call_reports_its_own_rows_alone():
    """Another call's bad target is neither raised by a checked call nor taken from gm_loss_status."""
    h, w, target = make("bf16", 200, 72, 300, ignored=0.0)
    bad = target.clone()
    bad[11] = 300
    one_h, one_target = h[:1], target[:1]
    losses.xent_forward(h, w, bad)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    loss, lse = losses.xent_forward(h, w, target, check=True)
    losses.xent_forward(one_h, w, one_target, check=True, stream=other)
    (gl,), _ = weights(200, 1, 0)
    losses.xent_backward(h, w, target, lse, gl, check=True)
    none = h[:0]
    losses.xent_forward(none, w, target[:0], check=True)
    with pytest.raises(binding.GmError) as e:
        losses.gm_loss_status()
    assert e.value.status == 9  # GM_ERR_BAD_INDEX
    losses.gm_loss_status()
    for step in (lambda: losses.xent_forward(h, w, bad, check=True), lambda: losses.xent_backward(h, w, bad, lse, gl, check=True),
                 lambda: losses.xent_backward(one_h, w, bad[11:12], lse[:1], gl[:1], check=True)):
        with pytest.raises(binding.GmError) as e:
            step()
        assert e.value.status == 9
        losses.gm_loss_status()  # told once, by the call itself


@pytest.mark.parametrize("kind,n", [("bf16", 200), ("f16", 60), ("f32", 140), ("f32", 5), ("bf16", 1)])
def test_rows_without_a_target_and_the_gradient_by_lse(kind, n):
    """An ignored row's lse has its gradient; a row whose target is out of range has none at all."""
    h, w, target = make(kind, n, 72, 300, ignored=0.0)
    loss, lse = losses.xent_forward(h, w, target, check=True)
    (gl, gs), (gl_n, gs_n) = weights(n, 2, 0, scale=64.0 if kind == "f16" else 1.0)
    row = n // 2
    target[row] = -100
    tn = target.cpu().numpy()
    f = lo.forward(wide(h), wide(w), tn)
    dh, dw = losses.xent_backward(h, w, target, lse, gl, gs, check=True)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n, gs_n), h, w, kind, 1.0, dh, dw)
    assert torch.any(dh[row] != 0)
    target[row] = 300
    gs_n[row] = 0.0
    dh, dw = losses.xent_backward(h, w, target, lse, gl, gs)
    with pytest.raises(binding.GmError):
        losses.gm_loss_status()
    assert torch.all(dh[row] == 0)
    check_grads(f, lo.logit_grads(f, tn, -100, gl_n, gs_n), h, w, kind, 1.0, dh, dw)


@pytest.mark.parametrize("offset", [1e9, -3e12, 1e300])
@pytest.mark.parametrize("longest", [40, 3000])
def test_teachers_values_are_large_and_close(offset, longest):
    """64-bit values count by their distance to the row's largest, however large they are."""
    n, v = 50, 3000
    h, w, _ = make("bf16", n, 40, v)
    dev, host = make_teacher(n, v, longest=longest, val=torch.float64)
    dev.val.add_(offset)
    host = lo.Teacher(host.row_ptr, host.col, dev.val.cpu().numpy())
    o = losses.distill_forward(h, w, dev, 1.5, check=True)
    f = lo.forward(wide(h), wide(w), None, -100, host, 1.5)
    # the oracle divides by the temperature before it subtracts: as far apart as that rounds
    spread = 2.0 ** -51 * abs(offset)
    if spread < 1e-2:
        bounds = lo.forward_bounds(f, wide(h), wide(w), 1.5)
        near(o.kl, f["kl"], bounds["kl"] + 8 * spread * (np.abs(f["z"]).max(1) + np.abs(f["kl"]) + 1), "kl")
    else:  # the values' own differences are rounded away: -inf and one value
        q, base = lo.teacher_rows(lo.Teacher(host.row_ptr, host.col, np.where(np.isinf(host.val), host.val, 0.0)), 1.5, n, v)
        kl = np.where(q.sum(1) > 0, base - (q * f["z"]).sum(1) / 1.5 + f["lse_t"], 0.0)
        near(o.kl, kl, lo.forward_bounds(f, wide(h), wide(w), 1.5)["kl"], "kl")


def test_teachers_lowest_values_over_a_small_temperature():
    """Rows of nothing but the type's lowest value are uniform, as rows of any one value are."""
    n, v = 40, 300
    h, w, _ = make("bf16", n, 40, v)
    dev, host = make_teacher(n, v, empty=0.0)
    dev.val.fill_(torch.finfo(torch.float32).min)
    host = lo.Teacher(host.row_ptr, host.col, np.zeros_like(host.val))
    o = losses.distill_forward(h, w, dev, 0.5, check=True)
    f = lo.forward(wide(h), wide(w), None, -100, host, 0.5)
    check_forward(f, h, w, 0.5, kl=o.kl, lse_t=o.lse_t)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lowest", [False, True])
@pytest.mark.parametrize("n,d", [(1, 65), (5, 65), (140, 65), (300, 129), (60, 200), (140, 1100)])
def test_classes_masked_by_their_bias(kind, lowest, n, d):
    """The last column of h is 1, that of w a bias: -inf, or the type's lowest value, takes a class out, and the rest are
    as if it were not there."""
    v = 400
    h, w, target = make(kind, n, d, v)
    h[:, -1] = 1
    w[:, -1] = 0
    keep = torch.arange(v) % 3 != 1
    w[(~keep).cuda(), -1] = torch.finfo(w.dtype).min if lowest else -torch.inf
    new = (torch.cumsum(keep, 0) - 1).numpy()
    target = torch.where(target < 0, target, target // 3 * 3)
    tn = target.cpu().numpy()
    tn = np.where(tn < 0, tn, new[tn])
    dev, host = make_teacher(n, v, longest=20)
    dev.col.copy_(dev.col)
    # entries on masked classes have probability 0
    masked = ~keep.numpy()[host.col]
    dev.val[torch.from_numpy(masked).cuda()] = -torch.inf
    rows = np.repeat(np.arange(n), np.diff(host.row_ptr))[~masked]
    rp = np.concatenate([[0], np.cumsum(np.bincount(rows, minlength=n))])
    host = lo.Teacher(rp, new[host.col[~masked]], host.val[~masked])
    wk = w[keep.cuda()]
    o = losses.distill_forward(h, w, dev, 2.0, target=target, check=True)
    f = lo.forward(wide(h), wide(wk), tn, -100, host, 2.0)
    check_forward(f, h, wk, 2.0, kl=o.kl, lse_t=o.lse_t, loss=o.loss, lse=o.lse)
    (gk, gl), (gk_n, gl_n) = weights(n, 2, d, scale=64.0 if kind == "f16" else 1.0)
    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, 2.0, target=target, lse=o.lse, grad_loss=gl, check=True)
    assert torch.all(dw[(~keep).cuda()] == 0)
    # 0 times -inf spoils the column of biases, as in any product; f16's lowest times a G of 2^-24 does not
    (eh, bh), (ew, bw) = lo.gradient_bounds(f, lo.logit_grads(f, tn, -100, gl_n, None, 2.0, gk_n), wide(h), wide(wk), kind, 2.0)
    near(dh[:, :-1], eh[:, :-1], bh[:, :-1], "dh")
    near(dw[keep.cuda()], ew, bw, "dw")


@pytest.mark.parametrize("n,d,v", [(140, 64, 5000), (300, 1100, 3000), (90, 130, 5000), (12, 1100, 4000), (300, 200, 20000)])
@pytest.mark.parametrize("cap", [0, 1])
@pytest.mark.parametrize("labels", [True, False])
def test_half_precision_with_weights_far_apart(n, d, v, cap, labels):
    """Each row's dH is as near as its own weight asks, not the largest one's: what f16 cannot hold of a row's G is at
    most 2^-11 of the row's weight, over all classes. dW's G is scaled by the largest weight, to at least 2^13, and loses
    half a unit of 2^-24."""
    h, w, target = make("f16", n, d, v, ignored=0.0)
    h *= 0.25
    w *= 4.0
    tn = target.cpu().numpy()
    weight = 2.0 ** (11 - np.arange(n) % 24)
    given = torch.from_numpy(weight.astype(np.float32)).cuda()
    if labels:
        _, lse = losses.xent_forward(h, w, target, check=True)
        f = lo.forward(wide(h), wide(w), tn)
        dh, dw = losses.xent_backward(h, w, target, lse, given, workspace_cap_bytes=cap, check=True)
        g, soft, hard = lo.logit_grads(f, tn, -100, weight)
        weight, top = 2 * weight, np.abs(f["lse"])
    else:
        dev, host = make_teacher(n, v)
        o = losses.distill_forward(h, w, dev, 1.0, check=True)
        f = lo.forward(wide(h), wide(w), None, -100, host, 1.0)
        dh, dw = losses.distill_backward(h, w, dev, o.lse_t, given, 1.0, workspace_cap_bytes=cap, check=True)
        g, soft, hard = lo.logit_grads(f, temperature=1.0, g_kl=weight)
        top = np.abs(f["lse_t"])
    u = lo.ROUND["f16"]
    dx = 2 * lo.logit_error(wide(h), wide(w)).max(1) + 2.0 ** -22 * (72 + 8 * np.abs(f["z"]).max(1) + 4 * top)
    dg = soft * np.expm1(dx)[:, None] + 2.0 ** -22 * (soft + hard) + u * np.abs(g) * (1 + 2.0 ** -8)
    small = weight[:, None] * 2.0 ** -11 * np.abs(wide(w)).max(0)
    for got, a, x, da, lost, what in ((dh, g, wide(w), dg, small, "dh"), (dw, g.T, wide(h), dg.T + weight.max() * 2.0 ** -38, 0.0, "dw")):
        exact = a @ x
        bound = da @ np.abs(x) + (6 * (a.shape[1] / 16 + 1) + 16) * 2.0 ** -23 * (np.abs(a) @ np.abs(x)) + lost
        near(got, exact, bound + u * np.abs(exact) * (1 + 2.0 ** -8) + 2.0 ** -24, what)


@pytest.mark.parametrize("n", [60, 200])
def test_half_precision_with_a_weight_that_is_not_finite(n):
    """It spoils its own row of dH alone; weights of 0 beside it leave nothing."""
    h, w, target = make("f16", n, 72, 300, ignored=0.0)
    _, lse = losses.xent_forward(h, w, target)
    (gl,), _ = weights(n, 1, 0, scale=64.0)
    want, _ = losses.xent_backward(h, w, target, lse, gl)
    gl[3] = 0
    for x in (float("inf"), float("nan")):
        gl[7] = x
        dh, _ = losses.xent_backward(h, w, target, lse, gl, check=True)
        assert not torch.isfinite(dh[7]).any() and torch.all(dh[3] == 0)
        keep = [i for i in range(n) if i not in (3, 7)]
        # another scale of G alone: two roundings of 11 bits at most
        assert (dh[keep].double() - want[keep].double()).abs().max() <= 2.0 ** -9 * want.double().abs().max()


def test_workspace_of_a_forward_call_is_bounded():
    lib = losses.load()
    p = 1 << 20
    for rows, classes in ((1 << 20, 1 << 20), (1 << 22, 1 << 22), (8192, 1 << 30)):
        z = losses.gm_logits(rows, classes, 8, p, 8, p, 8, losses.GM_LOSS_BF16)
        need = ctypes.c_int64()
        assert lib.gm_loss_workspace(z, -1, 0, None, need) == 0
        # the statistics' piece, and 64 bytes a row
        assert need.value <= (512 << 20) + 64 * rows + 4096


@pytest.mark.parametrize("kind,n,d,v", [("bf16", 40000, 16, 262221), ("f32", 40000, 8, 262221), ("bf16", 2000, 40, 2200001),
                                        ("f16", 2000, 16, 4400001), ("bf16", 300, 8, 14400001), ("f32", 100, 8, 22000001)])
def test_forward_in_pieces_of_the_classes(kind, n, d, v):
    """Row statistics of more than 512 MiB: two to three pieces, whose sums are joined. The caller's workspace has
    gm_loss_workspace's bytes, and the memory around it is left alone."""
    g = torch.Generator(device="cuda").manual_seed(n)
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}[kind]
    h = torch.randn(n, d, generator=g, device="cuda").to(dtype)
    w = (torch.randn(v, d, generator=g, device="cuda") * (2.0 / d ** 0.5)).to(dtype)
    target = torch.randint(0, v, (n,), generator=g, device="cuda")
    target[0], target[-1], target[5] = 0, v - 1, -100
    dev, _ = make_teacher(n, v // 64)
    dev = binding.DeviceCSR(n, v, dev.row_ptr, dev.col * 64 + 63, dev.val)
    temperature = 2.0
    out = losses.distill_forward(h, w, dev, temperature, target=target, check=True)
    lib = losses.load()
    z = losses.gm_logits(n, v, d, h.data_ptr(), d, w.data_ptr(), d, losses.TYPES[dtype])
    lab = losses.gm_labels(target.data_ptr(), -100, 0)
    need = ctypes.c_int64()
    assert lib.gm_loss_workspace(z, dev.nnz, 0, None, need) == 0
    memory = torch.full((need.value + 8192,), 0xa5, dtype=torch.uint8, device="cuda")
    cfg = losses.gm_loss_config(0, 0, memory.data_ptr() + 4096, need.value)
    again = [torch.empty_like(t) for t in out]
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.gm_distill_forward(z, dev.desc(), 1, 0, temperature, lab, cfg, stream, *(t.data_ptr() for t in again)) == 0
    torch.cuda.synchronize()
    assert torch.all(memory[:4096] == 0xa5) and torch.all(memory[4096 + need.value:] == 0xa5)
    assert all(torch.equal(a, b) for a, b in zip(again, out)) and all(torch.isfinite(t).all() for t in out)
    loss, lse = losses.xent_forward(h, w, target, check=True)
    W, rp = w.double(), dev.row_ptr.tolist()
    for i in sorted({*range(0, n, max(1, n // 40)), 5, n - 1}):
        zi = W @ h[i].double()
        dz = (6 * (d / 16 + 1) + 8) * 2.0 ** -23 * float((W.abs() @ h[i].double().abs()).max())
        big, want, want_t = float(zi.abs().max()), float(torch.logsumexp(zi, 0)), float(torch.logsumexp(zi / temperature, 0))
        # loss_oracle.forward_bounds
        bound = dz + 2.0 ** -22 * (64 + 4 * big + abs(want))
        assert abs(float(lse[i]) - want) <= bound and abs(float(out.lse[i]) - want) <= bound
        bound_t = dz / temperature + 2.0 ** -22 * (64 + 4 * big / temperature + abs(want_t))
        assert abs(float(out.lse_t[i]) - want_t) <= bound_t
        want_loss = 0.0 if i == 5 else want - float(zi[target[i]])
        for x in (loss[i], out.loss[i]):
            assert abs(float(x) - want_loss) <= bound + dz + 2.0 ** -22 * (big + abs(want))
        val = dev.val[rp[i]:rp[i + 1]].double() / temperature
        kl = 0.0
        if val.numel() and not torch.all(val == -torch.inf):
            q = torch.softmax(val, 0)
            kl = float(torch.xlogy(q, q).sum() - q @ zi[dev.col[rp[i]:rp[i + 1]].long()] / temperature + want_t)
        assert abs(float(out.kl[i]) - kl) <= bound_t + dz / temperature + 2.0 ** -20 * (8 + big / temperature + abs(want_t) + abs(kl))


@pytest.mark.parametrize("n,at", [(8, 0), (300, 7), (300, 290), (4097, 3), (4097, 4090), (9000, 5000), (200000, 199000)])
@pytest.mark.parametrize("row_ptr", [torch.int64, torch.int32])
@pytest.mark.parametrize("length", [10, 2500])
def test_teacher_rows_that_share_entries(n, at, row_ptr, length):
    """Row pointers fall back into the middle of row `at`: the rows that lie in it are refused, and it is not spoilt by
    them, nor are those before and after. Row at + 3 is empty and has nothing to share."""
    v = 3000
    h, w, target = make("bf16", n, 16, v, ignored=0.0)
    lens = np.full(n, 2)
    lens[at] = length
    lens[at + 1:at + 5] = (0, length // 2, 0, length - length // 2)
    rp = np.concatenate([[0], np.cumsum(lens)])
    g = torch.Generator().manual_seed(n)
    # ascending in every row, those that share entries too
    col = np.concatenate([np.arange(k) for k in lens])
    val = torch.randn(int(rp[-1]), generator=g)
    good = binding.DeviceCSR(n, v, torch.from_numpy(rp).to(row_ptr).cuda(), torch.from_numpy(col).int().cuda(), val.cuda())
    want = losses.distill_forward(h, w, good, 2.0, check=True)
    gk = torch.ones(n, device="cuda")
    gk[at + 1:at + 5] = 0
    want_h, want_w = losses.distill_backward(h, w, good, want.lse_t, gk, 2.0, check=True)
    start = int(rp[at])
    fall = rp.copy()
    fall[at + 2:at + 5] = (start, start + length // 2, start + length // 2)
    fall[at + 5:] -= length
    fall = torch.from_numpy(fall).to(row_ptr).cuda()
    # what row at held, then the rows after the four that lie in it
    keep = torch.cat([torch.arange(start + length), torch.arange(start + 2 * length, int(rp[-1]))]).cuda()
    bad = binding.DeviceCSR(n, v, fall, good.col[keep], good.val[keep])
    assert fall[at + 1] == start + length and fall[at + 5] == start + length
    spoilt = [at + 1, at + 2, at + 4]
    for _ in range(3):
        o = losses.distill_forward(h, w, bad, 2.0)
        with pytest.raises(binding.GmError) as e:
            losses.gm_loss_status()
        assert e.value.status == 9  # GM_ERR_BAD_INDEX
        assert torch.nonzero(torch.isnan(o.kl)).flatten().tolist() == spoilt
        rest = torch.ones(n, dtype=torch.bool, device="cuda")
        rest[at + 1:at + 5] = False
        assert torch.equal(o.kl[rest], want.kl[rest]) and o.kl[at + 3] == 0 and torch.equal(o.lse_t, want.lse_t)
        dh, dw = losses.distill_backward(h, w, bad, o.lse_t, torch.ones(n, device="cuda"), 2.0)
        with pytest.raises(binding.GmError):
            losses.gm_loss_status()
        assert torch.equal(dh, want_h) and torch.equal(dw, want_w)

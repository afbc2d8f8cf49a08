"""The losses at sizes where blocks walk several tiles or turns of classes: every element of the results against 64
bits, formed on the GPU by torch from the definitions, under the bounds of loss_oracle."""
import pytest
import torch

from loss_oracle import ROUND
from sparse_gemm_irregular_gm_gb300 import losses
from test_gpu_losses import make, make_teacher

pytestmark = pytest.mark.gpu


def rows_max(x):
    return x.abs().amax(1)


def teacher_q(dev, temperature, n, v):
    """Dense q and sum q log q of each row."""
    q, base = torch.zeros(n, v, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    rp = dev.row_ptr.tolist()
    for i in range(n):
        val = dev.val[rp[i]:rp[i + 1]].double() / temperature
        if val.numel() and not torch.all(val == -torch.inf):
            p = torch.softmax(val, 0)
            q[i, dev.col[rp[i]:rp[i + 1]].long()] = p
            base[i] = torch.xlogy(p, p).sum()
    return q, base


def logit_error(h, w):
    """loss_oracle.logit_error's bound, the largest of each row."""
    return (6 * (h.shape[1] / 16 + 1) + 8) * 2.0 ** -23 * (h.abs() @ w.abs().T).amax(1)


def check(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    over = (got.double() - want).abs() - bound
    assert bool((over <= 0).all()), f"{what}: {float(over.max()):.3g} over the bound"


def run(kind, n, d, v, temperature=2.0, cap=0, longest=40, **layout):
    """A distillation with labels and a cross entropy, forward and backward."""
    h, w, target = make(kind, n, d, v, seed=n + d, **layout)
    dev, _ = make_teacher(n, v, seed=d, longest=longest)
    g = torch.Generator().manual_seed(v)
    gk, gl, gs = ((torch.rand(3, n, generator=g) + 0.5) * ((64.0 if kind == "f16" else 1.0) / n)).cuda()
    H, W = h.double(), w.double()
    z = H @ W.T
    dz, big = logit_error(H, W), rows_max(z)
    use = target >= 0
    at = target.clamp(min=0).long()
    lse, lse_t = torch.logsumexp(z, 1), torch.logsumexp(z / temperature, 1)
    loss = torch.where(use, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    q, base = teacher_q(dev, temperature, n, v)
    has = q.sum(1) > 0
    kl = torch.where(has, base - (q * z).sum(1) / temperature + lse_t, 0.0)
    # loss_oracle.forward_bounds
    b_lse = dz + 2.0 ** -22 * (64 + 4 * big) + 2.0 ** -22 * lse.abs()
    b_lse_t = dz / temperature + 2.0 ** -22 * (64 + 4 * big / temperature) + 2.0 ** -22 * lse_t.abs()
    b_loss = b_lse + dz + 2.0 ** -22 * (big + lse.abs())
    b_kl = b_lse_t + dz / temperature + 2.0 ** -20 * (8 + big / temperature + lse_t.abs() + kl.abs())
    o = losses.distill_forward(h, w, dev, temperature, target=target, check=True)
    x_loss, x_lse = losses.xent_forward(h, w, target, check=True)
    for got, want, bound, what in ((o.kl, kl, b_kl, "kl"), (o.lse_t, lse_t, b_lse_t, "lse_t"), (o.loss, loss, b_loss, "loss"),
                                   (o.lse, lse, b_lse, "lse"), (x_loss, loss, b_loss, "xent loss"), (x_lse, lse, b_lse, "xent lse")):
        check(got, want, bound, what)

    def grads(with_kl):
        """loss_oracle.logit_grads and gradient_bounds."""
        wl = torch.where(use, gl.double(), 0.0)
        a = wl + gs.double()
        soft = a[:, None] * torch.exp(z - lse[:, None])
        hard = torch.zeros_like(z)
        hard.scatter_add_(1, at[:, None], -wl[:, None])
        top = lse.abs()
        t = 1.0
        if with_kl:
            b = torch.where(has, gk.double() / temperature, 0.0)
            soft += b[:, None] * torch.exp(z / temperature - lse_t[:, None])
            hard -= b[:, None] * q
            top = torch.maximum(top, lse_t.abs())
            t = min(1.0, temperature)
        G, soft, hard = soft + hard, soft.abs(), hard.abs()
        u = ROUND[kind]
        dx = 2 * dz / t + 2.0 ** -22 * (72 + 8 * big / t + 4 * top)
        dg = soft * torch.expm1(dx)[:, None] + 2.0 ** -22 * (soft + hard) + u * G.abs() * (1 + 2.0 ** -8)
        if kind == "f16":
            dg += 8 * float(hard.amax()) * 2.0 ** -37 + float((soft + hard).amax()) * 2.0 ** -36
        out = []
        for A, X, dA in ((G, W, dg), (G.T, H, dg.T)):
            exact = A @ X
            bound = dA @ X.abs() + (6 * (A.shape[1] / 16 + 1) + 16) * 2.0 ** -23 * (A.abs() @ X.abs())
            out.append((exact, bound + u * exact.abs() * (1 + 2.0 ** -8) + (2.0 ** -24 if kind == "f16" else 1e-37)))
        return out

    dh, dw = losses.distill_backward(h, w, dev, o.lse_t, gk, temperature, target=target, lse=o.lse, grad_loss=gl, grad_lse=gs,
                                     workspace_cap_bytes=cap, check=True)
    for got, (want, bound), what in zip((dh, dw), grads(True), ("dh", "dw")):
        check(got, want, bound, what)
    dh, dw = losses.xent_backward(h, w, target, x_lse, gl, gs, workspace_cap_bytes=cap, check=True)
    for got, (want, bound), what in zip((dh, dw), grads(False), ("xent dh", "xent dw")):
        check(got, want, bound, what)


# Tiles of 256 by 256 over a pair of SMs (76 pairs) or 128 by 256 over one (152): the logits of 300 x 40000 are 314 of
# the first kind, so that each of a pair's two reader groups takes a tile twice; of 100 x 160003 626 (f32: 1251) of the
# second. 24000 classes: 188 tiles with the sums in registers. dW of 40000 x 600 has 471 tiles, dH of 20000 x 300 158.
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,d,v", [(300, 64, 40000), (100, 64, 160003), (300, 1100, 24000), (100, 1100, 60001), (300, 600, 40000),
                                   (20000, 300, 300), (257, 200, 40001)])
def test_blocks_that_walk_several_tiles(kind, n, d, v):
    run(kind, n, d, v)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_pieces_of_several_tiles(kind):
    """16 MiB of G: pieces of some 4000 to 28000 classes, whose dH is added up."""
    run(kind, 300, 200, 60007, cap=16 << 20)


# 100003 classes over at most 1216 blocks: each has several turns of its warps. The dims take 1, 2 and 16 bytes a load,
# and one, several or all columns a thread; the table's alignment too.
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [33, 130, 1024, 2056, 4096])
def test_one_row_over_many_classes(kind, d):
    run(kind, 1, d, 100003, longest=3000)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,pad,shift", [(1024, 1, 0), (1024, 0, 1), (130, 2, 2), (4096, 0, 3)])
def test_one_row_over_many_classes_off_16_byte_boundaries(kind, d, pad, shift):
    run(kind, 1, d, 100003, longest=500, pad=pad, shift=shift)


@pytest.mark.parametrize("n", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("d,pad", [(305, 0), (1024, 0), (4096, 0), (2056, 1)])
def test_few_f32_rows_over_many_classes(n, d, pad):
    run("f32", n, d, 100003, longest=3000, pad=pad)

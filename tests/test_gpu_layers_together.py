"""The layers with the losses after them and the draw, as a model uses them: a block's norms and products, trained through
the cross entropy over a class table, then classes drawn from its logits."""
import copy

import pytest
import torch
import torch.nn.functional as F

from sparse_gemm_irregular_gm_gb300 import layers, losses, sampling

pytestmark = pytest.mark.gpu
ROWS, DIM, WIDE, CLASSES = 200, 136, 328, 1003


def weights(kind, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g, device="cuda") * std + mean).to(kind)  # noqa: E731
    p = {"first": n(DIM, std=0.1, mean=1.0), "up": n(WIDE, DIM, std=DIM ** -0.5), "up_bias": n(WIDE, std=0.1), "down": n(DIM, WIDE, std=WIDE ** -0.5),
         "after": n(DIM, std=0.1, mean=1.0), "gate": n(DIM, std=0.1, mean=0.5), "last": n(DIM, std=0.1, mean=1.0), "table": n(CLASSES, DIM, std=0.3)}
    return p, n(ROWS, DIM, std=2.0), torch.randint(0, CLASSES, (ROWS,), generator=g, device="cuda")


def block(p, x):
    """x plus a gated, normed two-layer block of its norm; the norm of that."""
    _, y = layers.residual_norm(x, before=p["first"])
    h = layers.linear(y, p["up"], p["up_bias"], activation="gelu")
    f = layers.linear(h, p["down"], residual=y)
    return layers.residual_norm(x, f, after=p["after"], gate=p["gate"], scale=0.8, before=p["last"])


def plain(p, x):
    rms = lambda v, w: v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    y = rms(x, p["first"])
    f = F.gelu(y @ p["up"].T + p["up_bias"]) @ p["down"].T + y
    x2 = x + 0.8 * p["gate"] * rms(f, p["after"])
    return x2, rms(x2, p["last"])


def step(p, x, target):
    x2, h = block(p, x)
    loss, _ = losses.cross_entropy(h, p["table"], target)
    total = loss.mean() + 0.01 * x2.float().square().mean()
    return [total, *torch.autograd.grad(total, [x, *p.values()])]


@pytest.mark.parametrize("kind,room", [(torch.float32, 2e-5), (torch.bfloat16, 2.5e-2), (torch.float16, 3.2e-3)])
def test_training_step(kind, room):
    """Against 64 bits. room: of each gradient's norm. bf16's half step is 2^-8, f16's 2^-11: about six of them one after another between
    an input and its gradient (the two norms, the two products, their gradients), each on values that are sums of many."""
    p, x, target = weights(kind)
    p = {k: v.requires_grad_() for k, v in p.items()}
    x.requires_grad_()
    got = step(p, x, target)
    p64 = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    x64 = x.detach().double().requires_grad_()
    x2, h = plain(p64, x64)
    total = F.cross_entropy(h @ p64["table"].T, target) + 0.01 * x2.square().mean()
    ref = [total, *torch.autograd.grad(total, [x64, *p64.values()])]
    for name, a, b in zip(["loss", "x", *p], got, ref):
        assert (a.double() - b).norm() <= room * b.norm(), (name, ((a.double() - b).norm() / b.norm()).item())


def test_two_blocks_in_a_graph_replayed():
    p, x, target = weights(torch.bfloat16)
    p = {k: v.requires_grad_() for k, v in p.items()}
    x.requires_grad_()

    def run():
        x2, _ = block(p, x)
        _, h = block(p, x2)
        loss, _ = losses.cross_entropy(h, p["table"], target)
        return [loss, *torch.autograd.grad(loss.sum(), [x, *p.values()])]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = run()
    q, x2, t2 = weights(torch.bfloat16, seed=7)
    with torch.no_grad():
        for k in p:
            p[k].copy_(q[k])
        x.copy_(x2)
        target.copy_(t2)
    g.replay()
    now = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(now, run()))


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_answering(rows):
    p, x, _ = weights(torch.bfloat16)
    _, h = block(p, x[:rows])
    z, _ = layers.linear_forward(h, p["table"])
    u = torch.rand(rows, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    d = sampling.draw(z, u, temperature=0.7, top_k=30, top_p=0.9)
    assert ((d.index >= 0) & (d.index < CLASSES)).all() and ((d.kept >= 1) & (d.kept <= 30)).all()
    greedy = sampling.draw(z, u, temperature=0.0)
    best = z.float().amax(1)
    assert torch.equal(z.float().gather(1, greedy.index[:, None])[:, 0], best)
    # the log-probability by the losses' log-sum, of the same logits before they were rounded: a step of bf16 is 2^-8 of a logit
    whole = sampling.draw(z, u)
    loss, _ = losses.xent_forward(h, p["table"], whole.index)
    assert ((whole.logprob + loss).abs() <= 2.0 ** -8 * (z.float().abs().amax(1) + 1) * 2).all()


def test_a_copied_module_of_parameters_trains():
    """Parameters that are views, copies or frozen make no difference to the others' gradients."""
    p, x, target = weights(torch.bfloat16)
    p = {k: v.requires_grad_() for k, v in p.items()}
    x.requires_grad_()
    ref = dict(zip(["loss", "x", *p], step(p, x, target)))
    q = {k: copy.deepcopy(v) for k, v in p.items()}
    for k in ("up", "gate"):
        q[k].requires_grad_(False)
    x2, h = block(q, x)
    loss, _ = losses.cross_entropy(h, q["table"], target)
    (loss.mean() + 0.01 * x2.float().square().mean()).backward()
    for k in ("down", "after", "table", "first"):
        assert torch.equal(q[k].grad, ref[k]) or (q[k].grad.double() - ref[k].double()).norm() <= 1e-6 * ref[k].double().norm(), k
    assert q["up"].grad is None and q["gate"].grad is None


def test_gradients_of_leaves_in_a_graph():
    """backward() captured with no eager graph of the leaves alive: each replay writes their gradients."""
    p, x, target = weights(torch.bfloat16)
    p = {k: v.requires_grad_() for k, v in p.items()}

    def step():
        _, h = block(p, x)
        losses.cross_entropy(h, p["table"], target)[0].sum().backward()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    ref = {k: v.grad.clone() for k, v in p.items() if v.grad is not None}
    for v in p.values():
        v.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        g.replay()
        assert ref and all(torch.equal(p[k].grad, r) for k, r in ref.items())

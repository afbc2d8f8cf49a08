"""Cases of the losses over a large vocabulary: what is timed, on which inputs, and the plain form of each.

Two operators, both on logits that are the product of a hidden state and a class table, Z = H W^T (H: rows x dim,
W: classes x dim), and that are never kept:

* softmax cross entropy (xent): loss_i = lse_i - z_i,t(i) with lse_i = log sum_j exp(z_ij), and its gradient;
* distillation from a teacher's top logits (distill): the teacher's row i is a CSR row, q_i the softmax of its stored
  values over the temperature T, kl_i = sum_k q_ik (log q_ik - log_softmax(z_i / T)_k), and its gradient; with labels
  too, the same pass also returns the cross entropy of the rows.

A row whose target is -100 has no loss and no gradient; so has a teacher's row without entries.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100


def listed():
    """Classes are the vertices of the repository's R-MAT graphs (2^16, 2^18, 2^20) or a generic vocabulary."""
    return [
        # log-probability of one token while serving: reading the class table once is all there is to do
        {"name": "xent-token", "op": "xent", "step": False, "type": "bf16", "rows": 1, "dim": 1024, "classes": 32768},
        # scoring a batch of text without a gradient, vocabulary not a multiple of anything
        {"name": "xent-scoring", "op": "xent", "step": False, "type": "bf16", "rows": 2000, "dim": 1024, "classes": 131071},
        # a small model's step with every size odd, rows of H and W not on 16-byte boundaries, scaled half precision
        {"name": "xent-step-odd", "op": "xent", "step": True, "type": "f16", "rows": 333, "dim": 129, "classes": 10007},
        # an ordinary training step of the head
        {"name": "xent-step", "op": "xent", "step": True, "type": "bf16", "rows": 4096, "dim": 1024, "classes": 50021},
        # vertices of a scale-16 graph embedded in 32 bits, next vertex predicted
        {"name": "xent-vertices-f32", "op": "xent", "step": True, "type": "f32", "rows": 1000, "dim": 128, "classes": 65536},
        # all vertices of a scale-20 graph as classes: the class table's gradient is most of the traffic
        {"name": "xent-vertices-long", "op": "xent", "step": True, "type": "bf16", "rows": 512, "dim": 256, "classes": 1048576},
        # the largest step: a batch of 8192 tokens on a large model's head
        {"name": "xent-step-large", "op": "xent", "step": True, "type": "bf16", "rows": 8192, "dim": 4096, "classes": 131072},
        # how far the model is from its teacher on four tokens, while serving
        {"name": "distill-token", "op": "distill", "step": False, "type": "bf16", "rows": 4, "dim": 2048, "classes": 32768,
         "top": 32, "ragged": False, "labels": False, "temp": 1.0},
        # a distillation step on half-precision weights, odd sizes
        {"name": "distill-step-odd", "op": "distill", "step": True, "type": "f16", "rows": 777, "dim": 520, "classes": 32003,
         "top": 17, "ragged": False, "labels": False, "temp": 2.0},
        # an ordinary distillation step: teacher's top 64, and the labels too
        {"name": "distill-step", "op": "distill", "step": True, "type": "bf16", "rows": 2048, "dim": 1024, "classes": 65536,
         "top": 64, "ragged": False, "labels": True, "temp": 2.0},
        # rows of a sparse product of graphs as the teacher: power-law lengths, empty rows among them, 32 bits
        {"name": "distill-ragged-f32", "op": "distill", "step": True, "type": "f32", "rows": 1500, "dim": 64, "classes": 262144,
         "top": 100, "ragged": True, "labels": False, "temp": 1.0},
        # the largest distillation step
        {"name": "distill-step-large", "op": "distill", "step": True, "type": "bf16", "rows": 8192, "dim": 2048, "classes": 131072,
         "top": 128, "ragged": False, "labels": True, "temp": 2.0},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["bf16", "bf16", "f16", "f32"])
    while True:
        rows, dim, classes = _log_uniform(rng, 1, 8192), _log_uniform(rng, 32, 4096), _log_uniform(rng, 1000, 1048576)
        if rng.random() < 0.5:  # half of the tables have rows on 16-byte boundaries, as most models' have
            dim = max(32, dim // 8 * 8)
        most = 1.5e12 if kind == "f32" else 1.2e13
        if 6.0 * rows * dim * classes <= most and rows * classes <= 1 << 30 and classes * dim <= 1 << 29:
            break
    case = {"op": rng.choice(["xent", "distill"]), "step": rng.random() < 0.75, "type": kind, "rows": rows, "dim": dim, "classes": classes}
    if case["op"] == "distill":
        case.update(top=_log_uniform(rng, 1, 256), ragged=rng.random() < 0.4, labels=rng.random() < 0.5, temp=rng.choice([0.75, 1.0, 2.0, 4.0]))
    return case


def _teacher(g, case):
    """A teacher's rows as CSR: column ids distinct and ascending in a row, more of them low (frequent) than high."""
    rows, classes, top = case["rows"], case["classes"], case["top"]
    dev = g.device
    if case["ragged"]:
        u = torch.rand(rows, generator=g, device=dev, dtype=torch.float64)
        lens = (0.3 * top * (1.0 / (1.0 - u * 0.9999)).pow(0.8)).long()  # power law: most short, a few very long
        lens = torch.where(torch.rand(rows, generator=g, device=dev) < 0.1, 0, lens)
        lens = lens.clamp(max=classes // 2)
    else:
        lens = torch.full((rows,), min(top, classes), device=dev, dtype=torch.int64)
    row_ptr = torch.zeros(rows + 1, dtype=torch.int64, device=dev)
    row_ptr[1:] = lens.cumsum(0)
    nnz = int(row_ptr[-1])
    row = torch.repeat_interleave(torch.arange(rows, device=dev), lens, output_size=nnz)
    x = torch.rand(nnz, generator=g, device=dev, dtype=torch.float64) ** 3
    x = (row + x * 0.999999).sort().values - row
    at = torch.arange(nnz, device=dev) - row_ptr[row]
    col = (at + torch.floor((classes - lens[row]) * x.clamp(0, 0.999999)).long()).to(torch.int32)
    val = torch.randn(nnz, generator=g, device=dev) * 2.0 + 8.0
    return row_ptr, col, val


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 17)
    kind = TYPES[case["type"]]
    rows, dim, classes = case["rows"], case["dim"], case["classes"]
    h = torch.randn(rows, dim, generator=g, device=dev).to(kind)  # after a norm
    w = torch.empty(classes, dim, device=dev, dtype=kind)
    for lo in range(0, classes, 65536):  # logits of a deviation of 2
        n = min(65536, classes - lo)
        w[lo:lo + n] = (torch.randn(n, dim, generator=g, device=dev) * (2.0 / math.sqrt(dim))).to(kind)
    s = {"case": dict(case), "h": h, "w": w}
    target = (torch.rand(rows, generator=g, device=dev, dtype=torch.float64) ** 3 * classes).long().clamp(max=classes - 1)
    drop = torch.rand(rows, generator=g, device=dev) < (0.06 if rows > 8 else 0.0)  # padding has no label
    s["target"] = torch.where(drop, IGNORE, target)
    if case["op"] == "distill":
        s["row_ptr"], s["col"], s["val"] = _teacher(g, case)
    # weights of the rows' losses in the step's mean; half precision runs with a scaled loss, as such training does
    scale = 65536.0 if case["type"] == "f16" else 1.0
    weight = torch.rand(rows, generator=g, device=dev) + 0.5
    s["grad_loss"] = (weight * (scale / rows)).float()
    s["grad_kl"] = (torch.rand(rows, generator=g, device=dev) * (scale / rows)).float()
    return s


def _labels(case):
    return case["op"] == "xent" or case["labels"]


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from sparse_gemm_irregular_gm_gb300 import binding, losses
    case, h, w = s["case"], s["h"], s["w"]
    if case["op"] == "xent":
        loss, lse = losses.xent_forward(h, w, s["target"], ignore_index=IGNORE)
        out = {"loss": loss, "lse": lse}
        if case["step"]:
            out["dh"], out["dw"] = losses.xent_backward(h, w, s["target"], lse, s["grad_loss"], ignore_index=IGNORE)
        return out
    teacher = binding.DeviceCSR(case["rows"], case["classes"], s["row_ptr"], s["col"], s["val"])
    target = s["target"] if case["labels"] else None
    f = losses.distill_forward(h, w, teacher, case["temp"], target=target, ignore_index=IGNORE)
    out = {"kl": f.kl, "lse_t": f.lse_t}
    if case["labels"]:
        out.update(loss=f.loss, lse=f.lse)
    if case["step"]:
        out["dh"], out["dw"] = losses.distill_backward(
            h, w, teacher, f.lse_t, s["grad_kl"], case["temp"], target=target, lse=f.lse,
            grad_loss=s["grad_loss"] if case["labels"] else None, ignore_index=IGNORE)
    return out


def _plain_lse(z):
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    t = e.sum(1, keepdim=True)
    return e.div_(t), (m + torch.log(t)).squeeze(1)


def _plain(s):
    case, h, w = s["case"], s["h"].float(), s["w"].float()
    z = h @ w.T
    grad, out = None, {}
    if _labels(case):
        p, lse = _plain_lse(z)
        valid = s["target"] != IGNORE
        at = s["target"].clamp(min=0).unsqueeze(1)
        out["loss"] = (lse - z.gather(1, at).squeeze(1)) * valid
        out["lse"] = lse
        if case["step"]:
            gl = (s["grad_loss"] * valid).unsqueeze(1)
            grad = p.mul_(gl)
            grad.scatter_add_(1, at, -gl)
    if case["op"] == "distill":
        temp, rows = case["temp"], case["rows"]
        p, lse = _plain_lse(z / temp)
        lens = s["row_ptr"][1:] - s["row_ptr"][:-1]
        row = torch.repeat_interleave(torch.arange(rows, device=z.device), lens, output_size=s["col"].numel())
        col = s["col"].long()
        v = s["val"] / temp
        m = torch.full((rows,), -torch.inf, device=z.device).scatter_reduce(0, row, v, "amax")
        e = torch.exp(v - m[row])
        t = torch.zeros(rows, device=z.device).index_add(0, row, e)
        q = e / t[row]
        log_q = v - m[row] - torch.log(t)[row]
        has = lens > 0
        out["kl"] = torch.zeros(rows, device=z.device).index_add(0, row, q * (log_q - z[row, col] / temp + lse[row]))
        out["lse_t"] = lse
        if case["step"]:
            gk = s["grad_kl"] / temp * has
            p = p.mul_(gk.unsqueeze(1))
            p.index_put_((row, col), -(q * gk[row]), accumulate=True)
            grad = p if grad is None else grad.add_(p)
    if case["step"]:
        out["dh"] = (grad @ w).to(s["h"].dtype)
        out["dw"] = (grad.T @ h).to(s["w"].dtype)
    return out


def work(case):
    rows, dim, classes = case["rows"], case["dim"], case["classes"]
    size = 4 if case["type"] == "f32" else 2
    both = (rows + classes) * dim * size
    n = both + 8 * rows  # H, W; loss and lse
    if _labels(case):
        n += 8 * rows + (8 * rows if case["op"] == "distill" else 0)
    if case["op"] == "distill":
        n += 8 * (rows + 1) + 8 * _entries(case)
    if case["step"]:
        n += both + 4 * rows
    # the logits, and for a step the two products of their gradient; a second product for the logits, which a step that
    # does not keep them makes, is not counted
    return {"bytes": float(n), "flops": (6.0 if case["step"] else 2.0) * rows * dim * classes}


def _entries(case):
    """Entries of the teacher: its rows' lengths summed (ragged ones: about the power law's mean)."""
    top = min(case["top"], case["classes"])
    return int(case["rows"] * top * (0.9 * 0.3 * 4.2 if case["ragged"] else 1.0))


def exact(case, seed):
    rows, dim, classes = case["rows"], case["dim"], case["classes"]
    if 6.0 * rows * dim * classes > 3e12 or rows * classes > 1 << 29:
        return None
    s = prepare(case, seed)
    step = case["step"]
    h = s["h"].double().requires_grad_(step)
    w = s["w"].double().requires_grad_(step)
    z = torch.nn.functional.linear(h, w)
    total, out = 0.0, {}
    if _labels(case):
        lse = torch.logsumexp(z, 1)
        use = torch.nonzero(s["target"] >= 0).squeeze(1)
        loss = torch.zeros(rows, dtype=torch.float64, device=z.device)
        loss = loss.index_put((use,), lse[use] - z[use, s["target"][use]])
        out.update(loss=loss, lse=lse)
        total = total + (loss * s["grad_loss"].double()).sum()
    if case["op"] == "distill":
        y = z / case["temp"]
        lse_t = torch.logsumexp(y, 1)
        ptr = s["row_ptr"].tolist()
        full = [i for i in range(rows) if ptr[i + 1] > ptr[i]]
        longest = max([ptr[i + 1] - ptr[i] for i in full], default=1)
        lens = (s["row_ptr"][1:] - s["row_ptr"][:-1]).unsqueeze(1)
        k = torch.arange(longest, device=z.device).unsqueeze(0)
        inside = k < lens
        at = (s["row_ptr"][:-1].unsqueeze(1) + k).clamp(max=max(ptr[-1] - 1, 0))
        at = torch.where(inside, at, 0)
        if ptr[-1]:
            v = torch.where(inside, s["val"].double()[at] / case["temp"], -torch.inf)
            log_q = torch.where(lens > 0, torch.log_softmax(torch.where(lens > 0, v, 0.0), 1), 0.0)
            col = torch.where(inside, s["col"].long()[at], 0)
            log_p = y.gather(1, col) - lse_t.unsqueeze(1)
            kl = torch.where(inside, torch.exp(log_q) * (torch.where(inside, log_q, 0.0) - log_p), 0.0).sum(1)
        else:
            kl = 0.0 * lse_t
        out.update(kl=kl, lse_t=lse_t)
        total = total + (kl * s["grad_kl"].double()).sum()
    out = {n: t.detach() for n, t in out.items()}
    if step:
        out["dh"], out["dw"] = torch.autograd.grad(total, (h, w))
    return out

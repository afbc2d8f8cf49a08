"""Cases of the operators before and after the class table: what is timed, on which inputs, and the plain form of each.

Three operators. Two make the rows H that the losses read, the third answers from the logits:

* product (linear): y = r + act(x W^T + b), with its gradient by x, W and b (by r it is the gradient of y itself);
* norms around a residual (norm): x' = x + s g p with p = n(f) w_a + c_a, and y = n(x') w_b + c_b, where n divides a row by
  its root mean square (rms) or takes its mean off first (layer), and g is a vector or a matrix; with its gradient by x,
  f, g and the norms' weights;
* a class drawn from logits (draw) with one given random number a row: softmax(z / T) is cut to the top_k largest
  logits, then to the shortest run of the largest whose share reaches top_p, then to those of at least min_p times the
  largest's probability; equal logits are taken from the lowest class on. The class is the first, in class order, at which the
  probability summed passes u. T = 0 takes the largest. Returned with the log of its probability and how many were kept.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    """Dims and classes are those of the losses' cases, or generic."""
    return [
        # the projection of one token while serving: the weights are read once
        {"name": "linear-token", "op": "linear", "step": False, "type": "bf16", "rows": 1, "dim": 4096, "outs": 4096, "act": "silu", "bias": True, "residual": True},
        # logits of a batch of 24 sequences over a class table
        {"name": "linear-logits", "op": "linear", "step": False, "type": "f16", "rows": 24, "dim": 1024, "outs": 32768, "act": "none", "bias": False, "residual": False},
        # a small model's layer with every size odd, rows not on 16-byte boundaries
        {"name": "linear-step-odd", "op": "linear", "step": True, "type": "f16", "rows": 333, "dim": 129, "outs": 517, "act": "relu", "bias": True, "residual": True},
        # embeddings of vertices in 32 bits through a hidden layer
        {"name": "linear-step-f32", "op": "linear", "step": True, "type": "f32", "rows": 1000, "dim": 128, "outs": 512, "act": "gelu_tanh", "bias": True, "residual": False},
        # the wide layer of a block in training
        {"name": "linear-step", "op": "linear", "step": True, "type": "bf16", "rows": 8192, "dim": 1024, "outs": 4096, "act": "gelu", "bias": True, "residual": False},
        # the narrow layer of a large block, added to the residual
        {"name": "linear-step-large", "op": "linear", "step": True, "type": "bf16", "rows": 8192, "dim": 16384, "outs": 4096, "act": "none", "bias": False, "residual": True},
        # between two blocks for one token
        {"name": "norm-token", "op": "norm", "step": False, "type": "bf16", "rows": 1, "dim": 4096, "norm": "rms", "after": True, "gate": "vector", "bias": False},
        # rows that are not on 16-byte boundaries, means taken off, a gate for every element
        {"name": "norm-step-odd", "op": "norm", "step": True, "type": "f16", "rows": 1001, "dim": 517, "norm": "layer", "after": True, "gate": "matrix", "bias": True},
        # between two blocks in training
        {"name": "norm-step", "op": "norm", "step": True, "type": "bf16", "rows": 8192, "dim": 4096, "norm": "rms", "after": True, "gate": "vector", "bias": False},
        # the next token of one sequence
        {"name": "draw-token", "op": "draw", "type": "bf16", "rows": 1, "classes": 131072, "rule": "all", "per_row": False},
        # the next tokens of a batch whose requests each have their own rule, logits in 32 bits, classes not a multiple of anything
        {"name": "draw-batch-mixed", "op": "draw", "type": "f32", "rows": 37, "classes": 50021, "rule": "all", "per_row": True},
        # a large batch, cut by share alone
        {"name": "draw-batch", "op": "draw", "type": "bf16", "rows": 256, "classes": 131072, "rule": "top_p", "per_row": False},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op, kind = rng.choice(["linear", "norm", "draw"]), rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "linear":
        while True:
            rows, dim, outs = _log_uniform(rng, 1, 8192), _log_uniform(rng, 16, 16384), _log_uniform(rng, 16, 32768)
            if rng.random() < 0.6:  # most layers' rows lie on 16-byte boundaries
                dim, outs = max(16, dim // 8 * 8), max(16, outs // 8 * 8)
            if 6.0 * rows * dim * outs <= (2e11 if kind == "f32" else 3e12):
                break
        return {"op": op, "step": rng.random() < 0.7, "type": kind, "rows": rows, "dim": dim, "outs": outs,
                "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), "bias": rng.random() < 0.6, "residual": rng.random() < 0.5}
    if op == "norm":
        while True:
            rows, dim = _log_uniform(rng, 1, 16384), _log_uniform(rng, 16, 8192)
            if rng.random() < 0.6:
                dim = max(16, dim // 8 * 8)
            if rows * dim <= 1 << 25:
                break
        return {"op": op, "step": rng.random() < 0.7, "type": kind, "rows": rows, "dim": dim, "norm": rng.choice(["rms", "layer"]),
                "after": rng.random() < 0.7, "gate": rng.choice(["none", "vector", "matrix"]), "bias": rng.random() < 0.5}
    while True:
        rows, classes = _log_uniform(rng, 1, 4096), _log_uniform(rng, 100, 262144)
        if rows * classes <= 1 << 25:
            break
    return {"op": op, "type": kind, "rows": rows, "classes": classes, "rule": rng.choice(["none", "top_k", "top_p", "min_p", "all", "all"]),
            "per_row": rng.random() < 0.5}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 1000003 + 29)
    kind = TYPES[case["type"]]
    rows = case["rows"]

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).add_(mean).to(kind)

    def uniform(n):
        return torch.rand(n, generator=g, device=dev)

    s = {"case": dict(case)}
    if case["op"] == "linear":
        dim, outs = case["dim"], case["outs"]
        s["x"] = normal(rows, dim)  # after a norm
        s["w"] = normal(outs, dim, std=1.0 / math.sqrt(dim))
        s["b"] = normal(outs, std=0.5) if case["bias"] else None
        s["r"] = normal(rows, outs, std=2.0) if case["residual"] else None
        if case["step"]:
            s["grad"] = normal(rows, outs, std=0.1)
    elif case["op"] == "norm":
        dim = case["dim"]
        s["x"] = normal(rows, dim, std=3.0, mean=0.1)
        s["f"] = normal(rows, dim, std=0.7)
        s["after"] = normal(dim, std=0.1, mean=1.0) if case["after"] else None
        s["before"] = normal(dim, std=0.1, mean=1.0)
        s["after_bias"] = normal(dim, std=0.1) if case["after"] and case["bias"] else None
        s["before_bias"] = normal(dim, std=0.1) if case["bias"] else None
        s["gate"] = {"none": None, "vector": normal(dim, std=0.2, mean=0.5), "matrix": normal(rows, dim, std=0.3, mean=0.5)}[case["gate"]]
        if case["step"]:
            s["grad_x"] = normal(rows, dim, std=0.1)
            s["grad_y"] = normal(rows, dim, std=0.1)
    else:
        z = torch.randn(rows, case["classes"], generator=g, device=dev)
        z.mul_(1.0 + 3.0 * uniform(rows).unsqueeze(1))  # some rows are flat, some are sure
        masked = torch.rand(rows, case["classes"], generator=g, device=dev) < 0.03
        s["z"] = torch.where(masked, -torch.inf, z).to(kind)  # classes that a grammar forbids
        s["u"] = uniform(rows)
        rule, per_row = case["rule"], case["per_row"]
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.8, 0, 1.0, 0.0
        if per_row:
            s["temperature"] = torch.where(uniform(rows) < 0.1, 0.0, 0.4 + uniform(rows))  # some are greedy
        if rule in ("top_k", "all"):
            s["top_k"] = 50
            if per_row:
                s["top_k"] = torch.where(uniform(rows) < 0.2, 0, torch.exp(uniform(rows) * math.log(1000.0)).to(torch.int32))
        if rule in ("top_p", "all"):
            s["top_p"] = 0.95
            if per_row:
                s["top_p"] = torch.where(uniform(rows) < 0.2, 1.0, 0.3 + 0.69 * uniform(rows))
        if rule in ("min_p", "all"):
            s["min_p"] = 0.02
            if per_row:
                s["min_p"] = torch.where(uniform(rows) < 0.2, 0.0, 0.2 * uniform(rows) ** 2)
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return _own_draw(s) if op == "draw" else _own_norm(s) if op == "norm" else _own_linear(s)
    return _plain_draw(s) if op == "draw" else _plain_norm(s) if op == "norm" else _plain_linear(s)


# ---- product ------------------------------------------------------------------------------
def _own_linear(s):
    from sparse_gemm_irregular_gm_gb300 import layers
    act, step = s["case"]["act"], s["case"]["step"]
    y, z = layers.linear_forward(s["x"], s["w"], s["b"], activation=act, residual=s["r"], keep=step)
    out = {"y": y}
    if step:
        out["dx"], out["dw"], db = layers.linear_backward(s["x"], s["w"], s["grad"], activation=act, z=z, need_bias=s["b"] is not None)
        if db is not None:
            out["db"] = db
    return out


def _plain_act(z, act):
    """act(z) and its slope."""
    if act == "none":
        return z, None
    if act == "relu":
        return z.clamp(min=0), (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * p, p + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z * z)


def _plain_linear(s):
    kind, act = s["x"].dtype, s["case"]["act"]
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T
    if s["b"] is not None:
        z = z + s["b"].float()
    y, slope = _plain_act(z, act)
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"y": y.to(kind)}
    if s["case"]["step"]:
        dz = s["grad"].float()
        if slope is not None:
            dz = dz * slope
        out["dx"] = (dz @ w).to(kind)
        out["dw"] = (dz.T @ x).to(kind)
        if s["b"] is not None:
            out["db"] = dz.sum(0).to(kind)
    return out


# ---- norms around a residual -----------------------------------------------------------------
def _own_norm(s):
    from sparse_gemm_irregular_gm_gb300 import layers
    case = s["case"]
    rule = dict(norm=case["norm"], after=s["after"], after_bias=s["after_bias"], gate=s["gate"], scale=0.7, before=s["before"],
                before_bias=s["before_bias"], eps=EPS)
    x2, y, stats = layers.residual_norm_forward(s["x"], s["f"], **rule)
    out = {"x": x2, "y": y}
    if case["step"]:
        d = layers.residual_norm_backward(s["x"], s["f"], s["grad_x"], s["grad_y"], stats, **rule)
        out.update({"d" + k: v for k, v in d._asdict().items() if v is not None})
    return out


def _plain_unit(x, norm):
    """n(x) of each row, and what its rows were divided by."""
    if norm == "layer":
        x = x - x.mean(1, keepdim=True)
    size = torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    return x / size, size


def _plain_unit_grad(d, unit, size, norm):
    """The gradient by x, given that by n(x)."""
    g = d - unit * (d * unit).mean(1, keepdim=True)
    if norm == "layer":
        g = g - d.mean(1, keepdim=True)
    return g / size


def _plain_norm(s):
    case, norm, kind = s["case"], s["case"]["norm"], s["x"].dtype
    x, p, scale = s["x"].float(), s["f"].float(), 0.7
    if case["after"]:
        unit_f, size_f = _plain_unit(p, norm)
        p = unit_f * s["after"].float()
        if case["bias"]:
            p = p + s["after_bias"].float()
    gate = scale if s["gate"] is None else scale * s["gate"].float()
    x2 = x + gate * p
    unit, size = _plain_unit(x2, norm)
    y = unit * s["before"].float()
    if case["bias"]:
        y = y + s["before_bias"].float()
    out = {"x": x2.to(kind), "y": y.to(kind)}
    if case["step"]:
        gy = s["grad_y"].float()
        dx = s["grad_x"].float() + _plain_unit_grad(gy * s["before"].float(), unit, size, norm)
        out["dx"] = dx.to(kind)
        dp = dx * gate
        df = _plain_unit_grad(dp * s["after"].float(), unit_f, size_f, norm) if case["after"] else dp
        out["df"] = df.to(kind)
        if s["gate"] is not None:
            dg = scale * dx * p
            out["dgate"] = (dg.sum(0) if case["gate"] == "vector" else dg).to(kind)
        if case["after"]:
            out["dafter"] = (dp * unit_f).sum(0).to(kind)
            if case["bias"]:
                out["dafter_bias"] = dp.sum(0).to(kind)
        out["dbefore"] = (gy * unit).sum(0).to(kind)
        if case["bias"]:
            out["dbefore_bias"] = gy.sum(0).to(kind)
    return out


# ---- a class drawn from logits -----------------------------------------------------------------
def _own_draw(s):
    from sparse_gemm_irregular_gm_gb300 import sampling
    d = sampling.draw(s["z"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return {"index": d.index, "logprob": d.logprob, "kept": d.kept}


def _plain_column(v, like):
    """A rule's value, one a row, in 64 bits; 32-bit numbers as they are."""
    if isinstance(v, torch.Tensor):
        return v.double().unsqueeze(1)
    return torch.full((like.shape[0], 1), float(np.float32(v)), dtype=torch.float64, device=like.device)


def _plain_draw(s):
    # sums of up to 2^18 weights meet borders between classes: 64 bits
    z, order = s["z"].double().sort(dim=1, descending=True, stable=True)
    temp, top_k, top_p, min_p = (_plain_column(s[k], z) for k in ("temperature", "top_k", "top_p", "min_p"))
    greedy = temp == 0
    at = torch.arange(z.shape[1], device=z.device)
    top_k = torch.where(greedy, 1, torch.where(top_k == 0, z.shape[1], top_k))
    w = torch.exp((z - z[:, :1]) / torch.where(greedy, 1.0, temp))
    keep = (at < top_k) & (w > 0)
    w = w * keep
    total = w.cumsum(1)
    before = torch.cat([torch.zeros_like(total[:, :1]), total[:, :-1]], 1)
    keep &= (top_p >= 1) | (before < top_p * total[:, -1:]) | (at == 0)
    keep &= w >= min_p
    w = torch.zeros_like(w).scatter(1, order, w * keep)  # from here on by class
    total = w.cumsum(1)
    all_ = total[:, -1:]
    index = torch.searchsorted(total, s["u"].double().unsqueeze(1) * all_, right=True)
    p = w.gather(1, index) / all_
    return {"index": index.squeeze(1), "logprob": torch.log(p).squeeze(1).float(), "kept": keep.sum(1).to(torch.int32)}


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    size = 4 if case["type"] == "f32" else 2
    rows = case["rows"]
    if case["op"] == "linear":
        dim, outs = case["dim"], case["outs"]
        n = rows * dim + outs * dim + rows * outs * (2 if case["residual"] else 1) + (outs if case["bias"] else 0)
        if case["step"]:
            n += rows * outs + rows * dim + outs * dim + (outs if case["bias"] else 0)
        return {"bytes": float(size * n), "flops": (6.0 if case["step"] else 2.0) * rows * dim * outs}
    if case["op"] == "norm":
        dim = case["dim"]
        vectors = 1 + (1 if case["after"] else 0) * (2 if case["bias"] else 1) + (1 if case["bias"] else 0) + (1 if case["gate"] == "vector" else 0)
        matrices = 4 + (1 if case["gate"] == "matrix" else 0)
        if case["step"]:
            matrices += 4 + (1 if case["gate"] == "matrix" else 0)
            vectors *= 2
        return {"bytes": float(size * dim * (matrices * rows + vectors)), "flops": (40.0 if case["step"] else 12.0) * rows * dim}
    return {"bytes": float(rows * (case["classes"] * size + 4 + 16 + (16 if case["per_row"] else 0))), "flops": 4.0 * rows * case["classes"]}


# ---- the same from the definitions, in 64 bits --------------------------------------------------------
def exact(case, seed):
    rows = case["rows"]
    if case["op"] == "draw":
        return _exact_draw(case, prepare(case, seed)) if rows * case["classes"] <= 1 << 26 else None
    if case["op"] == "linear" and 6.0 * rows * case["dim"] * case["outs"] > 5e12:
        return None
    s = prepare(case, seed)
    leaf = {k: v.double().requires_grad_(case["step"]) for k, v in s.items() if isinstance(v, torch.Tensor) and not k.startswith("grad")}
    F = torch.nn.functional
    if case["op"] == "linear":
        z = F.linear(leaf["x"], leaf["w"], leaf.get("b"))
        y = {"none": lambda t: t, "relu": F.relu, "silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[case["act"]](z)
        if "r" in leaf:
            y = y + leaf["r"]
        out, total = {"y": y}, None
        if case["step"]:
            total = (y * s["grad"].double()).sum()
        names = ["x", "w", "b"]
    else:
        dim = case["dim"]

        def normed(t, weight, bias):
            if case["norm"] == "layer":
                return F.layer_norm(t, (dim,), weight, bias, EPS)
            r = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS) * weight
            return r if bias is None else r + bias

        p = normed(leaf["f"], leaf["after"], leaf.get("after_bias")) if case["after"] else leaf["f"]
        x2 = leaf["x"] + 0.7 * (p if "gate" not in leaf else leaf["gate"] * p)
        y = normed(x2, leaf["before"], leaf.get("before_bias"))
        out, total = {"x": x2, "y": y}, None
        if case["step"]:
            total = (x2 * s["grad_x"].double()).sum() + (y * s["grad_y"].double()).sum()
        names = ["x", "f", "gate", "after", "after_bias", "before", "before_bias"]
    out = {k: v.detach() for k, v in out.items()}
    if case["step"]:
        names = [n for n in names if n in leaf]
        for n, d in zip(names, torch.autograd.grad(total, [leaf[n] for n in names])):
            out["d" + n] = d
    return out


def _exact_draw(case, s):
    z = s["z"].double().cpu().numpy()
    u = s["u"].double().cpu().numpy()
    rule = []
    for k in ("temperature", "top_k", "top_p", "min_p"):
        v = s[k]
        rule.append(v.double().cpu().numpy() if isinstance(v, torch.Tensor) else np.full(len(u), np.float64(np.float32(v))))
    index, logprob, kept = (np.zeros(len(u), t) for t in (np.int64, np.float64, np.int32))
    for i, (row, temp, top_k, top_p, min_p) in enumerate(zip(z, *rule)):
        alive = np.flatnonzero(row > -np.inf)
        v = row[alive]
        if temp == 0:
            index[i], kept[i] = alive[int(np.argmax(v))], 1
            continue
        by_size = np.argsort(-v, kind="stable")
        if top_k:
            by_size = by_size[:int(top_k)]
        e = np.exp((v[by_size] - v[by_size[0]]) / temp)
        if top_p < 1:
            e = e[:max(1, 1 + int(np.searchsorted(np.cumsum(e), top_p * e.sum(), side="left")))]
        e = e[e >= min_p]
        by_size = by_size[:len(e)]
        by_class = np.argsort(alive[by_size], kind="stable")
        e, classes = e[by_class], alive[by_size][by_class]
        sums = np.cumsum(e)
        j = min(int(np.searchsorted(sums, u[i] * sums[-1], side="right")), len(e) - 1)
        index[i], logprob[i], kept[i] = classes[j], math.log(e[j] / sums[-1]), len(e)
    return {"index": torch.from_numpy(index), "logprob": torch.from_numpy(logprob), "kept": torch.from_numpy(kept)}

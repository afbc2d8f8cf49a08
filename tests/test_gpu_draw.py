"""Classes drawn from logits on the GPU, against the rule applied class by class in 64 bits."""
import math

import numpy as np
import pytest
import torch

from sparse_gemm_irregular_gm_gb300 import sampling
from sparse_gemm_irregular_gm_gb300.binding import GmError

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# of the sum of a row's weights: each is within 2^-28 of itself and 2^-40 of the largest (up to 2^22 classes), the plain sums within 1e-12
DOUBT = 2.0 ** -27


def oracle(z, u, temp, top_k, top_p, min_p):
    """(index, log of its share, kept, whether each of index and kept is within DOUBT of another answer)."""
    alive = np.flatnonzero(z > -np.inf)
    v = z[alive]
    order = np.argsort(-v, kind="stable")
    if temp == 0:
        return alive[order[0]], 0.0, 1, False, False
    if top_k:
        order = order[:top_k]
    top = v[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(v[order] == top, 1.0, np.exp((v[order] - top) / temp))
    unsure = False
    if top_p < 1:
        sums = np.cumsum(w)
        n = max(1, 1 + int(np.searchsorted(sums, top_p * sums[-1], side="left")))
        unsure = any(0 <= j < len(sums) - 1 and abs(sums[j] - top_p * sums[-1]) <= DOUBT * sums[-1] and sums[j] != top_p * sums[-1]
                     for j in (n - 2, n - 1))
        w, order = w[:n], order[:n]
    keep = w >= min_p
    if min_p > 0:
        unsure = unsure or bool((np.abs(w - min_p) <= DOUBT * min_p)[w != 1].any())
    w, order = w[keep], order[keep]
    by_class = np.argsort(order, kind="stable")
    w, cls = w[by_class], alive[order[by_class]]
    sums = np.cumsum(w)
    goal = float(u) * sums[-1]
    j = min(int(np.searchsorted(sums, goal, side="right")), len(w) - 1)
    tied = len(set(w)) == 1  # equal weights add up exactly
    near = not tied and any(0 <= k < len(w) - 1 and abs(sums[k] - goal) <= DOUBT * sums[-1] for k in (j - 1, j))
    return cls[j], math.log(w[j] / sums[-1]), len(w), near or unsure, unsure


def check(z, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, most_unsure=0, **how):
    d = sampling.draw(z, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p, **how)
    rows = z.shape[0]
    value = lambda v: v.cpu().numpy() if isinstance(v, torch.Tensor) else np.full(rows, np.float32(v))  # noqa: E731
    rules = [value(v) for v in (temperature, top_k, top_p, min_p)]
    zs, us = z.double().cpu().numpy(), u.double().cpu().numpy()
    index, logprob, kept = (t.cpu().numpy() for t in d)
    unsure = 0
    for i in range(rows):
        t, k, p, m = (float(r[i]) for r in rules)
        j, lp, n, near, maybe = oracle(zs[i], us[i], t, int(k), p, m)
        if near or maybe:
            unsure += 1
            continue
        assert (index[i], kept[i]) == (j, n), (i, index[i], j, kept[i], n)
        # fp32's rounding of the result, 2^-24; weights and sums: 2^-27 of the share
        assert abs(float(logprob[i]) - lp) <= 2.0 ** -24 * abs(lp) + 2.0 ** -26, (i, logprob[i], lp)
    assert unsure <= most_unsure, unsure
    return d


def make(rows, classes, kind, seed=0, spread=3.0, masked=0.05, wide=0, offset=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 11)
    big = torch.full((rows * (classes + wide) + offset,), float("nan"), device="cuda", dtype=TYPES[kind])
    z = big[offset:].view(rows, classes + wide)[:, :classes]
    z.copy_(torch.randn(rows, classes, generator=g, device="cuda") * spread)
    z[torch.rand(rows, classes, generator=g, device="cuda") < masked] = -torch.inf
    z[:, classes // 2] = 0.25  # one at least
    return z, torch.rand(rows, generator=g, device="cuda")


RULES = [dict(), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.0),
         dict(temperature=0.7, top_k=50, top_p=0.95, min_p=0.01), dict(temperature=3.0, top_p=0.5), dict(top_p=0.0), dict(min_p=1.0),
         dict(top_k=1 << 30, top_p=0.999)]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("classes", [1, 2, 9, 100, 1025, 20011])
def test_rules(rule, kind, classes):
    check(*make(13, classes, kind, seed=classes), most_unsure=1, **rule)


@pytest.mark.parametrize("rows,classes", [(1, 7), (1, 8193), (1, 131072), (2, 262147), (40, 33333), (3, 400001), (200, 4099), (700, 300)])
@pytest.mark.parametrize("kind", TYPES)
def test_sizes(rows, classes, kind):
    z, u = make(rows, classes, kind, seed=rows)
    check(z, u, temperature=0.8, top_p=0.95, most_unsure=1)
    check(z, u, temperature=0.8, top_k=50, top_p=0.9, min_p=0.02, most_unsure=1)


@pytest.mark.parametrize("kind", TYPES)
def test_a_row_too_long_for_shared_memory(kind):
    z, u = make(2, 1700003, kind)
    check(z, u, most_unsure=1)
    check(z, u, top_k=1000, top_p=0.9, most_unsure=1)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("wide,offset", [(8, 0), (1, 0), (0, 3), (6, 5)])
@pytest.mark.parametrize("classes", [10, 2000, 70001])
def test_strides(kind, wide, offset, classes):
    z, u = make(5, classes, kind, wide=wide, offset=offset)
    check(z, u, temperature=1.2, top_k=300, top_p=0.97, most_unsure=1)


def test_a_rule_for_each_row():
    rows = 96
    z, u = make(rows, 5003, "f32", seed=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda: torch.rand(rows, generator=g, device="cuda")  # noqa: E731
    check(z, u, temperature=torch.where(r() < 0.2, 0.0, 0.2 + 2 * r()), top_k=(r() * 60).int(),
          top_p=torch.where(r() < 0.3, 1.0, r()), min_p=torch.where(r() < 0.3, 0.0, 0.3 * r()), most_unsure=1)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("classes", [64, 4096, 20000, 131072])
def test_equal_logits_are_taken_from_the_lowest_class_up(kind, classes):
    z = torch.full((4, classes), -3.0, device="cuda", dtype=TYPES[kind])
    u = torch.tensor([0.0, 0.25, 0.5, 1 - 2.0 ** -24], device="cuda")
    d = check(z, u)
    assert d.index.tolist() == [0, classes // 4, classes // 2, classes - 1] and (d.kept == classes).all()
    d = check(z, u, top_k=10)
    assert d.index.tolist() == [0, 2, 5, 9] and (d.kept == 10).all()
    d = check(z, u, top_p=0.5)
    assert d.index.tolist() == [0, classes // 8, classes // 4, classes // 2 - 1] and (d.kept == classes // 2).all()
    z[:, ::2] = -4.0  # a border inside the ties: only odd classes are largest
    d = check(z, u, top_k=12, min_p=0.9)
    assert d.index.tolist() == [1, 7, 13, 23]
    z[:, 5] = 2.0  # largest alone, then the ties
    # borders lie exp(-5) apart in a sum of up to 300: a random number is within 2^-27 of the sum of one with a chance of 2 * 300 * 2^-27 * exp(5),
    # 1 in 1500
    g = torch.Generator(device="cuda").manual_seed(3)
    check(z, torch.rand(4, device="cuda", generator=g), top_k=classes // 3, top_p=0.75, most_unsure=1)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("mask", ["none", "lowest", "both"])
@pytest.mark.parametrize("rows", [2, 160])
def test_rows_of_which_most_is_masked(kind, mask, rows):
    """Tens of thousands of equal logits: more than a 16-bit count holds."""
    classes = 200000 if rows == 2 else 140001
    z, u = make(rows, classes, kind, masked=0.0, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    hide = torch.rand(rows, classes, generator=g, device="cuda") < 0.97
    hide[:, 1000] = False
    low = torch.finfo(TYPES[kind]).min
    z[hide] = -torch.inf if mask == "none" else low
    if mask == "both":
        z[:, ::3] = -torch.inf
    z[:, 1000] = 1.0
    check(z, u, temperature=0.9, top_p=0.9, most_unsure=1)
    check(z, u, temperature=0.9, top_k=20, top_p=0.95, min_p=0.01, most_unsure=1)
    check(z, u, most_unsure=1)
    z[0] = low  # nothing but the mask
    check(z[:2], u[:2], top_p=0.5)
    check(z[:2], u[:2], top_k=70001)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("tiny", [False, True])
def test_zeros_and_tiny_logits_between_others(kind, tiny):
    z, u = make(6, 30000, kind, spread=1.0, seed=12)
    z[:, ::7] = 0.0
    if tiny:
        z[:, 3::11] = 2.0 ** -100 if kind == "bf16" else 2.0 ** -24
        z[:, 5::13] = -2.0 ** -120 if kind == "bf16" else -2.0 ** -24
    check(z, u, top_p=0.97, most_unsure=1)
    check(z, u, temperature=0.5, most_unsure=1)
    check(z, u, min_p=0.001, top_k=25000, most_unsure=1)


def test_zeros_of_both_signs_are_equal():
    z = torch.tensor([[0.0, -0.0, 0.0, -0.0, -1.0]], device="cuda").repeat(4, 1)
    u = torch.tensor([0.1, 0.3, 0.6, 0.9], device="cuda")
    for kind in TYPES.values():
        d = sampling.draw(z.to(kind), u, top_k=4)
        assert d.index.tolist() == [0, 1, 2, 3] and (d.kept == 4).all()
        assert sampling.draw(-z[:, :4].to(kind), u, temperature=0.0).index.tolist() == [0] * 4


@pytest.mark.parametrize("kind", TYPES)
def test_infinite_and_lowest_logits(kind):
    t = TYPES[kind]
    z = torch.full((5, 300), -torch.inf, device="cuda", dtype=t)
    z[0, 17] = -5.0  # the only one
    z[1, [3, 250]] = torch.inf  # they share the weight
    z[1, 8] = 3.0
    z[2] = torch.finfo(t).min  # a mask of the type's lowest value, everywhere
    z[3] = torch.finfo(t).min
    z[3, 99] = 1.0
    z[4, 7], z[4, 8] = torch.finfo(t).max, torch.finfo(t).min
    u = torch.tensor([0.9, 0.75, 0.5, 0.999, 0.3], device="cuda")
    d = sampling.draw(z, u)
    assert d.index.tolist() == [17, 250, 150, 99, 7]
    assert d.kept.tolist() == [1, 3, 300, 300, 2]
    assert torch.allclose(d.logprob, torch.tensor([0.0, math.log(0.5), -math.log(300), 0.0, 0.0], device="cuda"), atol=2e-7)
    assert sampling.draw(z, u, min_p=0.5).kept.tolist() == [1, 2, 300, 1, 1]
    assert sampling.draw(z, u, top_p=0.9, top_k=4).kept.tolist() == [1, 2, 4, 1, 1]
    assert sampling.draw(z, u, temperature=0.0).index.tolist() == [17, 3, 0, 99, 7]


@pytest.mark.parametrize("classes", [5, 40000])
def test_rows_that_cannot_be_drawn_from_say_so_and_stay_alone(classes):
    z, u = make(8, classes, "bf16", masked=0.0)
    good = sampling.draw(z, u)
    z[1] = -torch.inf
    z[2, classes - 1] = torch.nan
    z[3, 0] = -torch.nan
    u[4], u[5], u[6] = 1.0, -0.1, torch.nan
    d = sampling.draw(z, u)
    assert d.index[1:7].tolist() == [-1] * 6 and d.kept[1:7].tolist() == [0] * 6 and d.logprob[1:7].isnan().all()
    for a, b in zip(d, good):
        assert torch.equal(a[[0, 7]], b[[0, 7]])
    z, u = make(8, classes, "bf16", masked=0.0)
    bad = torch.tensor([1.0, -1.0, torch.inf, torch.nan, 1e-39, 1.0, 1.0, 1.0], device="cuda")
    assert sampling.draw(z, u, temperature=bad).index[1:5].tolist() == [-1] * 4
    assert sampling.draw(z, u, top_p=torch.tensor([1.0, -0.1, 1.1, torch.nan] * 2, device="cuda")).kept[1:4].tolist() == [0] * 3
    assert sampling.draw(z, u, min_p=torch.tensor([0.0, -0.1, 1.1, torch.nan] * 2, device="cuda")).kept[1:4].tolist() == [0] * 3
    assert sampling.draw(z, u, top_k=torch.tensor([0, -1] * 4, device="cuda", dtype=torch.int32)).kept[1::2].tolist() == [0] * 4


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rows,classes", [(1, 131072), (8, 131072), (40, 131072), (64, 131072), (100, 131072), (9, 524288), (30, 300000)])
def test_shares_reached_only_by_some_of_the_classes_at_the_border(kind, rows, classes):
    """Of many equal logits top-k keeps some, and top-p needs them: the sums without them fall short."""
    z, u = make(rows, classes, kind, spread=1.0, seed=rows)
    z[z < 2.5] = 2.5  # most are equal, and lowest
    check(z, u, top_k=classes // 3, top_p=0.9, most_unsure=1)
    check(z, u, top_k=classes // 2, top_p=0.999, min_p=0.01, most_unsure=1)
    z[:, 40:] = -torch.inf  # fewer than top_k
    check(z, u, top_k=700, top_p=0.95, most_unsure=1)


def test_negative_zero_is_zero():
    z, u = make(3, 500, "f32")
    a = sampling.draw(z, torch.zeros_like(u), top_p=0.0, min_p=0.0)
    b = sampling.draw(z, -torch.zeros_like(u), top_p=torch.full((3,), -0.0, device="cuda"), min_p=torch.full((3,), -0.0, device="cuda"))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(sampling.draw(z, u, temperature=torch.full((3,), -0.0, device="cuda")).index, z.argmax(1))


def test_offsets_past_32_bits():
    rows, classes = 17000, 131072  # 2.2e9 logits
    z = torch.empty(rows, classes, device="cuda", dtype=torch.bfloat16)
    z[:-3] = 0.0
    z[-3:], u3 = make(3, classes, "bf16", seed=21)
    u = torch.zeros(rows, device="cuda")
    u[-3:] = u3
    d = sampling.draw(z, u, top_k=50, top_p=0.9)
    ref = sampling.draw(z[-3:].clone(), u3, top_k=50, top_p=0.9)
    assert all(torch.equal(a[-3:], b) for a, b in zip(d, ref))
    assert (d.index[:-3] == 0).all() and (d.kept[:-3] == 45).all()


def test_calls_at_once_on_two_streams():
    z, u = make(64, 50000, "bf16", seed=30)
    ref = sampling.draw(z, u, top_p=0.8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    out = [sampling.draw(z, u, top_p=0.8, stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for d in out for a, b in zip(d, ref))


def test_shares_are_those_of_the_softmax():
    """u through [0, 1) in even steps meets each class in proportion to its weight."""
    z = (torch.randn(1, 37, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) * 2).repeat(4096, 1)
    u = (torch.arange(4096, device="cuda") + 0.5) / 4096
    d = sampling.draw(z, u, temperature=1.5)
    share = torch.bincount(d.index, minlength=37).double() / 4096
    p = torch.softmax(z[0].double() / 1.5, 0)
    assert (share - p).abs().max() <= 1.0 / 4096  # a class's interval meets its length of steps, one more or less
    assert (d.logprob.double() - torch.log(p)[d.index]).abs().max() <= 1e-6


def test_streams_graphs_and_repeats():
    z, u = make(50, 30001, "bf16", seed=8)
    a = sampling.draw(z, u, top_p=0.9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = sampling.draw(z, u, top_p=0.9, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = sampling.draw(z, u, top_p=0.9)
    z2, u2 = make(50, 30001, "bf16", seed=9)
    z.copy_(z2)
    u.copy_(u2)
    g.replay()
    check(z, u, top_p=0.9, most_unsure=1)
    assert all(torch.equal(x, y) for x, y in zip(c, sampling.draw(z, u, top_p=0.9)))


def test_results_into_the_callers_tensors_and_refusals():
    z, u = make(6, 100, "bf16")
    out = [torch.full((8,), 7, device="cuda", dtype=t) for t in (torch.int64, torch.float32, torch.int32)]
    sampling.gm_draw(z, u, *(t[:6] for t in out))
    d = sampling.draw(z, u)
    for t, x in zip(out, d):
        assert torch.equal(t[:6], x) and (t[6:] == 7).all()
    assert sampling.draw(z[:0], u[:0]).index.shape == (0,)
    for bad in (dict(temperature=-1.0), dict(temperature=float("inf")), dict(temperature=1e-39), dict(top_k=-1), dict(top_p=1.5),
                dict(top_p=float("nan")), dict(min_p=-0.5)):
        with pytest.raises(GmError):
            sampling.draw(z, u, **bad)
    for bad in (dict(top_k=torch.zeros(6, device="cuda", dtype=torch.int64)), dict(temperature=torch.ones(5, device="cuda")),
                dict(top_p=torch.ones(6)), dict(top_k=1 << 40)):
        with pytest.raises(ValueError):
            sampling.draw(z, u, **bad)
    for bad in (u[:5], u.double(), u.cpu()):
        with pytest.raises(ValueError):
            sampling.draw(z, bad)
    with pytest.raises(ValueError):
        sampling.draw(z.t(), u)


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p"])
@pytest.mark.parametrize("value", [None, "a", [0.5]])
def test_values_that_are_no_numbers_are_refused(name, value):
    z, u = make(3, 100, "bf16")
    with pytest.raises(ValueError, match=name):
        sampling.draw(z, u, **{name: value})


def test_a_whole_number_of_top_k():
    z, u = make(3, 100, "bf16")
    with pytest.raises(ValueError, match="top_k"):
        sampling.draw(z, u, top_k=1.5)


# more rows than SMs: blocks of 128 to 512 threads share one
@pytest.mark.parametrize("rows,classes", [(310, 1029), (320, 9000), (500, 4100), (170, 16001), (160, 49152), (160, 12288)])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rule", [dict(), dict(top_k=70), dict(top_p=0.8), dict(min_p=0.01), dict(top_k=400, top_p=0.95)])
def test_rows_that_share_an_sm(rows, classes, kind, rule):
    check(*make(rows, classes, kind, seed=classes), temperature=0.9, most_unsure=1, **rule)


@pytest.mark.parametrize("missing", [(0,), (1,), (2,), (1, 2), (0, 1, 2)])
def test_results_that_are_missing_are_refused_and_the_others_left(missing):
    out = [torch.full((6,), 9, device="cuda", dtype=t) for t in (torch.int64, torch.float32, torch.int32)]
    given = [None if i in missing else t for i, t in enumerate(out)]
    with pytest.raises(ValueError):
        sampling.gm_draw(torch.zeros(6, 50, device="cuda"), torch.zeros(6, device="cuda"), *given)
    assert all((t == 9).all() for t in out)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("classes", [100, 20000])
@pytest.mark.parametrize("temperature", [1e30, 5e37, 3.4e38])
@pytest.mark.parametrize("min_p", [0.999, 0.5, 1e-10, 1e-44])
def test_temperatures_near_the_end_of_the_range(kind, classes, temperature, min_p):
    """All weights are 1 but for 1e-28 of them, whatever T ln(min_p) comes to."""
    z, u = make(3, classes, kind, seed=2)
    alive = (z > -torch.inf).sum(1)
    for rule in (dict(), dict(top_k=classes), dict(top_p=1.0)):
        d = sampling.draw(z, u, temperature=temperature, min_p=min_p, **rule)
        assert torch.equal(d.kept.long(), alive)
        assert (d.logprob + alive.float().log()).abs().max() <= 1e-6 * math.log(classes)


@pytest.mark.parametrize("name,value", [("temperature", 1e-46), ("temperature", 1e-300), ("top_p", 1e-46), ("min_p", 1e-60)])
def test_numbers_that_32_bits_take_to_zero_are_refused(name, value):
    """Else a temperature over 0 would take the first of equal logits always, and a min-p be off."""
    z, u = make(2, 50, "f32")
    with pytest.raises(ValueError, match=name):
        sampling.draw(z, u, **{name: value})
    sampling.draw(z, u, **{name: 0.0})

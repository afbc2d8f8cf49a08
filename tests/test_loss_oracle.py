"""The 64-bit losses of loss_oracle: gradients against central differences, and closed forms."""
import numpy as np
import pytest

import loss_oracle as lo


def problem(seed, n=5, d=4, v=7):
    rng = np.random.default_rng(seed)
    h, w = rng.normal(size=(n, d)), rng.normal(size=(v, d))
    target = rng.integers(0, v, size=n)
    target[1] = -100
    lens = rng.integers(0, v + 1, size=n)
    lens[0] = 0
    row_ptr = np.concatenate([[0], np.cumsum(lens)])
    col = np.concatenate([np.sort(rng.choice(v, k, replace=False)) for k in lens]).astype(np.int64)
    val = rng.normal(size=row_ptr[-1]) * 2
    if val.size > 2:
        val[-1] = -np.inf
    return h, w, target, lo.Teacher(row_ptr, col, val), rng


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_gradients_are_the_differences(seed, temperature):
    h, w, target, teacher, rng = problem(seed)
    g_loss, g_lse, g_kl = rng.normal(size=(3, h.shape[0]))

    def objective(h, w):
        f = lo.forward(h, w, target, -100, teacher, temperature)
        return g_loss @ f["loss"] + g_lse @ f["lse"] + g_kl @ f["kl"]

    f = lo.forward(h, w, target, -100, teacher, temperature)
    g, _, _ = lo.logit_grads(f, target, -100, g_loss, g_lse, temperature, g_kl)
    for x, grad, other in ((h, g @ w, 0), (w, g.T @ h, 1)):
        for _ in range(6):
            step = rng.normal(size=x.shape)
            e = 1e-5
            up, down = (objective(h + e * step, w), objective(h - e * step, w)) if other == 0 else \
                       (objective(h, w + e * step), objective(h, w - e * step))
            # the third derivative's part is under 1e-9 of a step of this size
            assert abs((up - down) / (2 * e) - np.sum(grad * step)) < 1e-7


def test_closed_forms():
    n, v = 3, 8
    h, w = np.zeros((n, 2)), np.ones((v, 2))
    target = np.array([0, 7, -100])
    f = lo.forward(h, w, target, -100, lo.Teacher(np.array([0, 2, 2, 4]), np.array([1, 3, 0, 5]),
                                                  np.array([0.0, 0.0, -np.inf, -np.inf])), 3.0)
    np.testing.assert_allclose(f["loss"], [np.log(8), np.log(8), 0], atol=1e-14)
    np.testing.assert_allclose(f["kl"], [np.log(8) - np.log(2), 0, 0], atol=1e-14)  # two of eight; no row; all -inf

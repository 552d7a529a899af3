"""The fp64 definitions of the operators beside the routed experts, pinned:
worked examples, gradients against central differences, statements that hold
for any input."""

import numpy as np
import pytest

from oracle import block as B


def test_selection_worked_example():
    # groups {0, 1} {2, 3} {4, 5}; c = s + bias
    l = np.log(np.array([[0.6, 0.2, 0.5, 0.5, 0.1, 0.65]]) / (1 - np.array([[0.6, 0.2, 0.5, 0.5, 0.1, 0.65]])))
    ids, w = B.select_experts(l, 2, n_group=3, topk_group=1, group_top=2)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, 0.5)          # 1.0 beats 0.8 and 0.75; a tie by index
    ids, w = B.select_experts(l, 2, n_group=3, topk_group=1, group_top=1)
    assert ids.tolist() == [[5, 4]] and np.allclose(w, [[0.65 / 0.75, 0.1 / 0.75]])
    bias = np.array([0, 0.5, -0.3, -0.3, 0.0, 0.0])
    ids, w = B.select_experts(l, 3, bias=bias, n_group=3, topk_group=2, group_top=2, renormalize=False, scale=2.0)
    assert ids.tolist() == [[1, 5, 0]] and np.allclose(w, [[0.4, 1.3, 1.2]])     # the bias is not in the weights


def test_selection_of_empty_rows_and_nan():
    l = np.array([[-np.inf] * 4, [1.0, np.nan, -np.inf, 2.0]])
    for scoring in ("softmax", "sigmoid"):
        with np.errstate(invalid="ignore"):
            ids, w = B.select_experts(l, 3, scoring)
        assert ids.tolist() == [[0, 1, 2], [3, 0, 1]] and np.all(w[0] == 0)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_selection_gradient_against_differences(scoring, renorm):
    rng = np.random.default_rng(0)
    l, dw = rng.normal(size=(3, 7)), rng.normal(size=(3, 3))
    ids = np.array([[6, 0, 3], [1, 2, 4], [5, 5, 1]])                # one id twice

    def f(x):
        total = 0.0
        for t in range(3):
            s = B.scores(x[t], scoring)[ids[t]]
            total += (dw[t] * 1.7 * (s / s.sum() if renorm else s)).sum()
        return total
    g = B.select_experts_backward(l, ids, dw, scoring, renorm, 1.7)
    for i in np.ndindex(*l.shape):
        h = np.zeros_like(l)
        h[i] = 1e-5
        assert abs((f(l + h) - f(l - h)) / 2e-5 - g[i]) < 1e-8


def test_adamw_worked_example_and_first_step():
    w, m, v = B.adamw(np.array([1.0]), np.array([2.0]), np.array([0.5]), np.array([3.0]), 2, 0.1, (0.5, 0.75), 1.0, 0.2)
    assert m[0] == 1.25 and v[0] == 3.25
    assert np.isclose(w[0], 1 - 0.02 - 0.1 * (1.25 / 0.75) / (np.sqrt(3.25 / 0.4375) + 1))
    # the first step from zero states moves every weight by lr, whatever its gradient's size
    g = np.array([1e-3, -5.0, 7e4])
    w, _, _ = B.adamw(np.zeros(3), g, np.zeros(3), np.zeros(3), 1, 0.01, eps=1e-30)
    assert np.allclose(w, -0.01 * np.sign(g))


def test_stochastic_bits_are_uniform_and_differ():
    """Means, and correlations between fields, neighbours, steps, tensors and seeds, within 5 standard deviations."""
    n = 1 << 18
    fields = [f.astype(np.float64) / 65536 for args in ((0, 1, 0), (0, 2, 0), (0, 1, 1), (9, 1, 0)) for f in B.dice(n, *args)]
    for f in fields:
        assert abs(f.mean() - 0.5) < 5 / np.sqrt(12 * n) + 2.0 ** -17
        for lag in (1, 2, 8, 128, 2048):
            assert abs(np.corrcoef(f[:-lag], f[lag:])[0, 1]) < 5 / np.sqrt(n - lag)
    for i, a in enumerate(fields):
        for b in fields[:i]:
            assert abs(np.corrcoef(a, b)[0, 1]) < 5 / np.sqrt(n)


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"])
def test_activations_against_differences_and_known_values(name):
    rng = np.random.default_rng(1)
    z, dy = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4 if name == "swiglu" else 8))
    g = B.activate_grad(z, dy, name)
    for i in np.ndindex(*z.shape):
        h = np.zeros_like(z)
        h[i] = 1e-5
        assert abs(((B.activate(z + h, name) - B.activate(z - h, name)) * dy).sum() / 2e-5 - g[i]) < 1e-8
    one = np.array([[1.0, 2.0]])
    known = dict(none=1.0, relu=1.0, gelu=0.8413447460685429, gelu_tanh=0.8411919906082768, silu=0.7310585786300049,
                 swiglu=2 * 0.7310585786300049)
    assert abs(B.activate(one, name)[0, 0] - known[name]) < 1e-12
    assert B.activate(np.zeros((1, 2)), name)[0, 0] == 0

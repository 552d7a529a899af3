"""The fp64 definitions of the training operators (oracle/training.py) pinned
on the CPU: gradients against central differences, and against torch's own
float64 autograd of the formulas."""

import numpy as np
import pytest
import torch

from oracle import training as R


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, H, eps = 3, 16, 1e-5
    x, gamma, beta, dy = rng.normal(size=(T, H)), rng.normal(size=H), rng.normal(size=H), rng.normal(size=(T, H))
    _, mean, rstd = R.layer_norm(x, gamma, beta, eps)
    dx, dgamma, dbeta = R.layer_norm_backward(x, gamma, mean, rstd, dy)
    f = lambda x, g, b: (R.layer_norm(x, g, b, eps)[0] * dy).sum()
    h = 1e-6
    for t, c in ((0, 0), (1, 7), (2, 15)):
        d = np.zeros((T, H))
        d[t, c] = h
        # central differences: truncation h^2, cancellation 2^-52 |f| / h, both below 1e-8 here
        assert abs((f(x + d, gamma, beta) - f(x - d, gamma, beta)) / (2 * h) - dx[t, c]) < 1e-7
        assert abs((f(x, gamma + d[t], beta) - f(x, gamma - d[t], beta)) / (2 * h) - dgamma[c]) < 1e-7
        assert abs((f(x, gamma, beta + d[t]) - f(x, gamma, beta - d[t])) / (2 * h) - dbeta[c]) < 1e-7


def _case(T, E, k, S, seed, masked):
    rng = np.random.default_rng(seed)
    l = rng.normal(size=(T, E))
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    off = np.sort(np.concatenate([[0], rng.integers(0, T - 1, S - 1), [T - 1]]))
    return l, ids, off, (rng.random(T) < 0.8) if masked else None


@pytest.mark.parametrize("S,masked", [(1, False), (3, True)])
def test_balance_gradient_against_differences_and_autograd(S, masked):
    T, E, k, alpha = 12, 7, 3, 0.3
    l, ids, off, mask = _case(T, E, k, S, 1, masked)
    r = R.balance_loss(l, ids, alpha, off, mask)
    h = 1e-6
    for t in range(T):
        for e in (0, 3, 6):
            d = np.zeros((T, E))
            d[t, e] = h
            fd = (R.balance_loss(l + d, ids, alpha, off, mask)["loss"] -
                  R.balance_loss(l - d, ids, alpha, off, mask)["loss"]) / (2 * h)
            assert abs(fd - r["dlogits"][t, e]) < 1e-8
    lt = torch.tensor(l, requires_grad=True)
    p = torch.softmax(lt, 1)
    keep = np.ones(T, bool) if mask is None else mask
    loss, used = 0, 0
    for s in range(S):
        rows = [t for t in range(off[s], off[s + 1]) if keep[t]]
        if rows:
            used += 1
            f = torch.tensor(np.bincount(ids[rows].ravel(), minlength=E) * E / (k * len(rows)))
            loss = loss + (f * p[rows].mean(0)).sum()
    (alpha * loss / used).backward()
    assert np.allclose(lt.grad.numpy(), r["dlogits"], rtol=1e-12, atol=1e-16)
    assert abs(float(alpha * loss / used) - r["loss"]) < 1e-14


def test_balance_of_an_even_routing_is_alpha():
    """Every expert chosen equally often: f = 1, so the loss is alpha
    whatever the probabilities, and the gradient is zero."""
    T, E, k = 8, 4, 2
    ids = np.array([[(2 * t + j) % E for j in range(k)] for t in range(T)])
    r = R.balance_loss(np.random.default_rng(2).normal(size=(T, E)), ids, 0.5)
    assert abs(r["loss"] - 0.5) < 1e-15 and np.all(r["dlogits"] == 0)


def test_balance_empty_sequences_and_masked_rows():
    l = np.array([[0.0, 1.0], [np.nan, np.nan], [-np.inf, -np.inf]])
    r = R.balance_loss(l, np.array([[1], [0], [0]]), 1.0, np.array([0, 0, 2, 2]), np.array([1, 0, 1]))
    assert r["tokens"].tolist() == [0, 1, 0] and r["counts"].tolist() == [[0, 0], [0, 1], [0, 0]]
    assert np.all(r["dlogits"][1:] == 0) and np.isfinite(r["loss"])
    # a token whose logits are all -inf counts, without probability
    r = R.balance_loss(l, np.array([[1], [0], [0]]), 1.0, np.array([0, 3]), np.array([1, 0, 1]))
    assert r["counts"].tolist() == [[1, 1]] and np.all(r["dlogits"][2] == 0)
    assert abs(r["probs"].sum() - 0.5) < 1e-15


@pytest.mark.parametrize("shape", [(6, 9), (9, 6), (5, 5)])
def test_orthogonalize_moves_singular_values_only(shape):
    """The iteration is an odd polynomial of the singular values: U p(S) V^T
    with the same singular vectors, p applied to the normalised values."""
    u = np.random.default_rng(3).normal(size=shape)
    a, s, b = np.linalg.svd(u, full_matrices=False)
    v = s / (np.linalg.norm(s) + 1e-7)
    for _ in range(5):
        c = R.NS_COEFFS
        v = c[0] * v + c[1] * v ** 3 + c[2] * v ** 5
    assert np.allclose(R.orthogonalize(u), (a * v) @ b, atol=1e-12)
    cubic = [(1.5, -0.5, 0.0)] * 40
    o = R.orthogonalize(u, 40, cubic)
    w = o @ o.T if shape[0] <= shape[1] else o.T @ o
    assert np.allclose(w, np.eye(min(shape)), atol=1e-9)

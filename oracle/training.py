"""fp64 numpy definitions of the operators around the layer in a training
step: layer norm and its backward pass, the router's load-balance loss with
its gradient, and the Newton-Schulz orthogonalisation of a matrix.  Written
from the formulas in include/moe_layer.h, element by element where that is
short, without the device code's groupings or orders of sums."""

import numpy as np

NS_COEFFS = (3.4445, -4.7750, 2.0315)


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) of x [T, H]; beta may be None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(axis=1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * gamma
    return (y if beta is None else y + beta), mean, rstd


def layer_norm_backward(x, gamma, mean, rstd, dy):
    """(dx, dgamma, dbeta) for the given statistics."""
    z = (np.asarray(x, np.float64) - mean[:, None]) * rstd[:, None]
    dy = np.asarray(dy, np.float64)
    g = dy * gamma
    dx = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - z * (g * z).mean(axis=1, keepdims=True))
    return dx, (dy * z).sum(axis=0), dy.sum(axis=0)


def balance_loss(logits, ids, alpha, offsets=None, mask=None):
    """dict(loss, counts [S, E], probs [S, E], dlogits [T, E], tokens [S])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = ids.shape[1]
    offsets = np.array([0, T]) if offsets is None else np.clip(np.asarray(offsets), 0, T)
    mask = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    S = len(offsets) - 1
    counts = np.zeros((S, E), np.int64)
    probs = np.zeros((S, E))
    dlogits = np.zeros((T, E))
    p = np.zeros((T, E))
    rows = []
    for s in range(S):
        r = np.array([t for t in range(offsets[s], offsets[s + 1]) if mask[t]], int)
        rows.append(r)
        for t in r:
            m = logits[t].max()
            if m == -np.inf:
                continue
            e = np.exp(logits[t] - m)
            p[t] = e / e.sum()
            for i in ids[t]:
                counts[s, min(max(int(i), 0), E - 1)] += 1
        for t in r:
            if logits[t].max() == -np.inf:
                for i in ids[t]:
                    counts[s, min(max(int(i), 0), E - 1)] += 1
        if len(r):
            probs[s] = p[r].sum(axis=0) / len(r)
    used = max(1, sum(len(r) > 0 for r in rows))
    loss = 0.0
    for s, r in enumerate(rows):
        if not len(r):
            continue
        f = counts[s] * E / (k * len(r))
        loss += alpha / used * (f * probs[s]).sum()
        for t in r:
            # sum_i p_i (c_e - c_i): the derivative p_e (delta - p_i) of the softmax, contracted with f / N
            diff = (counts[s][:, None] - counts[s][None, :]).astype(np.float64)
            dlogits[t] = alpha / used * E / (k * len(r)) / len(r) * p[t] * (diff @ p[t])
    return dict(loss=loss, counts=counts, probs=probs, dlogits=dlogits, tokens=np.array([len(r) for r in rows]))


def orthogonalize(u, steps=5, coeffs=None, eps=1e-7):
    """steps Newton-Schulz products of each matrix of u [..., M, N]."""
    u = np.asarray(u, np.float64)
    if u.ndim > 2:
        return np.stack([orthogonalize(v, steps, coeffs, eps) for v in u])
    x = u / (np.sqrt((u * u).sum()) + eps)
    if u.shape[0] > u.shape[1]:
        x = x.T
    for i in range(steps):
        a, b, c = NS_COEFFS if coeffs is None else coeffs[i]
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if u.shape[0] > u.shape[1] else x

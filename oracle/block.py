"""fp64 numpy definitions of the operators that stand beside the routed
experts in a block: the selection of experts by scores, a bias and groups
with its gradient, linear layers with an epilogue and their gradient, and the
AdamW step.  Written from the formulas in include/moe_layer.h, a token or an
element at a time where that is short, without the device code's groupings or
orders of sums."""

import math

import numpy as np

from . import formats as F


# ------------------------------------------------------------------ selection
def scores(row, scoring):
    """s of one token's fp64 logits."""
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-row))
    m = row.max()
    if m == -np.inf:
        return np.zeros_like(row)
    e = np.exp(row - m)
    return e / e.sum()


def _best(keys, n):
    """The n largest by key, descending, ties to the lower index; NaN as -infinity."""
    keys = [-math.inf if math.isnan(v) else float(v) for v in keys]
    return sorted(range(len(keys)), key=lambda i: (-keys[i], i))[:n]


def select_experts(logits, k, scoring="sigmoid", bias=None, n_group=1, topk_group=1, group_top=2, renormalize=True,
                   scale=1.0):
    """(ids [T, k], weights [T, k])."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    per = E // n_group
    ids, w = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        s = scores(logits[t], scoring)
        c = s if bias is None else s + np.asarray(bias, np.float64)
        order = logits[t] if bias is None else c
        groups = [-np.sort(-np.where(np.isnan(g), -np.inf, g))[:group_top].sum() for g in c.reshape(n_group, per)]
        kept = _best(groups, topk_group)
        members = sorted(e for g in kept for e in range(g * per, g * per + per))
        ids[t] = [members[i] for i in _best(order[members], k)]
        w[t] = s[ids[t]]
        if renormalize:
            w[t] = w[t] / w[t].sum() if w[t].sum() != 0 else 0.0
    return ids, scale * w


def select_experts_backward(logits, ids, dw, scoring="sigmoid", renormalize=True, scale=1.0):
    """dlogits [T, E] by the chain rule through every s of the token."""
    logits, dw = np.asarray(logits, np.float64), np.asarray(dw, np.float64)
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        s = scores(logits[t], scoring)
        sel = np.clip(ids[t], 0, E - 1)
        z = s[sel].sum()
        ds = np.zeros(E)
        for j, e in enumerate(sel):
            if renormalize:
                # w_i = scale s_i / z:  dw_i / ds_e = scale ([i = j] / z - s_i / z^2), i over the slots
                ds[e] += scale * (dw[t, j] - (dw[t] * s[sel]).sum() / z) / z if z else 0.0
            else:
                ds[e] += scale * dw[t, j]
        out[t] = ds * s * (1 - s) if scoring == "sigmoid" else s * (ds - (s * ds).sum())
    return out


# --------------------------------------------------------------------- AdamW
def mix(x):
    """The 32-bit mixing function of the stochastic rounding, on Python ints or uint64 arrays."""
    x = x & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0x6A09E667) & 0xFFFFFFFF
    x = x ^ (x >> 13)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def dice(n, seed, t, index):
    """16 random bits per element for m, for v and for the weight: three arrays [n]."""
    key = mix(mix(seed ^ (t * 0x9E3779B9 & 0xFFFFFFFF)) + index * 0xA54FF53B)
    i = np.arange(n, dtype=np.uint64)
    h = mix(i * np.uint64(0x9E3779B1) + np.uint64(key))
    return h & 0xFFFF, h >> np.uint64(16), ((h * np.uint64(0x3C6EF373)) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)


def state_values(codes, scales):
    """The numbers that E4M3 codes [n] with a scale per 128 stand for."""
    return F.e4m3_decode(np.asarray(codes)) * np.repeat(np.asarray(scales, np.float64), 128)[:len(codes)]


def adamw(w, g, m, v, t, lr, betas=(0.9, 0.999), eps=1e-8, decay=0.0, grad_scale=1.0):
    """(w', m', v') of fp64 arrays after step t."""
    g = grad_scale * g
    m = betas[0] * m + (1 - betas[0]) * g
    v = betas[1] * v + (1 - betas[1]) * g * g
    update = (m / (1 - betas[0] ** t)) / (np.sqrt(v / (1 - betas[1] ** t)) + eps)
    return w - lr * decay * w - lr * update, m, v


# -------------------------------------------------------------- linear layers
def act(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return np.maximum(z, 0)
    if name == "gelu":
        return z * 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def act_grad(z, name):
    z = np.asarray(z, np.float64)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-z / math.sqrt(2)) + \
            z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s + z * s * (1 - s)
    return np.ones_like(z)


def activate(z, name):
    """act(z); SwiGLU of gate and up side by side."""
    if name == "swiglu":
        n = z.shape[1] // 2
        return act(z[:, :n], "silu") * z[:, n:]
    return act(z, name)


def activate_grad(z, dy, name):
    """dz."""
    if name == "swiglu":
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        return np.concatenate([dy * u * act_grad(g, "silu"), dy * act(g, "silu")], axis=1)
    return dy * act_grad(z, name)

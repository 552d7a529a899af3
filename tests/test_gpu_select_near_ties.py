"""Selection by softmax scores and a bias where candidates are as near to each other as fp32's error in the sum of the
exponentials: the order is that of 64-bit scores.

The kernels form exp(l - m) with the product m log2(e) rounded once, a factor F that all of a row's exponentials share, and with them
their sum; F is largest where the product lies just above a power of two, half a unit from an fp32 number.  A logit m of
that kind is searched for here on the CPU; F - 1 is 4.3e-2 for m near 2^20 / log2(e) and 4.2e-5 near 2^10 / log2(e)."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

F = np.float32
LOG2E = float(F(1.44269504))


def _logits_of_a_large_factor(lo, hi, n):
    """fp32 numbers m in [lo, hi) whose product with log2(e) is rounded down by most, so that exp(l - m) is too large."""
    m = np.arange(F(lo).view(np.int32), F(hi).view(np.int32)).astype(np.int32).view(np.float32)
    exact = m.astype(np.float64) * LOG2E
    off = exact - exact.astype(np.float32)
    return m[np.argsort(-off)[:n]]


def _check(l, bias, k):
    from moe_layer_router_amd import layer as L
    ids, _ = B.select_experts(l, k, "softmax", bias=bias, renormalize=False)
    out = L.select_experts(torch.from_numpy(l).cuda(), k, scoring="softmax", bias=torch.from_numpy(bias).cuda(), renormalize=False)
    got = out["topk_ids"].cpu().numpy()
    assert np.array_equal(got, ids), (l.max(), got, ids)


def _below(x):
    """The largest fp32 number below x."""
    f = F(x)
    return f if float(f) < x else np.nextafter(f, F(-np.inf))


@pytest.mark.parametrize("E,at", [(8, (0, 3)), (200, (17, 150)), (256, (255, 4)), (300, (299, 256)), (1024, (5, 900))])
@pytest.mark.parametrize("d", [1.0, 2.0, 5.0])
def test_two_candidates_of_different_scores(gpu_lib, E, at, d):
    """s_0 - s_1 = b_1 - b_0 but for less than a unit of fp32; the logits as large as 7e5."""
    for m in _logits_of_a_large_factor(726_830, 727_500, 12):
        l = np.full((2, E), m - 400, F)
        l[:, at[0]], l[:, at[1]] = m, m - F(d)
        s = B.scores(l[0].astype(np.float64), "softmax")
        bias = np.zeros(E, F)
        bias[at[1]] = _below(s[at[0]] - s[at[1]])              # the first is ahead, by less than fp32 can tell
        _check(l, bias, 1)
        _check(l, bias, 2)


@pytest.mark.parametrize("E,at", [(8, (0, 3, 6)), (200, (17, 150, 40)), (256, (255, 4, 130)), (300, (299, 256, 7)), (1024, (5, 900, 333))])
@pytest.mark.parametrize("d", [1.0, 3.0])
def test_a_candidate_behind_two_of_equal_scores(gpu_lib, E, at, d):
    """The sum decides between the last place and the second one behind it; the one between them has the last place's score and
    a bias a unit lower."""
    a, b, c = at
    for m in _logits_of_a_large_factor(709.8, 712, 12):
        l = np.full((2, E), m - 300, F)
        l[:, a] = l[:, b] = m - F(d)
        l[:, c] = m
        s = B.scores(l[0].astype(np.float64), "softmax")
        bias = np.zeros(E, F)
        bias[a] = _below(s[c] - s[a])                          # c is ahead of a, and a of b
        bias[b] = np.nextafter(bias[a], F(0))
        _check(l, bias, 1)
        _check(l, bias, 2)

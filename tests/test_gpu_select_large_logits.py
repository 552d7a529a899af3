"""Selection by softmax scores of large finite logits on the GPU: rows masked with a large negative number, one
large logit among ordinary ones, all of them large.

Ids are equal to the fp64 definition's.  Weights, with u = 2^-24: an exponential whose argument is below -126 ln 2 is below
fp32's normal numbers, so the differences that matter are at most 88, each rounded once, as in the test of ordinary logits:
(2 88 + 60) u relative, and fp32's least normal numbers.  Renormalised weights are those of scores that may underflow
in 64 bits: they are formed relative to the largest selected one."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LOWEST = float(np.finfo(np.float32).min)


def _np(t):
    return t.detach().cpu().numpy().astype(np.float64)


def _renormalized(l, ids, scoring):
    s = np.take_along_axis(l.astype(np.float64), ids, 1)
    b = np.minimum(s, 0) if scoring == "sigmoid" else s
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(b), 0, np.exp(b - b.max(1, keepdims=True)))
    e = e / (1 + np.exp(-np.abs(s))) if scoring == "sigmoid" else e
    z = e.sum(1, keepdims=True)
    return np.where(z > 0, e / np.where(z > 0, z, 1), 0)


def _rows(E, rng):
    n = rng.normal(size=(20, E))
    l = n.copy()
    l[0], l[1], l[2], l[3] = -1e30, LOWEST, -LOWEST, -1e10         # a masked token, in several manners
    l[4], l[5], l[6] = 3e9 * n[4], 1e30 * n[5], 1e38 * n[6].clip(-3, 3)
    l[7, E // 2], l[8, E // 3] = 1e10, -1e10                       # one among ordinary ones
    l[9, 1:] = 1e10                                                # all of them but one
    l[10, :-1] = LOWEST                                            # all masked but one
    l[11], l[11, E // 5] = -np.inf, -1e30
    l[12], l[12, ::3] = -1e30, -np.inf
    l[13] = 2.0 ** 24 + 2 * rng.integers(0, 5, size=E)             # neighbours in fp32
    l[14] = -2.0 ** 25 + 4 * rng.integers(0, 3, size=E)
    l[15], l[16] = 2.0 ** 21 + 3 * n[15], -2.0 ** 20 + 3 * n[16]
    l[17], l[18] = 1e5 + n[17], -3e6 + 4 * n[18]
    return l.astype(np.float32)


@pytest.mark.parametrize("E,groups,keep", [(8, 2, 1), (96, 6, 3), (200, 10, 4), (256, 8, 4), (300, 6, 2), (1000, 10, 5)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_large_logits(gpu_lib, E, groups, keep, scoring, renorm):
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(E)
    l = _rows(E, rng)
    bias = (0.01 * rng.normal(size=E)).astype(np.float32)
    for b in (None, bias):
        for kw in (dict(), dict(n_group=groups, topk_group=keep)):
            kw.update(scoring=scoring, renormalize=renorm, scale=2.5)
            ids, w = B.select_experts(l, 4, bias=b, **kw)
            w = 2.5 * _renormalized(l, ids, scoring) if renorm else w
            out = L.select_experts(torch.from_numpy(l).cuda(), 4, bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
            got, g = _np(out["topk_ids"]).astype(np.int64), _np(out["topk_weights"])
            assert np.array_equal(got, ids), (b is not None, kw, np.flatnonzero((got != ids).any(1)))
            bad = ~(np.abs(g - w) <= (2 * 88 + 60) * U * np.abs(w) + 2.0 ** -124)
            assert not bad.any(), (b is not None, kw, np.flatnonzero(bad.any(1)), g[bad][:4], w[bad][:4])


@pytest.mark.parametrize("E", [60, 256, 300, 1024])
def test_a_token_does_not_see_its_neighbours_logits(gpu_lib, E):
    """Tokens that share a wave: the same bits beside a masked row as beside an ordinary one."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(E)
    l = rng.normal(size=(40, E)).astype(np.float32)
    bias = torch.from_numpy((0.01 * rng.normal(size=E)).astype(np.float32)).cuda()
    kw = dict(scoring="softmax", renormalize=False, bias=bias)
    ref = L.select_experts(torch.from_numpy(l).cuda(), 4, **kw)
    m = l.copy()
    m[1::4], m[2::4] = -1e30, 1e12 * m[2::4]
    out = L.select_experts(torch.from_numpy(m).cuda(), 4, **kw)
    for n in ref:
        assert torch.equal(ref[n][::4], out[n][::4]) and torch.equal(ref[n][3::4], out[n][3::4])


@pytest.mark.parametrize("E", [8, 96, 256, 300, 1000])
@pytest.mark.parametrize("renorm", [False, True])
def test_large_logits_gradient(gpu_lib, E, renorm):
    from tests.test_gpu_select import _check_bwd
    rng = np.random.default_rng(E)
    l = _rows(E, rng)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :4]
    _check_bwd(l, ids, rng.normal(size=ids.shape).astype(np.float32), scoring="softmax", renormalize=renorm, scale=2.5)

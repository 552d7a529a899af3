"""moe_orthogonalize on matrices with a side of at most 64, whose iteration runs in
64 bits, over many steps and on exactly low rank: the directions that a matrix
lacks must stay empty, however often a step lifts what rounding leaves there.

The matrices are products of integer factors (exact in fp32), the reference the
factors' singular vectors with the scalar polynomial in 64 bits.  Bounds, per
element: y's rounding, half a step, 2^-8 |y|; the singular values' own
perturbation, 2^-45 / s by the shift of the Gram matrix and 64 * 2^-53 / s per step by
its rounding, below 2^-42 / s together over 32 steps, times the derivative of the
polynomial's iterate; and in the directions that U lacks, where Q reaches 2^22, the rounding of
up to 64 terms in each of up to 32 products, 2^22 * 64 * 32 * 2^-53 = 2^-20."""

import numpy as np
import pytest
import torch

from oracle import training as R

pytestmark = pytest.mark.gpu


def _iterate(s, steps):
    a, b, c = (float(np.float32(v)) for v in R.NS_COEFFS)       # (as the library holds them)
    d = np.ones_like(s)
    for _ in range(steps):
        d = d * (a + 3 * b * s ** 2 + 5 * c * s ** 4)
        s = a * s + b * s ** 3 + c * s ** 5
    return s, d


@pytest.mark.parametrize("M,N,r", [(64, 2048, 8), (2048, 64, 8), (64, 200, 1), (33, 500, 5), (500, 32, 2), (16, 16, 3),
                                   (7, 30, 1), (64, 64, 63), (1, 40, 1)])
def test_exact_low_rank_over_many_steps(gpu_lib, M, N, r):
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(M + N)
    p, q = np.rint(4 * rng.normal(size=(M, r))) + 1, np.rint(4 * rng.normal(size=(N, r)))
    (qp, rp), (qq, rq) = np.linalg.qr(p), np.linalg.qr(q)
    a, s, b = np.linalg.svd(rp @ rq.T)
    left, right = qp @ a, b @ qq.T
    u = p @ q.T
    s = s / (np.linalg.norm(s) + 1e-7)
    ut = torch.from_numpy(np.stack([u, -u]).astype(np.float32)).cuda()
    assert np.array_equal(ut[0].cpu().double().numpy(), u)
    for steps in (1, 5, 10, 16, 20, 32):
        y = L.orthogonalize(ut, steps=steps).cpu().double().numpy()
        t, d = _iterate(s, steps)
        ref = (left * t) @ right
        bound = 2.0 ** -8 * np.abs(ref) + (np.abs(left) * (np.abs(d) * 2.0 ** -42 / s)) @ np.abs(right) + 2.0 ** -20
        assert np.all(np.isfinite(y)), steps
        worst = np.max(np.abs(y[0] - ref) / bound)
        assert worst <= 1.01 and np.array_equal(y[1], -y[0]), (steps, worst)


@pytest.mark.parametrize("E,H", [(32, 512), (64, 2048), (8, 256)])
def test_rows_that_sum_to_zero(gpu_lib, E, H):
    """A router's gradient: its columns sum to zero but for fp32's rounding, which
    is far below 2^-22 of the norm and must not be lifted into the update."""
    from moe_layer_router_amd import layer as L
    g = np.random.default_rng(E).normal(size=(E, H)) * 1e-3
    g = (g - g.mean(axis=0)).astype(np.float32)
    u = torch.from_numpy(g).cuda()
    a, s, b = np.linalg.svd(g.astype(np.float64), full_matrices=False)
    s = s / (np.linalg.norm(s) + 1e-7)
    assert s[-1] < 1e-7 < 1e-2 < s[-2]
    for steps in (5, 10, 16, 20, 32):
        y = L.orthogonalize(u, steps=steps).cpu().double().numpy()
        assert np.all(np.isfinite(y)), steps
        t, d = _iterate(s, steps)
        t[-1] = 0
        err = np.linalg.norm(y - (a * t) @ b)
        # y's rounding, at most 2^-8 / sqrt(3) of it at random, and the last value lifted 2^22-fold at most
        assert err <= 2.0 ** -8 * np.linalg.norm(t) + 2.0 ** 22 * s[-1] + np.linalg.norm(d[:-1] * 2.0 ** -42 / s[:-1]), steps


def test_norms_at_the_ends_of_fp32(gpu_lib):
    """Norms whose reciprocals leave fp32: tiny ones with a tiny eps, and the largest."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(3)
    for M, N in ((20, 50), (60, 16)):
        base = rng.normal(size=(M, N)).astype(np.float32)
        base /= np.abs(base).max()
        for scale in (2.0 ** -126, 2.0 ** -140, 2.0 ** 127):
            u = (base.astype(np.float64) * scale).astype(np.float32)
            y = L.orthogonalize(torch.from_numpy(u).cuda(), eps=1e-44).cpu().double().numpy()
            eps = float(np.float32(1e-44))
            ref = R.orthogonalize(u, 5, None, eps)
            assert np.all(np.abs(y - ref) <= 2.0 ** -8 * 1.01 * np.abs(ref) + 2.0 ** -24), (M, N, scale)

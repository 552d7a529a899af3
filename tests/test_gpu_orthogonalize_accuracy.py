"""The accuracy that moe_orthogonalize documents, on the updates that strain it
most: exactly low rank (the gradient of an expert that got few tokens), where
every direction that the matrix lacks holds nothing but what rounding puts
there, and matrices of one magnitude, whose elements all round alike.

The matrices are products of integer factors, so that fp32 holds them exactly
and their rank is exact; the iteration keeps their singular vectors, and the
reference follows in 64 bits from the factors' QR and the scalar polynomial.

Bounds (relative, Frobenius), for the wide path (sides above 64).  A step's roundings
are those of FP16 operands, half a step 2^-11 = 4.9e-4 of an element at most,
2.8e-4 in the root mean square: of A (in the polynomial 4.8 + 2 * 2.0 times), of
B' (its diagonal, 2 to 4, at most 2^-10 from its place) and of the FP16 part of X in
X X^T.  Simulated with these rounding points in 64 bits: 2.6e-3 after 5 steps and
4.1e-3 after 8 for rank 1 to 64, 1.1e-2 and 1.4e-2 for matrices of one magnitude.  With
the BF16 rounding of y, 2^-8 / sqrt(3) = 2.3e-3 at most and independent: 4e-3
(documented) >= sqrt(2.6^2 + 2.3^2) = 3.5e-3; 6e-3 for 8 steps; 1.3e-2 and 1.6e-2.

Beside it, in directions that U lacks, what the sums' own rounding leaves, lifted by
a = 3.4445 in each step that follows, as in an fp32 iteration.  A step's sum over m
terms is m / 32 additions of fp32 numbers, each off by up to 2^-24 of the sum, at
random sqrt(m / 32) 2^-24 together; behind K steps, with P = a^K, the sum over the steps
is P / a * 1.41 * sqrt(m / 32) 2^-24 = P sqrt(m) 2^-27.8, and X_0's 22 bits (half a step 2^-23
at most, 2^-23.8 at random) add P 2^-23.8, which is below P sqrt(m) 2^-26.8 from m = 65 on:
together P sqrt(m) 2^-26 (3.3e-4 after 5 steps at m = 2048, within the 4e-3; 1.3e-2 after 8)."""

import numpy as np
import pytest
import torch

from oracle import training as R

pytestmark = pytest.mark.gpu


def _poly(s, steps, coeffs=None):
    for i in range(steps):
        a, b, c = R.NS_COEFFS if coeffs is None else coeffs[i]
        s = a * s + b * s ** 3 + c * s ** 5
    return s


def low_rank(M, N, r, seed, ratio=None):
    """(U exact in fp32, function of the steps: the exact result); its eps is
    1e-7, or ratio |U|, as exact.eps."""
    rng = np.random.default_rng(seed)
    p, q = np.rint(4 * rng.normal(size=(M, r))), np.rint(4 * rng.normal(size=(N, r)))
    qp, rp = np.linalg.qr(p)
    qq, rq = np.linalg.qr(q)
    a, s, b = np.linalg.svd(rp @ rq.T)
    eps = 1e-7 if ratio is None else float(np.float32(ratio * np.linalg.norm(s)))
    s /= np.linalg.norm(s) + eps
    u = (p @ q.T).astype(np.float32)
    assert np.array_equal(u, p @ q.T)

    def exact(steps):
        return ((qp @ a) * _poly(s, steps)) @ (b @ qq.T)
    exact.eps = eps
    return torch.from_numpy(u).cuda(), exact


def _error(y, ref):
    got = y.cpu().double().numpy()
    assert np.all(np.isfinite(got))
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("M,N,ranks", [(65, 65, (1, 4)), (96, 160, (1, 3)), (300, 200, (1, 16)), (256, 512, (1, 2, 64)),
                                       (1024, 4096, (1, 2, 16)), (2048, 1024, (1, 8)), (2048, 7168, (1, 2, 16))])
def test_low_rank(gpu_lib, M, N, ranks):
    from moe_layer_router_amd import layer as L
    for r in ranks:
        u, exact = low_rank(M, N, r, M + r)
        for steps, bound in ((5, 4e-3), (8, 6e-3), (10, 8e-3)):
            lifted = R.NS_COEFFS[0] ** steps * min(M, N) ** 0.5 * 2.0 ** -26 if steps > 5 else 0
            e = _error(L.orthogonalize(u, steps=steps), exact(steps))
            assert e <= bound + lifted, (r, steps, e)


@pytest.mark.parametrize("M,N", [(65, 65), (127, 345), (350, 733), (200, 333), (2048, 1024)])
def test_elements_of_one_magnitude(gpu_lib, M, N):
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(1)
    for u in (np.ones((M, N)), np.sign(rng.normal(size=(M, 1))) * np.sign(rng.normal(size=(1, N)))):
        v = u / np.sqrt(M * N)
        for steps, bound in ((5, 1.3e-2), (8, 1.6e-2)):
            s = _poly(np.sqrt(M * N) / (np.sqrt(M * N) + 1e-7), steps)
            e = _error(L.orthogonalize(torch.from_numpy(u.astype(np.float32)).cuda(), steps=steps), s * v)
            assert e <= bound, (steps, e)


def test_the_cut_between_parts_of_a_batch(gpu_lib):
    """Rank-1 matrices around the cut of a batch that goes through in two parts."""
    from moe_layer_router_amd import layer as L, lib
    M, N, B = 1024, 4096, 400
    per = lib.moe_orthogonalize_workspace_size(2, M, N) - lib.moe_orthogonalize_workspace_size(1, M, N)
    assert lib.moe_orthogonalize_workspace_size(B, M, N) == lib.moe_orthogonalize_workspace_size(2 * B, M, N)
    cut = (8 << 30) // per
    some = [0, 1] + [i for i in range(cut - 12, cut + 3)] + [B - 1]
    assert cut + 3 < B
    u = torch.randn(B, M, N, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    exact = {}
    for i in some:
        u[i], exact[i] = low_rank(M, N, 1, i)
    y = L.orthogonalize(u)
    torch.cuda.synchronize()
    for i in some:
        assert _error(y[i], exact[i](5)) <= 4e-3, i


def test_norms_at_the_ends_of_fp32(gpu_lib):
    """Norms whose reciprocals leave fp32: tiny ones with a tiny eps, and the largest."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(3)
    for M, N in ((96, 160), (300, 70)):
        base = rng.normal(size=(M, N)).astype(np.float32)
        base /= np.abs(base).max()
        for scale in (2.0 ** -126, 2.0 ** -140, 2.0 ** 127):
            u = (base.astype(np.float64) * scale).astype(np.float32)
            y = L.orthogonalize(torch.from_numpy(u).cuda(), eps=1e-44)
            assert _error(y, R.orthogonalize(u, 5, None, float(np.float32(1e-44)))) <= 4e-3, (M, N, scale)


@pytest.mark.parametrize("M,N", [(65, 65), (96, 200), (256, 512)])
def test_many_steps(gpu_lib, M, N):
    """Full rank: the roundings of each step (7e-3 after 32 steps in the simulation
    above) and y's stay within 1e-2.  Low rank: what is lifted ends in the
    polynomial's range, singular values up to 1.2 and their roundings."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(5)
    u = torch.from_numpy(rng.normal(size=(M, N)).astype(np.float32)).cuda()
    low, _ = low_rank(M, N, 1, 7)
    for steps in (16, 32):
        assert _error(L.orthogonalize(u, steps=steps), R.orthogonalize(u.cpu().numpy(), steps)) <= 1e-2, steps
        y = L.orthogonalize(low, steps=steps).cpu().double().numpy()
        assert np.all(np.isfinite(y)) and np.linalg.norm(y, 2) <= 1.25, steps


@pytest.mark.parametrize("M,N", [(96, 160), (2048, 7168)])
def test_norms_below_eps(gpu_lib, M, N):
    """|U| = eps / 1024: X_0's elements are small FP16 numbers."""
    from moe_layer_router_amd import layer as L
    for r in (1, 16):
        u, exact = low_rank(M, N, r, 3, 1024)
        assert _error(L.orthogonalize(u, eps=exact.eps), exact(5)) <= 4e-3, r


@pytest.mark.parametrize("M,N", [(65, 65), (130, 100), (200, 333), (256, 1000), (512, 300), (960, 2100)])
def test_full_rank(gpu_lib, M, N):
    """Gaussian matrices and singular values 1 / r, held to the documented bounds."""
    from moe_layer_router_amd import layer as L
    g = np.random.default_rng(M).normal(size=(M, N))
    a, s, b = np.linalg.svd(g, full_matrices=False)
    for u in (g, (a / np.arange(1, len(s) + 1)) @ b):
        for dtype in (torch.float32, torch.bfloat16):
            t = torch.from_numpy(u).to(dtype).cuda()
            for steps, bound in ((5, 4e-3), (8, 6e-3)):
                ref = R.orthogonalize(t.double().cpu().numpy(), steps)
                assert _error(L.orthogonalize(t, steps=steps), ref) <= bound, (dtype, steps)

"""Newton-Schulz orthogonalisation on the GPU against the fp64 iteration.

Tolerances, as the relative error of the Frobenius norm of each matrix.  The
output's rounding to BF16 is at most half a step, 2^-8 of each element; over
many elements (here from 4096 on) it is spread evenly over the step, and its
root mean square is at most 2^-8 / sqrt(3).  Inside:
- short side up to 64: fp64 iteration, Q rounded to fp32 and a product of up to
  64 terms in fp32, |Q| |x| against |Q x|: 70 u |Q|_2 |X_0| with |Q|_2 up to
  3.4445^5 = 485 (on the small singular values that it lifts) and |X_0| = 1:
  70 * 2^-24 * 485 = 2e-3, while |y| is at least 0.6 (the largest singular value
  is at least 1 / sqrt(m) = 0.125, which the polynomial takes there): 3.4e-3;
- above: FP16 products, whose roundings, simulated in fp64 with the kernel's
  rounding points, stay below 2.3e-3 for sides from 65 on and spectra from flat to
  1 / r^2 (and fall with the size); 3e-3."""

import numpy as np
import pytest
import torch

from oracle import training as R

pytestmark = pytest.mark.gpu


def _mat(B, M, N, seed, kind="normal", dtype=torch.float32):
    rng = np.random.default_rng(seed)
    u = rng.normal(size=(B, M, N))
    if kind == "decay":                       # singular values 1 / r
        for b in range(B):
            p, s, q = np.linalg.svd(u[b], full_matrices=False)
            u[b] = (p / np.arange(1, len(s) + 1)) @ q
    elif kind == "low_rank":
        r = max(1, min(M, N) // 8)
        u = rng.normal(size=(B, M, r)) @ rng.normal(size=(B, r, N)) + 0.01 * u
    elif kind == "tiny":
        u *= 1e-4
    return torch.from_numpy(u.astype(np.float32)).to(dtype).cuda()


def _check(y, u, steps=5, coeffs=None, eps=1e-7, what=""):
    ref = R.orthogonalize(u.float().cpu().numpy(), steps, coeffs, eps)
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), what
    inner = 3.4e-3 if min(u.shape[1:]) <= 64 else 3e-3
    half = 2.0 ** -8 * (1 if u.shape[1] * u.shape[2] < 4096 else 3 ** -0.5)
    for b in range(len(ref)):
        n = np.linalg.norm(ref[b])
        err = np.linalg.norm(got[b] - ref[b])
        assert err <= (inner + half) * n + 1e-30, f"{what} matrix {b}: {err / n:.2e}"


# sides around the narrow limit, the padding, the tiles of both sizes; wide, tall, square, one row, one column
SHAPES = [(1, 1, 1), (2, 1, 300), (3, 70, 1), (5, 7, 16), (2, 17, 33), (4, 40, 40), (2, 64, 200), (3, 500, 64),
          (2, 33, 1025), (2, 65, 65), (3, 100, 130), (2, 200, 333), (1, 333, 200), (2, 128, 128), (2, 129, 257),
          (1, 256, 1000), (8, 256, 256), (1, 700, 300)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,M,N", SHAPES)
def test_against_definition(gpu_lib, B, M, N, dtype):
    from moe_layer_router_amd import layer as L
    u = _mat(B, M, N, M + N, dtype=dtype)
    y = L.orthogonalize(u)
    torch.cuda.synchronize()
    assert y.shape == u.shape and y.dtype == torch.bfloat16
    _check(y, u, what=(B, M, N))


@pytest.mark.parametrize("kind", ["decay", "low_rank", "tiny"])
@pytest.mark.parametrize("B,M,N", [(2, 48, 100), (2, 300, 48), (2, 96, 160), (1, 512, 300), (1, 300, 640)])
def test_spectra(gpu_lib, B, M, N, kind):
    from moe_layer_router_amd import layer as L
    u = _mat(B, M, N, 5, kind)
    y = L.orthogonalize(u)
    torch.cuda.synchronize()
    _check(y, u, what=kind)


@pytest.mark.parametrize("B,M,N", [
    (8, 960, 2100),      # 256 x 256 tiles, cut off on both sides
    (40, 520, 1100),     # 128 x 128 tiles, as the larger ones would cover a third more
    (7, 576, 1000),      # 128 x 128, up to one per CU (three stages) in the symmetric products
    (8, 450, 900),       # in all of them
    (4, 1000, 4300),     # not in X X^T, whose K is long: split
    (12, 520, 1100),
    (3, 520, 1100),      # 64 x 64
])
def test_tile_shapes(gpu_lib, B, M, N):
    """Batches for each tile shape and its variants, with padding and partial tiles on
    both sides and a partial round split along K, wide and tall."""
    from moe_layer_router_amd import layer as L
    for m, n in ((M, N), (N, M)):
        u = _mat(B, m, n, 9)
        y = L.orthogonalize(u)
        torch.cuda.synchronize()
        some = sorted({0, B - 1} if m * n > 10 ** 6 else {0, B // 2, B - 1})
        _check(y[some], u[some], what=(m, n))
        assert torch.equal(L.orthogonalize(u), y)


def test_batch_in_several_parts(gpu_lib):
    """A batch whose workspace would pass 8 GiB goes through in parts: the
    matrices on both sides of the cut, and the last."""
    from moe_layer_router_amd import layer as L, lib
    B, M, N = 3000, 512, 1000                        # (about 2300 in one part)
    assert lib.moe_orthogonalize_workspace_size(B, M, N) == lib.moe_orthogonalize_workspace_size(2 * B, M, N)
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(B, M, N, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    y = L.orthogonalize(u)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all()
    some = [0, 1500, 2290, 2300, 2303, 2304, 2310, B - 2, B - 1]
    _check(y[some], u[some])
    # every matrix was done: the squares sum to the number of singular values, roughly (0.68 .. 1.2 each)
    s = y.float().square().sum((1, 2))
    assert float(s.min()) > 0.4 * M and float(s.max()) < 1.5 * M


@pytest.mark.parametrize("B,M,N", [(40, 576, 1088), (40, 1100, 520), (8, 960, 2100), (8, 130, 1500), (3, 200, 333)])
def test_repeated_calls_agree(gpu_lib, B, M, N):
    """Sides that end inside a tile, of each tile shape: the same bits from every call."""
    from moe_layer_router_amd import layer as L
    u, ws = _mat(B, M, N, 7), L.Workspace("cuda")
    ys = [L.orthogonalize(u, workspace=ws) for _ in range(8)]
    torch.cuda.synchronize()
    _check(ys[0][:2], u[:2])
    for y in ys[1:]:
        assert torch.equal(y, ys[0])


@pytest.mark.parametrize("M,N", [(12, 30), (90, 200)])
def test_steps_and_coefficients(gpu_lib, M, N):
    from moe_layer_router_amd import layer as L
    u = _mat(2, M, N, 3)
    y = L.orthogonalize(u, steps=1)
    _check(y, u, steps=1)
    co = [(3.0, -3.2, 1.2), (2.5, -2.0, 0.6), (1.5, -0.5, 0.0)]
    y = L.orthogonalize(u, steps=3, coeffs=co, eps=1e-3)
    torch.cuda.synchronize()
    _check(y, u, steps=3, coeffs=co, eps=1e-3)


@pytest.mark.parametrize("M,N", [(20, 50), (130, 90)])
def test_zero_huge_and_non_finite_matrices(gpu_lib, M, N):
    """An expert without tokens has a zero gradient: its update is exactly
    zero.  A NaN or infinity stays within its matrix."""
    from moe_layer_router_amd import layer as L
    u = _mat(6, M, N, 1)
    u[1] = 0
    u[2] *= 1e25                               # its squares overflow fp32
    u[3, 4, 5] = float("nan")
    u[4, 0, 0] = float("inf")
    u[5] *= 1e-20                              # its squares underflow fp32; far below eps
    y = L.orthogonalize(u)
    torch.cuda.synchronize()
    assert torch.all(y[1] == 0)
    _check(y[[0, 2]], u[[0, 2]])
    assert torch.isnan(y[3]).any() and torch.isnan(y[4]).any()
    ref = R.orthogonalize(u[5].cpu().numpy())
    got = y[5].double().cpu().numpy()
    # far below eps the update is linear in u and tiny; FP16's smallest step (2^-24 of 2^-12 in each of five
    # steps that grow 3.44-fold) bounds what is lost
    assert np.abs(got - ref).max() <= 2.0 ** -36 * 485 + 2.0 ** -7 * np.abs(ref).max()


@pytest.mark.parametrize("M,N", [(24, 60), (150, 110)])
def test_single_matrix_strided_reused_and_deterministic(gpu_lib, M, N):
    from moe_layer_router_amd import layer as L
    big = _mat(3, N, 2 * M, 2)
    u = big[:, :, ::2].transpose(1, 2)         # [3, M, N], not contiguous
    a = L.orthogonalize(u)
    b = L.orthogonalize(u.contiguous())
    c = L.orthogonalize(u[1])
    flat = torch.empty(M * N + 1, device="cuda")
    flat[1:] = u[1].reshape(-1)
    off = flat[1:].view(M, N)
    assert off.data_ptr() % 16 != 0
    d = L.orthogonalize(off)
    out = torch.full((3, M, N), 7, dtype=torch.bfloat16, device="cuda")
    e = L.orthogonalize(u, out=out, workspace=L.Workspace("cuda"))
    torch.cuda.synchronize()
    assert e is out and torch.equal(a, b) and torch.equal(a[1], c) and torch.equal(c, d) and torch.equal(a, out)


def test_streams_and_captured_graphs_with_one_workspace(gpu_lib):
    from moe_layer_router_amd import layer as L
    us = [_mat(2, 30, 100, 1), _mat(2, 140, 90, 2)]
    ref = [L.orthogonalize(u) for u in us]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [L.orthogonalize(u, stream=s) for u, s in zip(us, ss)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, r) for g, r in zip(got, ref))
    ws = L.Workspace("cuda")
    ws.get(1 << 24)
    graphs, outs = [], []
    co = [[3.4445, -4.7750, 2.0315]] * 5
    for u in us:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(L.orthogonalize(u, coeffs=co, workspace=ws))     # (coefficients are read during the call)
        graphs.append(g)
    co[0][0] = 0.0
    for i in range(6):
        ws.buf.fill_(255)
        outs[i % 2].fill_(-1)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], ref[i % 2]), i


def test_wrapper_refusals(gpu_lib):
    from moe_layer_router_amd import layer as L, lib
    u = torch.zeros(2, 8, 8, device="cuda")
    for b in (dict(u=u.half()), dict(u=u.cpu()), dict(u=u[0, 0]), dict(coeffs=[(1, 2, 3)]), dict(out=u),
              dict(out=torch.zeros(2, 8, 9, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            L.orthogonalize(**{**dict(u=u), **b})
    for b in (dict(steps=0), dict(steps=33), dict(eps=0.0), dict(eps=-1.0), dict(steps=1, coeffs=[(0.0, 99.0, 0.0)]),
              dict(u=u[:0])):
        with pytest.raises(lib.MoeError):
            L.orthogonalize(**{**dict(u=u), **b})


@pytest.mark.parametrize("B,M,N", [(40_000, 1024, 60), (3, 16384, 20_000)])
def test_offsets_past_32_bits(gpu_lib, B, M, N):
    """Batches of narrow matrices, and of the largest, with elements past 2^31
    (and bytes of one matrix past 2^29): narrow ones against the definition,
    large ones by what they must be: U^T Y symmetric (same singular vectors) and Y's
    singular values in the polynomial's range, on random vectors."""
    from moe_layer_router_amd import layer as L
    u = torch.empty(B, M, N, dtype=torch.bfloat16, device="cuda")
    u.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    y = L.orthogonalize(u)
    torch.cuda.synchronize()
    if M == 1024:
        some = [0, 20_000, 35_000, B - 1]
        _check(y[some], u[some])
        return
    g = torch.Generator(device="cuda").manual_seed(2)
    for b in (0, B - 1):
        v = torch.randn(M, 8, generator=g, device="cuda")
        uf, yf = u[b].float(), y[b].float()
        # all singular values between 0.6 and 1.3: |Y^T v| = |v| within that
        ratio = (yf.t() @ v).norm(dim=0) / v.norm(dim=0)
        assert float(ratio.min()) > 0.6 and float(ratio.max()) < 1.3
        # Y U^T = V p(S) S V^T is symmetric
        a, c = (yf @ (uf.t() @ v)), (uf @ (yf.t() @ v))
        assert float((a - c).norm() / a.norm()) < 1e-2
        del uf, yf

"""dz's third BF16 part on the GPU, in every tile and way of working on it."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -23                     # what a sum of the matrix cores may lose at each addition, relative


# (with 256 CUs: small tiles, the 128-column ones with two workgroups per CU and with one, 256 columns; whole and in parts)
SHAPES = [(3, 72, 40), (64, 64, 64), (333, 1000, 488), (700, 640, 1032), (2048, 192, 2048), (2100, 1096, 2056), (4100, 1032, 4104),
          (1024, 2048, 2048), (300, 7168, 2048), (512, 1024, 7168), (4096, 512, 4096)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("want", [(True, True), (True, False), (False, True)], ids=["both", "dx", "dw"])
def test_all_24_bits_of_dz_count(gpu_lib, T, K, N, want):
    """One dz in a row and in a column, so that an element of dx or dW is one product: three exact terms, added in fp32, within
    4 units of 2^-23 (one an addition).  With two parts it would be up to 2^-17 off, 16 times that."""
    from moe_layer_router_amd import layer as L
    g = torch.Generator(device="cuda").manual_seed(T + K)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    n = min(T, N)
    rows, cols = torch.randperm(T, generator=g, device="cuda")[:n], torch.randperm(N, generator=g, device="cuda")[:n]
    dy = torch.zeros(T, N, device="cuda")
    dy[rows, cols] = torch.randn(n, generator=g, device="cuda")
    out = L.linear_backward(x, w, dy, want_dx=want[0], want_dw=want[1])
    d = dy[rows, cols].double()[:, None]
    for name, at, of in (("dx", rows, w[cols]), ("dw", cols, x[rows])):
        if out[name] is None:
            continue
        ref = torch.zeros(out[name].shape, dtype=torch.float64, device="cuda")
        ref[at] = d * of.double()
        off = (out[name].double() - ref).abs()
        assert bool((off <= 4 * U * ref.abs()).all()), (name, float((off / ref.abs().clamp(min=1e-300)).max()))

"""Gradients of linear layers on the GPU at the ends of fp32's range."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -23                     # what a sum of the matrix cores may lose at each addition, relative


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_derivatives_of_large_finite_z(gpu_lib, act):
    """act'(z) is 0 or 1 but for fp32's rounding from |z| = 20 on, up to fp32's largest numbers."""
    from moe_layer_router_amd import layer as L
    z = np.array([20, 100, 1e3, 1025, 1e5, 1e10, 1.8e19, 1.9e19, 1e20, 1e30, 3e38, 0], np.float32)
    z = np.concatenate([z, -z])
    N, K = len(z), 8
    dy = np.where(np.arange(N) % 3 == 1, -0.75, 1.5).astype(np.float32)
    with np.errstate(over="ignore"):
        ref = dy * B.act_grad(z, act)
    x, w = torch.ones(1, K, dtype=torch.bfloat16, device="cuda"), torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    out = L.linear_backward(x, w, torch.from_numpy(dy[None]).cuda(), act, torch.from_numpy(z[None]).cuda(), want_dbias=True)
    # (60 2^-23 (1 + |z|) of dy, as at ordinary z, up to where the derivative is 0 or 1)
    bound = 60 * U * np.abs(dy) * (1 + np.minimum(np.abs(z), 20))
    assert np.all(np.abs(_np(out["dbias"]) - ref) <= bound), (_np(out["dbias"]), ref)
    assert np.all(np.abs(_np(out["dw"])[:, 0] - ref) <= bound) and np.all(np.isfinite(_np(out["dx"])))


def test_swiglu_of_large_finite_factors(gpu_lib):
    """dy z_up and dy z_gate beyond fp32's largest number where SiLU or its derivative is zero."""
    from moe_layer_router_amd import layer as L
    gate = np.array([-3e38, -1e30, -200, -110, -3e38, 2, 2, 0], np.float32)
    up = np.array([3e38, 3e38, 3e38, -3e38, 1, 1e30, -1e30, 1], np.float32)
    dy = np.array([8, 1e10, 4, 100, 50, 1e-3, 1e-3, 3], np.float32)
    N, K = 8, 8
    x, w = torch.ones(1, K, dtype=torch.bfloat16, device="cuda"), torch.ones(2 * N, K, dtype=torch.bfloat16, device="cuda")
    pre = torch.from_numpy(np.concatenate([gate, up])[None]).cuda()
    out = L.linear_backward(x, w, torch.from_numpy(dy[None]).cuda(), "swiglu", pre, want_dbias=True)
    with np.errstate(over="ignore", under="ignore"):
        ref = B.activate_grad(_np(pre), dy[None].astype(np.float64), "swiglu")[0]
    size = np.concatenate([np.abs(dy * up.astype(np.float64)), np.abs(dy).astype(np.float64)])
    g2 = np.tile(np.minimum(np.abs(gate), 20), 2)
    got = _np(out["dbias"])
    # (sigmoid(-110) is below fp32's normal numbers: 2^-126 of dy z_up)
    bound = np.where(np.tile(gate, 2) < -88, 2.0 ** -126 * 128 * size, 60 * U * size * (1 + g2))
    assert np.all(np.abs(got - ref) <= bound), (got, ref)
    assert np.all(np.abs(_np(out["dw"])[:, 0] - ref) <= bound)


@pytest.mark.parametrize("T", [3, 70, 700])
def test_infinities_of_the_other_operand(gpu_lib, T):
    """An infinity in W (x) with a dz in parts: the elements of dx (dW) that it enters are not finite, an infinity or a NaN;
    the others are those of the call without it.  With a BF16 dy of no activation, one part, it is an infinity of the product's sign."""
    from moe_layer_router_amd import layer as L
    K, N = 200, 72
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn(T, N, generator=g, device="cuda")
    dy[dy == 0] = 1
    xi, wi = x.clone(), w.clone()
    xi[2, 5], wi[7, 9] = -float("inf"), float("inf")
    for d in (dy, dy.to(torch.bfloat16)):
        ref, out = L.linear_backward(x, w, d), L.linear_backward(xi, wi, d)
        for name, col in (("dx", 9), ("dw", 5)):
            other = torch.arange(K, device="cuda") != col
            assert torch.equal(out[name][:, other], ref[name][:, other]), name
            assert not bool(torch.isfinite(out[name][:, col]).any()), name
        if d.dtype == torch.bfloat16:
            assert torch.equal(out["dx"][:, 9], float("inf") * torch.sign(d[:, 7].float()))
            assert torch.equal(out["dw"][:, 5], -float("inf") * torch.sign(d[2].float()))

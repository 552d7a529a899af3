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

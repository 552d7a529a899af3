"""Layer norm of rows that are not finite: the NaN reaches every output of its
row, the scales of an FP8 output (whose codes have none) among them, and no
other row; a gamma or beta that is not finite reaches its own block only."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(5, 128), (9, 640), (6, 1024), (7, 2048), (5, 2176), (6, 4096), (5, 7168), (5, 16384)]


@pytest.mark.parametrize("scale_mode", ["f32", "pow2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_rows(gpu_lib, T, H, dtype, scale_mode):
    from moe_layer_router_amd import layer as L
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(H)).to(dtype).cuda()
    gamma, beta = torch.ones(H, device="cuda"), torch.zeros(H, device="cuda")
    clean = L.layer_norm(x, gamma, beta, out_dtype="fp8", scale_mode=scale_mode, want_stats=True)
    bad = x.clone()
    bad[1, H - 1] = float("nan")
    bad[3, 5] = float("inf")
    bad[4, 0] = -float("inf")
    r8 = L.layer_norm(bad, gamma, beta, out_dtype="fp8", scale_mode=scale_mode, want_stats=True)
    r16 = L.layer_norm(bad, gamma, beta)
    torch.cuda.synchronize()
    for t in range(T):
        if t in (1, 3, 4):
            assert torch.isnan(r8["y_scales"][t]).all() and torch.isnan(r8["rstd"][t]) and torch.isnan(r16["y"][t]).all(), t
        else:
            for k in clean:
                assert torch.equal(r8[k][t], clean[k][t]), (t, k)


def test_gamma_beta_and_rows_without_spread(gpu_lib):
    from moe_layer_router_amd import layer as L
    T, H = 6, 1152
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).cuda()
    x[2] = 1.5
    for name, at, value in (("gamma", 130, float("nan")), ("beta", 1151, float("inf")), ("gamma", 0, -float("inf"))):
        w = dict(gamma=torch.ones(H, device="cuda"), beta=torch.zeros(H, device="cuda"))
        clean = L.layer_norm(x, **w, out_dtype="fp8")
        w[name][at] = value
        r = L.layer_norm(x, **w, out_dtype="fp8")
        torch.cuda.synchronize()
        hit = np.arange(H // 128) == at // 128
        assert torch.isnan(r["y_scales"][:, hit]).all() and torch.equal(r["y_scales"][:, ~hit], clean["y_scales"][:, ~hit])
    # eps = 0: a row without spread is 0 / 0
    r = L.layer_norm(x, torch.ones(H, device="cuda"), eps=0.0, out_dtype="fp8")
    torch.cuda.synchronize()
    assert torch.isnan(r["y_scales"][2]).all() and torch.isfinite(r["y_scales"][[0, 1, 3, 4, 5]]).all()


def test_a_layer_fed_such_a_row_keeps_to_its_bounds(gpu_lib):
    """NaN scales in one token's input: the others' outputs are what they are
    without it, the token's routing stays in range."""
    from moe_layer_router_amd import layer as L
    from workloads import gen
    from tests._helpers import to_dev
    cfg = gen.LayerConfig("nan_row", 70, 512, 16, 4, 256, "fp8", "fp8")
    inp = L.pack_weights(to_dev(gen.make_inputs(cfg, seed=1)))
    h = torch.randn(cfg.T, cfg.H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    gamma = torch.ones(cfg.H, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            h[7, 3] = float("nan")
        n = L.layer_norm(h, gamma, out_dtype="fp8")
        x = n["y"].view(inp["x"].dtype) if inp["x"].dtype != torch.uint8 else n["y"]
        outs.append(L.forward({**inp, "x": x, "x_scales": n["y_scales"]}, cfg.k))
    torch.cuda.synchronize()
    keep = torch.arange(cfg.T, device="cuda") != 7
    assert torch.equal(outs[0]["y"][keep], outs[1]["y"][keep])
    ids = outs[1]["topk_ids"]
    assert int(ids.min()) >= 0 and int(ids.max()) < cfg.E

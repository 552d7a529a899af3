"""The layer, its backward pass and its conversions on a stream that is not the
current one, fed strided and misaligned views, while the current stream allocates and
writes."""

import pytest
import torch

from workloads import gen

from tests._helpers import to_dev

pytestmark = pytest.mark.gpu


def test_side_stream_with_views(gpu_lib):
    from moe_layer_router_amd import layer as L
    cfg = gen.LayerConfig("streams", 300, 256, 12, 3, 128, "bf16", "bf16")
    inp = to_dev(gen.make_inputs(cfg, seed=2))
    fwd = L.forward(L.pack_weights(inp), cfg.k)
    dl = L.balance_loss(L.logits(fwd).clone(), fwd["topk_ids"], alpha=2.0)["dlogits"]
    dy = torch.randn(cfg.T, cfg.H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    ref = L.backward(inp, fwd["topk_ids"], fwd["topk_weights"], dy, dlogits=dl)
    torch.cuda.synchronize()
    flat = torch.empty(dl.numel() + 1, device="cuda")
    flat[1:] = dl.reshape(-1)
    views = [dl.t().contiguous().t(), flat[1:].view_as(dl)]
    wide = torch.zeros(cfg.T, 2 * cfg.H, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2] = inp["x"]
    side = torch.cuda.Stream()
    for v in views:
        for s in (side, side.cuda_stream):
            torch.cuda.synchronize()
            got = L.backward({**inp, "x": wide[:, ::2]}, fwd["topk_ids"], fwd["topk_weights"], dy.t().contiguous().t(),
                             dlogits=v, stream=s)
            junk = [torch.full((1 << 22,), -1.0, device="cuda") for _ in range(24)]    # what the call freed may not be among it
            torch.cuda.synchronize()
            for k in ref:
                assert torch.equal(got[k], ref[k]), k
            del junk


def test_the_layer_and_its_conversions_on_a_side_stream(gpu_lib):
    from moe_layer_router_amd import layer as L
    cfg = gen.LayerConfig("side", 200, 512, 16, 4, 256, "fp8", "fp8")
    raw = to_dev(gen.make_inputs(cfg, seed=3))
    h = torch.randn(cfg.T, cfg.H, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    strided = h.t().contiguous().t()

    def run(s, x):
        inp = L.pack_weights(raw, stream=s)
        q, qs = L.quantize_input(x, stream=s)
        e, es = L.quantize_e5m6(x, stream=s)
        d = L.dequantize_e5m6(e, es, stream=s)
        f = L.forward({**inp, "x": q.view(inp["x"].dtype), "x_scales": qs}, cfg.k, stream=s)
        r = L.route({**inp, "x": q.view(inp["x"].dtype), "x_scales": qs}, cfg.k, cfg.E, stream=s)
        p = L.permute(r["topk_ids"], cfg.E, stream=s)
        g = L.forward({**inp, "x": q.view(inp["x"].dtype), "x_scales": qs}, cfg.k, stream=s,
                      routing=(r["topk_ids"], r["topk_weights"]))
        return [q, qs, d, f["y"], f["topk_ids"], r["logits"], r["topk_weights"], p["perm"], p["expert_offsets"], g["y"]]

    ref = run(None, h)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        got = run(s, strided)
        junk = [torch.full((1 << 22,), -1.0, device="cuda") for _ in range(16)]
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, ref)):
            assert torch.equal(a, b), i
        del junk

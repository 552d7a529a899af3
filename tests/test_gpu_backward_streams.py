"""The backward pass on a stream that is not the current one, fed strided and
misaligned views, while the current stream allocates and writes."""

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

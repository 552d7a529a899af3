"""Steps of AdamW that are left out because their gradients overflowed, with the count taken back as step()'s
documentation says: the others are, bit for bit, those of a run without them."""

import pytest
import torch

pytestmark = pytest.mark.gpu

SCALES = [float("inf"), float("nan"), 0.5, float("-inf"), 1.0, float("inf"), 2.0]


def _run(state):
    g = torch.Generator(device="cuda").manual_seed(1)
    p = [torch.randn(n, generator=g, device="cuda").to(torch.bfloat16) for n in (3000, 129, 8)]
    return p, [[torch.randn(q.shape, generator=g, device="cuda") for q in p] for _ in SCALES]


def _all(opt):
    return opt.params + [v for s in opt.states for v in s.values()]


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_count_on_the_host(gpu_lib, state):
    from moe_layer_router_amd import layer as L
    (p, gs), (q, hs) = _run(state), _run(state)
    a, b = L.AdamW(p, state=state), L.AdamW(q, state=state)
    for s, g, h in zip(SCALES, gs, hs):
        scale = torch.tensor([s], device="cuda")
        a.step(g, 1e-2, grad_scale=scale)
        if not bool(torch.isfinite(scale)):
            a.count -= 1
            continue
        b.step(h, 1e-2, grad_scale=scale)
    assert a.count == b.count == 3 and all(torch.equal(x, y) for x, y in zip(_all(a), _all(b)))


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_count_on_the_gpu_in_a_graph(gpu_lib, state):
    from moe_layer_router_amd import layer as L
    (p, gs), (q, hs) = _run(state), _run(state)
    a, b = L.AdamW(p, state=state, capturable=True), L.AdamW(q, state=state, capturable=True)
    now, scale = [torch.zeros_like(g) for g in gs[0]], torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(now, 1e-2, grad_scale=scale)
        a.count.add_(torch.isfinite(scale).long() - 1)
    for s, g, h in zip(SCALES, gs, hs):
        scale.fill_(s)
        for x, y in zip(now, g):
            x.copy_(y)
        graph.replay()
        if abs(s) < float("inf"):
            b.step(h, 1e-2, grad_scale=torch.tensor([s], device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(a.count, b.count) and all(torch.equal(x, y) for x, y in zip(_all(a), _all(b)))
    assert int(a.count) == 3

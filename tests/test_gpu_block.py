"""A training step of a block with routed and shared experts, the operators together as they are used:

  routing by a selection of the router's logits;  y = routed layer(x) + shared expert(x)
  backward of both;  AdamW over all of their weights

against the fp64 definitions fed what the device fed the next operator, and
captured in one graph with eager steps beside it.

Tolerances: the routed layer's gradients as in its own test (1e-3 of the larger of the element and the rms); products of the
shared expert's: (K / 32 + 40) 2^-23 of their terms' magnitudes, 2^-8 of the value where it is BF16, and for a gradient
through the activation 60 2^-23 (1 + |z|) of its factors, twice the terms' bound for its parts; a step's weights 2^-24 times 2 (|w| + |w'|)
+ 16 lr (m / sqrt(v) is at most 1 in a first step)."""

import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import moe_oracle as O
from workloads import gen

from tests._helpers import to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
SEL = dict(scoring="sigmoid", n_group=4, topk_group=2, scale=2.5)
NAMES = ("w_gate_up", "w_down", "router_w", "shared_in", "shared_out")


def _np(t):
    return t.detach().double().cpu().numpy()


def _block(cfg, S, seed):
    """Weights of a block in BF16, and their fp32 masters."""
    w = to_dev({k: v for k, v in gen.make_inputs(cfg, seed=seed).items()})
    g = torch.Generator().manual_seed(seed)
    w["shared_in"] = (torch.randn(2 * S, cfg.H, generator=g) / cfg.H ** 0.5).to(torch.bfloat16).cuda()
    w["shared_out"] = (torch.randn(cfg.H, S, generator=g) / S ** 0.5).to(torch.bfloat16).cuda()
    sel = dict(SEL, bias=(0.05 * torch.randn(cfg.E, generator=g)).cuda())
    return w, [w[n].float() for n in NAMES], sel


def _batch(cfg, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(cfg.T, cfg.H, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]


def _step(L, w, sel, k, x, dy, opt, lr):
    own = {n: v for n, v in w.items() if not n.startswith("shared") and n != "x"}
    fwd = L.forward({**L.pack_weights({**own, "x": x}), "x": x}, k, selection=sel)
    a = L.linear(x, w["shared_in"], act="swiglu", pre_dtype="bf16")
    y = L.linear(a["y"], w["shared_out"], residual=fwd["y"])
    out = L.linear_backward(a["y"], w["shared_out"], dy, dx_dtype="bf16")
    into = L.linear_backward(x, w["shared_in"], out["dx"], "swiglu", a["pre"])
    routed = L.backward({**own, "x": x}, fwd["topk_ids"], fwd["topk_weights"], dy, selection=sel, logits=fwd["logits"])
    dx = routed["dx"] + into["dx"]
    opt.step([routed["dw_gate_up"], routed["dw_down"], routed["dw_router"], into["dw"], out["dw"]], lr)
    return fwd, a, y, out, into, routed, dx


@pytest.mark.parametrize("cfg,S", [(gen.LayerConfig("block_small", 7, 256, 8, 2, 128, "bf16", "bf16"), 136),
                                   (gen.LayerConfig("block", 260, 384, 24, 4, 256, "bf16", "bf16"), 520)], ids=["small", "block"])
def test_a_step_of_a_block(gpu_lib, cfg, S):
    from moe_layer_router_amd import layer as L
    w, masters, sel = _block(cfg, S, 3)
    x, dy = _batch(cfg, 4)
    before = [m.clone() for m in masters]
    old = {n: w[n].clone() for n in NAMES}
    opt = L.AdamW([w[n] for n in NAMES], masters)
    fwd, a, y, out, into, routed, dx = _step(L, w, sel, cfg.k, x, dy, opt, 1e-2)
    torch.cuda.synchronize()
    ids, wt = B.select_experts(_np(fwd["logits"]), cfg.k, **{**SEL, "bias": _np(sel["bias"])})
    assert np.array_equal(_np(fwd["topk_ids"]), ids)
    assert np.all(np.abs(_np(fwd["topk_weights"]) - wt) <= 4 * U * wt + 1e-30)
    # the shared expert
    xn, dyn, an, win, wout = _np(x), _np(dy), _np(a["y"]), _np(old["shared_in"]), _np(old["shared_out"])
    yn = an @ wout.T + _np(fwd["y"])
    ey = (S / 32 + 40) * U * (np.abs(an) @ np.abs(wout).T) + 2 * U * np.abs(yn)
    assert np.all(np.abs(_np(y["y"]) - yn) <= ey + 2.0 ** -8 * (np.abs(yn) + ey))
    z = xn @ win.T
    ez = (cfg.H / 32 + 40) * U * (np.abs(xn) @ np.abs(win).T)
    assert np.all(np.abs(_np(a["pre"]) - z) <= ez + 2.0 ** -8 * (np.abs(z) + ez))
    da = dyn @ wout
    ea = (cfg.H / 32 + 40) * U * (np.abs(dyn) @ np.abs(wout))
    assert np.all(np.abs(_np(out["dx"]) - da) <= ea + 2.0 ** -8 * (np.abs(da) + ea))
    dz = B.activate_grad(_np(a["pre"]), _np(out["dx"]), "swiglu")
    g, up = np.split(_np(a["pre"]), 2, axis=1)
    d = np.abs(_np(out["dx"]))
    edz = 60 * U * np.concatenate([d * np.abs(up) * (1 + np.abs(g)), d * (1 + np.abs(g))], 1) + 2.0 ** -17 * np.abs(dz)
    for got, ref, err, terms, n in ((into["dx"], dz @ win, edz @ np.abs(win), np.abs(dz) @ np.abs(win), 2 * S),
                                    (into["dw"], dz.T @ xn, edz.T @ np.abs(xn), np.abs(dz).T @ np.abs(xn), cfg.T),
                                    (out["dw"], dyn.T @ an, 0, np.abs(dyn).T @ np.abs(an), cfg.T)):
        assert np.all(np.abs(_np(got) - ref) <= err + 2 * (n / 32 + 40) * U * terms)
    # the routed experts: dx of the whole block
    assert torch.equal(dx, routed["dx"] + into["dx"])
    dl = B.select_experts_backward(_np(fwd["logits"]), ids, _dweights(old, fwd, xn, dyn, ids, cfg),
                                   **{n: SEL[n] for n in ("scoring", "scale")})
    ref = dl.T @ xn
    rms = np.sqrt((ref ** 2).mean())
    assert np.max(np.abs(_np(routed["dw_router"]) - ref) / np.maximum(np.abs(ref), rms)) <= 1e-3
    # the weights
    grads = [routed["dw_gate_up"], routed["dw_down"], routed["dw_router"], into["dw"], out["dw"]]
    for n, b, m, gr in zip(NAMES, before, masters, grads):
        new, _, _ = B.adamw(_np(b), _np(gr), 0.0, 0.0, 1, 1e-2)
        assert np.all(np.abs(_np(m) - new) <= 2.0 ** -24 * (2 * (np.abs(new) + np.abs(_np(b))) + 16 * 1e-2)), n
        assert torch.equal(w[n], m.to(torch.bfloat16)), n
    assert opt.count == 1


def _dweights(old, fwd, xn, dyn, ids, cfg):
    """Gradient of the routed experts' weights: dy . expert(x)."""
    wgu, wd = _np(old["w_gate_up"]), _np(old["w_down"])
    dw = np.zeros(ids.shape)
    for t in range(cfg.T):
        for j, e in enumerate(ids[t]):
            gu = wgu[e] @ xn[t]
            dw[t, j] = dyn[t] @ (wd[e] @ O.swiglu(gu[:cfg.I], gu[cfg.I:]))
    return dw


def test_steps_of_a_block_in_one_graph(gpu_lib):
    """Captured while an eager block of the same values lives, replayed several times on new batches with eager steps of the other
    block in between: every result, weight and state bit for bit."""
    from moe_layer_router_amd import layer as L
    cfg = gen.LayerConfig("block_graph", 200, 256, 8, 2, 128, "bf16", "bf16")
    S, blocks = 264, []
    for _ in range(2):
        w, masters, sel = _block(cfg, S, 6)
        blocks.append((w, masters, sel, L.AdamW([w[n] for n in NAMES], masters, capturable=True, weight_decay=0.01)))
    (w0, m0, sel0, opt0), (w1, m1, sel1, opt1) = blocks
    x, dy = _batch(cfg, 7)
    lr = torch.full((1,), 1e-2, device="cuda")
    eager = _step(L, w0, sel0, cfg.k, x, dy, opt0, lr)
    first = _step(L, w1, sel1, cfg.k, x, dy, opt1, lr)
    torch.cuda.synchronize()
    assert torch.equal(eager[-1], first[-1])
    xs, dys = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = _step(L, w1, sel1, cfg.k, xs, dys, opt1, lr)
    for i in range(4):
        x, dy = _batch(cfg, 30 + i)
        lr.fill_(1e-2 / (1 + i))
        eager = _step(L, w0, sel0, cfg.k, x, dy, opt0, lr)
        torch.cuda.synchronize()
        xs.copy_(x)
        dys.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager[-1], cap[-1]), i
        for e, c in zip(eager[:-1], cap[:-1]):
            for n in e:
                if isinstance(e[n], torch.Tensor) and n != "workspace":
                    assert torch.equal(e[n], c[n]), (i, n)
        assert int(opt0.count) == int(opt1.count) == i + 2
        for n, a, b in zip(NAMES, m0, m1):
            assert torch.equal(a, b) and torch.equal(w0[n], w1[n]), (i, n)
        for s0, s1 in zip(opt0.states, opt1.states):
            assert torch.equal(s0["m"], s1["m"]) and torch.equal(s0["v"], s1["v"])

"""One training step of a block, the operators together as they are used:

  x = LN(h);  y = layer(x);  loss = sum(dy * y) + balance loss of the routing
  backward: d logits of the balance loss -> the layer's backward -> the norm's
  update: the orthogonalised weight gradients

against the fp64 definitions fed what the device fed the next operator (the
BF16 x, the routing, the statistics), and captured in one graph.

Tolerances: dx and the router's gradients as in the backward pass's own test
(1e-3 of the larger of the element and the rms: sums of two-part BF16 products);
dh and dgamma, linear in dx with fp32 sums, the same; the updates as the
orthogonalisation's own test has them, on the device's gradients."""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import moe_oracle as O
from oracle import training as R
from workloads import gen

from tests._helpers import to_dev

pytestmark = pytest.mark.gpu

ALPHA = 0.05


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(got, ref, axes, what):
    rms = np.sqrt((ref ** 2).mean(axis=axes, keepdims=True))
    err = np.abs(got - ref) / np.maximum(np.maximum(np.abs(ref), rms), 1e-30)
    assert np.all(np.isfinite(got)) and err.max() <= 1e-3, f"{what}: {err.max():.2e}"


def _step(L, h, gamma, beta, weights, packed, cfg, dy, off, mask, ws):
    """The calls of a training step; `ws`: a Workspace per operator, or None."""
    w = ws or dict.fromkeys(("fwd", "bal", "bwd", "ln", "orth"))
    norm = L.layer_norm(h, gamma, beta, want_stats=True)
    fwd = L.forward({**packed, "x": norm["y"]}, cfg.k, workspace=w["fwd"])
    bal = L.balance_loss(L.logits(fwd), fwd["topk_ids"], alpha=ALPHA, seq_offsets=off, token_mask=mask,
                         workspace=w["bal"])
    grads = L.backward({**weights, "x": norm["y"]}, fwd["topk_ids"], fwd["topk_weights"], dy, workspace=w["bwd"],
                       dlogits=bal["dlogits"])
    back = L.layer_norm_backward(h, gamma, norm["mean"], norm["rstd"], grads["dx"], workspace=w["ln"])
    E, I2, H = grads["dw_gate_up"].shape
    upd = dict(gate_up=L.orthogonalize(grads["dw_gate_up"].view(2 * E, I2 // 2, H), workspace=w["orth"]),
               down=L.orthogonalize(grads["dw_down"], workspace=w["orth"]),
               router=L.orthogonalize(grads["dw_router"], workspace=w["orth"]))
    return norm, fwd, bal, grads, back, upd


def _inputs(cfg, seed):
    weights = to_dev({k: v for k, v in gen.make_inputs(cfg, seed=seed).items()})
    g = torch.Generator().manual_seed(seed)
    h = (2 * torch.randn(cfg.T, cfg.H, generator=g) + 0.5).to(torch.bfloat16).cuda()
    dy = torch.randn(cfg.T, cfg.H, generator=g).to(torch.bfloat16).cuda()
    return weights, h, dy


@pytest.mark.parametrize("cfg,masked", [
    (gen.LayerConfig("step_small", 70, 256, 6, 2, 128, "bf16", "bf16"), False),
    (gen.LayerConfig("step_zipf", 260, 384, 24, 4, 256, "bf16", "bf16", zipf=1.1), True),
], ids=["small", "zipf"])
def test_training_step(gpu_lib, cfg, masked):
    from moe_layer_router_amd import layer as L
    weights, h, dy = _inputs(cfg, 3)
    gamma = 1 + 0.1 * torch.randn(cfg.H, generator=torch.Generator().manual_seed(1)).cuda()
    beta = 0.1 * torch.randn(cfg.H, generator=torch.Generator().manual_seed(2)).cuda()
    off = torch.tensor([0, cfg.T // 3, cfg.T - 4], dtype=torch.int32, device="cuda") if masked else None
    mask = (torch.arange(cfg.T, device="cuda") % 9 != 4) if masked else None
    packed = L.pack_weights(weights)
    norm, fwd, bal, grads, back, upd = _step(L, h, gamma, beta, weights, packed, cfg, dy, off, mask, None)
    torch.cuda.synchronize()
    # the norm's output in BF16 is the layer's input
    y_ref, mean, rstd = R.layer_norm(_np(h), _np(gamma), _np(beta), 1e-5)
    assert np.abs(_np(norm["y"]) - y_ref).max() <= 2.0 ** -8 * np.abs(y_ref).max() * 1.01
    ids = fwd["topk_ids"].cpu().numpy().astype(np.int64)
    b = R.balance_loss(fwd_logits := _np(L.logits(fwd)), ids, ALPHA, None if off is None else off.cpu().numpy(),
                       None if mask is None else mask.cpu().numpy())
    assert fwd_logits.shape == (cfg.T, cfg.E) and np.array_equal(bal["counts"].cpu().numpy(), b["counts"])
    if off is None:                                    # every token counts: the permutation has the same counts
        assert np.array_equal(np.diff(fwd["expert_offsets"].cpu().numpy()), b["counts"][0])
    # the layer's gradients, with the balance loss's share
    view = gen.oracle_view({k: (None if v is None else v.cpu()) for k, v in {**weights, "x": norm["y"]}.items()})
    ref = O.layer_backward(gen.spec_of(cfg), view, ids,
                           F.bf16_decode(dy.cpu().view(torch.int16).numpy().view(np.uint16)))
    x, wr = _np(norm["y"]), _np(weights["router_w"])
    dx = ref["dx"] + b["dlogits"] @ wr
    _close(_np(grads["dx"]), dx, (1,), "dx")
    _close(_np(grads["dw_router"]), ref["dw_router"] + b["dlogits"].T @ x, (0, 1), "dw_router")
    _close(_np(grads["dbias"]), ref["dbias"] + b["dlogits"].sum(0), (0,), "dbias")
    # the norm's
    dh, dgamma, dbeta = R.layer_norm_backward(_np(h), _np(gamma), mean, rstd, dx)
    _close(_np(back["dx"]), dh, (1,), "dh")
    _close(_np(back["dgamma"]), dgamma, (0,), "dgamma")
    _close(_np(back["dbeta"]), dbeta, (0,), "dbeta")
    # the updates; an expert without tokens gets none
    E, I2, H = grads["dw_gate_up"].shape
    for name, g, u in (("gate_up", grads["dw_gate_up"].view(2 * E, I2 // 2, H), upd["gate_up"]),
                       ("down", grads["dw_down"], upd["down"]), ("router", grads["dw_router"][None], upd["router"][None])):
        r, got = R.orthogonalize(_np(g)), _np(u)
        for i in range(len(r)):
            n = np.linalg.norm(r[i])
            if n == 0:
                assert np.all(got[i] == 0)
            else:
                # 3.4e-3 inside (short sides up to 64) and the rounding to BF16 of thousands of elements
                assert np.linalg.norm(got[i] - r[i]) <= (3.4e-3 + 2.0 ** -8) * n, (name, i)


def test_training_step_in_one_graph(gpu_lib):
    """The step captured with a workspace per operator (one for the three
    orthogonalisations), while eager results of the same tensors live, and
    replayed on new activations and gradients."""
    from moe_layer_router_amd import layer as L
    cfg = gen.LayerConfig("step_graph", 300, 256, 8, 2, 128, "bf16", "bf16")
    weights, h, dy = _inputs(cfg, 5)
    gamma, beta = torch.ones(cfg.H, device="cuda"), torch.zeros(cfg.H, device="cuda")
    packed = L.pack_weights(weights)
    eager = _step(L, h, gamma, beta, weights, packed, cfg, dy, None, None, None)
    torch.cuda.synchronize()
    ws = {k: L.Workspace("cuda") for k in ("fwd", "bal", "bwd", "ln", "orth")}
    for w in ws.values():
        w.get(64 << 20)
    hs, dys = h.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = _step(L, hs, gamma, beta, weights, packed, cfg, dys, None, None, ws)
    for i in range(4):
        if i:
            _, hn, dyn = _inputs(cfg, 20 + i)
            hs.copy_(hn)
            dys.copy_(dyn)
            eager = _step(L, hn, gamma, beta, weights, packed, cfg, dyn, None, None, None)
        graph.replay()
        torch.cuda.synchronize()
        for e, c in zip(eager, cap):
            for k in e:
                if isinstance(e[k], torch.Tensor) and k != "workspace":
                    assert torch.equal(e[k], c[k]), (i, k)

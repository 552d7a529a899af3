"""The balance loss, the experts' counts and the gradient in the logits on
the GPU against the fp64 definition; the gradient's way through the layer's
backward pass.

Tolerances, with u = 2^-24: a probability p = exp(l - m) / sum has the
rounding of its argument (|l - m| u), two of the exponential, those of the
sum over E (at most 16 in a lane and 6 across lanes) and of the quotient:
(R + 40) u with R = max |l - m| over the logits that matter (p > 2^-40: 28).
  probs    (R + 40 + N_s) u P       (a mean over N_s tokens, any order)
  loss     the same bound, relative (its sum is in fp64)
  dlogits  |err| <= (R + 80) u kappa p (|h_e| + sum_i p_i |h_i|), h_e = c_e - c_top
Counts are equal."""

import numpy as np
import pytest
import torch

from oracle import training as R
from workloads import gen

from tests._helpers import to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _case(T, E, k, S, masked, seed, spread=2.0):
    rng = np.random.default_rng(seed)
    l = (rng.normal(size=(T, E)) * spread + rng.normal(size=E)).astype(np.float32)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    off = None
    if S:
        last = T - T // 8
        off = np.sort(np.concatenate([[min(1, last)], rng.integers(min(1, last), last + 1, S - 1), [last]])).astype(np.int32)
    mask = (rng.random(T) < 0.8) if masked else None
    return l, ids, off, mask


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _check(out, l, ids, alpha, off, mask, what=""):
    ref = R.balance_loss(l, ids, alpha, off, mask)
    T, E = l.shape
    k = ids.shape[1]
    assert np.array_equal(out["counts"].cpu().numpy(), ref["counts"]), f"{what}: counts"
    lim = np.where(np.isfinite(l), l.astype(np.float64), 0)
    rng_l = min(28.0, float((lim.max(1) - lim.min(1)).max()))
    n = ref["tokens"]
    probs = out["probs"].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(probs - ref["probs"]) <= ((rng_l + 40 + n) * U)[:, None] * ref["probs"] + 2.0 ** -60), f"{what}: probs"
    loss = float(out["loss"].cpu()[0])
    assert abs(loss - ref["loss"]) <= (rng_l + 41 + n.max()) * U * abs(ref["loss"]) + 1e-30, f"{what}: loss"
    if out["dlogits"] is None:
        return ref
    offs = np.array([0, T]) if off is None else np.clip(off, 0, T)
    used = max(1, int((n > 0).sum()))
    bound = np.zeros((T, E))
    keep = np.ones(T, bool) if mask is None else mask
    for s in range(len(n)):
        for t in range(offs[s], offs[s + 1]):
            if keep[t] and l[t].max() > -np.inf:
                e = np.exp(l[t].astype(np.float64) - l[t].max())
                p = e / e.sum()
                h = ref["counts"][s] - ref["counts"][s][np.flatnonzero(l[t] == l[t].max())].max()
                kappa = abs(alpha) * E / (used * k * float(n[s]) ** 2)
                bound[t] = kappa * p * (np.abs(h) + p @ np.abs(h))
    d = out["dlogits"].cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(d)), f"{what}: non-finite gradient"
    # (2^-130: products below fp32's normal range)
    assert np.all(np.abs(d - ref["dlogits"]) <= (rng_l + 80) * U * bound + 2.0 ** -130), f"{what}: dlogits"
    return ref


# one token to several blocks; expert counts at and around every lane layout, odd ones among them
@pytest.mark.parametrize("T,E,k,S,masked", [
    (1, 1, 1, 0, False), (1, 8, 2, 0, False), (1, 256, 8, 0, True), (3, 2, 1, 2, False), (64, 8, 2, 0, False),
    (65, 63, 4, 3, True), (130, 64, 6, 0, True), (257, 65, 16, 5, False), (300, 128, 8, 4, True), (77, 129, 3, 0, False),
    (1000, 256, 8, 7, True), (90, 257, 8, 2, True), (513, 512, 2, 0, False), (210, 515, 16, 3, True),
    (1500, 1024, 16, 4, True), (40, 1023, 5, 40, False), (900, 70, 3, 300, True), (5000, 16, 4, 64, True), (3, 4, 4, 0, False),
    # one workgroup does it all (few tokens, at most 4 sequences), and the first that it does not
    (60, 300, 8, 2, True), (64, 1024, 16, 3, False), (50, 515, 4, 0, True), (512, 128, 4, 2, True),
    (513, 100, 4, 2, True), (400, 200, 4, 4, False),
])
@pytest.mark.parametrize("grad", [True, False])
def test_against_definition(gpu_lib, T, E, k, S, masked, grad):
    from moe_layer_router_amd import layer as L
    l, ids, off, mask = _case(T, E, k, S, masked, T + E)
    out = L.balance_loss(_dev(l), _dev(ids), alpha=0.02, seq_offsets=_dev(off), token_mask=_dev(mask), want_grad=grad)
    torch.cuda.synchronize()
    _check(out, l, ids, 0.02, off, mask)


def test_several_blocks_of_one_sequence(gpu_lib):
    """Enough ids for several count blocks and several passes per workgroup,
    sequences that end inside blocks, and a skewed routing."""
    from moe_layer_router_amd import layer as L
    T, E, k = 20011, 12, 4
    l, ids, _, mask = _case(T, E, k, 0, True, 5)
    off = np.array([0, 5, 5, 9000, 9001, 20011], np.int32)
    out = L.balance_loss(_dev(l), _dev(ids), alpha=1.0, seq_offsets=_dev(off), token_mask=_dev(mask))
    torch.cuda.synchronize()
    _check(out, l, ids, 1.0, off, mask)


@pytest.mark.parametrize("E", [8, 300])
def test_masked_infinite_and_saturated_rows(gpu_lib, E):
    from moe_layer_router_amd import layer as L
    T, k = 40, 2
    l, ids, _, _ = _case(T, E, k, 0, False, 3)
    l[4, :] = -np.inf                        # no probability at all
    l[5, 1:] = -np.inf                       # certain of one expert
    l[6] = -200
    l[6, 3] = 200                            # saturated: the other probabilities vanish in fp32
    l[7, 2] = 30                             # nearly saturated
    l[8, 5] = -np.finfo(np.float32).max      # a mask of the type's lowest value
    l[9] = 1.0                               # all alike
    mask = np.ones(T, bool)
    mask[[0, 10, 39]] = False
    l[10] = np.nan                           # masked: never looked at
    l[0] = np.inf
    off = np.array([0, 1, 20, 38], np.int32)         # sequence 0 has no token that counts, two rows belong to none
    l[38] = np.nan
    out = L.balance_loss(_dev(l), _dev(ids), alpha=0.1, seq_offsets=_dev(off), token_mask=_dev(mask))
    torch.cuda.synchronize()
    m = mask.copy()
    ref = l.copy()
    ref[[0, 10, 38]] = 0
    _check(out, ref, ids, 0.1, off, m)
    assert torch.all(out["dlogits"][[0, 4, 10, 38, 39]] == 0)


def test_no_token_counts(gpu_lib):
    from moe_layer_router_amd import layer as L
    l, ids, _, _ = _case(33, 20, 4, 0, False, 1)
    for off, mask in ((None, np.zeros(33, bool)), (np.array([9, 9, 9], np.int32), None)):
        out = L.balance_loss(_dev(l), _dev(ids), seq_offsets=_dev(off), token_mask=_dev(mask))
        torch.cuda.synchronize()
        for v in out.values():
            assert torch.all(v == 0)


def test_nan_reaches_its_own_sequence_only(gpu_lib):
    from moe_layer_router_amd import layer as L
    l, ids, _, _ = _case(30, 20, 4, 0, False, 1)
    l[25, 7] = np.nan
    off = np.array([0, 20, 30], np.int32)
    out = L.balance_loss(_dev(l), _dev(ids), seq_offsets=_dev(off))
    torch.cuda.synchronize()
    assert torch.isfinite(out["probs"][0]).all() and torch.isnan(out["probs"][1]).all() and torch.isnan(out["loss"]).all()
    d = out["dlogits"]
    assert torch.isnan(d[25]).all() and torch.isfinite(d[:25]).all() and torch.isfinite(d[26:]).all()
    l[25] = np.nan                           # a row of nothing else
    out = L.balance_loss(_dev(l), _dev(ids), seq_offsets=_dev(off))
    torch.cuda.synchronize()
    assert torch.isnan(out["dlogits"][25]).all() and torch.isnan(out["loss"]).all()


def test_offsets_and_ids_out_of_range_stay_in_bounds(gpu_lib):
    """Offsets are clamped to the tokens, ids to the experts (as in
    moe_permute); ids may repeat within a token and come as int64."""
    from moe_layer_router_amd import layer as L
    l, ids, _, _ = _case(50, 9, 3, 0, False, 2)
    ids[3] = [-5, 100, 2]
    ids[4] = [1, 1, 1]
    off = np.array([-7, 20, 1000], np.int64)
    out = L.balance_loss(_dev(l), _dev(ids.astype(np.int64)), seq_offsets=_dev(off))
    torch.cuda.synchronize()
    _check(out, l, ids, 1.0, off, None)


def test_gradient_against_differences(gpu_lib):
    from moe_layer_router_amd import layer as L
    T, E, k = 40, 24, 3
    l, ids, off, mask = _case(T, E, k, 2, True, 11)
    out = L.balance_loss(_dev(l), _dev(ids), alpha=1.0, seq_offsets=_dev(off), token_mask=_dev(mask))
    d = out["dlogits"].cpu().numpy().astype(np.float64)
    h = 1e-5                                  # (of the definition in 64 bits: truncation h^2, cancellation 1e-16 / h)
    for t, e in ((1, 0), (7, int(ids[7, 0])), (20, 23), (33, int(ids[33, 2]))):
        up, dn = l.astype(np.float64), l.astype(np.float64)
        up[t, e] += h
        dn[t, e] -= h
        fd = (R.balance_loss(up, ids, 1.0, off, mask)["loss"] - R.balance_loss(dn, ids, 1.0, off, mask)["loss"]) / (2 * h)
        assert abs(fd - d[t, e]) <= 1e-8 + 100 * U * abs(fd)


def test_deterministic_strided_and_reused_outputs(gpu_lib):
    from moe_layer_router_amd import layer as L
    l, ids, off, mask = _case(700, 60, 6, 5, True, 4)
    wide = torch.zeros(700, 121, device="cuda")
    wide[:, 1::2] = _dev(l)
    a = L.balance_loss(_dev(l), _dev(ids), seq_offsets=_dev(off), token_mask=_dev(mask))
    b = L.balance_loss(wide[:, 1::2], _dev(ids).t().contiguous().t(), seq_offsets=_dev(off).long(),
                       token_mask=_dev(mask).to(torch.uint8) * 255)
    torch.cuda.synchronize()
    for key in a:
        assert torch.equal(a[key], b[key]), key
    kept = {key: v.clone() for key, v in a.items()}
    for v in a.values():
        v.fill_(-1)
    c = L.balance_loss(_dev(l), _dev(ids), seq_offsets=_dev(off), token_mask=_dev(mask), out=a,
                       workspace=L.Workspace("cuda"))
    torch.cuda.synchronize()
    assert c is a and all(torch.equal(a[key], kept[key]) for key in a)


def test_two_streams_and_captured_graphs_with_one_workspace(gpu_lib):
    from moe_layer_router_amd import layer as L
    cases = [_case(900, 256, 8, 3, True, 6), _case(65, 30, 2, 2, False, 7)]
    dev = [tuple(_dev(v) for v in c) for c in cases]
    run = lambda c, **kw: L.balance_loss(c[0], c[1], seq_offsets=c[2], token_mask=c[3], **kw)
    ref = [run(c) for c in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [run(c, stream=s) for c, s in zip(dev, streams)]          # two calls at once, a workspace each
    torch.cuda.synchronize()
    for g, r in zip(got, ref):
        assert all(torch.equal(g[k], r[k]) for k in r)
    ws = L.Workspace("cuda")
    ws.get(1 << 24)                                                  # both graphs use it, one after the other
    graphs, outs = [], []
    for c in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(c, workspace=ws))
        graphs.append(g)
    for i in range(6):
        ws.buf.fill_(255)                                            # whatever another call left there
        for o in outs[i % 2].values():
            o.fill_(-1)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i % 2][k], ref[i % 2][k]) for k in ref[i % 2]), i


def test_wrapper_refusals(gpu_lib):
    from moe_layer_router_amd import layer as L, lib
    l, i = torch.zeros(6, 8, device="cuda"), torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    for b in (dict(logits=l.bfloat16()), dict(topk_ids=i[:5]), dict(topk_ids=i.float()), dict(topk_ids=i.cpu()),
              dict(seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
              dict(seq_offsets=torch.zeros(3, device="cuda")), dict(token_mask=torch.ones(5, dtype=torch.bool, device="cuda")),
              dict(token_mask=torch.ones(6, device="cuda"))):
        with pytest.raises(ValueError):
            L.balance_loss(**{**dict(logits=l, topk_ids=i), **b})
    with pytest.raises(lib.MoeError):
        L.balance_loss(l, torch.zeros(6, 9, dtype=torch.int32, device="cuda"))
    r = L.balance_loss(l, i, want_grad=False)
    with pytest.raises(ValueError):
        L.balance_loss(l, i, out=r)
    with pytest.raises(lib.MoeError):
        L.balance_loss(l, i, out={**r, "dlogits": l})


def test_gradient_through_the_layers_backward(gpu_lib):
    """moe_backward_aux: the additional logit gradient reaches dW_router, dbias
    and dx on top of the layer's own, by the formulas dW_r += d^T x,
    db += sum_t d, dx += d W_r (operands in two BF16 parts: 2^-16 relative per
    term, and fp32 sums; 1e-3 of the rms as for the rest of the backward
    pass), and leaves the expert gradients as they are, bit for bit."""
    from moe_layer_router_amd import layer as L
    cfg = gen.LayerConfig("aux", 150, 256, 11, 3, 128, "bf16", "bf16")
    inp = to_dev(gen.make_inputs(cfg, seed=4))
    fwd = L.forward(L.pack_weights(inp), cfg.k)
    logits = L.logits(fwd).clone()
    rt = L.route(inp, cfg.k, cfg.E)
    torch.cuda.synchronize()
    assert torch.allclose(logits, rt["logits"], atol=1e-4)
    aux = L.balance_loss(logits, fwd["topk_ids"], alpha=5.0)["dlogits"]
    dy = torch.randn(cfg.T, cfg.H, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    a = L.backward(inp, fwd["topk_ids"], fwd["topk_weights"], dy)
    b = L.backward(inp, fwd["topk_ids"], fwd["topk_weights"], dy, dlogits=aux)
    z = L.backward(inp, fwd["topk_ids"], fwd["topk_weights"], dy, dlogits=torch.zeros_like(aux))
    torch.cuda.synchronize()
    for k in ("dw_gate_up", "dw_down"):
        assert torch.equal(a[k], b[k])
    for k in a:
        assert torch.equal(a[k], z[k]), k
    d, x, w = aux.double().cpu(), inp["x"].double().cpu(), inp["router_w"].double().cpu()
    for k, add in (("dw_router", d.t() @ x), ("dbias", d.sum(0)), ("dx", d @ w)):
        ref = a[k].double().cpu() + add
        assert add.abs().max() > 0
        err = (b[k].double().cpu() - ref).abs().max() / ref.square().mean().sqrt()
        assert err < 1e-3, (k, float(err))
    with pytest.raises(ValueError):
        L.backward(inp, fwd["topk_ids"], fwd["topk_weights"], dy, dlogits=aux[:, :5])


def test_offsets_past_32_bits(gpu_lib):
    """More than 2^31 logits: the gradient of rows at both ends from the counts
    and the softmax of the rows themselves."""
    from moe_layer_router_amd import layer as L
    T, E, k = 2_200_000, 1000, 2
    l = torch.empty(T, E, device="cuda")
    l.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    ids = torch.stack([torch.arange(T, device="cuda") ** 2 % E, torch.arange(T, device="cuda") % 7], 1).to(torch.int32)
    out = L.balance_loss(l, ids, alpha=1.0)
    torch.cuda.synchronize()
    c = torch.bincount(ids.long().reshape(-1), minlength=E)
    assert torch.equal(out["counts"][0].long(), c)
    for t in (0, 1_000_003, T - 1):
        p = torch.softmax(l[t].double(), 0)
        h = (c - c[l[t].argmax()]).double()
        ref = E / (k * float(T) ** 2) * p * (h - p @ h)
        bound = E / (k * float(T) ** 2) * p * (h.abs() + p @ h.abs())
        assert bool(((out["dlogits"][t].double() - ref).abs() <= 108 * U * bound + 2.0 ** -130).all()), t
    mean = torch.zeros(E, dtype=torch.float64, device="cuda")
    for i in range(0, T, 100_000):
        mean += torch.softmax(l[i:i + 100_000].double(), 1).sum(0)
    # sums over blocks of about T / 1024 tokens, then over the blocks: (28 + 40 + T / 1024 + 64) roundings
    err = (out["probs"][0].double() - mean / T).abs() / (mean / T)
    assert float(err.max()) <= (132 + T / 1024) * U

"""Selection of experts and its gradient on the GPU against the fp64
definition, through the layer's forward and backward pass too.

Ids are equal: the device compares scores in 64 bits, ties go to the lower
index, and random inputs have no two experts within fp64's rounding.
Tolerances, with u = 2^-24.  A weight is a quotient of exponentials: each has
its argument's rounding (|l - m| u, at most R u with R the row's range) and
that of the function (2 u), a sum of E terms 16 + 6 levels of u, the quotient
and the scale 2 u each: (2 R + 60) u relative.  A gradient is formed in fp64
and rounded once (u); with softmax scores over all experts its products take
fp32 exponentials: (R + 16) u of the terms it is the difference of."""

import numpy as np
import pytest
import torch

from oracle import block as B
from oracle import moe_oracle as O
from workloads import gen

from tests._helpers import to_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _np(t):
    return t.detach().cpu().numpy().astype(np.float64)


def _range(l):
    f = np.where(np.isfinite(l), l, np.nan)
    with np.errstate(all="ignore"):
        r = np.nanmax(f, axis=1) - np.nanmin(f, axis=1)
    return np.where(np.isnan(r), 0, r)[:, None]


def _check(l, k, bias, **kw):
    from moe_layer_router_amd import layer as L
    dev = None if bias is None else torch.from_numpy(bias).cuda()
    out = L.select_experts(torch.from_numpy(l).cuda(), k, bias=dev, **kw)
    ids, w = B.select_experts(l, k, bias=bias, **kw)
    got = _np(out["topk_ids"]).astype(np.int64)
    assert np.array_equal(got, ids), np.flatnonzero((got != ids).any(1))[:5]
    g = _np(out["topk_weights"])
    assert np.all(np.abs(g - w) <= (2 * _range(l) + 60) * U * np.abs(w) + 1e-37)
    return out, ids, w


CASES = [
    # T, E, k, groups, keep, top
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (3, 2, 2, 1, 1, 1), (5, 8, 2, 8, 2, 1), (65, 63, 4, 7, 3, 2),
    (64, 64, 6, 64, 9, 1), (130, 65, 16, 13, 4, 2), (77, 128, 8, 4, 1, 2), (300, 129, 3, 3, 2, 1), (257, 256, 8, 8, 4, 2),
    (40, 257, 16, 1, 1, 1), (33, 512, 16, 32, 5, 2), (70, 544, 16, 2, 1, 2), (21, 1000, 10, 50, 50, 2),
    (200, 1024, 16, 16, 4, 2), (9, 1024, 1, 64, 1, 1),
]


@pytest.mark.parametrize("T,E,k,groups,keep,top", CASES)
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
def test_select(gpu_lib, T, E, k, groups, keep, top, scoring, biased):
    rng = np.random.default_rng(T * E + k)
    popular = rng.normal(size=E)
    l = (1.5 * rng.normal(size=(T, E)) + popular).astype(np.float32)
    bias = ((0.1 if scoring == "sigmoid" else 0.5 / E) * (rng.normal(size=E) - popular)).astype(np.float32) if biased else None
    _check(l, k, bias, scoring=scoring, n_group=groups, topk_group=keep, group_top=top, renormalize=bool(T % 2), scale=2.5)


@pytest.mark.parametrize("E,groups", [(8, 1), (60, 4), (256, 8), (1024, 16)])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_index(gpu_lib, E, groups, biased):
    """Logits of five values, and all of one; a bias that makes sums equal again."""
    rng = np.random.default_rng(E)
    l = rng.integers(-2, 3, size=(50, E)).astype(np.float32)
    l[7] = 0.5
    bias = np.full(E, 0.25, np.float32) if biased else None
    for scoring in ("sigmoid", "softmax"):
        for renorm in (False, True):
            _check(l, 4, bias, scoring=scoring, n_group=groups, topk_group=max(1, groups // 2), group_top=2,
                   renormalize=renorm)


def test_scores_that_fp32_cannot_tell_apart(gpu_lib):
    """Scores a few 2^-30 apart, far below an fp32 sigmoid's rounding, at the border of the selection and of the groups."""
    rng = np.random.default_rng(3)
    T, E = 200, 256
    l = np.full((T, E), 2.0, np.float32)
    step = rng.integers(0, 1 << 10, size=(T, E)).astype(np.float32)
    l += step * np.float32(2.0 ** -22)                 # sigmoid'(2) = 0.105: differences of 2^-25
    bias = np.zeros(E, np.float32)
    s = 1 / (1 + np.exp(-l.astype(np.float64)))
    assert all(len(np.unique(s[t].astype(np.float32))) < len(np.unique(s[t])) for t in range(3))
    _check(l, 8, bias, n_group=8, topk_group=4)
    _check(l, 8, None, n_group=8, topk_group=4)
    _check(l, 16, bias, scoring="softmax", renormalize=False)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_extreme_logits(gpu_lib, scoring, renorm):
    """Rows of -infinity, masked experts, logits whose scores underflow or saturate fp32."""
    rng = np.random.default_rng(5)
    l = rng.normal(size=(12, 96)).astype(np.float32)
    l[0] = -np.inf
    l[1, 5:] = -np.inf                                 # fewer experts than asked for
    l[2, ::2] = -np.inf
    l[3] -= 80                                         # sigmoid below fp32's normal range
    l[4] -= 300
    l[5] += 30                                         # 1 - s below fp32's resolution
    l[6, 10] = 90
    for bias in (None, (0.01 * rng.normal(size=96)).astype(np.float32)):
        _check(l, 8, bias, scoring=scoring, renormalize=renorm, n_group=6, topk_group=3)
        _check(l, 8, bias, scoring=scoring, renormalize=renorm)


def test_a_bias_of_minus_infinity_takes_experts_out(gpu_lib):
    rng = np.random.default_rng(6)
    l = rng.normal(size=(30, 40)).astype(np.float32)
    bias = np.where(np.arange(40) % 3 == 0, -np.inf, 0.0).astype(np.float32)
    out, ids, _ = _check(l, 6, bias)
    assert np.all(ids % 3 != 0)
    _check(l, 6, bias, n_group=4, topk_group=2)
    _check(l, 6, np.full(40, -np.inf, np.float32), n_group=4, topk_group=2)


def test_nan_is_last_and_stays_in_its_token(gpu_lib):
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(7)
    l = rng.normal(size=(9, 64)).astype(np.float32)
    clean = L.select_experts(torch.from_numpy(l).cuda(), 4, n_group=8, topk_group=4)
    l[4, 13] = np.nan
    for kw in (dict(n_group=8, topk_group=4), dict(), dict(bias=torch.zeros(64, device="cuda"))):
        out = L.select_experts(torch.from_numpy(l).cuda(), 4, **kw)
        assert 13 not in _np(out["topk_ids"])[4] and np.all(np.isfinite(_np(out["topk_weights"])))
    rest = [t for t in range(9) if t != 4]
    out = L.select_experts(torch.from_numpy(l).cuda(), 4, n_group=8, topk_group=4)
    for n in clean:
        assert torch.equal(clean[n][rest], out[n][rest])
    l[4] = np.nan
    out = L.select_experts(torch.from_numpy(l).cuda(), 4, scoring="softmax")
    assert _np(out["topk_ids"])[4].tolist() == [0, 1, 2, 3] and np.all(np.isnan(_np(out["topk_weights"])[4]))
    out = L.select_experts(torch.from_numpy(l).cuda(), 4, scoring="softmax", renormalize=False, bias=torch.zeros(64, device="cuda"))
    assert _np(out["topk_ids"])[4].tolist() == [0, 1, 2, 3] and np.all(np.isfinite(_np(out["topk_weights"])[rest]))


def _check_bwd(l, ids, dw, **kw):
    from moe_layer_router_amd import layer as L
    got = _np(L.select_experts_backward(torch.from_numpy(l).cuda(), torch.from_numpy(ids.astype(np.int32)).cuda(),
                                        torch.from_numpy(dw).cuda(), **kw))
    ref = B.select_experts_backward(l, ids, dw, **kw)
    bound = U * np.abs(ref) + 2.0 ** -44 * np.abs(dw).max(1, keepdims=True) * abs(kw.get("scale", 1.0))
    if kw.get("scoring") == "softmax" and not kw.get("renormalize", True):
        for t in range(len(l)):
            s = B.scores(l[t].astype(np.float64), "softmax")
            part = np.zeros_like(s)
            np.add.at(part, np.clip(ids[t], 0, len(s) - 1), np.abs(dw[t]) * abs(kw.get("scale", 1.0)))
            bound[t] += (min(_range(l)[t, 0], 28) + 16) * U * s * (part + (s * part).sum())
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) / np.maximum(bound, 1e-300))
    return got


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (65, 63, 4), (64, 64, 6), (130, 65, 16), (77, 128, 8),
                                   (300, 129, 3), (257, 256, 8), (40, 257, 16), (33, 512, 1), (21, 1000, 10), (100, 1024, 16)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_select_backward(gpu_lib, T, E, k, scoring, renorm):
    rng = np.random.default_rng(E + k)
    l = (1.5 * rng.normal(size=(T, E))).astype(np.float32)
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    dw = rng.normal(size=(T, k)).astype(np.float32)
    _check_bwd(l, ids, dw, scoring=scoring, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_select_backward_of_unusual_ids_and_logits(gpu_lib, scoring, renorm):
    """An id twice, all the same, out of range (clamped); rows of -infinity; sure and underflowing experts."""
    rng = np.random.default_rng(8)
    l = rng.normal(size=(8, 70)).astype(np.float32)
    ids = rng.integers(0, 70, size=(8, 5))
    ids[0] = [3, 9, 3, 3, 9]
    ids[1] = 69
    ids[2] = [-5, 70, 1 << 30, -(1 << 31), 7]
    l[3] = -np.inf
    l[4, 20:] = -np.inf
    l[5] -= 200
    l[6, ids[6, 0]] = 40
    with np.errstate(invalid="ignore"):
        _check_bwd(l, ids, rng.normal(size=(8, 5)).astype(np.float32), scoring=scoring, renormalize=renorm)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_select_gradient_against_differences_of_the_device(gpu_lib, scoring):
    """Central differences of the device's own weights: fp32 weights (1e-7 off) over steps of 2^-6."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(9)
    l = rng.normal(size=(1, 12)).astype(np.float32)
    dw = rng.normal(size=(1, 12)).astype(np.float32)
    for renorm in (False, True):
        kw = dict(scoring=scoring, renormalize=renorm)
        ids = torch.arange(12, dtype=torch.int32, device="cuda")[None]
        g = _np(L.select_experts_backward(torch.from_numpy(l).cuda(), ids, torch.from_numpy(dw).cuda(), **kw))[0]
        h = np.float32(2.0 ** -6)
        for e in range(12):
            f = []
            for sign in (1, -1):
                x = l.copy()
                x[0, e] += sign * h
                r = L.select_experts(torch.from_numpy(x).cuda(), 12, **kw)     # all experts: no border
                f.append((_np(r["topk_weights"]) * dw[:, _np(r["topk_ids"]).astype(int)[0]]).sum())
            # third derivatives of s are below 1/8 (of the quotient below 1), fp32 weights 2^-22 off
            assert abs((f[0] - f[1]) / (2 * float(h)) - g[e]) < 12 * (2.0 ** -12 / 6 + 2.0 ** -22 / float(h))


def test_offsets_past_32_bits(gpu_lib):
    """T E = 2^31 + 2^21 logits: the last token's row lies past 2^33 bytes."""
    from moe_layer_router_amd import layer as L
    E = 1024
    T = (1 << 21) + 2048
    l = torch.zeros(T, E, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = [0, 1 << 20, (1 << 21) - 1, 1 << 21, T - 1]
    for t in rows:
        l[t] = torch.randn(E, generator=g, device="cuda")
    out = L.select_experts(l, 8, n_group=8, topk_group=4)
    ids, w = B.select_experts(_np(l[rows]), 8, n_group=8, topk_group=4)
    assert np.array_equal(_np(out["topk_ids"][rows]), ids)
    assert bool((out["topk_ids"][1:1000] == torch.arange(8, device="cuda")).all())
    d = L.select_experts_backward(l, out["topk_ids"], out["topk_weights"])
    ref = B.select_experts_backward(_np(l[rows]), ids, _np(out["topk_weights"][rows]))
    assert np.all(np.abs(_np(d[rows]) - ref) <= 2 * U * np.abs(ref) + 1e-12)


def test_select_streams_views_and_reused_outputs(gpu_lib):
    """Logits that are no dense matrix, on a side stream, into the outputs of a call before."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(10)
    l = rng.normal(size=(50, 96)).astype(np.float32)
    wide = torch.from_numpy(np.concatenate([l, l], 1)).cuda()[:, 1:97]
    assert not wide.is_contiguous()
    ref = L.select_experts(wide.contiguous(), 6, n_group=4, topk_group=2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = {n: torch.full_like(v, 7) for n, v in ref.items()}
    side.wait_stream(torch.cuda.current_stream())
    got = L.select_experts(wide, 6, n_group=4, topk_group=2, stream=side, out=out)
    d = L.select_experts_backward(wide, got["topk_ids"], got["topk_weights"], stream=side)
    side.synchronize()
    assert got is out and all(torch.equal(ref[n], out[n]) for n in ref)
    assert torch.equal(d, L.select_experts_backward(wide.contiguous(), ref["topk_ids"], ref["topk_weights"]))
    for bad in (dict(bias=torch.zeros(95, device="cuda")), dict(bias=torch.zeros(96)), dict(scoring="relu"),
                dict(out=dict(topk_ids=out["topk_weights"], topk_weights=out["topk_weights"]))):
        with pytest.raises(ValueError):
            L.select_experts(wide, 6, **bad)
    with pytest.raises(gpu_lib.MoeError):
        L.select_experts(wide, 17)
    with pytest.raises(ValueError):
        L.select_experts_backward(wide, ref["topk_ids"].long(), ref["topk_weights"])


SELECTIONS = [dict(scoring="sigmoid", n_group=4, topk_group=2, scale=2.5),
              dict(scoring="softmax", renormalize=False), dict(scoring="sigmoid", renormalize=False, scale=0.5)]


@pytest.mark.parametrize("kw", SELECTIONS, ids=["groups", "softmax", "plain"])
@pytest.mark.parametrize("aux", [False, True])
def test_layer_routed_by_a_selection(gpu_lib, kw, aux):
    """forward(selection=) and backward(selection=): the routed layer for those weights, and the router's gradient through
    them.  Tolerance as the backward pass's own test: 1e-3 of the larger of the element and the rms."""
    from moe_layer_router_amd import layer as L
    cfg = gen.LayerConfig("sel", 130, 256, 16, 3, 128, "bf16", "bf16")
    raw = gen.make_inputs(cfg, seed=21)
    dev = to_dev(raw)
    rng = np.random.default_rng(2)
    bias = (0.05 * rng.normal(size=cfg.E)).astype(np.float32)
    sel = dict(kw, bias=torch.from_numpy(bias).cuda())
    fwd = L.forward(L.pack_weights(dev), cfg.k, selection=sel)
    ids, w = B.select_experts(_np(fwd["logits"]), cfg.k, bias=bias, **kw)
    assert np.array_equal(_np(fwd["topk_ids"]), ids)
    spec, view = gen.spec_of(cfg), gen.oracle_view(raw)
    xh, logits, _, _ = O.route(spec, view)
    assert np.abs(_np(fwd["logits"]) - logits).max() <= 1e-4
    given = L.forward(L.pack_weights(dev), cfg.k, routing=(fwd["topk_ids"], fwd["topk_weights"]))
    assert torch.equal(given["y"], fwd["y"])
    dy = torch.randn(cfg.T, cfg.H, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    dl = (1e-2 * torch.randn(cfg.T, cfg.E, generator=torch.Generator().manual_seed(4))) if aux else None
    got = L.backward(dev, fwd["topk_ids"], fwd["topk_weights"], dy.cuda(), selection=sel, logits=fwd["logits"],
                     dlogits=None if dl is None else dl.cuda())
    # fp64: the experts' part by definition, the router's by the selection's gradient
    wgu, wd, wr = (O.decode_weight(spec, view[n]) if n != "router_w" else _np(dev[n].float()) for n in ("w_gate_up", "w_down", "router_w"))
    dyn, x, I = _np(dy.float()), _np(dev["x"].float()), cfg.I
    dx, dgu, dd, dw = np.zeros((cfg.T, cfg.H)), np.zeros_like(wgu), np.zeros_like(wd), np.zeros((cfg.T, cfg.k))
    for t in range(cfg.T):
        for j, e in enumerate(ids[t]):
            gu = wgu[e] @ x[t]
            g, u = gu[:I], gu[I:]
            a = O.swiglu(g, u)
            dw[t, j] = dyn[t] @ (wd[e] @ a)
            dd[e] += w[t, j] * np.outer(dyn[t], a)
            da = w[t, j] * (dyn[t] @ wd[e])
            d = np.concatenate([da * u * O.silu_grad(g), da * O.silu(g)])
            dgu[e] += np.outer(d, x[t])
            dx[t] += d @ wgu[e]
    dlog = B.select_experts_backward(logits, ids, dw, **{n: v for n, v in kw.items() if n in ("scoring", "renormalize", "scale")})
    if aux:
        dlog = dlog + dl.numpy().astype(np.float64)
    ref = dict(dx=dx + dlog @ wr, dw_gate_up=dgu, dw_down=dd, dw_router=dlog.T @ x, dbias=dlog.sum(0))
    for name, axes in (("dx", (1,)), ("dw_gate_up", (1, 2)), ("dw_down", (1, 2)), ("dw_router", (0, 1)), ("dbias", (0,))):
        r, v = ref[name], _np(got[name])
        rms = np.sqrt((r ** 2).mean(axis=axes, keepdims=True))
        assert np.all(np.isfinite(v)) and np.max(np.abs(v - r) / np.maximum(np.maximum(np.abs(r), rms), 1e-30)) <= 1e-3, name


def test_two_tokens_per_wave_past_32_bits(gpu_lib):
    """More than 2^32 logits of 256 experts, an odd number of tokens."""
    from moe_layer_router_amd import layer as L
    T, E = (1 << 24) + 7, 256
    l = torch.zeros(T, E, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = [0, (1 << 22) + 1, (1 << 23) - 1, 1 << 23, 1 << 24, T - 2, T - 1]
    for t in rows:
        l[t] = torch.randn(E, generator=g, device="cuda")
    out = L.select_experts(l, 8, n_group=8, topk_group=4)
    ids, w = B.select_experts(_np(l[rows]), 8, n_group=8, topk_group=4)
    assert np.array_equal(_np(out["topk_ids"][rows]), ids)
    assert np.all(np.abs(_np(out["topk_weights"][rows]) - w) <= 80 * U * w)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert bool((out["topk_ids"][rest] == torch.arange(8, device="cuda")).all())


def test_more_tokens_than_one_launch_takes(gpu_lib):
    from moe_layer_router_amd import layer as L
    T, E = (1 << 26) + 3, 3
    l = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    out = L.select_experts(l, 2, scoring="softmax", renormalize=False)
    top = torch.topk(l, 2, dim=1)
    same = (torch.gather(l, 1, out["topk_ids"].long()) == top.values).all(1)
    assert bool(same.all())
    p = torch.softmax(l[-5:].double(), 1)
    assert float((out["topk_weights"][-5:].double() - torch.gather(p, 1, out["topk_ids"][-5:].long())).abs().max()) <= 80 * U


def test_many_tokens_that_fp32_does_not_settle(gpu_lib):
    """Every token of a large batch near a tie, in one of its halves, in both, or in its groups; and more candidates than lanes."""
    rng = np.random.default_rng(12)
    for E, groups, keep in ((256, 8, 4), (128, 4, 2), (64, 16, 5), (200, 1, 1), (1000, 10, 4)):
        T = 331
        l = rng.normal(size=(T, E)).astype(np.float32)
        l[::3] = np.round(l[::3] * 2) / 2                  # a few values: ties everywhere
        l[1::3] = 1.0 + rng.integers(0, 64, size=l[1::3].shape).astype(np.float32) * np.float32(2.0 ** -23)
        bias = (1e-9 * rng.normal(size=E)).astype(np.float32)
        for scoring in ("sigmoid", "softmax"):
            for b in (None, bias):
                _check(l, 7, b, scoring=scoring, n_group=groups, topk_group=keep, group_top=2, renormalize=True)
                _check(l, 16, b, scoring=scoring, n_group=groups, topk_group=keep, group_top=1, renormalize=False)


@pytest.mark.parametrize("E,groups,keep", [(256, 8, 4), (96, 3, 2), (512, 4, 2), (1024, 8, 3)])
@pytest.mark.parametrize("at", [-6.0, -20.0, -60.0, -85.0])
def test_small_scores_a_unit_of_the_logits_apart(gpu_lib, E, groups, keep, at):
    """Logits that differ by a few of their last bits, where an fp32 exponential's argument is off by as much: without a bias the
    order is the logits', whatever their scores round to; with one smaller than the scores it is that of 64-bit scores."""
    rng = np.random.default_rng(E + int(at))
    T = 400
    unit = float(np.spacing(np.float32(abs(at))))
    step = rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)
    l = (at + step * unit).astype(np.float32)
    assert len(np.unique(l[0])) == E
    _check(l, 8, None, n_group=groups, topk_group=keep, group_top=2)
    _check(l, 8, None, n_group=groups, topk_group=keep, group_top=1, renormalize=False)
    s = 1 / (1 + np.exp(-float(at)))
    bias = (1e-7 * s * rng.normal(size=E)).astype(np.float32)
    _check(l, 8, bias, n_group=groups, topk_group=keep, group_top=2)
    # softmax: the same differences far below one large logit
    l[:, 0] = l[:, 0] + 2 * abs(at)
    _check(l, 8, None, scoring="softmax", n_group=groups, topk_group=keep, group_top=2)
    _check(l, 8, np.float32(0.5) * bias, scoring="softmax", renormalize=False)


@pytest.mark.parametrize("E", [100, 256, 1000])
@pytest.mark.parametrize("at", [0.0, 300.0])
def test_biases_that_even_out_softmax_scores(gpu_lib, E, at):
    """A bias that makes all c of some rows equal but for its own rounding: their order is that of the fp64 sum."""
    rng = np.random.default_rng(E)
    rows = (rng.normal(size=(3, E)) + at).astype(np.float32)
    for i in range(3):
        s = np.exp(rows[i].astype(np.float64) - rows[i].max())
        s /= s.sum()
        bias = (s.max() + 0.01 - s).astype(np.float32)
        l = np.concatenate([rows, rows + rng.integers(-1, 2, size=rows.shape).astype(np.float32) * np.float32(2.0 ** -15), rows])
        _check(l, 8, bias, scoring="softmax", renormalize=False)
        _check(l, 16, bias, scoring="softmax")

"""The AdamW step on the GPU against the fp64 definition.

Tolerances, with u = 2^-24 and the states that the call read: m' = b1 m + a1 g
takes the roundings of its two constants, of the product and of the fused sum:
4 u (|b1 m| + |a1 g|), and one more for a grad_scale; v' the same and g^2's: 5 u v'.
The update lr m'/(...) takes m' 's and half of v' 's error, two units of the reciprocal, two of the
root, and those of its constants and products: 16 u of |lr| (|b1 m| + |a1 g|) / c1 / (...);
w' the decay's and the last sum's: 2 u (|w| + |w'|).  What is then rounded to BF16 is
within half a step (2^-8 of the value) to nearest, a whole one stochastically.
8-bit states: the scale is the largest magnitude / 448, 2 u more; a code is one of
the two around value / scale, the upper one where the dropped fraction and the
random bits reach 1, either one where they do so within 16 steps of 8 u."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
GRID = np.sort(np.unique(np.abs(B.F.e4m3_decode(np.arange(127, dtype=np.uint8)))))      # 0 .. 448


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _tensors(sizes, p, master, g, state, seed=0):
    """params, grads, masters, states as the wrapper takes them."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    params, grads, masters, states = [], [], [], []
    for i, n in enumerate(sizes):
        w = 0.1 * rn(n)
        params.append(w.to(torch.bfloat16) if p == "bf16" else w)
        masters.append(w.clone() if master else None)
        size = 10.0 ** (i % 5 - 3)
        gr = size * rn(n)
        grads.append(gr.to(torch.bfloat16) if g == "bf16" else gr)
        if state == "f32":
            states.append(dict(m=0.3 * size * rn(n), v=(size * rn(n)) ** 2))
        else:
            nb = (n + 127) // 128
            codes = torch.randint(0, 127, (n,), generator=gen, device="cuda", dtype=torch.uint8)
            sign = 128 * torch.randint(0, 2, (n,), generator=gen, device="cuda", dtype=torch.uint8)
            states.append(dict(m=codes | sign, v=torch.randint(0, 127, (n,), generator=gen, device="cuda", dtype=torch.uint8),
                               m_scales=size / 448 * (0.5 + rn(nb).abs()), v_scales=size / 448 * (0.5 + rn(nb).abs())))
    return params, grads, masters, states


def _moments(s, state):
    if state == "f32":
        return _np(s["m"]), _np(s["v"])
    m = B.state_values(s["m"].cpu().numpy(), _np(s["m_scales"]))
    return m, B.state_values(s["v"].cpu().numpy(), _np(s["v_scales"])) ** 2


def _check_codes(codes, scales, ref, err, bits, root, few):
    """8-bit states against fp64 values `ref` that the device has within `err`."""
    n = len(ref)
    pad = lambda a: np.concatenate([a, np.zeros(-n % 128)]).reshape(-1, 128)
    amax = np.abs(pad(ref)).max(1)
    want = np.where(amax < 2.0 ** -100, 1.0, amax / 448)
    assert np.all(np.abs(scales - want) <= pad(err).max(1) / 448 + 2 * U * want), "scales"
    s = np.repeat(scales, 128)[:n]
    x, dx = np.abs(ref) / s, err / s + 3 * U * np.abs(ref) / s
    x = np.minimum(x, 448)
    lo = GRID[np.searchsorted(GRID, x, side="right") - 1]
    hi = GRID[np.minimum(np.searchsorted(GRID, x, side="right"), len(GRID) - 1)]
    frac = np.where(hi > lo, (x - lo) / np.where(hi > lo, hi - lo, 1), 0)
    edge = np.where(hi > lo, dx / np.where(hi > lo, hi - lo, 1), 0) + 2.0 ** -20
    up = frac + bits / 65536
    got = np.abs(B.F.e4m3_decode(codes))
    expect = np.where(up >= 1, hi, lo)
    if root:
        expect = np.where((expect == 0) & (ref > 0), 2.0 ** -9, expect)
    near = (np.abs(up - 1) <= edge) | (frac <= edge) | (frac >= 1 - edge)
    steps = np.abs(np.searchsorted(GRID, got) - np.searchsorted(GRID, expect))
    assert np.all(got[~near] == expect[~near]), np.flatnonzero(~near & (got != expect))[:5]
    assert np.all(steps[near] <= 1)
    # few elements are left to either code: those within edge (about 1e-5) of a border, and each block's largest,
    # which is at the code 448 by construction (value / (largest / 448)).  (Not so where scaled-down gradients leave
    # all of a block shrinking by one factor, each value / scale at the code that it came from.)
    if few:
        assert (near & (x < 448 * (1 - 8 * U))).sum() <= 2 + 0.05 * n
    sign = np.signbit(B.F.e4m3_decode(codes))
    assert np.all(sign[got > 0] == (ref < 0)[got > 0])


def _step_and_check(sizes, p, master, g, state, t=3, lr=1e-2, betas=(0.9, 0.999), eps=1e-8, decay=0.1, scale=None, seed=5):
    from moe_layer_router_amd import layer as L
    params, grads, masters, states = _tensors(sizes, p, master, g, state)
    before = [( _np(w if w is not None else q), *_moments(s, state)) for q, w, s in zip(params, masters, states)]
    decays = [decay * (i % 2) for i in range(len(sizes))]
    opt = L.AdamW(params, masters=masters if master else None, states=states, betas=betas, eps=eps, weight_decay=decays, seed=seed,
                  count=t - 1)
    assert opt.state == state
    opt.step(grads, lr, grad_scale=None if scale is None else torch.tensor([scale], device="cuda"))
    torch.cuda.synchronize()
    assert opt.count == t
    gs = 1.0 if scale is None else float(np.float32(scale))
    for i, (w, m, v) in enumerate(before):
        n, gr = len(w), _np(grads[i])
        rw, rm, rv = B.adamw(w, gr, m, v, t, lr, betas, eps, decays[i], gs)
        both = np.abs(betas[0] * m) + np.abs((1 - betas[0]) * gs * gr)
        em, ev = 5 * U * both, 7 * U * rv
        den = np.sqrt(rv / (1 - betas[1] ** t)) + eps
        ew = 16 * U * abs(lr) * both / (1 - betas[0] ** t) / den + 2 * U * (np.abs(w) + np.abs(rw)) + 1e-38
        bm, bv, bw = (b.astype(np.float64) for b in B.dice(n, seed, t, i))
        s = states[i]
        if state == "f32":
            assert np.all(np.abs(_np(s["m"]) - rm) <= em + 1e-38) and np.all(np.abs(_np(s["v"]) - rv) <= ev + 1e-38), i
        else:
            _check_codes(s["m"].cpu().numpy(), _np(s["m_scales"]), rm, em, bm, False, scale is None)
            r = np.sqrt(rv)
            _check_codes(s["v"].cpu().numpy(), _np(s["v_scales"]), r, 5 * U * r, bv, True, scale is None)
        got = _np(params[i])
        if p == "f32":
            assert np.all(np.abs(got - rw) <= ew), i
        elif master:
            fresh = _np(masters[i])
            assert np.all(np.abs(fresh - rw) <= ew)
            assert torch.equal(params[i], masters[i].to(torch.bfloat16))
        else:
            # bits above the dropped 16 of the fp32 value, one more where they and the random bits carry
            x = rw.astype(np.float32).view(np.uint32).astype(np.uint64)
            want = B.F.bf16_decode(((x + bw.astype(np.uint64)) >> np.uint64(16)).astype(np.uint16))
            ulp = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(rw), 1e-37))) - 7)
            drop = (x & np.uint64(0xFFFF)).astype(np.float64) + bw
            near = np.minimum(np.abs(drop - 65536), np.minimum(drop - bw, 65536 - (drop - bw))) * ulp / 65536 <= ew + U * np.abs(rw)
            assert np.all(got[~near] == want[~near]), i
            assert np.all(np.abs(got - rw)[near] <= ulp[near] * 1.01 + ew[near])
    return params, states


SIZES = [1, 7, 8, 9, 127, 128, 129, 1000, 2047, 2048, 2049, 4096, 8200, 20001]


@pytest.mark.parametrize("p,master", [("f32", False), ("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_adamw(gpu_lib, p, master, g, state):
    _step_and_check(SIZES, p, master, g, state)


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_adamw_large_chunks(gpu_lib, state):
    """Enough elements for the larger workgroups, sizes that end inside one."""
    _step_and_check([17_000_003, 8191, 8193, 40], "bf16", state == "f32", "f32", state)


@pytest.mark.parametrize("over", [dict(t=1), dict(t=100_000), dict(betas=(0.0, 0.0)), dict(betas=(0.95, 0.9)), dict(decay=0.0),
                                  dict(lr=0.0), dict(lr=-1e-3), dict(eps=1.0), dict(scale=0.125), dict(scale=0.0),
                                  dict(seed=(1 << 32) - 1, t=(1 << 33) + 7)],
                         ids=lambda o: "-".join(f"{k}={v}" for k, v in o.items()))
@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_adamw_hyperparameters(gpu_lib, over, state):
    _step_and_check([300, 2500], "f32", False, "f32", state, **over)


def test_adamw_of_many_tensors_in_several_launches(gpu_lib):
    """130 tensors of each kind mixed: three launches' worth, each with its own random bits."""
    from moe_layer_router_amd import layer as L
    kinds = [("f32", False, "f32"), ("bf16", False, "f32"), ("bf16", True, "bf16")]
    parts = [_tensors([1 + (i * 37) % 700 for i in range(130)], p, w, g, "f32", seed=k) for k, (p, w, g) in enumerate(kinds)]
    order = [(k, i) for i in range(130) for k in range(3)]
    pick = lambda j: [parts[k][j][i] for k, i in order]
    params, grads, masters, states = (pick(j) for j in range(4))
    ref = [[_np(w if w is not None else q), *_moments(s, "f32")] for q, w, s in zip(params, masters, states)]
    opt = L.AdamW(params, masters=masters, states=states, weight_decay=0.01, count=9)
    opt.step(grads, 1e-3)
    for i in range(len(params)):
        rw, rm, rv = B.adamw(ref[i][0], _np(grads[i]), ref[i][1], ref[i][2], 10, 1e-3, decay=0.01)
        assert np.all(np.abs(_np(states[i]["m"]) - rm) <= 5 * U * (np.abs(ref[i][1]) + np.abs(_np(grads[i])))), i
        assert np.all(np.abs(_np(states[i]["v"]) - rv) <= 7 * U * rv), i
        tol = {torch.float32: 1e-6}.get(params[i].dtype, 2.0 ** -7)
        assert np.all(np.abs(_np(params[i]) - rw) <= tol * np.maximum(np.abs(rw), 1e-3)), i


def test_adamw_states_from_zero_over_many_steps(gpu_lib):
    """300 steps on a quadratic: 8-bit states and BF16 weights follow the fp64 run on average, where rounding to nearest
    would stand still.  Stochastic rounding's noise averages over the 4096 weights: their mean is held to 2%, v's mean to 5%."""
    from moe_layer_router_amd import layer as L
    n = 4096
    gen = torch.Generator(device="cuda").manual_seed(3)
    target = 1 + 0.1 * torch.randn(n, generator=gen, device="cuda")
    noise = [0.5 * torch.randn(n, generator=gen, device="cuda") for _ in range(300)]
    runs = {}
    for name in ("f32", "fp8"):
        w = torch.zeros(n, device="cuda", dtype=torch.float32 if name == "f32" else torch.bfloat16)
        opt = L.AdamW([w], state=name, betas=(0.9, 0.99))
        for z in noise:
            opt.step([w.float() - target + z], 2e-3)
        runs[name] = (_np(w), _moments(opt.states[0], name)[1])
    w64, m, v = np.zeros(n), np.zeros(n), np.zeros(n)
    for t, z in enumerate(noise):
        w64, m, v = B.adamw(w64, w64 - _np(target) + _np(z), m, v, t + 1, 2e-3, (0.9, 0.99))
    assert np.abs(runs["f32"][0] - w64).max() <= 1e-3 and np.abs(runs["f32"][1] / v - 1).max() <= 1e-2
    assert abs(runs["fp8"][0].mean() / w64.mean() - 1) <= 0.02
    assert abs(runs["fp8"][1].mean() / v.mean() - 1) <= 0.05


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_adamw_leaves_out_overflowed_steps(gpu_lib, state):
    from moe_layer_router_amd import layer as L
    for bad in (float("inf"), float("-inf"), float("nan")):
        params, grads, masters, states = _tensors([777, 5000], "bf16", True, "f32", state)
        keep = [t.clone() for t in params + masters + [v for s in states for v in s.values()]]
        opt = L.AdamW(params, masters=masters, states=states)
        opt.step(grads, 1e-3, grad_scale=torch.tensor([bad], device="cuda"))
        torch.cuda.synchronize()
        now = params + masters + [v for s in states for v in s.values()]
        assert all(torch.equal(a, b) for a, b in zip(keep, now)) and opt.count == 1


def test_adamw_what_is_not_finite_stays_in_its_place(gpu_lib):
    """NaN and infinity in a gradient: fp32 states lose that element, 8-bit ones its block of 128, visibly."""
    from moe_layer_router_amd import layer as L
    for state, lost in (("f32", 1), ("fp8", 128)):
        for bad in (float("nan"), float("inf")):
            params, grads, _, states = _tensors([1000], "f32", False, "f32", state)
            grads[0][300] = bad
            opt = L.AdamW(params, states=states)
            opt.step(grads, 1e-3)
            opt.step([torch.ones(1000, device="cuda")], 1e-3)
            m, v = _moments(states[0], state)
            block = slice(256, 384) if lost == 128 else slice(300, 301)
            rest = np.ones(1000, bool)
            rest[block] = False
            assert not np.any(np.isfinite(m[block])) and np.all(np.isfinite(m[rest])) and np.all(np.isfinite(v[rest]))
            assert np.all(np.isfinite(_np(params[0])[rest])) and not np.isfinite(_np(params[0])[300])


def test_adamw_zeros_and_tiny_values(gpu_lib):
    """Blocks of zeros keep a scale of 1; gradients down to fp32's smallest never divide by zero or make NaN."""
    from moe_layer_router_amd import layer as L
    for state in ("f32", "fp8"):
        w = torch.ones(1024, device="cuda")
        g = torch.zeros(1024, device="cuda")
        g[128:256] = 1e-36
        g[256:384] = 1e-42
        g[384:512] = 1e-18
        g[512:640] = 1e18
        opt = L.AdamW([w], state=state)
        for _ in range(3):
            opt.step([g], 1e-3)
        assert np.all(np.isfinite(_np(w))) and np.all(_np(w)[:128] == 1)
        for k in ("m", "v"):
            assert np.all(np.isfinite(_moments(opt.states[0], state)[0 if k == "m" else 1]))
        if state == "fp8":
            assert float(opt.states[0]["m_scales"][0]) == 1 and float(opt.states[0]["v_scales"][0]) == 1
            assert not opt.states[0]["m"][:128].any() and not opt.states[0]["v"][:128].any()
        assert np.all(np.abs(_np(w)[512:640] - (1 - 3e-3)) < 1e-4)


def test_adamw_same_call_same_bits_and_other_seeds_other_ones(gpu_lib):
    from moe_layer_router_amd import layer as L

    def go(seed, count=0):
        params, grads, _, states = _tensors([5000, 300], "bf16", False, "f32", "fp8")
        L.AdamW(params, states=states, seed=seed, count=count).step(grads, 1e-2)
        return params + [v for s in states for v in s.values()]
    a, b, c, d = go(1), go(1), go(2), go(1, 1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not torch.equal(a[0], c[0]) and not torch.equal(a[2], c[2]) and not torch.equal(a[3], d[3])


@pytest.mark.parametrize("state", ["f32", "fp8"])
def test_adamw_in_a_graph(gpu_lib, state):
    """A captured step with the count and lr on the device: every replay counts on and equals the eager step."""
    from moe_layer_router_amd import layer as L
    sizes = [3000, 129, 70_000]
    mk = lambda: _tensors(sizes, "bf16", False, "f32", state)
    pe, ge, _, se = mk()
    pc, gc, _, sc = mk()
    eager = L.AdamW(pe, states=se, weight_decay=0.1, count=4)
    cap = L.AdamW(pc, states=sc, weight_decay=0.1, count=4, capturable=True)
    lr, gs = torch.tensor([1e-2], device="cuda"), torch.tensor([1.0], device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.step(gc, lr, grad_scale=gs)
    torch.cuda.synchronize()
    assert int(cap.count) == 4
    for i in range(4):
        rate = 1e-2 / (i + 1)
        lr.fill_(rate)
        gs.fill_(0.5 * (i + 1) if i != 2 else float("inf"))
        for a, b in zip(gc, ge):
            a.copy_(b.mul_(0.9))
        graph.replay()
        # (fp32 lr, as the device has it)
        eager.step(ge, float(np.float32(rate)), grad_scale=gs.clone())
        torch.cuda.synchronize()
        assert int(cap.count) == eager.count == 5 + i
        for a, b in zip(pc, pe):
            # the bias corrections are formed on the device: the last bit of a step's size may differ
            assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -8 * float(b.float().abs().max())
        for a, b in zip(sc, se):
            ma, va = _moments(a, state)
            mb, vb = _moments(b, state)
            assert np.array_equal(ma, mb) and np.array_equal(va, vb)


def test_adamw_wrapper(gpu_lib):
    """States and shapes of any dimension, a side stream, gradients that are no dense tensors, memory exchanged between
    steps, refusals."""
    from moe_layer_router_amd import layer as L
    w = torch.randn(30, 50, device="cuda")
    x = w.clone()
    a, b = L.AdamW([w], state="fp8"), L.AdamW([x], state="fp8")
    assert a.states[0]["m"].shape == w.shape and a.states[0]["m_scales"].shape == (12,)
    g = torch.randn(50, 30, device="cuda").t()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.step([g], 1e-2, stream=side)
    b.step([g.contiguous()], 1e-2)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(w, x)
    old = w.clone()
    w.data = w.data.clone()                            # the step has to find the new memory
    a.step([g], 1e-2)
    b.step([g], 1e-2)
    assert torch.equal(w, x) and not torch.equal(w, old)
    for bad in (dict(params=[w.t()]), dict(params=[w], masters=[w.clone()]), dict(params=[w], states=[dict(m=w, v=w.half())]),
                dict(params=[w.cpu()]), dict(params=[w.bfloat16()], masters=[w.bfloat16()]),
                dict(params=[w], state="fp8", states=[dict(m=w, v=w, m_scales=w, v_scales=w)])):
        with pytest.raises((ValueError, KeyError)):
            L.AdamW(**bad).step([g], 1e-2)
    for args in (([g, g], 1e-2), ([g.half()], 1e-2), ([g[:10]], 1e-2), ([g.cpu()], 1e-2)):
        with pytest.raises(ValueError):
            a.step(*args)
    with pytest.raises(gpu_lib.MoeError):              # the same weights twice
        L.AdamW([w, w]).step([g, g], 1e-2)
    with pytest.raises(gpu_lib.MoeError):
        L.AdamW([torch.zeros(9, device="cuda")[1:]]).step([torch.zeros(8, device="cuda")], 1e-2)   # not on 16 bytes
    L.AdamW([torch.zeros(0, device="cuda"), w]).step([torch.zeros(0, device="cuda"), g], 0.0)


def test_adamw_moments_and_roots_are_rounded_once_per_operation(gpu_lib):
    """The states bit for bit as fp32 operations one at a time give them (the root correctly rounded), over all magnitudes down to
    the smallest: a last bit may decide a stochastic rounding."""
    from moe_layer_router_amd import layer as L
    rng = np.random.default_rng(1)
    n = 128 * 4000
    f = np.float32
    size = (10.0 ** rng.uniform(-22, 15, n // 128)).astype(f).repeat(128)
    g = (size * rng.normal(size=n)).astype(f)
    m0, r0 = (size * rng.normal(size=n)).astype(f), np.abs(size * rng.normal(size=n)).astype(f)
    c = dict(dtype=torch.float32, device="cuda")
    st = dict(m=torch.tensor(m0, **c), v=torch.tensor(r0 * r0, **c))
    L.AdamW([torch.zeros(n, **c)], states=[st]).step([torch.tensor(g, **c)], 1e-3)
    m = f(0.9) * m0 + f(1 - 0.9) * g
    v = f(0.999) * (r0 * r0) + f(1 - 0.999) * (g * g)
    assert np.array_equal(st["m"].cpu().numpy(), m) and np.array_equal(st["v"].cpu().numpy(), v)
    one = lambda: torch.ones(n // 128, **c)
    st = dict(m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"), m_scales=one(), v_scales=one())
    L.AdamW([torch.zeros(n, **c)], states=[st]).step([torch.tensor(g, **c)], 1e-3)
    root = np.sqrt(f(1 - 0.999) * (g * g))
    for k, x in (("m_scales", np.abs(f(1 - 0.9) * g)), ("v_scales", root)):
        top = x.reshape(-1, 128).max(1)
        assert np.array_equal(st[k].cpu().numpy(), np.where(top < 2.0 ** -100, f(1), top * f(1 / 448))), k


def test_adamw_scales_in_one_buffer(gpu_lib):
    """Scales of several tensors one after another: only the first lies on 16 bytes."""
    from moe_layer_router_amd import layer as L
    sizes = [130, 200, 1000, 90]
    params, grads, _, states = _tensors(sizes, "f32", False, "f32", "fp8")
    other = [p.clone() for p in params]
    flat = torch.cat([s[k] for k in ("m_scales", "v_scales") for s in states])
    views, at = [], 0
    for k in ("m_scales", "v_scales"):
        for s in states:
            views.append(flat[at:at + s[k].numel()])
            at += s[k].numel()
    shared = [dict(m=s["m"].clone(), v=s["v"].clone(), m_scales=views[i], v_scales=views[4 + i]) for i, s in enumerate(states)]
    L.AdamW(params, states=states).step(grads, 1e-2)
    L.AdamW(other, states=shared).step(grads, 1e-2)
    for i in range(4):
        assert torch.equal(params[i], other[i]) and all(torch.equal(states[i][k], shared[i][k]) for k in states[i])


def test_adamw_offsets_past_32_bits(gpu_lib):
    """2^31 + 1000 elements: byte offsets past 2^33, element indices past 2^31."""
    from moe_layer_router_amd import layer as L
    n = (1 << 31) + 1000
    w = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    opt = L.AdamW([w], state="fp8")
    opt.step([g], 0.25)
    s = opt.states[0]
    # -lr within a few fp32 units, so -0.25 or, once in thousands, the BF16 number 2^-10 below or 2^-9 above it in magnitude; the
    # states' values are their blocks' largest, the code 448 or the one below
    off = float((w + 0.25).abs().max())
    assert off <= 2.0 ** -9
    wrong = sum(int((s[k] < 125).sum()) + int((s[k] > 126).sum()) for k in ("m", "v"))
    assert wrong == 0
    for k, value in (("m_scales", 0.1 * 0.5 / 448), ("v_scales", (1e-3 * 0.25) ** 0.5 / 448)):
        assert float((s[k] - value).abs().max()) <= 1e-6 * value

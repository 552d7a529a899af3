"""Linear layers with an epilogue and their gradients on the GPU against fp64.

Tolerances, with u = 2^-23 (a unit of fp32, which the matrix cores' sums may lose once per addition): a product's sum
over k is off by at most (K / 32 + 40) u of its terms' magnitudes (32 additions in an instruction, one per instruction, up
to 8 for the parts of a split sum).  Activations have slopes of at most 1.13 and add their functions' units:
40 u (|z| + 1) of fp32 (exponentials' arguments are rounded: |z| u each, |z| < 16).  SwiGLU: the product rule's terms.  A BF16
output is within 2^-8 of its value.  dz, two BF16 parts, is within 2^-17 of its fp32 value, whose own
activation's derivative is off by 60 u (1 + |z|) of its factors."""

import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]


def _np(t):
    return t.detach().double().cpu().numpy()


def _mm(a, b):
    """fp64 product of device tensors (dense operands)."""
    return torch.matmul(a.double().contiguous(), b.double().contiguous())


def _inputs(T, K, N, act, seed=0, bias=True, res=None):
    g = torch.Generator(device="cuda").manual_seed(seed + T + K + N)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    R = 2 * N if act == "swiglu" else N
    x = rn(T, K).to(torch.bfloat16)
    w = (rn(R, K) / K ** 0.5).to(torch.bfloat16)
    b = 0.3 * rn(R) if bias else None
    r = None if res is None else rn(T, N).to(torch.bfloat16 if res == "bf16" else torch.float32)
    return x, w, b, r


def _check(x, w, b, r, act, out_dtype, out, pre_dtype=None):
    K = x.shape[1]
    z = _np(_mm(x, w.t()))
    ez = (K / 32 + 40) * U * _np(_mm(x.abs(), w.abs().t()))
    if b is not None:
        z = z + _np(b)
        ez = ez + U * np.abs(z)
    if pre_dtype is not None:
        p = _np(out["pre"])
        assert np.all(np.abs(p - z) <= ez + (2.0 ** -8 * np.abs(z) if pre_dtype == "bf16" else 0)), "pre"
    y = B.activate(z, act)
    if act == "swiglu":
        n = y.shape[1]
        g, up, eg, eu = z[:, :n], z[:, n:], ez[:, :n], ez[:, n:]
        sg = np.abs(B.act(g, "silu"))
        ey = (1.13 * eg + 40 * U * (np.abs(g) + 1)) * (np.abs(up) + eu) + sg * eu
    elif act == "none":
        ey = ez
    else:
        ey = 1.13 * ez + 40 * U * (np.abs(z) + 1)
    if r is not None:
        y = y + _np(r)
    ey = ey + 2 * U * np.abs(y)
    if out_dtype == "bf16":
        ey = ey + 2.0 ** -8 * (np.abs(y) + ey)
    got = _np(out["y"])
    assert np.all(np.isfinite(got)) and got.shape == y.shape
    bad = np.abs(got - y) > ey
    assert not bad.any(), (np.argwhere(bad)[:4], float((np.abs(got - y) / ey).max()))


# one row to many, every tile shape, whole tiles and such that end inside, sums in one piece and in parts
SHAPES = [(1, 8, 8), (1, 64, 64), (2, 72, 40), (3, 7168, 136), (16, 128, 24), (17, 4096, 64), (33, 200, 136), (63, 64, 64),
          (64, 1000, 488), (65, 72, 520), (100, 4096, 256), (128, 136, 128), (129, 512, 264), (255, 264, 1000),
          (257, 2048, 512), (333, 1000, 488), (700, 640, 1032), (2048, 192, 2048), (2100, 1096, 2056), (4096, 136, 4096),
          (4100, 1032, 4104)]


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear(gpu_lib, T, K, N, act):
    from moe_layer_router_amd import layer as L
    x, w, b, r = _inputs(T, K, N, act, res="bf16")
    _check(x, w, b, r, act, "bf16", L.linear(x, w, b, act, r))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("pre", [None, "bf16", "f32"])
def test_linear_epilogues(gpu_lib, act, out, pre):
    from moe_layer_router_amd import layer as L
    for T, K, N in ((5, 320, 72), (70, 2048, 136)):
        for bias in (False, True):
            for res in (None, "bf16", "f32"):
                x, w, b, r = _inputs(T, K, N, act, bias=bias, res=res)
                got = L.linear(x, w, b, act, r, out_dtype=out, pre_dtype=pre)
                assert (got["pre"] is None) == (pre is None)
                _check(x, w, b, r, act, out, got, pre)


@pytest.mark.parametrize("T,K,N", [(1, 7168, 512), (40, 1024, 200), (300, 4096, 712), (4100, 520, 4104)])
def test_whole_numbers_are_exact(gpu_lib, T, K, N):
    """Operands of -2 .. 2: every sum is a whole number below 2^24, whichever way it is split."""
    from moe_layer_router_amd import layer as L
    g = torch.Generator(device="cuda").manual_seed(1)
    ri = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").to(torch.bfloat16)
    x, w, dy = ri(T, K), ri(N, K), ri(T, N)
    y = L.linear(x, w, act="relu", out_dtype="f32")["y"]
    assert bool((y.double() == _mm(x, w.t()).clamp(min=0)).all())
    d = L.linear_backward(x, w, dy, want_dbias=True)
    assert bool((d["dx"].double() == _mm(dy, w)).all()) and bool((d["dw"].double() == _mm(dy.t(), x)).all())
    assert bool((d["dbias"].double() == dy.double().sum(0)).all())
    d2 = L.linear_backward(x, w, dy.float() + 2.0 ** -9, act="none")
    assert float((d2["dx"].double() - _mm(dy.float() + 2.0 ** -9, w)).abs().max()) <= (N / 32 + 40) * U * 4.1 * N


def _check_bwd(x, w, dy, act, pre, dx_dtype, out):
    T, K = x.shape
    R = w.shape[0]
    z = None if pre is None else _np(pre)
    dyn = _np(dy)
    dz = dyn if act == "none" else B.activate_grad(z, dyn, act)
    if act == "none":
        edz = np.zeros_like(dz) if dy.dtype == torch.bfloat16 else 2.0 ** -17 * np.abs(dz)
        esum = np.zeros_like(dz)
    else:
        if act == "swiglu":
            n = dyn.shape[1]
            g, up = z[:, :n], z[:, n:]
            size = np.concatenate([np.abs(dyn * up) * (1 + np.abs(g)), np.abs(dyn) * (1 + np.abs(g))], 1)
        else:
            size = np.abs(dyn) * (1 + np.abs(z))
        esum = 60 * U * size
        edz = esum + 2.0 ** -17 * np.abs(dz)
    t = lambda a: torch.from_numpy(a).cuda()
    D, E = t(dz), t(edz)
    for name, ref, err, terms, n in (
            ("dx", _mm(D, w), _mm(E, w.abs()), _mm(D.abs(), w.abs()), R),
            ("dw", _mm(D.t(), x), _mm(E.t(), x.abs()), _mm(D.abs().t(), x.abs()), T)):
        if out[name] is None:
            continue
        # (two parts: two sums in one)
        bound = err + (2 * (n / 32 + 40)) * U * terms
        if name == "dx" and dx_dtype == "bf16":
            bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        got = out[name].double()
        assert bool(torch.isfinite(got).all())
        worst = float(((got - ref).abs() / bound.clamp(min=1e-300)).max())
        assert worst <= 1, (name, worst)
    if out["dbias"] is not None:
        bound = esum.sum(0) + (T + 8) * U * np.abs(dz).sum(0)
        assert np.all(np.abs(_np(out["dbias"]) - dz.sum(0)) <= bound), "dbias"


def _bwd_inputs(T, K, N, act, dy, pre):
    x, w, _, _ = _inputs(T, K, N, act)
    g = torch.Generator(device="cuda").manual_seed(9)
    dt = lambda n: torch.bfloat16 if n == "bf16" else torch.float32
    d = torch.randn(T, N, generator=g, device="cuda").to(dt(dy))
    p = None if act == "none" else torch.randn(T, w.shape[0], generator=g, device="cuda").to(dt(pre))
    return x, w, d, p


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_backward(gpu_lib, T, K, N, act):
    from moe_layer_router_amd import layer as L
    x, w, dy, pre = _bwd_inputs(T, K, N, act, "bf16", "bf16")
    out = L.linear_backward(x, w, dy, act, pre, want_dbias=True)
    _check_bwd(x, w, dy, act, pre, "f32", out)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("dx", ["bf16", "f32"])
def test_linear_backward_types(gpu_lib, act, dy, dx):
    from moe_layer_router_amd import layer as L
    for T, K, N in ((5, 320, 72), (333, 136, 520)):
        for pre in ("bf16", "f32"):
            for want in ((True, True, True), (True, False, False), (False, True, False), (False, False, True)):
                x, w, d, p = _bwd_inputs(T, K, N, act, dy, pre)
                out = L.linear_backward(x, w, d, act, p, dx_dtype=dx, want_dx=want[0], want_dw=want[1], want_dbias=want[2])
                assert [out[n] is not None for n in ("dx", "dw", "dbias")] == list(want)
                _check_bwd(x, w, d, act, p, dx, out)


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences_of_the_device(gpu_lib, act):
    """Central differences of the device's own fp32 outputs along random directions of x, W and b: steps of 2^-4 in x and W
    keep BF16 operands exact; the differences' third-order term is below h^2 of the directional derivative's scale."""
    from moe_layer_router_amd import layer as L
    T, K, N = 6, 64, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    R = 2 * N if act == "swiglu" else N
    ri = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").float() / 16
    x, w, b = ri(T, K), ri(R, K), ri(R)
    dy = torch.randn(T, N, generator=g, device="cuda")

    def f(x, w, b):
        return float((L.linear(x.to(torch.bfloat16), w.to(torch.bfloat16), b, act, out_dtype="f32")["y"].double() * dy.double()).sum())
    fwd = L.linear(x.to(torch.bfloat16), w.to(torch.bfloat16), b, act, pre_dtype="f32")
    out = L.linear_backward(x.to(torch.bfloat16), w.to(torch.bfloat16), dy, act, fwd["pre"], want_dbias=True)
    h = 2.0 ** -8
    for n, (v, grad) in enumerate((("x", "dx"), ("w", "dw"), ("b", "dbias"))):
        args = dict(x=x, w=w, b=b)
        for k in range(4):
            d = torch.zeros_like(args[v]).flatten()
            d[(37 * k + 11 * n) % d.numel()] = 1
            d = d.view_as(args[v])
            hi, lo = f(**{**args, v: args[v] + h * d}), f(**{**args, v: args[v] - h * d})
            got = float((out[grad].double() * d.double()).sum())
            scale = float(dy.abs().sum()) * 4
            assert abs((hi - lo) / (2 * h) - got) <= (h * h + 2.0 ** -20 / h) * scale + (1e-2 * scale if act == "relu" else 0), (v, k)


def test_rows_behind_and_beside_stay(gpu_lib):
    """Outputs inside larger buffers: nothing before or behind them is touched."""
    from moe_layer_router_amd import layer as L
    for T, K, N, act in ((5, 136, 72, "none"), (130, 1024, 264, "swiglu"), (2100, 200, 2056, "gelu")):
        x, w, b, r = _inputs(T, K, N, act)
        R = w.shape[0]

        def room(rows, cols, dt):
            buf = torch.full(((rows + 64) * cols + 256,), 7.0, dtype=dt, device="cuda")
            return buf, buf[128:128 + rows * cols].view(rows, cols)
        yb, y = room(T, N, torch.bfloat16)
        pb, p = room(T, R, torch.bfloat16)
        L.linear(x, w, b, act, out=dict(y=y, pre=p), pre_dtype="bf16")
        ref = L.linear(x, w, b, act, pre_dtype="bf16")
        assert torch.equal(ref["y"], y) and torch.equal(ref["pre"], p)
        dxb, dx = room(T, K, torch.float32)
        dwb, dw = room(R, K, torch.float32)
        L.linear_backward(x, w, y, act, None if act == "none" else p, out=dict(dx=dx, dw=dw, dbias=None))
        for buf, v in ((yb, y), (pb, p), (dxb, dx), (dwb, dw)):
            assert bool((buf[:128] == 7).all()) and bool((buf[128 + v.numel():] == 7).all())


def test_nan_stays_in_its_row_and_is_not_lost(gpu_lib):
    from moe_layer_router_amd import layer as L
    for act in ACTS:
        x, w, b, r = _inputs(70, 200, 72, act, res="bf16")
        x[33, 199] = float("nan")
        y = L.linear(x, w, b, act, r)["y"]
        assert bool(torch.isnan(y[33]).all()) and bool(torch.isfinite(y[torch.arange(70, device="cuda") != 33]).all())
        x, w, dy, pre = _bwd_inputs(70, 200, 72, act, "f32", "f32")
        dy[12, 5] = float("nan")
        out = L.linear_backward(x, w, dy, act, pre, want_dbias=True)
        assert bool(torch.isnan(out["dx"][12]).all()) and bool(torch.isfinite(out["dx"][torch.arange(70, device="cuda") != 12]).all())
        assert bool(torch.isnan(out["dw"][5]).all()) and bool(torch.isnan(out["dbias"][5]))
        assert bool(torch.isfinite(out["dw"][6:72]).all())


def test_linear_is_deterministic_and_residual_in_place(gpu_lib):
    from moe_layer_router_amd import layer as L
    for T, K, N in ((3, 7168, 264), (300, 4096, 512), (2100, 1096, 2056)):
        x, w, b, r = _inputs(T, K, N, "none", res="bf16")
        a = L.linear(x, w, b, residual=r)["y"]
        for _ in range(3):
            assert torch.equal(a, L.linear(x, w, b, residual=r)["y"])
        dy = torch.randn(T, N, device="cuda")
        g = L.linear_backward(x, w, dy, want_dbias=True)
        for _ in range(3):
            h = L.linear_backward(x, w, dy, want_dbias=True)
            assert all(torch.equal(g[n], h[n]) for n in g)
        L.linear(x, w, b, residual=r, out=dict(y=r, pre=None))
        assert torch.equal(a, r)


def test_linear_views_streams_and_workspaces(gpu_lib):
    """Operands that are no dense matrices, a side stream, one workspace for calls of different sizes, refusals."""
    from moe_layer_router_amd import layer as L
    x, w, b, r = _inputs(50, 136, 72, "gelu", res="f32")
    ref = L.linear(x, w, b, "gelu", r, pre_dtype="f32")
    back = L.linear_backward(x, w, r, "gelu", ref["pre"], want_dbias=True)
    torch.cuda.synchronize()
    xt, wt, rt = x.t().contiguous().t(), w.t().contiguous().t(), torch.cat([r, r], 1)[:, :72]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = L.Workspace("cuda")
    for _ in range(2):
        got = L.linear(xt, wt, b, "gelu", rt, pre_dtype="f32", stream=side, workspace=ws)
        gb = L.linear_backward(xt, wt, rt, "gelu", got["pre"], want_dbias=True, stream=side, workspace=ws)
        L.linear(x[:3], w, act="gelu", stream=side, workspace=ws)
    side.synchronize()
    assert all(torch.equal(ref[n], got[n]) for n in ref) and all(torch.equal(back[n], gb[n]) for n in back)
    for bad in (dict(w=w[:, :128]), dict(w=w.float()), dict(bias=b[:8]), dict(bias=b.bfloat16()), dict(residual=r[:, :64]),
                dict(act="tanh"), dict(out_dtype="fp8"), dict(pre_dtype="fp8"), dict(residual=r.cpu()),
                dict(out=dict(y=ref["y"], pre=ref["pre"])), dict(out=dict(y=ref["y"].float(), pre=None))):
        kw = dict(x=x, w=w, act="gelu")
        kw.update(bad)
        with pytest.raises(ValueError):
            L.linear(**kw)
    for bad in (dict(pre=None), dict(dy=r[:9]), dict(dx_dtype="fp8"), dict(pre=ref["pre"][:, :64]), dict(act="swish")):
        kw = dict(x=x, w=w, dy=r, act="gelu", pre=ref["pre"])
        kw.update(bad)
        with pytest.raises(ValueError):
            L.linear_backward(**kw)
    with pytest.raises(gpu_lib.MoeError):
        L.linear(x[:, :132].contiguous(), w[:, :132].contiguous())
    with pytest.raises(gpu_lib.MoeError):
        L.linear_backward(x, w, r, want_dx=False, want_dw=False)


def test_linear_in_a_graph(gpu_lib):
    """Forward and backward captured with workspaces of their own while eager results of the same tensors live; replayed on
    new inputs with eager work in between."""
    from moe_layer_router_amd import layer as L
    x, w, b, _ = _inputs(300, 1024, 264, "swiglu")
    dy = torch.randn(300, 264, device="cuda")

    def both(ws):
        f = L.linear(x, w, b, "swiglu", pre_dtype="bf16", workspace=ws and ws[0])
        g = L.linear_backward(x, w, dy, "swiglu", f["pre"], want_dbias=True, workspace=ws and ws[1])
        return [f["y"], f["pre"], g["dx"], g["dw"], g["dbias"]]
    eager = both(None)
    ws = [L.Workspace("cuda"), L.Workspace("cuda")]
    ws[0].get(gpu_lib.moe_linear_workspace_size(300, 1024, 264, "swiglu"))
    ws[1].get(gpu_lib.moe_linear_backward_workspace_size(300, 1024, 264, "swiglu"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = both(ws)
    for i in range(4):
        if i:
            x.copy_(torch.randn(300, 1024, device="cuda"))
            dy.normal_()
            eager = both(None)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(eager, cap)), i


def test_offsets_past_32_bits(gpu_lib):
    """x, dz and y past 2^32 bytes: the last rows are right."""
    from moe_layer_router_amd import layer as L
    torch.manual_seed(2)
    T, K, N = 300_000, 8200, 8
    x = torch.zeros(T, K, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(N, K, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([0, 1, 131072, 261888, 262144, T - 1], device="cuda")
    x[rows] = torch.randn(len(rows), K, device="cuda").to(torch.bfloat16)
    y = L.linear(x, w, out_dtype="f32")["y"]
    ref = _mm(x[rows], w.t())
    assert float((y[rows].double() - ref).abs().max()) <= (K / 32 + 40) * U * float(_mm(x[rows].abs(), w.abs().t()).max())
    y[rows] = 0
    assert float(y.abs().max()) == 0
    dy = torch.zeros(T, N, device="cuda")
    dy[rows] = torch.randn(len(rows), N, device="cuda")
    d = L.linear_backward(x, w, dy, dx_dtype="bf16")
    ref = _mm(dy[rows].t(), x[rows])
    assert float((d["dw"].double() - ref).abs().max()) <= 2.0 ** -15 * float(_mm(dy[rows].abs().t(), x[rows].abs()).max())
    ref = _mm(dy[rows], w)
    assert float((d["dx"][rows].double() - ref).abs().max()) <= 2.0 ** -7 * float(ref.abs().max())
    del d, x, y
    # the other way round: dz and W wide, dx and y narrow
    T, K, N = 20_000, 8, 131_072
    x = torch.randn(T, K, device="cuda").to(torch.bfloat16)
    w = torch.randn(N, K, device="cuda").to(torch.bfloat16)
    y = L.linear(x, w)["y"]
    ref = _mm(x[-3:], w.t())
    assert float((y[-3:].double() - ref).abs().max()) <= 2.0 ** -7 * float(ref.abs().max())
    dy = torch.zeros(T, N, device="cuda")
    dy[-3:] = torch.randn(3, N, device="cuda")
    d = L.linear_backward(x, w, dy)
    ref = _mm(dy[-3:], w)
    assert float((d["dx"][-3:].double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max()) and float(d["dx"][:-3].abs().max()) == 0
    ref = _mm(dy[-3:].t(), x[-3:])
    assert float((d["dw"].double() - ref).abs().max()) <= 2.0 ** -14 * float(ref.abs().max())


@pytest.mark.parametrize("T,K,N", [s for s in SHAPES if s[0] >= 33] + [(2048, 2048, 7168), (300, 7168, 2048)])
@pytest.mark.parametrize("dx,want_dw", [("bf16", False), ("bf16", True), ("f32", True)])
def test_linear_backward_in_parts_with_every_tile(gpu_lib, T, K, N, dx, want_dw):
    """dz in two parts, in two of three, in three."""
    from moe_layer_router_amd import layer as L
    x, w, d, p = _bwd_inputs(T, K, N, "silu", "f32", "bf16")
    out = L.linear_backward(x, w, d, "silu", p, dx_dtype=dx, want_dw=want_dw, want_dbias=True)
    _check_bwd(x, w, d, "silu", p, dx, out)


@pytest.mark.parametrize("T", [3, 70, 700])
def test_infinities_and_the_largest_numbers(gpu_lib, T):
    """An infinity in x, W or dy gives infinities (of its products' signs) where it enters, in whichever part, and nothing beside; dy
    above the largest BF16 number is no infinity."""
    from moe_layer_router_amd import layer as L
    K, N = 200, 72
    x, w, _, _ = _inputs(T, K, N, "none")
    x, w = torch.where(x == 0, 1.0, x).to(torch.bfloat16), torch.where(w == 0, 1.0, w).to(torch.bfloat16)
    inf = float("inf")
    rest = torch.arange(T, device="cuda") != 2
    xi = x.clone()
    xi[2, 5] = inf
    y = L.linear(xi, w)["y"]
    assert torch.equal(y[2].float(), inf * torch.sign(w[:, 5].float())) and bool(torch.isfinite(y[rest]).all())
    wi = w.clone()
    wi[7, 5] = -inf
    y = L.linear(x, wi)["y"]
    assert torch.equal(y[:, 7].float(), -inf * torch.sign(x[:, 5].float())) and bool(torch.isfinite(y[:, 8:]).all())
    dy = torch.randn(T, N, device="cuda")
    dy[2, 4] = -inf
    d = L.linear_backward(x, w, dy, want_dbias=True)
    assert torch.equal(d["dx"][2], -inf * torch.sign(w[4].float())) and bool(torch.isfinite(d["dx"][rest]).all())
    assert torch.equal(d["dw"][4], -inf * torch.sign(x[2].float())) and bool(torch.isfinite(d["dw"][5:]).all())
    assert float(d["dbias"][4]) == -inf and bool(torch.isfinite(d["dbias"][5:]).all())
    dy = torch.zeros(T, N, device="cuda")
    dy[2, 4] = 3.4e38
    ws, xs = (w.float() * 2.0 ** -12).to(torch.bfloat16), (x.float() * 2.0 ** -12).to(torch.bfloat16)
    d = L.linear_backward(xs, ws, dy)
    # (one product each: three exact terms, added in fp32)
    for got, of in ((d["dx"][2], ws[4]), (d["dw"][4], xs[2])):
        ref = of.double() * float(dy[2, 4])
        assert bool(((got.double() - ref).abs() <= 4 * U * ref.abs()).all())


def test_two_calls_at_once(gpu_lib):
    """Two streams, each with a workspace of its own, tiles in parts in both."""
    from moe_layer_router_amd import layer as L
    sets = [_bwd_inputs(300, 2048, 512, "silu", "f32", "bf16"), _bwd_inputs(130, 4096, 264, "silu", "f32", "bf16")]
    ref = [(L.linear(x, w), L.linear_backward(x, w, d, "silu", p, want_dbias=True)) for x, w, d, p in sets]
    torch.cuda.synchronize()
    streams, spaces, got = [torch.cuda.Stream(), torch.cuda.Stream()], [L.Workspace("cuda"), L.Workspace("cuda")], []
    for _ in range(4):
        for s, ws, (x, w, d, p) in zip(streams, spaces, sets):
            got.append((L.linear(x, w, stream=s, workspace=ws),
                        L.linear_backward(x, w, d, "silu", p, want_dbias=True, stream=s, workspace=ws)))
    for s in streams:
        s.synchronize()
    for i, (f, g) in enumerate(got):
        assert torch.equal(f["y"], ref[i % 2][0]["y"]) and all(torch.equal(g[n], ref[i % 2][1][n]) for n in g)

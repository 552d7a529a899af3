"""Layer norm and its backward pass on the GPU against the fp64 definition.

Tolerances, with u = 2^-24 (a fp32 rounding): a sum over a row goes through
at most 32 additions in a thread, 6 across a wave and 16 across the waves, so
its error is below 54 u of the sum of magnitudes; with the few roundings of
the element itself C = 128 covers each element:
  y   |err| <= C u (|z gamma| + |beta| + |gamma| (1 + mean|x| rstd))
      (the last term: the mean's error, 54 u mean|x|, scaled to z)
  dx  |err| <= C u rstd (|g| + mean|g| + |z| mean|g z|)
  dgamma, dbeta: (T + 64) u of the sum of magnitudes, any order of sums.
BF16 outputs add half a step, 2^-8 |y|; E4M3 outputs 2^-4 |y| (2^-10 of the
scale where they are subnormal)."""

import numpy as np
import pytest
import torch

from oracle import training as R

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -24, 128
# one token to several rows per workgroup, every row layout, chunk counts that leave lanes idle
SHAPES = [(1, 128), (3, 384), (5, 512), (17, 640), (9, 1024), (33, 1152), (4, 2048), (70, 2176), (3, 4096),
          (30, 4224), (2, 7168), (3, 8192), (2, 8320), (3, 16384), (9001, 256), (2500, 1664), (2100, 4096)]


def _rows(T, H, dtype, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g)
    if kind == "offset":
        x = 100 + x                       # a mean far above the spread
    return x.to(dtype).cuda()


def _vec(H, seed, base):
    return (base + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).cuda()


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _check(got, ref, bound, what):
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), what
    worst = np.max(err / bound)
    assert worst <= 1, f"{what}: error {worst:.2f} of its bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"


def _y_bound(x, gamma, beta, rstd, y):
    b = 0 if beta is None else np.abs(beta)
    spread = np.abs(x).mean(1, keepdims=True) * rstd[:, None]
    return C * U * (np.abs(y) + b + np.abs(gamma) * (1 + spread)) + 1e-30


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(gpu_lib, T, H, dtype):
    from moe_layer_router_amd import layer as L
    x, gamma, beta = _rows(T, H, dtype, T + H), _vec(H, 1, 1.0), _vec(H, 2, 0.0)
    r32 = L.layer_norm(x, gamma, beta, out_dtype="f32", want_stats=True)
    r16 = L.layer_norm(x, gamma, beta, out_dtype="bf16")
    r8 = L.layer_norm(x, gamma, beta, out_dtype="fp8")
    torch.cuda.synchronize()
    y, mean, rstd = R.layer_norm(_np(x), _np(gamma), _np(beta), 1e-5)
    bound = _y_bound(_np(x), _np(gamma), _np(beta), rstd, y)
    _check(_np(r32["y"]), y, bound, "y")
    _check(_np(r32["mean"]), mean, C * U * np.abs(_np(x)).mean(1) + 1e-30, "mean")
    _check(_np(r32["rstd"]), rstd, C * U * rstd * (1 + (np.abs(mean) * rstd) ** 2), "rstd")
    _check(_np(r16["y"]), y, bound * 1.01 + 2.0 ** -8 * np.abs(y), "bf16 y")
    s = _np(r8["y_scales"])
    amax = np.abs(y).reshape(T, H // 128, 128).max(2)
    bb = bound.reshape(T, H // 128, 128).max(2)
    _check(s, amax / 448, (bb + 2 * U * amax) / 448, "scales")
    v = _np(r8["y"].view(torch.float8_e4m3fn)).reshape(T, -1, 128) * s[:, :, None]
    v = v.reshape(T, H)
    se = np.repeat(s, 128, 1)
    _check(v, y, 1.1 * bound + np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * se) * (1 + 2.0 ** -10), "fp8 y")
    # the codes are those of the layer's own quantiser on the fp32 output
    q, qs = L.quantize_input(r32["y"])
    torch.cuda.synchronize()
    assert torch.equal(q, r8["y"]) and torch.equal(qs, r8["y_scales"])


def test_forward_power_of_two_scales_and_no_beta(gpu_lib):
    from moe_layer_router_amd import layer as L
    x, gamma = _rows(37, 768, torch.bfloat16, 5), _vec(768, 3, 1.0)
    r = L.layer_norm(x, gamma, out_dtype="fp8", scale_mode="pow2")
    y32 = L.layer_norm(x, gamma, out_dtype="f32")["y"]
    q, s = L.quantize_input(y32, "pow2")
    torch.cuda.synchronize()
    assert torch.equal(r["y"], q) and torch.equal(r["y_scales"], s)
    y, _, rstd = R.layer_norm(_np(x), _np(gamma), None, 1e-5)
    _check(_np(y32), y, _y_bound(_np(x), _np(gamma), None, rstd, y), "y")


@pytest.mark.parametrize("T,H", [(5, 512), (6, 7168)])
def test_rows_with_a_large_mean_and_constant_rows(gpu_lib, T, H):
    from moe_layer_router_amd import layer as L
    x, gamma = _rows(T, H, torch.float32, 7, "offset"), _vec(H, 3, 1.0)
    x[1] = 3.25                            # no spread: z = 0
    x[2] = 0
    r = L.layer_norm(x, gamma, out_dtype="f32", want_stats=True)
    torch.cuda.synchronize()
    y, _, rstd = R.layer_norm(_np(x), _np(gamma), None, 1e-5)
    _check(_np(r["y"]), y, _y_bound(_np(x), _np(gamma), None, rstd, y), "y")
    assert torch.all(r["y"][2] == 0)


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dyd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(gpu_lib, T, H, xd, dyd):
    from moe_layer_router_amd import layer as L
    x, gamma, dy = _rows(T, H, xd, T + H), _vec(H, 1, 1.0), _rows(T, H, dyd, 3 * T + H)
    st = L.layer_norm(x, gamma, want_stats=True)
    r = L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy)
    torch.cuda.synchronize()
    xn, gn, dn, mean, rstd = _np(x), _np(gamma), _np(dy), _np(st["mean"]), _np(st["rstd"])
    dx, dgamma, dbeta = R.layer_norm_backward(xn, gn, mean, rstd, dn)
    z, g = (xn - mean[:, None]) * rstd[:, None], dn * gn
    bound = C * U * rstd[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True) +
                                     np.abs(z) * np.abs(g * z).mean(1, keepdims=True))
    _check(_np(r["dx"]), dx, bound, "dx")
    _check(_np(r["dgamma"]), dgamma, (T + 64) * U * np.abs(dn * z).sum(0) + 1e-30, "dgamma")
    _check(_np(r["dbeta"]), dbeta, (T + 64) * U * np.abs(dn).sum(0) + 1e-30, "dbeta")


def test_backward_in_place_without_weights_and_deterministic(gpu_lib):
    from moe_layer_router_amd import layer as L
    for T, H in ((600, 384), (530, 7168)):
        x, gamma, dy = _rows(T, H, torch.bfloat16, 1), _vec(H, 1, 1.0), _rows(T, H, torch.float32, 2)
        st = L.layer_norm(x, gamma, want_stats=True)
        a = L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy)
        b = L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy)
        c = L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy, want_weights=False)
        torch.cuda.synchronize()
        assert c["dgamma"] is None and c["dbeta"] is None and torch.equal(a["dx"], c["dx"])
        for k in a:
            assert torch.equal(a[k], b[k]), k
        out = dict(dx=dy, dgamma=torch.empty_like(gamma), dbeta=torch.empty_like(gamma))
        L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy, out=out)
        torch.cuda.synchronize()
        assert torch.equal(dy, a["dx"]) and torch.equal(out["dgamma"], a["dgamma"])


def test_only_one_weight_gradient_through_the_c_entry(gpu_lib):
    from moe_layer_router_amd import layer as L, lib
    T, H = 40, 256
    x, gamma, dy = _rows(T, H, torch.float32, 1), _vec(H, 1, 1.0), _rows(T, H, torch.float32, 2)
    st = L.layer_norm(x, gamma, want_stats=True)
    a = L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy)
    dx, db = torch.empty(T, H, device="cuda"), torch.empty(H, device="cuda")
    ws = torch.empty(lib.moe_layer_norm_backward_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    lib.moe_layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy, dx, None, db, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, a["dx"]) and torch.equal(db, a["dbeta"])


def test_strided_and_misaligned_inputs(gpu_lib):
    """Views that are not contiguous, or start off a 16-byte boundary, give
    what their copies give."""
    from moe_layer_router_amd import layer as L
    T, H = 11, 256
    big = _rows(T, 2 * H, torch.bfloat16, 4)
    x = big[:, ::2]
    flat = torch.randn(H + 1, device="cuda")
    gamma = flat[1:]
    assert gamma.data_ptr() % 16 != 0
    r = L.layer_norm(x, gamma, want_stats=True)
    s = L.layer_norm(x.clone().contiguous(), gamma.clone(), want_stats=True)
    dy = _rows(H, T, torch.float32, 5).t()
    a = L.layer_norm_backward(x, gamma, r["mean"], r["rstd"], dy)
    b = L.layer_norm_backward(x.contiguous(), gamma.clone(), r["mean"], r["rstd"], dy.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(r["y"], s["y"])
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_rows_behind_the_batch_are_left_alone(gpu_lib):
    from moe_layer_router_amd import lib
    T, H = 7, 384
    x, gamma = _rows(T, H, torch.bfloat16, 4), _vec(H, 1, 1.0)
    y = torch.full((T + 3, H), 7.0, dtype=torch.bfloat16, device="cuda")
    mean = torch.full((T + 3,), 7.0, device="cuda")
    rstd = mean.clone()
    lib.moe_layer_norm(x, gamma, None, 1e-5, y[:T], None, mean[:T], rstd[:T])
    torch.cuda.synchronize()
    assert torch.all(y[T:] == 7) and torch.all(mean[T:] == 7) and torch.all(rstd[T:] == 7)


def test_side_stream_and_captured_graph(gpu_lib):
    from moe_layer_router_amd import layer as L
    T, H = 260, 1152
    x, gamma, dy = _rows(T, H, torch.bfloat16, 8), _vec(H, 1, 1.0), _rows(T, H, torch.float32, 9)
    st = L.layer_norm(x, gamma, want_stats=True)
    ref = L.layer_norm_backward(x, gamma, st["mean"], st["rstd"], dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        r = L.layer_norm(x, gamma, want_stats=True, stream=s)
        b = L.layer_norm_backward(x, gamma, r["mean"], r["rstd"], dy, stream=s)
        side.synchronize()
        assert torch.equal(r["y"], st["y"]) and all(torch.equal(b[k], ref[k]) for k in b)
    graph = torch.cuda.CUDAGraph()
    xs, dys = x.clone(), dy.clone()
    ws = L.Workspace("cuda")
    ws.get(1 << 24)
    with torch.cuda.graph(graph):
        r = L.layer_norm(xs, gamma, want_stats=True)
        b = L.layer_norm_backward(xs, gamma, r["mean"], r["rstd"], dys, workspace=ws)
    for i in range(4):
        xi, di = _rows(T, H, torch.bfloat16, 20 + i), _rows(T, H, torch.float32, 30 + i)
        xs.copy_(xi)
        dys.copy_(di)
        graph.replay()
        e = L.layer_norm(xi, gamma, want_stats=True)
        f = L.layer_norm_backward(xi, gamma, e["mean"], e["rstd"], di)
        torch.cuda.synchronize()
        assert torch.equal(r["y"], e["y"]) and all(torch.equal(b[k], f[k]) for k in b)


def test_wrapper_refusals(gpu_lib):
    from moe_layer_router_amd import layer as L, lib
    x, g = torch.zeros(4, 256, device="cuda"), torch.ones(256, device="cuda")
    bad = [dict(x=x.half()), dict(gamma=g[:128]), dict(gamma=g.double()), dict(gamma=g.cpu()), dict(out_dtype="fp4"),
           dict(scale_mode="no"), dict(beta=g[None])]
    for b in bad:
        with pytest.raises(ValueError):
            L.layer_norm(**{**dict(x=x, gamma=g), **b})
    with pytest.raises(lib.MoeError):
        L.layer_norm(torch.zeros(4, 200, device="cuda"), torch.ones(200, device="cuda"))
    with pytest.raises(lib.MoeError):
        L.layer_norm(torch.zeros(0, 256, device="cuda"), g)
    r = L.layer_norm(x, g)
    with pytest.raises(ValueError):
        L.layer_norm(x, g, out_dtype="f32", out=r)
    with pytest.raises(ValueError):
        L.layer_norm(x, g, want_stats=True, out=r)
    with pytest.raises(ValueError):
        L.layer_norm_backward(x, g, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"), x)


def test_offsets_past_32_bits(gpu_lib):
    """More than 2^31 elements: the rows at both ends, forward and backward."""
    from moe_layer_router_amd import layer as L
    T, H = 300_000, 7680
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    gamma = _vec(H, 1, 1.0)
    r = L.layer_norm(x, gamma, out_dtype="bf16", want_stats=True)
    b = L.layer_norm_backward(x, gamma, r["mean"], r["rstd"], x)
    torch.cuda.synchronize()
    some = [0, 1, 123_456, T - 2, T - 1]
    xn = _np(x[some])
    y, mean, rstd = R.layer_norm(xn, _np(gamma), None, 1e-5)
    _check(_np(r["y"][some]), y, 1.01 * _y_bound(xn, _np(gamma), None, rstd, y) + 2.0 ** -8 * np.abs(y), "y")
    m, s = _np(r["mean"][some]), _np(r["rstd"][some])
    dx, _, _ = R.layer_norm_backward(xn, _np(gamma), m, s, xn)
    z, g = (xn - m[:, None]) * s[:, None], xn * _np(gamma)
    bound = C * U * s[:, None] * (np.abs(g) + np.abs(g).mean(1, keepdims=True) +
                                  np.abs(z) * np.abs(g * z).mean(1, keepdims=True))
    _check(_np(b["dx"][some]), dx, bound, "dx")
    ref, mag = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, T, 50_000):
        c = x[i:i + 50_000].double()
        ref += c.sum(0)
        mag += c.abs().sum(0)
    # a workgroup sums its T / 256 rows, then the workgroups' sums are joined
    assert bool(((b["dbeta"].double() - ref).abs() <= (T / 256 + 64) * U * mag).all())


def test_default_stream_by_handle(gpu_lib):
    from moe_layer_router_amd import layer as L
    x, gamma = _rows(9, 256, torch.bfloat16, 1), _vec(256, 1, 1.0)
    a, b = L.layer_norm(x, gamma), L.layer_norm(x, gamma, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(a["y"], b["y"])

"""Refusals of the operators beside the routed experts on the host (no GPU):
every argument check of the C entry points, and those of the Python wrappers,
before any device call."""

import ctypes

import pytest
import torch

from moe_layer_router_amd import layer as L, lib

A = 0x100000                       # a fake, 16-byte-aligned address: the checks never dereference
INVALID, UNSUPPORTED, SMALL = lib.MOE_ERR_INVALID_ARGUMENT, lib.MOE_ERR_UNSUPPORTED, lib.MOE_ERR_WORKSPACE_TOO_SMALL


def _sel(over):
    s = dict(T=10, E=64, k=4, scoring=1, groups=8, keep=2, top=2, renorm=1, scale=1.0)
    for n in s:
        s[n] = over.pop(n, s[n])
    return lib.MoeSelection(*s.values())


def _select(**over):
    s = _sel(over)
    a = dict(logits=A, bias=2 * A, ids=3 * A, w=4 * A)
    a.update(over)
    return lib._lib.moe_select_experts(ctypes.byref(s), *a.values(), None)


BAD_SELECTIONS = [
    (dict(T=0), INVALID), (dict(T=-4), INVALID), (dict(E=0), INVALID), (dict(E=1040, groups=1, keep=1), UNSUPPORTED),
    (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(k=17, keep=8), UNSUPPORTED), (dict(scoring=2), INVALID),
    (dict(scoring=-1), INVALID), (dict(groups=0), INVALID), (dict(groups=7), INVALID), (dict(groups=-8), INVALID),
    (dict(E=1024, groups=128), UNSUPPORTED), (dict(keep=0), INVALID), (dict(keep=9), INVALID), (dict(top=0), INVALID),
    (dict(top=3), INVALID), (dict(groups=64, keep=4), INVALID),       # groups of one expert have no second
    (dict(groups=32, keep=1), INVALID),                               # four experts asked of two
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
]


@pytest.mark.parametrize("over,status", BAD_SELECTIONS + [
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(bias=A + 4), INVALID),
    (dict(logits=A + 8), INVALID), (dict(ids=A), INVALID), (dict(w=A + 10 * 64 * 4 - 16), INVALID), (dict(ids=4 * A), INVALID),
    (dict(w=2 * A), INVALID), (dict(ids=2 * A + 64), INVALID),
])
def test_select_refusals(over, status):
    assert _select(**over) == status
    assert lib.moe_last_error() != ""


def test_select_null_selection():
    assert lib._lib.moe_select_experts(None, A, None, 2 * A, 3 * A, None) == INVALID
    assert lib._lib.moe_select_experts_backward(None, A, 2 * A, 3 * A, 4 * A, None) == INVALID


def _select_bwd(**over):
    s = _sel(over)
    a = dict(logits=A, ids=2 * A, dw=3 * A, dl=4 * A)
    a.update(over)
    return lib._lib.moe_select_experts_backward(ctypes.byref(s), *a.values(), None)


@pytest.mark.parametrize("over,status", BAD_SELECTIONS + [
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(dw=None), INVALID), (dict(dl=None), INVALID),
    (dict(dl=4 * A + 4), INVALID), (dict(dl=A), INVALID), (dict(dl=2 * A + 16), INVALID), (dict(dl=3 * A), INVALID),
])
def test_select_backward_refusals(over, status):
    assert _select_bwd(**over) == status
    assert lib.moe_last_error() != ""


@pytest.mark.parametrize("over,status", [
    (dict(logits=None), INVALID), (dict(sel=dict(T=11)), INVALID), (dict(sel=dict(E=32, groups=4)), INVALID),
    (dict(sel=dict(k=2)), INVALID), (dict(sel=dict(scoring=5)), INVALID), (dict(ids=None), INVALID),
    (dict(nbytes=16), SMALL),
])
def test_backward_selected_refusals(over, status):
    over = dict(over)
    s = _sel(over.pop("sel", {}))
    d = lib.make_desc(10, 256, 64, 128, 4, "bf16", "bf16", layout="row_major")
    a = dict(x=A, wr=A, wgu=A, wd=A, logits=A, ids=A, w=A, dy=A, dlogits=None, dx=A, dwgu=A, dwd=A, dwr=A, db=A, ws=A,
             nbytes=1 << 40)
    a.update(over)
    assert lib._lib.moe_backward_selected(ctypes.byref(d), ctypes.byref(s), *a.values(), None) == status
    assert lib._lib.moe_backward_selected(ctypes.byref(d), None, *a.values(), None) == INVALID


def test_select_wrappers_refuse():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="on a GPU"):
        L.select_experts(x, 2)
    with pytest.raises(ValueError, match="on a GPU"):
        L.select_experts_backward(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="exclude"):
        L.forward({"weights_packed": True}, 2, routing=(x, x), selection={})


BF, F32, FP8, FP4 = lib.MOE_DTYPE_BF16, lib.MOE_DTYPE_F32, lib.MOE_DTYPE_FP8_E4M3, lib.MOE_DTYPE_FP4_E2M1


def _adamw(tensors=({},), n_tensors=None, f8=False, table=True, options=True, **over):
    o = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, grad_scale=None, lr_dev=None, step_dev=None,
             state_dtype=FP8 if f8 else F32, seed=0)
    o.update(over)
    ts = (lib.MoeAdamwTensor * max(1, len(tensors)))()
    for i, t in enumerate(tensors):
        b = A * 16 * (i + 1)
        d = dict(param=b, grad=b + A, m=b + 2 * A, v=b + 3 * A, m_scales=b + 4 * A if f8 else None,
                 v_scales=b + 5 * A if f8 else None, master=None, n=1000, param_dtype=F32, grad_dtype=F32,
                 weight_decay=0.0, reserved=0)
        d.update(t)
        ts[i] = lib.MoeAdamwTensor(*d.values())
    opts = lib.MoeAdamwOptions(*o.values())
    return lib._lib.moe_adamw(len(tensors) if n_tensors is None else n_tensors, ts if table else None,
                              ctypes.byref(opts) if options else None, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("over,status", [
    (dict(n_tensors=-1), INVALID), (dict(n_tensors=(1 << 24) + 1), UNSUPPORTED), (dict(table=False), INVALID),
    (dict(options=False), INVALID), (dict(beta1=1.0), INVALID), (dict(beta1=-0.1), INVALID), (dict(beta2=1.0), INVALID),
    (dict(beta2=NAN), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=INF), INVALID), (dict(lr=NAN), INVALID), (dict(lr=INF), INVALID), (dict(step=0), INVALID),
    (dict(step=-3), INVALID), (dict(state_dtype=BF), UNSUPPORTED), (dict(state_dtype=9), UNSUPPORTED),
    (dict(grad_scale=A + 2), INVALID), (dict(lr_dev=A + 1), INVALID), (dict(step_dev=A + 4), INVALID),
    (dict(tensors=[dict(n=-1)]), INVALID), (dict(tensors=[dict(n=(1 << 40) + 1)]), UNSUPPORTED),
    (dict(tensors=[dict(param_dtype=FP8)]), UNSUPPORTED), (dict(tensors=[dict(grad_dtype=FP4)]), UNSUPPORTED),
    (dict(tensors=[dict(weight_decay=INF)]), INVALID), (dict(tensors=[dict(master=A)]), INVALID),
    (dict(tensors=[dict(m_scales=A)]), INVALID), (dict(tensors=[dict(m_scales=None)], f8=True), INVALID),
    (dict(tensors=[dict(v_scales=None)], f8=True), INVALID), (dict(tensors=[dict(v_scales=A + 2)], f8=True), INVALID), (dict(tensors=[dict(param=None)]), INVALID),
    (dict(tensors=[dict(grad=None)]), INVALID), (dict(tensors=[dict(m=None)]), INVALID),
    (dict(tensors=[dict(v=None)]), INVALID), (dict(tensors=[dict(param=A + 4)]), INVALID),
    (dict(tensors=[dict(grad=A + 8)]), INVALID), (dict(tensors=[dict(param_dtype=BF, master=A + 4)]), INVALID),
    (dict(tensors=[{}, dict(param=A * 16)]), INVALID),                     # one tensor twice
    (dict(tensors=[{}, dict(grad=A * 16 + 16)]), INVALID),                 # a gradient that is another's weights
    (dict(tensors=[dict(m=A * 18, v=A * 18 + 3984)]), INVALID),            # the last bytes of m
    (dict(tensors=[dict(grad=A * 16)]), INVALID), (dict(tensors=[dict(m_scales=A * 16 + 16)], f8=True), INVALID),
])
def test_adamw_refusals(over, status):
    assert _adamw(**over) == status
    assert lib.moe_last_error() != ""


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: the call must end at the missing device")
def test_adamw_shared_gradients_are_no_overlap():
    """Past its checks of the arguments a call without a GPU fails at the device."""
    for ts in ([dict(grad=A), dict(grad=A)], [dict(n=0, param=None, grad=None, m=None, v=None)],
               [dict(m=A * 18, v=A * 18 + 4000)]):
        assert _adamw(ts) not in (INVALID, lib.MOE_ERR_WORKSPACE_TOO_SMALL)


def test_adamw_wrapper_refuses():
    with pytest.raises(ValueError, match="not be empty"):
        L.AdamW([])
    with pytest.raises(ValueError, match="on a GPU"):
        L.AdamW([torch.zeros(4)])


def _linear(**over):
    a = dict(T=10, K=64, N=24, act=0, x=A, w=2 * A, bias=3 * A, res=4 * A, rd=BF, y=5 * A, yd=BF, pre=6 * A, pd=BF,
             ws=16 * A, nbytes=1 << 20)
    a.update(over)
    return lib._lib.moe_linear(*a.values(), None)


SHAPES = [(dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(K=60), INVALID), (dict(N=0), INVALID),
          (dict(N=20), INVALID), (dict(K=-8), INVALID), (dict(act=6), INVALID), (dict(act=-1), INVALID),
          (dict(K=131080), UNSUPPORTED), (dict(N=131080), UNSUPPORTED), (dict(N=65544, act=5), UNSUPPORTED)]


@pytest.mark.parametrize("over,status", SHAPES + [
    (dict(yd=FP8), UNSUPPORTED), (dict(rd=FP8), UNSUPPORTED), (dict(pd=FP4), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(x=A + 2), INVALID),
    (dict(bias=A + 4), INVALID), (dict(res=A + 8), INVALID), (dict(pre=A + 1), INVALID), (dict(nbytes=0), SMALL),
    (dict(y=A), INVALID), (dict(y=2 * A + 24 * 64 * 2 - 16), INVALID), (dict(y=3 * A), INVALID), (dict(y=4 * A + 16), INVALID),
    (dict(y=4 * A, yd=F32), INVALID), (dict(pre=4 * A), INVALID), (dict(pre=5 * A), INVALID), (dict(ws=A - 128), INVALID),
    (dict(ws=5 * A), INVALID), (dict(pre=16 * A), INVALID),
])
def test_linear_refusals(over, status):
    assert _linear(**over) == status
    assert lib.moe_last_error() != ""


def _linear_bwd(**over):
    a = dict(T=10, K=64, N=24, act=2, x=A, w=2 * A, pre=3 * A, pd=BF, dy=4 * A, dyd=BF, dx=5 * A, dxd=BF, dw=6 * A,
             db=7 * A, ws=16 * A, nbytes=1 << 24)
    a.update(over)
    return lib._lib.moe_linear_backward(*a.values(), None)


@pytest.mark.parametrize("over,status", SHAPES + [
    (dict(dyd=FP8), UNSUPPORTED), (dict(dxd=FP8), UNSUPPORTED), (dict(pd=FP4), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(w=None), INVALID), (dict(pre=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None, dw=None, db=None), INVALID),
    (dict(dx=A + 2), INVALID), (dict(dw=A + 4), INVALID), (dict(db=A + 8), INVALID), (dict(nbytes=64), SMALL),
    (dict(dx=A), INVALID), (dict(dx=4 * A), INVALID), (dict(dw=2 * A), INVALID), (dict(dw=5 * A), INVALID),
    (dict(db=3 * A), INVALID), (dict(db=6 * A + 64), INVALID), (dict(ws=4 * A), INVALID), (dict(ws=7 * A), INVALID),
])
def test_linear_backward_refusals(over, status):
    assert _linear_bwd(**over) == status
    assert lib.moe_last_error() != ""


def test_linear_workspace_sizes():
    for f in (lib.moe_linear_workspace_size, lib.moe_linear_backward_workspace_size):
        assert f(0, 64, 64, "none") == 0 and f(1, 60, 64, "none") == 0 and f(1, 64, 65544, "swiglu") == 0
        assert 0 < f(1, 8, 8, "none") < 1 << 16
    assert lib.moe_linear_workspace_size(8192, 7168, 2048, "swiglu") <= 128 << 20
    T, K, N = 8192, 7168, 2048
    assert lib.moe_linear_backward_workspace_size(T, K, N, "swiglu") <= 6 * T * 2 * N + 256 * 2 * N * 4 + (128 << 20) + 1024


def test_linear_wrappers_refuse():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on a GPU"):
        L.linear(x, x)
    with pytest.raises(ValueError, match="on a GPU"):
        L.linear_backward(x, x, x)

"""Refusals of the training operators on the host (no GPU): every argument
check of the C entry points, and those of the Python wrappers, before any
device call."""

import ctypes

import pytest
import torch

from moe_layer_router_amd import layer as L, lib

A = 0x100000                       # a fake, 16-byte-aligned address: the checks never dereference
BF, F32, FP8, FP4 = lib.MOE_DTYPE_BF16, lib.MOE_DTYPE_F32, lib.MOE_DTYPE_FP8_E4M3, lib.MOE_DTYPE_FP4_E2M1
INVALID, UNSUPPORTED, SMALL = lib.MOE_ERR_INVALID_ARGUMENT, lib.MOE_ERR_UNSUPPORTED, lib.MOE_ERR_WORKSPACE_TOO_SMALL


def _norm(**over):
    a = dict(T=4, H=256, i=BF, o=BF, mode=0, x=A, gamma=A, beta=A, eps=1e-5, y=2 * A, ys=None, mean=A, rstd=A)
    a.update(over)
    return lib._lib.moe_layer_norm(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=0), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=200), INVALID),
    (dict(H=16512), UNSUPPORTED), (dict(i=FP8), UNSUPPORTED), (dict(o=FP4), UNSUPPORTED), (dict(o=9), UNSUPPORTED),
    (dict(o=FP8, ys=A, mode=7), INVALID), (dict(o=FP8), INVALID), (dict(ys=A), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=None), INVALID), (dict(gamma=None), INVALID), (dict(y=None), INVALID),
    (dict(beta=A + 4), INVALID), (dict(x=A + 2), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(y=A), INVALID), (dict(y=A + 4 * 256 * 2 - 16), INVALID), (dict(y=A - 16), INVALID),
])
def test_layer_norm_refusals(over, status):
    assert _norm(**over) == status
    assert lib.moe_last_error() != ""


def _norm_bwd(**over):
    a = dict(T=4, H=256, i=BF, o=F32, x=A, gamma=A, mean=A, rstd=A, dy=A, dx=2 * A, dgamma=A, dbeta=A, ws=A,
             nbytes=lib.moe_layer_norm_backward_workspace_size(4, 256))
    a.update(over)
    return lib._lib.moe_layer_norm_backward(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=0), INVALID), (dict(H=130), INVALID), (dict(H=32768), UNSUPPORTED), (dict(i=FP8), UNSUPPORTED),
    (dict(o=FP8), UNSUPPORTED), (dict(x=None), INVALID), (dict(gamma=None), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dgamma=A + 8), INVALID),
    (dict(ws=None), INVALID), (dict(ws=None, dgamma=None), INVALID), (dict(nbytes=64), SMALL),
    (dict(o=BF, dx=A), INVALID),             # dx over a BF16 dy
    (dict(x=4 * A, dx=A + 16), INVALID),     # dx over a part of an fp32 dy
    (dict(dy=4 * A, dx=A), INVALID),         # dx over x
])
def test_layer_norm_backward_refusals(over, status):
    assert _norm_bwd(**over) == status
    assert lib.moe_last_error() != ""


def _balance(**over):
    a = dict(T=10, E=8, k=2, S=1, logits=A, ids=A, off=None, mask=None, alpha=1.0, counts=A, probs=A, loss=A,
             dlogits=2 * A, ws=A, nbytes=1 << 40)
    a.update(over)
    return lib._lib.moe_balance_loss(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(T=0), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID), (dict(S=0), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(E=64, k=17), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED),
    (dict(S=2), INVALID), (dict(S=(1 << 20) + 1, off=A), UNSUPPORTED), (dict(logits=None), INVALID),
    (dict(ids=None), INVALID), (dict(counts=None), INVALID), (dict(probs=None), INVALID), (dict(loss=None), INVALID),
    (dict(loss=A + 4), INVALID), (dict(dlogits=A), INVALID), (dict(dlogits=A + 16), INVALID), (dict(mask=A + 1), INVALID), (dict(ws=None), INVALID),
    (dict(nbytes=0), SMALL),
])
def test_balance_loss_refusals(over, status):
    assert _balance(**over) == status
    assert lib.moe_last_error() != ""


def _orth(**over):
    a = dict(batch=2, M=8, N=300, i=F32, u=A, steps=5, coeffs=None, eps=1e-7, y=8 * A, ws=A, nbytes=1 << 40)
    a.update(over)
    if a["coeffs"] is not None:
        flat = [v for row in a["coeffs"] for v in row]
        a["coeffs"] = (ctypes.c_float * len(flat))(*flat)
    return lib._lib.moe_orthogonalize(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INVALID), (dict(batch=65536), UNSUPPORTED), (dict(M=0), INVALID), (dict(N=-3), INVALID),
    (dict(N=32769), UNSUPPORTED), (dict(M=16385, N=16385), UNSUPPORTED), (dict(i=FP8), UNSUPPORTED),
    (dict(steps=0), INVALID), (dict(steps=33), UNSUPPORTED), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(u=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID),
    (dict(u=A + 4), INVALID), (dict(y=A), INVALID), (dict(y=A + 16), INVALID), (dict(nbytes=16), SMALL),
    (dict(steps=1, coeffs=[(1, 20, 0)]), UNSUPPORTED),                  # b A past the range
    (dict(steps=2, coeffs=[(9, 0, 0), (9, 0, 0)]), UNSUPPORTED),        # X grows past it
    (dict(steps=1, coeffs=[(float("nan"), 0, 0)]), UNSUPPORTED),
    (dict(steps=1, coeffs=[(1, float("inf"), 0)]), UNSUPPORTED),
])
def test_orthogonalize_refusals(over, status):
    assert _orth(**over) == status
    assert lib.moe_last_error() != ""


def test_orthogonalize_workspace_is_bounded():
    one = lib.moe_orthogonalize_workspace_size(1, 2048, 7168)
    assert one >= 8 * 2048 * 7168 + 4 * 2048 * 2048
    assert lib.moe_orthogonalize_workspace_size(512, 2048, 7168) <= (8 << 30) + (1 << 20)
    assert lib.moe_orthogonalize_workspace_size(0, 4, 4) == 0 and lib.moe_orthogonalize_workspace_size(1, 4, 40000) == 0
    assert lib.moe_orthogonalize_workspace_size(1, 1, 1) > 0


def test_workspace_sizes_of_refused_shapes_are_zero():
    assert lib.moe_layer_norm_backward_workspace_size(0, 256) == 0
    assert lib.moe_layer_norm_backward_workspace_size(4, 100) == 0
    assert lib.moe_layer_norm_backward_workspace_size(4, 256) > 0
    assert lib.moe_balance_loss_workspace_size(10, 8, 9, 1) == 0
    assert lib.moe_balance_loss_workspace_size(10, 2000, 2, 1) == 0
    assert lib.moe_balance_loss_workspace_size(1, 1, 1, 1) > 0


def test_backward_aux_checks_its_gradient():
    d = lib.make_desc(64, 256, 8, 128, 2, "bf16", "bf16", layout="row_major")
    with pytest.raises(lib.MoeError) as ex:
        lib.moe_backward_aux(d, A, A, A, A, A, A, A, A + 4, A, A, A, A, None, None, stream=0)
    assert ex.value.status == INVALID and "dlogits" in str(ex.value)


def test_wrappers_refuse_host_tensors():
    """A host pointer would fault on the device: the wrappers refuse it."""
    x, g = torch.zeros(4, 256), torch.ones(256)
    with pytest.raises(ValueError):
        L.layer_norm(x, g)
    with pytest.raises(ValueError):
        L.layer_norm_backward(x, g, torch.zeros(4), torch.ones(4), x)
    with pytest.raises(ValueError):
        L.balance_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        L.orthogonalize(torch.zeros(2, 8, 8))

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

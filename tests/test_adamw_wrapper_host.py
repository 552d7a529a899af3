"""The optimiser on the host (no GPU): what its wrapper hands to moe_adamw after a step that was refused, by stand-ins
for the library's entry point and for the GPU's tensors; moe_adamw's refusal of what it does not know."""

import contextlib
import ctypes

import pytest
import torch

from moe_layer_router_amd import layer as L, lib


class P(torch.Tensor):                                                     # a tensor that says that it is on a GPU
    is_cuda = True


def _host(monkeypatch):
    """Calls of moe_adamw: per tensor (n, param, grad, m, v, param_dtype, grad_dtype)."""
    calls = []
    monkeypatch.setattr(L, "_on", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(lib, "moe_adamw", lambda table, options: calls.append(
        [(r.n, r.param, r.grad, r.m, r.v, r.param_dtype, r.grad_dtype) for r in table]))
    return calls


def _rows(params, grads, states):
    t = {torch.float32: lib.MOE_DTYPE_F32, torch.bfloat16: lib.MOE_DTYPE_BF16}
    return [(p.numel(), p.data_ptr(), g.data_ptr(), s["m"].data_ptr(), s["v"].data_ptr(), t[p.dtype], t[g.dtype])
            for p, g, s in zip(params, grads, states)]


@pytest.mark.parametrize("bad", [0, 1, 2])
@pytest.mark.parametrize("why", ["not dense", "state's type", "state's size"])
def test_a_step_after_a_refused_one(monkeypatch, bad, why):
    """Weights or states that are refused and then put right: the next step is that of all tensors again."""
    calls = _host(monkeypatch)
    params = [torch.randn(16, 16).as_subclass(P) for _ in range(3)]
    params[1] = params[1].to(torch.bfloat16)
    grads = [torch.randn(16, 16), torch.randn(16, 16).to(torch.bfloat16), torch.randn(16, 16)]
    opt = L.AdamW(params)
    opt.step(grads, 1e-3)
    assert calls[-1] == _rows(params, grads, opt.states)
    keep = dict(opt.states[bad])
    if why == "not dense":
        params[bad].data = params[bad].data.t()
    elif why == "state's type":
        opt.states[bad] = dict(keep, v=torch.zeros(16, 16, dtype=torch.bfloat16))
    else:
        opt.states[bad] = dict(keep, m=torch.zeros(16, 8))
    for _ in range(2):
        with pytest.raises(ValueError):
            opt.step(grads, 1e-3)
    assert len(calls) == 1 and opt.count == 1
    if why == "not dense":
        params[bad].data = params[bad].data.t()
    else:
        opt.states[bad] = keep
    new = [torch.randn(16, 16) for _ in range(3)]
    opt.step(new, 1e-3)
    assert len(calls) == 2 and calls[-1] == _rows(params, new, opt.states) and opt.count == 2


def test_a_first_step_that_is_refused(monkeypatch):
    calls = _host(monkeypatch)
    params = [torch.randn(8, 8).as_subclass(P) for _ in range(2)]
    params[1].data = params[1].data.t()
    opt = L.AdamW(params, states=[dict(m=torch.zeros(8, 8), v=torch.zeros(8, 8)) for _ in range(2)])
    with pytest.raises(ValueError):
        opt.step([torch.ones(8, 8)] * 2, 1e-3)
    params[1].data = params[1].data.t()
    opt.step([torch.ones(8, 8)] * 2, 1e-3)
    assert len(calls) == 1 and [r[0] for r in calls[0]] == [64, 64] and all(r[1] and r[2] for r in calls[0])


@pytest.mark.parametrize("reserved", [1, -1, 1 << 30])
@pytest.mark.parametrize("n", [0, 100])
def test_reserved_has_to_be_zero(reserved, n):
    a = 0x100000                                                           # made-up addresses: the checks never dereference
    ts = (lib.MoeAdamwTensor * 1)(lib.MoeAdamwTensor(a, 2 * a, 3 * a, 4 * a, None, None, None, n, lib.MOE_DTYPE_F32, lib.MOE_DTYPE_F32, 0.0, reserved))
    o = lib.MoeAdamwOptions(1e-3, 0.9, 0.999, 1e-8, 1, None, None, None, lib.MOE_DTYPE_F32, 0)
    assert lib._lib.moe_adamw(1, ts, ctypes.byref(o), None) == lib.MOE_ERR_INVALID_ARGUMENT
    assert "reserved" in lib.moe_last_error()

"""The Python wrappers of the selection, the linear layers and AdamW on the host
(no GPU): copies, outputs, workspaces and the launch are made in the context of
the stream that the call is given, and tensors or streams of another device are
refused.  The library's entry points, the context and the allocation are stand-ins."""

import contextlib

import pytest
import torch

from moe_layer_router_amd import layer as L, lib

T, K, N = 6, 16, 24
BF = dict(dtype=torch.bfloat16)


def _t(*shape, **kw):
    """A matrix that is not dense: the wrapper has to copy it."""
    return torch.zeros(shape[1], shape[0], **kw).t()


CALLS = {
    "select_experts": lambda s: L.select_experts(_t(T, 8), 2, stream=s),
    "select_experts_backward": lambda s: L.select_experts_backward(_t(T, 8), _t(T, 2, dtype=torch.int32), _t(T, 2), stream=s),
    "linear": lambda s: L.linear(_t(T, K, **BF), _t(N, K, **BF), torch.zeros(N), "gelu", _t(T, N), pre_dtype="f32", stream=s),
    "linear_backward": lambda s: L.linear_backward(_t(T, K, **BF), _t(N, K, **BF), _t(T, N), "gelu", _t(T, N), want_dbias=True,
                                                   stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_everything_happens_on_the_stream_of_the_call(monkeypatch, name):
    stream, where, calls = object(), [], []

    @contextlib.contextmanager
    def on(device, s):
        where.append(s)
        yield
        where.pop()

    def inside(f):
        def g(*a, **kw):
            assert where == [stream]
            return f(*a, **kw)
        return g

    def entry(*a, **kw):
        assert where == [stream] and stream not in a and not kw
        assert all(t.is_contiguous() for t in a if isinstance(t, torch.Tensor))
        calls.append(1)

    monkeypatch.setattr(L, "_on", on)
    monkeypatch.setattr(L, "_matrix", lambda *a: None)                     # (asks for a GPU)
    for f in ("moe_select_experts", "moe_select_experts_backward", "moe_linear", "moe_linear_backward"):
        monkeypatch.setattr(lib, f, entry)
    dense = L._dense
    monkeypatch.setattr(L, "_dense", inside(dense))
    monkeypatch.setattr(L, "_scratch", inside(L._scratch))
    CALLS[name](stream)
    assert calls and not where


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_the_host_are_refused(name):
    with pytest.raises(ValueError):
        CALLS[name](None)


def test_optimiser_on_the_stream_of_the_call(monkeypatch):
    stream, where, calls = object(), [], []

    @contextlib.contextmanager
    def on(device, s):
        where.append(s)
        yield
        where.pop()

    def entry(table, options):
        assert where == [stream]
        calls.append([(r.n, r.param, r.grad) for r in table])

    class P(torch.Tensor):                                                 # a tensor that says that it is on a GPU
        is_cuda = True

    p = torch.zeros(9, 5).as_subclass(P)
    monkeypatch.setattr(L, "_on", on)
    monkeypatch.setattr(lib, "moe_adamw", entry)
    monkeypatch.setattr(L, "_is", lambda *a: None)
    opt = L.AdamW([p])
    g = torch.ones(5, 9).t()
    opt.step([g], 1e-3, stream=stream)
    assert calls[0][0][0] == 45 and calls[0][0][1] == p.data_ptr() and calls[0][0][2] != g.data_ptr() and opt.count == 1
    p.data = p.data[:4].contiguous()                                       # the weights' memory and size were exchanged
    opt.states[0] = {n: v[:4].contiguous() for n, v in opt.states[0].items()}
    opt.step([g[:4]], 1e-3, stream=stream)
    assert calls[1][0][0] == 20 and calls[1][0][1] == p.data_ptr() and opt.count == 2
    p.data = p.data[:2]                                                    # the same address, fewer weights
    opt.states[0] = {n: v[:2] for n, v in opt.states[0].items()}
    opt.step([g[:2]], 1e-3, stream=stream)
    assert calls[2][0][0] == 10 and calls[2][0][1] == p.data_ptr()
    looked = []
    monkeypatch.setattr(L, "_is", lambda *a: looked.append(a[1]))
    p.data = torch.zeros(5, 5)
    opt.states[0] = {n: torch.zeros(5, 5) for n in ("m", "v")}
    opt.step([torch.ones(5, 5)], 1e-3, stream=stream)
    del looked[:]
    opt.step([torch.ones(5, 5)], 1e-3, stream=stream)
    assert not looked
    p.data = p.data.t()                                                    # the same address and shape, no longer dense
    opt.step([torch.ones(5, 5)], 1e-3, stream=stream)
    assert "params[0]" in looked


def test_a_refused_step_does_not_count(monkeypatch):
    class P(torch.Tensor):
        is_cuda = True

    def entry(*a):
        raise lib.MoeError(1, "moe_adamw")

    monkeypatch.setattr(L, "_on", lambda *a: contextlib.nullcontext())
    monkeypatch.setattr(lib, "moe_adamw", entry)
    for capturable in (False, True):
        opt = L.AdamW([torch.zeros(8).as_subclass(P)], capturable=capturable, count=3)
        with pytest.raises(lib.MoeError):
            opt.step([torch.zeros(8)], 1e-3)
        assert int(opt.count) == 3

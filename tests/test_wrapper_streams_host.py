"""The Python wrappers of the layer and its conversions on the host (no GPU):
copies, outputs, workspaces and the launch itself are made in the context of
the stream that the call is given.  The library's entry points, the context
and the allocation are stand-ins."""

import contextlib

import pytest
import torch

from moe_layer_router_amd import layer as L, lib

T, H, E, I, K = 6, 128, 4, 128, 2
BF = dict(dtype=torch.bfloat16)


def _inputs():
    return dict(x=torch.zeros(T, H, **BF), router_w=torch.zeros(E, H, **BF), w_gate_up=torch.zeros(E, 2 * I, H, **BF),
                w_down=torch.zeros(E, H, I, **BF))


def _packed():
    return {**_inputs(), "weights_packed": True}


CALLS = {
    "pack_weights": lambda s: L.pack_weights(_inputs(), stream=s),
    "forward": lambda s: L.forward(_packed(), K, stream=s),
    "forward_routed": lambda s: L.forward(_packed(), K, stream=s, routing=(torch.zeros(T, K), torch.zeros(T, K))),
    "forward_trace": lambda s: L.forward(_packed(), K, stream=s, trace=True),
    "quantize_input": lambda s: L.quantize_input(torch.zeros(H, T, **BF).t(), stream=s),
    "quantize_e5m6": lambda s: L.quantize_e5m6(torch.zeros(H, T, **BF).t(), stream=s),
    "dequantize_e5m6": lambda s: L.dequantize_e5m6(torch.zeros(T, 192, dtype=torch.uint8), torch.zeros(T, 1), stream=s),
    "route": lambda s: L.route(_inputs(), K, E, stream=s),
    "permute": lambda s: L.permute(torch.zeros(T, K, dtype=torch.int64), E, stream=s),
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
        calls.append(1)

    monkeypatch.setattr(L, "_on", on)
    for f in ("moe_pack_weights", "moe_forward", "moe_quantize_input", "moe_quantize_e5m6", "moe_dequantize_e5m6",
              "moe_route", "moe_permute"):
        monkeypatch.setattr(lib, f, entry)
    real = torch.empty
    monkeypatch.setattr(L.torch, "empty", inside(real))
    monkeypatch.setattr(torch.Tensor, "copy_", inside(torch.Tensor.copy_))
    CALLS[name](stream)
    assert calls and not where

"""The Python wrapper of the backward pass on the host (no GPU): whatever it
copies, allocates and launches belongs to the stream it is given.  The library
call and the stream's context are stand-ins."""

import contextlib

import torch

from moe_layer_router_amd import layer as L, lib


def test_copies_and_buffers_belong_to_the_stream_of_the_call(monkeypatch):
    T, H, E, I, k = 6, 128, 4, 128, 2
    stream, where, seen = object(), [], {}

    @contextlib.contextmanager
    def on(device, s):
        where.append(s)
        yield
        where.pop()

    def scratch(workspace, device, nbytes):
        assert where == [stream] and workspace is None and device == torch.device("cpu")
        return torch.empty(256, dtype=torch.uint8)

    def aux(desc, x, router_w, w_gate_up, w_down, ids, w, dy, dlogits, dx, dgu, dd, dr, db, ws, s=None):
        assert where == [stream] and s is None         # the context's own stream
        for t in (x, router_w, w_gate_up, w_down, ids, w, dy, dlogits):
            assert t.is_contiguous() and t.data_ptr() % 16 == 0
        seen.update(x=x, dlogits=dlogits, dy=dy)

    contiguous = torch.Tensor.contiguous
    monkeypatch.setattr(torch.Tensor, "contiguous", lambda t: (where == [stream] or t.is_contiguous() or 1 / 0) and
                        contiguous(t))
    monkeypatch.setattr(L, "_on", on)
    monkeypatch.setattr(L, "_scratch", scratch)
    monkeypatch.setattr(lib, "moe_backward_aux", aux)
    bf = dict(dtype=torch.bfloat16)
    inputs = dict(x=torch.randn(T, 2 * H).to(torch.bfloat16)[:, ::2], router_w=torch.zeros(E, H, **bf),
                  w_gate_up=torch.zeros(E, 2 * I, H, **bf), w_down=torch.zeros(E, H, I, **bf))
    dl = torch.randn(E, T).t()
    L.backward(inputs, torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(H, T, **bf).t(),
               dlogits=dl, stream=stream)
    assert torch.equal(seen["dlogits"], dl) and torch.equal(seen["x"], inputs["x"])
    flat = torch.randn(T * E + 1)                       # a view off a 16-byte boundary is copied, not refused
    off = flat[1:].view(T, E)
    assert off.data_ptr() % 16
    L.backward(inputs, torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(T, H, **bf), dlogits=off,
               stream=stream)
    assert torch.equal(seen["dlogits"], off)

"""Convenience wrapper: allocate outputs and workspace with PyTorch and call
moe_forward / moe_route / moe_permute, and the operators of a training step
around the layer (layer_norm, balance_loss, backward, orthogonalize).  No
arithmetic happens here."""

import contextlib

import torch

from . import lib


def pack_weights(inputs: dict, top_k: int = 1, stream=None) -> dict:
    """Copy of `inputs` whose expert weights (and FP4 scales) are in the
    MFMA-tiled layout moe_forward reads (moe_pack_weights).  The input dict
    is not modified; the result carries "weights_packed": True."""
    if inputs.get("weights_packed"):
        return inputs
    desc = desc_from_inputs(inputs, top_k, layout="row_major")
    fp4 = desc.weight_dtype == lib.MOE_DTYPE_FP4_E2M1
    out = dict(inputs)
    with _on(inputs["x"].device, stream):
        for which, w, sc in ((lib.MOE_WEIGHTS_GATE_UP, "w_gate_up", "w_gate_up_scales"),
                             (lib.MOE_WEIGHTS_DOWN, "w_down", "w_down_scales")):
            dst = torch.empty_like(inputs[w])
            dst_sc = torch.empty_like(inputs[sc]) if fp4 else None
            lib.moe_pack_weights(desc, which, inputs[w].contiguous(), inputs[sc].contiguous() if fp4 else None,
                                 dst, dst_sc)
            out[w] = dst
            if fp4:
                out[sc] = dst_sc
    out["weights_packed"] = True
    return out


def desc_from_inputs(inputs: dict, top_k: int, mode: str = "mega", flags: int = 0, I=None, layout=None,
                     inter_scale: str = "f32") -> lib.MoeDesc:
    x = inputs["x"]
    T, H = x.shape
    E = inputs["w_gate_up"].shape[0]
    if I is None:
        I = inputs["w_gate_up"].shape[1] // 2
    act = "bf16" if x.dtype == torch.bfloat16 else "fp8"
    wgu = inputs["w_gate_up"]
    if wgu.dtype == torch.bfloat16:
        weight = "bf16"
    elif wgu.shape[2] == H:
        weight = "fp8"
    else:
        weight = "fp4"
    if layout is None:
        layout = "tiled" if inputs.get("weights_packed") else "row_major"
    # FP8 weight scales: [E][N/128][K/128] per block, [E][N] per output channel
    sc = inputs.get("w_gate_up_scales")
    wscale = "channel" if weight == "fp8" and sc is not None and sc.dim() == 2 else "block"
    return lib.make_desc(T, H, E, I, top_k, act, weight, mode, flags, layout, inter_scale, wscale)


class Workspace:
    """A cached device workspace, grown on demand."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = None

    def get(self, nbytes: int) -> torch.Tensor:
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        return self.buf


def forward(inputs: dict, top_k: int, mode: str = "mega", workspace: Workspace = None,
            routing=None, want_perm: bool = True, stream=None, out=None, inter_scale: str = "f32",
            trace: bool = False) -> dict:
    """Run the layer on inputs whose weights went through pack_weights().
    routing=(topk_ids, topk_weights) feeds given routing
    (MOE_FLAG_ROUTING_GIVEN).  Returns dict(y, topk_ids, topk_weights,
    expert_offsets, perm)."""
    if not inputs.get("weights_packed"):
        raise ValueError("forward() needs MFMA-tiled weights: pass the inputs through pack_weights() first")
    flags = (lib.MOE_FLAG_ROUTING_GIVEN if routing is not None else 0) | (lib.MOE_FLAG_TRACE if trace else 0)
    desc = desc_from_inputs(inputs, top_k, mode, flags, inter_scale=inter_scale)
    dev = inputs["x"].device
    T, H, E, k = desc.T, desc.H, desc.E, desc.top_k
    with _on(dev, stream):
        if out is None:
            out = dict(y=torch.empty(T, H, dtype=torch.bfloat16, device=dev),
                       topk_ids=torch.empty(T, k, dtype=torch.int32, device=dev),
                       topk_weights=torch.empty(T, k, dtype=torch.float32, device=dev),
                       expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev) if want_perm else None,
                       perm=torch.empty(T * k, dtype=torch.int32, device=dev) if want_perm else None)
        if routing is not None:
            out["topk_ids"].copy_(routing[0])
            out["topk_weights"].copy_(routing[1])
        ws = _scratch(workspace, dev, lib.moe_workspace_size(desc))
        if trace:      # rows of workgroups that do not run must read as unused
            reg = lib.moe_get_workspace_regions(desc)
            ws[reg["trace"]: reg["trace"] + lib.MOE_TRACE_GROUPS * lib.MOE_TRACE_FIELDS * 8].zero_()
        lib.moe_forward(desc, inputs["x"], inputs.get("x_scales"), inputs["router_w"], inputs.get("router_bias"),
                        inputs["w_gate_up"], inputs.get("w_gate_up_scales"), inputs["w_down"],
                        inputs.get("w_down_scales"), out["y"], out["topk_ids"], out["topk_weights"],
                        out["expert_offsets"], out["perm"], ws)
    out["workspace"] = ws
    out["desc"] = desc
    return out


def intermediate(out: dict):
    """Views of the intermediate activations of a finished forward() call:
    (codes or BF16 values [T*k][I] in permuted row order, scales [T*k][I/128]
    or None)."""
    desc, ws = out["desc"], out["workspace"]
    reg = lib.moe_get_workspace_regions(desc)
    rows, I = desc.T * desc.top_k, desc.I
    if desc.weight_dtype != lib.MOE_DTYPE_BF16:     # FP8 / FP4 experts: E4M3 intermediate
        codes = ws[reg["inter"]: reg["inter"] + rows * I].view(rows, I)
        sc = ws[reg["inter_scales"]: reg["inter_scales"] + rows * (I // 128) * 4].view(torch.float32)
        return codes, sc.view(I // 128, rows).t()       # stored K block major
    vals = ws[reg["inter"]: reg["inter"] + rows * I * 2].view(torch.bfloat16).view(rows, I)
    return vals, None


def quantize_input(x: torch.Tensor, scale_mode: str = "f32", stream=None):
    """Per-token FP8 quantisation of [T, H] BF16 / fp32 activations
    (moe_quantize_input): returns (codes uint8 [T, H], scales float32 [T, H/128])."""
    T, H = x.shape
    with _on(x.device, stream):
        xq = torch.empty(T, H, dtype=torch.uint8, device=x.device)
        xs = torch.empty(T, H // 128, dtype=torch.float32, device=x.device)
        lib.moe_quantize_input(x.contiguous(), xq, xs, scale_mode)
    return xq, xs


def quantize_e5m6(x: torch.Tensor, scale_mode: str = "f32", stream=None):
    """Per-token, per-128-channel E5M6 quantisation (moe_quantize_e5m6) of a
    [T, H] bfloat16 / float32 tensor: (codes [T, 3H/2] uint8, scales
    [T, H/128] float32)."""
    T, H = x.shape
    with _on(x.device, stream):
        xq = torch.empty(T, H // 2 * 3, dtype=torch.uint8, device=x.device)
        xs = torch.empty(T, H // 128, dtype=torch.float32, device=x.device)
        lib.moe_quantize_e5m6(x.contiguous(), xq, xs, scale_mode)
    return xq, xs


def dequantize_e5m6(xq: torch.Tensor, xs: torch.Tensor, stream=None) -> torch.Tensor:
    """float32 [T, H] values of E5M6 codes and their scales (moe_dequantize_e5m6)."""
    T, H = xq.shape[0], xq.shape[1] // 3 * 2
    with _on(xq.device, stream):
        out = torch.empty(T, H, dtype=torch.float32, device=xq.device)
        lib.moe_dequantize_e5m6(xq.contiguous(), xs.contiguous(), out)
    return out


def backward(inputs: dict, topk_ids: torch.Tensor, topk_weights: torch.Tensor, dy: torch.Tensor,
             workspace: Workspace = None, stream=None, want_dbias: bool = True, out: dict = None,
             dlogits: torch.Tensor = None) -> dict:
    """Gradients of a BF16 layer (moe_backward) for the routing a forward
    call returned, from row-major weights (inputs as generated, not packed).
    dlogits: an additional gradient of the router logits [T, E] float32
    (balance_loss's; moe_backward_aux).  Returns dict(dx, dw_gate_up, dw_down,
    dw_router, dbias), fp32 (`out`, a previous result, is reused)."""
    if inputs.get("weights_packed"):
        raise ValueError("backward() reads the row-major weights: pass the inputs before pack_weights()")
    x = inputs["x"]
    T, H = x.shape
    k = topk_ids.shape[1]
    desc = desc_from_inputs(inputs, k, layout="row_major")
    E, I = desc.E, desc.I
    dev = x.device
    if dlogits is not None:
        _is(dlogits, "dlogits", (T, E), _F32, dev)
    with _on(dev, stream):
        f32 = dict(dtype=torch.float32, device=dev)
        if out is None:
            out = dict(dx=torch.empty(T, H, **f32), dw_gate_up=torch.empty(E, 2 * I, H, **f32),
                       dw_down=torch.empty(E, H, I, **f32), dw_router=torch.empty(E, H, **f32),
                       dbias=torch.empty(E, **f32) if want_dbias else None)
        ws = _scratch(workspace, dev, lib.moe_backward_workspace_size(desc))
        lib.moe_backward_aux(desc, _dense(x), _dense(inputs["router_w"]), _dense(inputs["w_gate_up"]),
                             _dense(inputs["w_down"]), _dense(topk_ids), _dense(topk_weights), _dense(dy),
                             None if dlogits is None else _dense(dlogits), out["dx"], out["dw_gate_up"],
                             out["dw_down"], out["dw_router"], out["dbias"], ws)
    return out


def logits(out: dict) -> torch.Tensor:
    """View of the router logits [T, E] (float32, bias included) of a forward()
    call that did the routing itself, valid until its workspace is used again."""
    desc, ws = out["desc"], out["workspace"]
    _need(not desc.flags & lib.MOE_FLAG_ROUTING_GIVEN, "the call was given its routing: it has no logits")
    at = lib.moe_get_workspace_regions(desc)["logits"]
    return ws[at: at + desc.T * desc.E * 4].view(torch.float32).view(desc.T, desc.E)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """Context in which `device` is the current device and `stream` (None: the
    device's current stream) its current stream, so that copies, outputs and
    workspaces of a call belong to the stream that the call runs on."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(stream, device)
        _need(stream.device == device, f"stream must be one of {device} (got one of {stream.device})")
        return torch.cuda.stream(stream)
    return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _scratch(workspace, device, nbytes):
    """The caller's workspace, or one of the call's own; on the call's device."""
    if workspace is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    ws = workspace.get(nbytes)
    _need(ws.device == device, f"workspace must be on {device} (got {ws.device})")
    return ws


def _dense(t):
    """t, or a copy of it that is contiguous and starts on a 16-byte boundary."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _is(t, name, shape, dtypes, device, out=False):
    """Check an argument; outputs must be laid out as the library writes them.
    (One test on the way that every call takes, the message only when it fails.)"""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.device == device and \
            (not out or t.is_contiguous()):
        return
    _need(isinstance(t, torch.Tensor) and t.shape == shape, f"{name} must be a tensor {list(shape)}")
    _need(t.dtype in dtypes, f"{name} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    _need(t.device == device, f"{name} must be on {device} (got {t.device})")
    _need(t.is_contiguous(), f"{name} must be contiguous")


def _matrix(t, name, dtypes):
    """Check a 2-d input on a GPU, which the other arguments are checked against."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 2 and t.is_cuda and t.dtype in dtypes):
        raise ValueError(f"{name} must be a 2-d tensor on a GPU, {' or '.join(str(d) for d in dtypes)}")


_FLOATS = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)
_OUT_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}


def layer_norm(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor = None, eps: float = 1e-5,
               out_dtype: str = "bf16", scale_mode: str = "f32", want_stats: bool = False, stream=None,
               out: dict = None) -> dict:
    """Layer norm of [T, H] bfloat16 / float32 activations (moe_layer_norm),
    gamma and beta [H] float32.  out_dtype "bf16", "f32", or "fp8": the layer's
    quantised input (E4M3 codes as uint8, with scales).  Returns dict(y,
    y_scales, mean, rstd): y [T, H], y_scales [T, H/128] float32 ("fp8", else
    None), mean and rstd [T] float32 (want_stats, for layer_norm_backward, else
    None); `out`, a previous result, is reused."""
    _matrix(x, "x", _FLOATS)
    T, H = x.shape
    dev = x.device
    if out_dtype not in _OUT_DTYPES or scale_mode not in lib.INTER_SCALES:
        raise ValueError(f"unknown out_dtype {out_dtype!r} or scale_mode {scale_mode!r}")
    _is(gamma, "gamma", (H,), _F32, dev)
    if beta is not None:
        _is(beta, "beta", (H,), _F32, dev)
    dt = _OUT_DTYPES[out_dtype]
    fp8 = out_dtype == "fp8"
    with _on(dev, stream):
        if out is None:
            out = dict(y=torch.empty(T, H, dtype=dt, device=dev),
                       y_scales=torch.empty(T, H // 128, dtype=torch.float32, device=dev) if fp8 else None,
                       mean=torch.empty(T, dtype=torch.float32, device=dev) if want_stats else None,
                       rstd=torch.empty(T, dtype=torch.float32, device=dev) if want_stats else None)
        else:
            _is(out["y"], "out['y']", (T, H), (dt,), dev, True)
            for name, shape, wanted in (("y_scales", (T, H // 128), fp8), ("mean", (T,), want_stats),
                                        ("rstd", (T,), want_stats)):
                _need((out[name] is not None) == wanted, "out does not fit the call")
                if wanted:
                    _is(out[name], name, shape, _F32, dev, True)
        lib.moe_layer_norm(_dense(x), _dense(gamma), None if beta is None else _dense(beta), eps, out["y"],
                           out["y_scales"], out["mean"], out["rstd"], scale_mode)
    return out


def layer_norm_backward(x: torch.Tensor, gamma: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        dy: torch.Tensor, want_weights: bool = True, workspace: Workspace = None, stream=None,
                        out: dict = None) -> dict:
    """Backward pass of layer_norm (moe_layer_norm_backward) for dy [T, H]
    bfloat16 / float32 and the statistics of the forward call.  Returns
    dict(dx [T, H], dgamma [H], dbeta [H]), float32; without want_weights
    dgamma and dbeta are None.  `out`, a previous result, is reused (out["dx"]
    may be dy)."""
    _matrix(x, "x", _FLOATS)
    T, H = x.shape
    dev = x.device
    _is(gamma, "gamma", (H,), _F32, dev)
    _is(mean, "mean", (T,), _F32, dev)
    _is(rstd, "rstd", (T,), _F32, dev)
    _is(dy, "dy", (T, H), _FLOATS, dev)
    with _on(dev, stream):
        f32 = dict(dtype=torch.float32, device=dev)
        if out is None:
            out = dict(dx=torch.empty(T, H, **f32), dgamma=torch.empty(H, **f32) if want_weights else None,
                       dbeta=torch.empty(H, **f32) if want_weights else None)
        else:
            _is(out["dx"], "out['dx']", (T, H), _F32, dev, True)
            for name in ("dgamma", "dbeta"):
                _need((out[name] is not None) == want_weights, "out does not fit the call")
                if want_weights:
                    _is(out[name], name, (H,), _F32, dev, True)
        ws = None
        if want_weights:
            ws = _scratch(workspace, dev, lib.moe_layer_norm_backward_workspace_size(T, H))
        lib.moe_layer_norm_backward(_dense(x), _dense(gamma), _dense(mean), _dense(rstd), _dense(dy), out["dx"],
                                    out["dgamma"], out["dbeta"], ws)
    return out


def balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, alpha: float = 1.0, seq_offsets: torch.Tensor = None,
                 token_mask: torch.Tensor = None, want_grad: bool = True, workspace: Workspace = None, stream=None,
                 out: dict = None) -> dict:
    """Load-balance loss of a routing (moe_balance_loss): logits [T, E] float32
    and topk_ids [T, k] int32 or int64 as route() returns them, seq_offsets
    [S + 1] int32 or int64 (None: one sequence; both clamped to their range), token_mask [T] bool or uint8 (None: every token
    counts).  Returns dict(loss [1] float32, counts [S, E] int32, probs [S, E]
    float32, dlogits [T, E] float32 or, without want_grad, None); `out`, a
    previous result, is reused."""
    _matrix(logits, "logits", _F32)
    T, E = logits.shape
    dev = logits.device
    _need(topk_ids.dim() == 2, "topk_ids must be [T, k]")
    _is(topk_ids, "topk_ids", (T, topk_ids.shape[1]), (torch.int32, torch.int64), dev)
    S = 1
    if seq_offsets is not None:
        _need(seq_offsets.dim() == 1 and seq_offsets.shape[0] >= 2, "seq_offsets must be [n_seq + 1]")
        S = seq_offsets.shape[0] - 1
        _is(seq_offsets, "seq_offsets", (S + 1,), (torch.int32, torch.int64), dev)
    if token_mask is not None:
        _is(token_mask, "token_mask", (T,), (torch.bool, torch.uint8), dev)
    with _on(dev, stream):
        f32 = dict(dtype=torch.float32, device=dev)
        if out is None:
            out = dict(loss=torch.empty(1, **f32), counts=torch.empty(S, E, dtype=torch.int32, device=dev),
                       probs=torch.empty(S, E, **f32), dlogits=torch.empty(T, E, **f32) if want_grad else None)
        else:
            _need((out["dlogits"] is not None) == want_grad, "out['dlogits'] does not fit the call")
            for name, shape, dt in (("loss", (1,), torch.float32), ("counts", (S, E), torch.int32),
                                    ("probs", (S, E), torch.float32), ("dlogits", (T, E), torch.float32)):
                if out[name] is not None:
                    _is(out[name], name, shape, (dt,), dev, True)
        ws = _scratch(workspace, dev, lib.moe_balance_loss_workspace_size(T, E, topk_ids.shape[1], S))
        # (the library clamps 32-bit values: wider ones must not wrap round into the range)
        if topk_ids.dtype == torch.int64:
            topk_ids = topk_ids.clamp(0, E - 1).to(torch.int32)
        if seq_offsets is not None and seq_offsets.dtype == torch.int64:
            seq_offsets = seq_offsets.clamp(0, T).to(torch.int32)
        lib.moe_balance_loss(_dense(logits), _dense(topk_ids), None if seq_offsets is None else _dense(seq_offsets),
                             None if token_mask is None else _dense(token_mask), alpha, out["counts"], out["probs"],
                             out["loss"], out["dlogits"], ws)
    return out


def trace_phases(out: dict) -> dict:
    """Phase timing of a finished forward(..., trace=True) call in the
    persistent kernel, from the per-workgroup stamps (100 MHz clock):
    microseconds from the first workgroup's entry to each phase boundary
    (first / median / last workgroup), and the items per workgroup."""
    import numpy as np
    desc, ws = out["desc"], out["workspace"]
    reg = lib.moe_get_workspace_regions(desc)
    n = lib.MOE_TRACE_GROUPS * lib.MOE_TRACE_FIELDS
    raw = ws[reg["trace"]: reg["trace"] + n * 8].view(torch.int64).cpu().numpy().reshape(lib.MOE_TRACE_GROUPS, -1)
    used = raw[:, 0] > 0
    t = raw[used, :6].astype(np.float64)
    t0 = t[:, 0].min()
    us = (t - t0) / 100.0
    names = ["entry", "routing_end", "gateup_start", "gateup_end", "down_end", "exit"]
    res = {nm: {"first": round(float(us[:, i].min()), 1), "median": round(float(np.median(us[:, i])), 1),
                "last": round(float(us[:, i].max()), 1)} for i, nm in enumerate(names)}
    res["gateup_items_per_wg"] = [int(raw[used, 6].min()), int(raw[used, 6].max())]
    res["down_items_per_wg"] = [int(raw[used, 7].min()), int(raw[used, 7].max())]
    res["workgroups"] = int(used.sum())
    return res


def route(inputs: dict, top_k: int, E: int, I: int = 128, workspace: Workspace = None, stream=None) -> dict:
    x = inputs["x"]
    T, H = x.shape
    act = "bf16" if x.dtype == torch.bfloat16 else "fp8"
    desc = lib.make_desc(T, H, E, I, top_k, act, "bf16" if act == "bf16" else "fp8")
    dev = x.device
    with _on(dev, stream):
        out = dict(logits=torch.empty(T, E, dtype=torch.float32, device=dev),
                   topk_ids=torch.empty(T, top_k, dtype=torch.int32, device=dev),
                   topk_weights=torch.empty(T, top_k, dtype=torch.float32, device=dev))
        ws = _scratch(workspace, dev, lib.moe_route_workspace_size(desc))
        lib.moe_route(desc, x, inputs.get("x_scales"), inputs["router_w"], inputs.get("router_bias"),
                      out["logits"], out["topk_ids"], out["topk_weights"], ws)
    return out


def permute(topk_ids: torch.Tensor, E: int, H: int = 128, I: int = 128, workspace: Workspace = None,
            stream=None) -> dict:
    T, k = topk_ids.shape
    desc = lib.make_desc(T, H, E, I, k, "fp8", "fp8")
    dev = topk_ids.device
    with _on(dev, stream):
        out = dict(expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                   perm=torch.empty(T * k, dtype=torch.int32, device=dev),
                   row_of=torch.empty(T * k, dtype=torch.int32, device=dev))
        ws = _scratch(workspace, dev, lib.moe_permute_workspace_size(desc))
        lib.moe_permute(desc, topk_ids.to(torch.int32).contiguous(), out["expert_offsets"], out["perm"],
                        out["row_of"], ws)
    return out


def orthogonalize(u: torch.Tensor, steps: int = 5, coeffs=None, eps: float = 1e-7, workspace: Workspace = None,
                  stream=None, out: torch.Tensor = None) -> torch.Tensor:
    """Newton-Schulz orthogonalisation (moe_orthogonalize) of a matrix [M, N] or
    a batch [batch, M, N], bfloat16 or float32: bfloat16 of u's shape.  coeffs:
    `steps` triples (a, b, c), or None.  backward()'s gradients: dw_down and
    dw_router as they are; dw_gate_up [E, 2I, H] as .view(2 * E, I, H), gate
    and up being matrices of their own."""
    _need(u.dim() in (2, 3) and u.is_cuda, "u must be [M, N] or [batch, M, N] on a GPU")
    _need(u.dtype in _FLOATS, "u must be bfloat16 or float32")
    _need(coeffs is None or (len(coeffs) == steps and all(len(c) == 3 for c in coeffs)),
          "coeffs must be one triple per step")
    dev = u.device
    with _on(dev, stream):
        if out is None:
            out = torch.empty(u.shape, dtype=torch.bfloat16, device=dev)
        else:
            _is(out, "out", u.shape, (torch.bfloat16,), dev, True)
        v = _dense(u)
        v, y = (v, out) if u.dim() == 3 else (v[None], out[None])
        ws = _scratch(workspace, dev, lib.moe_orthogonalize_workspace_size(*v.shape))
        lib.moe_orthogonalize(v, steps, coeffs, eps, y, ws)
    return out

"""Workloads of the operators that stand beside the routed experts of a layer:
the selection of experts from router logits (softmax or sigmoid scores, a bias
for balance, groups of experts) with its gradient, linear layers (a shared
expert's, a dense block's) with bias, activation and residual in their epilogue
and their gradient, and the AdamW step over a layer's tensors.  `run` computes a
case in plain torch, or, with `own` set, through `moe_layer_router_amd.layer`."""

import math
import random

import torch

own = False

SCALE = 2.5                     # of the routing weights
E4M3_MAX = 448.0
BETAS = (0.9, 0.999)
EPS = 1e-8
LR = 1e-4
DECAY = 0.1
COUNT = 1000                    # steps done before: the middle of a training run
LAYER = 3 * 2048 * 7168         # weights of one expert


def _ragged(n, total, seed):
    """n tensor sizes of about `total` elements together: a few large ones, most of them small and odd."""
    r = random.Random(seed)
    parts = [math.exp(r.uniform(0, 7)) for _ in range(n)]
    return ",".join(str(max(1, int(total * p / sum(parts)) | 1)) for p in parts)


def listed():
    return [
        # one decoded token, 256 experts in 8 groups: latency counts
        dict(name="select_token", op="select", T=1, E=256, k=8, scoring="sigmoid", bias=True, groups=8, keep=4, top=2, renorm=True),
        # the same routing for a prefill-sized batch
        dict(name="select_prefill", op="select", T=8192, E=256, k=8, scoring="sigmoid", bias=True, groups=8, keep=4, top=2, renorm=True),
        # 1024 experts without groups, softmax scores and a bias for balance
        dict(name="select_e1024", op="select", T=16384, E=1024, k=16, scoring="softmax", bias=True, groups=1, keep=1, top=1, renorm=False),
        # the training step's gradient of the same routings: sparse with sigmoid scores, dense with softmax
        dict(name="select_bwd_prefill", op="select_bwd", T=8192, E=256, k=8, scoring="sigmoid", renorm=True),
        dict(name="select_bwd_e1024", op="select_bwd", T=16384, E=1024, k=16, scoring="softmax", renorm=False),
        # one decoded token through a shared expert's gate and up projections
        dict(name="linear_token", op="linear", T=1, K=7168, N=2048, act="swiglu", bias=False, residual=False, y="bf16", pre=False),
        # a prefill-sized batch through them in a training step, which keeps what the activation took
        dict(name="linear_shared", op="linear", T=8192, K=7168, N=2048, act="swiglu", bias=False, residual=False, y="bf16", pre=True),
        # a small dense block with bias, odd sizes, FP32 gradient of what follows
        dict(name="linear_bwd_ragged", op="linear_bwd", T=333, K=1000, N=488, act="gelu", bias=True, dy="f32", dx="f32"),
        # the training step's backward of linear_shared
        dict(name="linear_bwd_shared", op="linear_bwd", T=8192, K=7168, N=2048, act="swiglu", bias=False, dy="bf16", dx="f32"),
        # the tensors of a tiny layer: norm, router, experts
        dict(name="adamw_tiny", op="adamw", sizes="256,256,2048,524288,262144", p="f32", master=False, state="f32"),
        # a dense block's tensors of all sizes, BF16 weights alone, states in 8 bits
        dict(name="adamw_ragged_fp8", op="adamw", sizes=_ragged(37, 40_000_000, 1), p="bf16", master=False, state="fp8"),
        # eight experts with FP32 master weights and states
        dict(name="adamw_experts", op="adamw", sizes=",".join([str(2 * LAYER // 3), str(LAYER // 3)] * 8), p="bf16", master=True, state="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "select", "select_bwd", "linear", "linear", "linear_bwd", "linear_bwd", "adamw", "adamw"])
    if op in ("select", "select_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * _log_int(rng, 2, 1024 // groups)
        keep = rng.randint(1, groups)
        c = dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=rng.randint(1, min(16, keep * (E // groups))),
                 scoring=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.5)
        if op == "select":
            c.update(bias=rng.random() < 0.7, groups=groups, keep=keep, top=rng.choice([1, 2]))
        return c
    if op == "adamw":
        n = _log_int(rng, 1, 60)
        return dict(op=op, sizes=_ragged(n, _log_int(rng, 64, 8 * LAYER), rng.randrange(1 << 30)), p=rng.choice(["f32", "bf16"]),
                    master=rng.random() < 0.5, state=rng.choice(["f32", "fp8"]))
    big = max(work(c)["flops"] for c in listed() if c["op"] == op)
    while True:
        c = dict(op=op, T=_log_int(rng, 1, 8192), K=8 * _log_int(rng, 1, 896), N=8 * _log_int(rng, 1, 896),
                 act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "swiglu"]), bias=rng.random() < 0.5)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, y=rng.choice(["bf16", "f32"]), pre=rng.random() < 0.3)
        else:
            c.update(dy=rng.choice(["bf16", "f32"]), dx=rng.choice(["bf16", "f32"]))
        if work(c)["flops"] <= big:
            return c


def _rows(case):
    """Rows of a linear layer's weights: gate and up for SwiGLU."""
    return case["N"] * (2 if case["act"] == "swiglu" else 1)


def work(case):
    op, size = case["op"], {"bf16": 2, "f32": 4}
    if op == "select":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 8 * T * E}
    if op == "select_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        # without a softmax over all experts the selected logits are enough
        dense = case["scoring"] == "softmax" and not case["renorm"]
        return {"bytes": 4 * T * E + 8 * T * k + 4 * T * (E if dense else k), "flops": T * (8 * E if dense else 16 * k)}
    if op == "linear":
        T, K, N, R = case["T"], case["K"], case["N"], _rows(case)
        b = 2 * T * K + 2 * R * K + T * N * size[case["y"]]
        b += 4 * R if case["bias"] else 0
        b += 2 * T * N if case["residual"] else 0
        b += 2 * T * R if case["pre"] else 0
        return {"bytes": b, "flops": 2 * T * K * R}
    if op == "linear_bwd":
        T, K, N, R = case["T"], case["K"], case["N"], _rows(case)
        b = 2 * T * K + 2 * R * K + T * N * size[case["dy"]] + T * K * size[case["dx"]] + 4 * R * K
        b += 4 * R if case["bias"] else 0
        b += 2 * T * R if case["act"] != "none" else 0
        return {"bytes": b, "flops": 4 * T * K * R}
    n = sum(int(s) for s in case["sizes"].split(","))
    state = 8 if case["state"] == "f32" else 2 + 8 / 128
    # BF16 weights with FP32 master weights are written, and only the master weights read
    p = 8 if case["p"] == "f32" else 2 + 8 if case["master"] else 4
    return {"bytes": int(n * (2 * state + p + 4)), "flops": 16 * n}


# ------------------------------------------------------------------- inputs
def _e4m3(v):
    """A state of 8 bits: E4M3 codes of |v| <= 448 s and the scales s of 128 elements each."""
    b = torch.nn.functional.pad(v, (0, -v.numel() % 128)).view(-1, 128)
    amax = b.abs().amax(1)
    s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    q = (b / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(-1)[:v.numel()].clone(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def typed(v, name):
        return v.to(torch.bfloat16) if name == "bf16" else v

    st, op = {"case": case}, case["op"]
    if op in ("select", "select_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        # popular and unpopular experts; a bias that has begun to even them out
        popular = randn(E)
        st["logits"] = 1.2 * randn(T, E) + popular
        if op == "select":
            spread = 0.1 if case["scoring"] == "sigmoid" else 0.2 / E
            st["bias"] = spread * (randn(E) - popular) if case["bias"] else None
        else:
            st["topk_ids"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
            st["dweights"] = 1e-2 * randn(T, k)
    elif op in ("linear", "linear_bwd"):
        T, K, N, R = case["T"], case["K"], case["N"], _rows(case)
        st["x"] = randn(T, K).to(torch.bfloat16)
        st["w"] = (randn(R, K) / math.sqrt(K)).to(torch.bfloat16)
        if op == "linear":
            st["bias"] = 0.1 * randn(R) if case["bias"] else None
            st["residual"] = randn(T, N).to(torch.bfloat16) if case["residual"] else None
        else:
            st["pre"] = randn(T, R).to(torch.bfloat16) if case["act"] != "none" else None
            st["dy"] = typed(1e-2 * randn(T, N), case["dy"])
    else:
        sizes = [int(s) for s in case["sizes"].split(",")]
        pdt = torch.bfloat16 if case["p"] == "bf16" else torch.float32
        st["params"], st["grads"], st["masters"], st["states"] = [], [], [], []
        # the tensors of each kind lie in one buffer, as a program keeps them that reduces or saves them at once
        pad = [-(-s // 128) * 128 for s in sizes]
        total = sum(pad)
        st["flat_p"] = torch.zeros(total, dtype=pdt, device="cuda")
        st["flat_master"] = torch.zeros(total, device="cuda") if case["master"] and case["p"] == "bf16" else None
        f8 = case["state"] == "fp8"
        for name in ("m", "v"):
            st["flat_" + name] = torch.zeros(total, dtype=torch.uint8 if f8 else torch.float32, device="cuda")
            st["flat_%s_scales" % name] = torch.ones(total // 128, device="cuda") if f8 else None
        grads = torch.empty(total, device="cuda")
        at = 0
        for i, (n, room) in enumerate(zip(sizes, pad)):
            # gradients of different scale from tensor to tensor and from row to row
            rows = (1 + randn(-(-n // 1024)).abs()).repeat_interleave(1024)[:n] * 10.0 ** (-4 + i % 3)
            w = 0.02 * randn(n)
            st["flat_p"][at:at + n] = w
            st["params"].append(st["flat_p"][at:at + n])
            if st["flat_master"] is not None:
                st["flat_master"][at:at + n] = w
            st["masters"].append(st["flat_master"][at:at + n] if st["flat_master"] is not None else None)
            grads[at:at + n] = rows * randn(n)
            st["grads"].append(grads[at:at + n])
            m, root = 0.3 * rows * randn(n), rows * (0.7 + 0.2 * randn(n)).abs()
            s = {}
            for name, v in (("m", m), ("v", root if f8 else root * root)):
                part = st["flat_" + name][at:at + n]
                s[name] = part
                if f8:
                    sc = st["flat_%s_scales" % name][at // 128:(at + room) // 128]
                    codes, scales = _e4m3(v)
                    part.copy_(codes)
                    sc.copy_(scales)
                    s[name + "_scales"] = sc
                else:
                    part.copy_(v)
            st["states"].append(s)
            at += room
        st["decay"] = [DECAY if n >= 4096 else 0.0 for n in sizes]
        st["seed"] = seed & 0xFFFFFFFF
        st["count"] = COUNT
    return st


# --------------------------------------------------------------- the passes
def _opts(case):
    return dict(scoring=case["scoring"], renormalize=case["renorm"], scale=SCALE)


def _adamw_outputs(st):
    """What a step wrote: weights, and states as the numbers they stand for (8 bits: in units of their scales)."""
    out = [st["flat_p"]] + ([st["flat_master"]] if st["flat_master"] is not None else [])
    for name in ("m", "v"):
        if st["flat_%s_scales" % name] is None:
            out.append(st["flat_" + name])
        else:
            out += [st["flat_" + name].view(torch.float8_e4m3fn), st["flat_%s_scales" % name]]
    return out


def run(st):
    case = st["case"]
    if own:
        from moe_layer_router_amd import layer
        if case["op"] == "select":
            r = layer.select_experts(st["logits"], case["k"], bias=st["bias"], n_group=case["groups"], topk_group=case["keep"],
                                     group_top=case["top"], **_opts(case))
            return [r["topk_ids"], r["topk_weights"]]
        if case["op"] == "select_bwd":
            return [layer.select_experts_backward(st["logits"], st["topk_ids"], st["dweights"], **_opts(case))]
        if case["op"] == "linear":
            r = layer.linear(st["x"], st["w"], bias=st["bias"], act=case["act"], residual=st["residual"], out_dtype=case["y"],
                             pre_dtype="bf16" if case["pre"] else None)
            return [r["y"], r["pre"]] if case["pre"] else [r["y"]]
        if case["op"] == "linear_bwd":
            r = layer.linear_backward(st["x"], st["w"], st["dy"], act=case["act"], pre=st["pre"], dx_dtype=case["dx"], want_dbias=case["bias"])
            return [r["dx"], r["dw"], r["dbias"]] if case["bias"] else [r["dx"], r["dw"]]
        if "optimizer" not in st:
            st["optimizer"] = layer.AdamW(st["params"], masters=st["masters"] if st["flat_master"] is not None else None, states=st["states"],
                                          betas=BETAS, eps=EPS, weight_decay=st["decay"], seed=st["seed"], count=st["count"])
        st["optimizer"].step(st["grads"], lr=LR)
        return _adamw_outputs(st)
    return {"select": _select, "select_bwd": _select_bwd, "linear": _linear, "linear_bwd": _linear_bwd, "adamw": _adamw}[case["op"]](st)


def _scores(l, scoring):
    if scoring == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _select(st):
    # (64 bits: two experts' scores and a bias may lie close to each other)
    case, l = st["case"], st["logits"]
    T, E = l.shape
    s = _scores(l.double(), case["scoring"])
    c = s if st["bias"] is None else s + st["bias"].double()
    # without a bias the experts' scores are ordered as their logits are
    key = l.double() if st["bias"] is None else c
    if case["groups"] > 1:
        of = c.view(T, case["groups"], -1)
        best = torch.sort(of, dim=2, descending=True).values[:, :, :case["top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        mask = torch.zeros(T, case["groups"], dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = torch.where(mask.repeat_interleave(E // case["groups"], 1), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [ids.to(torch.int32), (SCALE * w).float()]


def _select_bwd(st):
    # (64 bits: dw - sum q dw, and 1 - s of a sure expert, cancel)
    case, l, ids = st["case"], st["logits"], st["topk_ids"].long()
    s = _scores(l.double(), case["scoring"])
    d = SCALE * st["dweights"].double()
    if case["renorm"]:
        z = s.gather(1, ids)
        q = z / z.sum(1, keepdim=True)
        d = (d - (q * d).sum(1, keepdim=True)) / z.sum(1, keepdim=True)
    ds = torch.zeros_like(s).scatter_(1, ids, d)
    if case["scoring"] == "sigmoid":
        return [(ds * s * (1.0 - s)).float()]
    return [(s * (ds - (s * ds).sum(1, keepdim=True))).float()]


def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = 2.0 * math.sqrt(2.0 / math.pi)
        p = 1.0 / (1.0 + torch.exp(-a * (z + 0.044715 * z * z * z)))
        return p + z * p * (1.0 - p) * a * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _linear(st):
    case = st["case"]
    z = torch.matmul(st["x"].float(), st["w"].float().t())
    if st["bias"] is not None:
        z = z + st["bias"]
    n = case["N"]
    y = _act(z[:, :n], "silu") * z[:, n:] if case["act"] == "swiglu" else _act(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    y = y.to(torch.bfloat16) if case["y"] == "bf16" else y
    return [y, z.to(torch.bfloat16)] if case["pre"] else [y]


def _linear_bwd(st):
    case, dy = st["case"], st["dy"].float()
    n = case["N"]
    if case["act"] == "swiglu":
        g, u = st["pre"][:, :n].float(), st["pre"][:, n:].float()
        dz = torch.cat([dy * u * _act_grad(g, "silu"), dy * _act(g, "silu")], 1)
    else:
        dz = dy if case["act"] == "none" else dy * _act_grad(st["pre"].float(), case["act"])
    dx = torch.matmul(dz, st["w"].float())
    dw = torch.matmul(dz.t(), st["x"].float())
    out = [dx.to(torch.bfloat16) if case["dx"] == "bf16" else dx, dw]
    return out + [dz.sum(0)] if case["bias"] else out


def _mix(x):
    """A 32-bit hash (of an int, or of an int32 tensor whose products wrap round)."""
    if isinstance(x, int):
        x ^= x >> 15
        x = x * 0x6A09E667 & 0xFFFFFFFF
        x ^= x >> 13
        x = x * 0xBB67AE85 & 0xFFFFFFFF
        return x ^ x >> 16
    x = x ^ ((x >> 15) & 0x1FFFF)
    x = x * 0x6A09E667
    x = x ^ ((x >> 13) & 0x7FFFF)
    x = x * (0xBB67AE85 - (1 << 32))
    return x ^ ((x >> 16) & 0xFFFF)


def _dice(n, key, device):
    """16 random bits for the first moment, the second one and the weight of each of n elements."""
    i = torch.arange(n, dtype=torch.int32, device=device)
    h = _mix(i * (0x9E3779B1 - (1 << 32)) + (key - (1 << 32) if key >= 1 << 31 else key))
    return h & 0xFFFF, (h >> 16) & 0xFFFF, (h * 0x3C6EF373 >> 16) & 0xFFFF


def _to_e4m3(v, dice):
    """Codes and scales of v, rounded up as often as the dropped part says."""
    n = v.numel()
    b = torch.nn.functional.pad(v, (0, -n % 128)).view(-1, 128)
    amax = b.abs().amax(1)
    s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    x = (b * (1.0 / s)[:, None]).view(-1)[:n].clamp(-E4M3_MAX, E4M3_MAX)
    a = x.abs()
    normal = ((a.view(torch.int32) + (dice << 4)) & -(1 << 20)).view(torch.float32)
    small = torch.floor(a * 512.0 + dice.float() / 65536.0) / 512.0
    return torch.copysign(torch.where(a < 2.0 ** -6, small, normal), x), s


def _adamw(st):
    case = st["case"]
    st["count"] += 1
    t = st["count"]
    c1, c2 = 1.0 - BETAS[0] ** t, 1.0 - BETAS[1] ** t
    call = _mix(st["seed"] ^ (t * 0x9E3779B9 & 0xFFFFFFFF))
    for i, (p, g, master, s) in enumerate(zip(st["params"], st["grads"], st["masters"], st["states"])):
        f8 = "m_scales" in s
        n = p.numel()
        # what is held in fewer bits is rounded stochastically
        rounds = f8 or (master is None and case["p"] == "bf16")
        dice = _dice(n, _mix(call + i * 0xA54FF53B & 0xFFFFFFFF), p.device) if rounds else None
        w = p.float() if master is None else master
        if f8:
            m = s["m"].view(torch.float8_e4m3fn).float() * s["m_scales"].repeat_interleave(128)[:n]
            root = s["v"].view(torch.float8_e4m3fn).float() * s["v_scales"].repeat_interleave(128)[:n]
            v = root * root
        else:
            m, v = s["m"], s["v"]
        m = BETAS[0] * m + (1.0 - BETAS[0]) * g
        v = BETAS[1] * v + (1.0 - BETAS[1]) * (g * g)
        w = w * (1.0 - LR * st["decay"][i]) - (LR / c1) * m / (torch.sqrt(v) / math.sqrt(c2) + EPS)
        if f8:
            codes, scales = _to_e4m3(m, dice[0])
            s["m"].copy_(codes.to(torch.float8_e4m3fn).view(torch.uint8))
            s["m_scales"].copy_(scales)
            root = torch.sqrt(v)
            codes, scales = _to_e4m3(root, dice[1])
            codes = torch.where(root > 0, codes.clamp(min=2.0 ** -9), codes)      # never zero where the root is not
            s["v"].copy_(codes.to(torch.float8_e4m3fn).view(torch.uint8))
            s["v_scales"].copy_(scales)
        else:
            m, v = s["m"].copy_(m), s["v"].copy_(v)
        if master is not None:
            master.copy_(w)
            p.copy_(w.to(torch.bfloat16))
        elif case["p"] == "bf16":
            p.copy_(((w.contiguous().view(torch.int32) + dice[2]) & -(1 << 16)).view(torch.float32))
        else:
            p.copy_(w)
    return _adamw_outputs(st)


# ------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op in ("select", "select_bwd"):
        l = st["logits"].double()
        s = torch.sigmoid(l) if case["scoring"] == "sigmoid" else torch.softmax(l, 1)
        if op == "select":
            E, G = case["E"], case["groups"]
            choice = s + (st["bias"].double() if case["bias"] else 0.0)
            order = choice if case["bias"] else l
            if G > 1:
                tops = torch.topk(choice.reshape(case["T"], G, E // G), min(case["top"], E // G), dim=2).values.sum(2)
                worst = torch.topk(tops, case["keep"], dim=1).values[:, -1:]
                order = order.masked_fill((tops < worst).repeat_interleave(E // G, 1), -math.inf)
            picked = s.gather(1, torch.topk(order, case["k"], dim=1).indices)
            if case["renorm"]:
                picked = picked / picked.sum(1)[:, None]
            return [None, SCALE * picked]
        # the derivative of sum(dw * w) by each selected score, then of the score by the logits
        ids, dw = st["topk_ids"].long(), st["dweights"].double()
        z = s.gather(1, ids)
        if case["renorm"]:
            total = z.sum(1)[:, None]
            by = SCALE * (dw / total - (dw * z).sum(1)[:, None] / total ** 2)
        else:
            by = SCALE * dw
        if case["scoring"] == "sigmoid":
            return [torch.zeros_like(l).scatter(1, ids, by * z * torch.sigmoid(-l).gather(1, ids))]
        inner = torch.linalg.vecdot(by, z)[:, None]
        return [(-s * inner).scatter_add(1, ids, by * z)]
    if op == "linear":
        n = case["N"]
        pre = torch.nn.functional.linear(st["x"].double(), st["w"].double(), None if st["bias"] is None else st["bias"].double())
        y = _exact_act(pre, case["act"], n)
        if case["residual"]:
            y = y + st["residual"].double()
        return [y, pre] if case["pre"] else [y]
    if op == "linear_bwd":
        dy = st["dy"].double()
        if case["act"] == "none":
            dz = dy
        else:
            pre = st["pre"].double().requires_grad_()
            with torch.enable_grad():
                dz, = torch.autograd.grad(_exact_act(pre, case["act"], case["N"]), pre, dy)
        out = [dz @ st["w"].double(), dz.t().contiguous() @ st["x"].double()]
        return out + [torch.ones(1, case["T"], dtype=torch.float64, device="cuda").matmul(dz)[0]] if case["bias"] else out
    t = COUNT + 1
    p = torch.zeros(st["flat_p"].numel(), dtype=torch.float64, device="cuda")
    m, v, ms, vs = p.clone(), p.clone(), [], []
    at = 0
    for i, g in enumerate(st["grads"]):
        n, s = g.numel(), st["states"][i]
        here = slice(at, at + n)
        at += -(-n // 128) * 128
        old = (st["params"] if st["masters"][i] is None else st["masters"])[i].double()
        if case["state"] == "fp8":
            wide = [torch.nn.functional.pad(s[k].view(torch.float8_e4m3fn).double(), (0, -n % 128)).view(-1, 128) * s[k + "_scales"].double()[:, None]
                    for k in ("m", "v")]
            m0, v0 = wide[0].reshape(-1)[:n], wide[1].reshape(-1)[:n] ** 2
        else:
            m0, v0 = s["m"].double(), s["v"].double()
        m[here] = torch.lerp(g.double(), m0, BETAS[0])
        v[here] = torch.lerp(g.double() ** 2, v0, BETAS[1])
        mhat, vhat = m[here] / (1 - BETAS[0] ** t), v[here] / (1 - BETAS[1] ** t)
        p[here] = old - LR * (mhat / (vhat ** 0.5 + EPS) + st["decay"][i] * old)
    out = [p] * (2 if st["flat_master"] is not None else 1)
    if case["state"] == "f32":
        return out + [m, v]
    for x in (m, v ** 0.5):
        amax = x.reshape(-1, 128).abs().max(1).values
        out += [None, torch.where(amax == 0, 1.0, amax / E4M3_MAX)]
    return out


def _exact_act(z, act, n):
    f = torch.nn.functional
    if act == "swiglu":
        return f.silu(z[:, :n]) * z[:, n:]
    return {"none": lambda v: v, "relu": torch.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"), "silu": f.silu}[act](z)

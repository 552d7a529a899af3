"""Workloads of the training and serving operators around the MoE layer: the
router's balance loss with its gradient, layer norm in front of the layer
(forward and backward), and the Newton-Schulz orthogonalisation of a weight
matrix's update.  `run` computes a case in plain torch, or, with `own` set,
through `moe_layer_router_amd.layer`."""

import math

import torch

own = False

E4M3_MAX = 448.0
NS_COEFFS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
LN_EPS = 1e-5
ALPHA = 1e-2


def listed():
    return [
        # the balance loss of a tiny layer's batch: latency counts
        dict(name="balance_tiny", op="balance", T=64, E=8, k=2, S=1, mask=False, grad=True),
        # a prefill-sized training batch of 256 experts, one balance loss over the whole batch
        dict(name="balance_prefill", op="balance", T=8192, E=256, k=8, S=1, mask=False, grad=True),
        # 1024 experts, a loss per packed sequence, padding tokens masked
        dict(name="balance_e1024_seqs", op="balance", T=16384, E=1024, k=16, S=13, mask=True, grad=True),
        # one decoded token: normalise and quantise the layer's FP8 input
        dict(name="ln_token_fp8", op="ln", T=1, H=7168, x="bf16", y="fp8"),
        # the layer's input in a training step, with the statistics the backward pass reads
        dict(name="ln_prefill", op="ln", T=8192, H=7168, x="bf16", y="bf16"),
        # a ragged batch of a small layer
        dict(name="ln_bwd_small", op="ln_bwd", T=300, H=384, x="f32", dy="bf16"),
        # the training step's backward: fp32 gradient of the layer's input
        dict(name="ln_bwd_prefill", op="ln_bwd", T=8192, H=7168, x="bf16", dy="f32"),
        # the experts' gate|up updates of a tiny layer
        dict(name="orth_tiny", op="orth", B=8, M=256, N=256, x="f32"),
        # odd matrices
        dict(name="orth_odd", op="orth", B=3, M=200, N=333, x="f32"),
        # the router's update: one wide matrix
        dict(name="orth_router", op="orth", B=1, M=256, N=7168, x="f32"),
        # down projections of four experts (tall), BF16 momentum
        dict(name="orth_down", op="orth", B=4, M=7168, N=2048, x="bf16"),
        # gate and up projections of four experts
        dict(name="orth_gate_up", op="orth", B=8, M=2048, N=7168, x="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "ln", "ln_bwd", "orth"])
    if op == "balance":
        E = _log_int(rng, 2, 1024)
        k = rng.randint(1, min(16, E))
        T = _log_int(rng, 1, 16384)
        S = min(T, _log_int(rng, 1, 64))
        return dict(op=op, T=T, E=E, k=k, S=S, mask=rng.random() < 0.5, grad=rng.random() < 0.8)
    if op in ("ln", "ln_bwd"):
        H = 128 * _log_int(rng, 1, 128)
        T = _log_int(rng, 1, min(16384, 8192 * 7168 // H))
        c = dict(op=op, T=T, H=H, x=rng.choice(["bf16", "f32"]))
        if op == "ln":
            c["y"] = rng.choice(["bf16", "f32", "fp8"])
        else:
            c["dy"] = rng.choice(["bf16", "f32"])
        return c
    big = max(work(c)["flops"] for c in listed())
    while True:
        c = dict(op=op, B=_log_int(rng, 1, 64), M=_log_int(rng, 8, 7168), N=_log_int(rng, 8, 7168),
                 x=rng.choice(["bf16", "f32"]))
        if work(c)["flops"] <= big and c["B"] * c["M"] * c["N"] <= 8 * 2048 * 7168:
            return c


def work(case):
    op = case["op"]
    if op == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        b = 4 * T * E * (2 if case["grad"] else 1) + 4 * T * k + 8 * S * E + 4 * (S + 1) + (T if case["mask"] else 0)
        return {"bytes": b, "flops": T * E * (10 if case["grad"] else 5)}
    if op == "ln":
        T, H = case["T"], case["H"]
        out = {"bf16": 2, "f32": 4, "fp8": 1 + 4 / 128}[case["y"]]
        return {"bytes": T * H * ((2 if case["x"] == "bf16" else 4) + out) + 8 * H + 8 * T, "flops": 8 * T * H}
    if op == "ln_bwd":
        T, H = case["T"], case["H"]
        size = {"bf16": 2, "f32": 4}
        return {"bytes": T * H * (size[case["x"]] + size[case["dy"]] + 4) + 12 * H + 8 * T, "flops": 14 * T * H}
    m, n = sorted((case["M"], case["N"]))
    # per step: X X^T and A A (symmetric: half of the products), then B X
    return {"bytes": case["B"] * m * n * ((2 if case["x"] == "bf16" else 4) + 2),
            "flops": case["B"] * NS_STEPS * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)}


# ------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def typed(v, name):
        return v.to(torch.bfloat16) if name == "bf16" else v

    st = {"case": case}
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        # popular and unpopular experts, as a router meets them in training
        st["logits"] = 1.5 * randn(T, E) + randn(E)
        st["topk_ids"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        # packed sequences of ragged lengths; behind them up to an eighth of the rows belongs to none
        last = T - T // 8 if case["mask"] else T
        cuts = torch.rand(S - 1, generator=g, device="cuda").mul(last).long().sort().values
        ends = torch.tensor([last], device="cuda")
        st["seq_offsets"] = torch.cat([ends * 0, cuts, ends]).to(torch.int32)
        st["token_mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9) if case["mask"] else None
    elif case["op"] in ("ln", "ln_bwd"):
        T, H = case["T"], case["H"]
        # a residual stream: rows of different scale, a few strong channels
        x = randn(T, H) * (1 + randn(T, 1).abs()) * (1 + 4 * (torch.rand(H, generator=g, device="cuda") < 0.01)) + 0.2 * randn(H)
        st["x"] = typed(x, case["x"])
        st["gamma"] = 1 + 0.1 * randn(H)
        st["beta"] = 0.1 * randn(H)
        if case["op"] == "ln_bwd":
            xf = st["x"].double()
            mean = xf.mean(1)
            st["mean"] = mean.float()
            st["rstd"] = ((xf - mean[:, None]).square().mean(1) + LN_EPS).rsqrt().float()
            st["dy"] = typed(1e-2 * randn(T, H), case["dy"])
    else:
        B, M, N = case["B"], case["M"], case["N"]
        # a gradient: a decaying low-rank part and noise
        r = max(1, min(M, N) // 16)
        decay = torch.arange(1, r + 1, device="cuda").float().rsqrt()
        low = torch.matmul(randn(B, M, r) * decay, randn(B, r, N))
        st["u"] = typed(1e-3 * (low + 0.5 * randn(B, M, N)), case["x"])
    return st


# --------------------------------------------------------------- the passes
def run(st):
    case = st["case"]
    if own:
        from moe_layer_router_amd import layer
        if case["op"] == "balance":
            r = layer.balance_loss(st["logits"], st["topk_ids"], alpha=ALPHA, seq_offsets=st["seq_offsets"],
                                   token_mask=st["token_mask"], want_grad=case["grad"])
            return [r["loss"], r["counts"], r["probs"], r["dlogits"]] if case["grad"] else [r["loss"], r["counts"], r["probs"]]
        if case["op"] == "ln":
            r = layer.layer_norm(st["x"], st["gamma"], st["beta"], eps=LN_EPS, out_dtype=case["y"], want_stats=True)
            if case["y"] == "fp8":
                # the E4M3 codes as the numbers they stand for, in units of their scales
                return [r["y"].view(torch.float8_e4m3fn).to(torch.bfloat16), r["y_scales"], r["mean"], r["rstd"]]
            return [r["y"], r["mean"], r["rstd"]]
        if case["op"] == "ln_bwd":
            r = layer.layer_norm_backward(st["x"], st["gamma"], st["mean"], st["rstd"], st["dy"])
            return [r["dx"], r["dgamma"], r["dbeta"]]
        return [layer.orthogonalize(st["u"], steps=NS_STEPS, eps=NS_EPS)]
    return {"balance": _balance, "ln": _ln, "ln_bwd": _ln_bwd, "orth": _orth}[case["op"]](st)


def _balance(st):
    l, ids, off, mask, case = st["logits"], st["topk_ids"].long(), st["seq_offsets"].long(), st["token_mask"], st["case"]
    (T, E), k, S = l.shape, ids.shape[1], case["S"]
    t = torch.arange(T, device=l.device)
    member = (t >= off[:-1, None]) & (t < off[1:, None])                    # [S, T]
    if mask is not None:
        member = member & mask
    valid = member.any(0)
    seq = member.int().argmax(0)
    n = member.sum(1)                                                       # tokens of each sequence
    hits = torch.zeros(S, E, dtype=torch.int32, device=l.device)
    ones = valid[:, None].expand(T, k).to(torch.int32).reshape(-1)
    hits.view(-1).index_add_(0, (seq[:, None] * E + ids).reshape(-1), ones)
    e = torch.exp(l - l.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True)
    nf = n.clamp(min=1).float()[:, None]
    probs = torch.matmul(member.float(), p) / nf
    f = hits.float() * (E / k) / nf
    used = (n > 0).sum().clamp(min=1).float()
    loss = (ALPHA * (f * probs).sum() / used).reshape(1)
    if not case["grad"]:
        return [loss, hits, probs]
    g = (ALPHA * f / nf / used)[seq]
    # relative to the likeliest expert's: sum_i p_i (g_e - g_i) without cancellation
    g = g - g.gather(1, l.argmax(1, keepdim=True))
    d = p * (g - (p * g).sum(1, keepdim=True))
    return [loss, hits, probs, torch.where(valid[:, None], d, torch.zeros_like(d))]


def _ln(st):
    x, case = st["x"].float(), st["case"]
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + LN_EPS)
    y = d * rstd * st["gamma"] + st["beta"]
    if case["y"] == "fp8":
        T, H = y.shape
        b = y.view(T, H // 128, 128)
        amax = b.abs().amax(2)
        s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
        q = (b * (1.0 / s)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return [q.view(T, H).to(torch.bfloat16), s, mean[:, 0], rstd[:, 0]]
    return [y.to(torch.bfloat16) if case["y"] == "bf16" else y, mean[:, 0], rstd[:, 0]]


def _ln_bwd(st):
    x, dy = st["x"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    xhat = (x - st["mean"][:, None]) * rstd
    g = dy * st["gamma"]
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return [dx, (dy * xhat).sum(0), dy.sum(0)]


def _orth(st):
    u = st["u"].float()
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2).contiguous() if tall else u
    x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NS_EPS)
    a, b, c = NS_COEFFS
    for _ in range(NS_STEPS):
        gram = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * gram + c * torch.matmul(gram, gram), x)
    return [(x.transpose(1, 2).contiguous() if tall else x).to(torch.bfloat16)]


# ------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["S"]
        p = torch.softmax(st["logits"].double(), 1)
        ids = st["topk_ids"].long()
        off = st["seq_offsets"].tolist()
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["token_mask"] is None else st["token_mask"]
        counts = torch.zeros(S, E, dtype=torch.int32, device="cuda")
        probs = torch.zeros(S, E, dtype=torch.float64, device="cuda")
        grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        rows = [off[s] + keep[off[s]:off[s + 1]].nonzero()[:, 0] for s in range(S)]
        used = max(1, sum(r.numel() > 0 for r in rows))
        loss = 0.0
        for s, r in enumerate(rows):
            if r.numel() == 0:
                continue
            counts[s] = torch.bincount(ids[r].reshape(-1), minlength=E).to(torch.int32)
            probs[s] = p[r].mean(0)
            f = counts[s].double() * E / (k * r.numel())
            loss = loss + (f * probs[s]).sum()
            g = ALPHA / used * f / r.numel()
            g = g - g[p[r].max(1).indices][:, None]           # (a token's gradient knows differences of g alone)
            grad[r] = p[r] * (g - (p[r] * g).sum(1)[:, None])
        loss = torch.as_tensor(loss, dtype=torch.float64, device="cuda").reshape(1) * ALPHA / used
        return [loss, None, probs, grad] if case["grad"] else [loss, None, probs]
    if case["op"] in ("ln", "ln_bwd"):
        x, gamma = st["x"].double(), st["gamma"].double()
        if case["op"] == "ln":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + LN_EPS) ** -0.5
            y = gamma * (x - mean[:, None]) * rstd[:, None] + st["beta"].double()
            if case["y"] == "fp8":
                amax = y.abs().reshape(case["T"], -1, 128).amax(2)
                return [None, torch.where(amax == 0, 1.0, amax / 448), mean, rstd]
            return [y, mean, rstd]
        dy, mean, rstd = st["dy"].double(), st["mean"].double(), st["rstd"].double()
        z = (x - mean[:, None]) * rstd[:, None]
        h = case["H"]
        gy = gamma * dy
        dx = rstd[:, None] / h * (h * gy - gy.sum(1)[:, None] - z * (z * gy).sum(1)[:, None])
        return [dx, torch.linalg.vecdot(dy, z, dim=0), dy.sum(0)]
    u = st["u"].double()
    y = u / (torch.linalg.matrix_norm(u)[:, None, None] + NS_EPS)
    if case["M"] > case["N"]:
        y = y.mT.contiguous()
    a, b, c = NS_COEFFS
    for _ in range(NS_STEPS):
        w = y @ y.mT
        wy = w @ y
        y = a * y + b * wy + c * (w @ wy)
    return [y.mT.contiguous() if case["M"] > case["N"] else y]

"""Workloads of the operators of a whole block, each in two forms.

* ``layer``: a whole mixture-of-experts layer for a few tokens: the router's choice, the chosen
  experts' gated feed-forward and the weighted sum, in bf16 or with 8-bit rows and gate/up weights.
* ``block_norm`` and its gradient: the norm of a block's output, its gate, the scaled residual and
  the norm before the next block, with an 8-bit output (e4m3, one scale a row) for the next layer.

With ``own`` false ``run`` computes the plain form from elementary torch operations in 32 bits; with
``own`` true it calls the package.  ``exact`` evaluates the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
SCALING = 2.5       # the routed scaling of the layers with sigmoid scores


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token through 8 of 128 experts: latency
        dict(name="layer_token", op="layer", N=1, E=128, K=8, H=2048, I=768, bits=16, scoring="softmax", groups=1),
        # one new token through 2 of 8 wide experts
        dict(name="layer_token_wide", op="layer", N=1, E=8, K=2, H=4096, I=4096, bits=16, scoring="softmax", groups=1),
        # three sequences at the widest hidden size, group-limited routing, 8-bit rows and weights
        dict(name="layer_few_8bit", op="layer", N=3, E=256, K=8, H=7168, I=1024, bits=8, scoring="sigmoid", groups=8),
        # a small model's batch, sizes that fill no tile, scores that are not normalised
        dict(name="layer_odd", op="layer", N=17, E=60, K=4, H=1000, I=712, bits=16, scoring="sigmoid", groups=1,
             renormalize=False),
        # a decoding batch over few wide experts: the most rows an expert
        dict(name="layer_batch_wide", op="layer", N=32, E=8, K=2, H=4096, I=4096, bits=16, scoring="softmax", groups=1),
        # a decoding batch whose tokens reach nearly every expert: the largest layer
        dict(name="layer_batch", op="layer", N=61, E=64, K=6, H=4096, I=1280, bits=16, scoring="softmax", groups=1),
        # between two blocks of a decoding step of a handful of sequences: latency
        dict(name="between_decode_8bit", op="block_norm", N=4, H=2048, residual="bf16", gate="none", quantize=True),
        # between two blocks of a long prompt at the widest hidden size, a gate for each token
        dict(name="between_prompt_8bit", op="block_norm", N=8192, H=7168, residual="bf16", gate="token", quantize=True),
        # a training step's forward pass: residual stream in 32 bits, a gate for each element
        dict(name="between_train", op="block_norm", N=16384, H=4096, residual="fp32", gate="full", quantize=False),
        # the gradient of a small batch, odd sizes
        dict(name="between_backward_small", op="block_norm_backward", N=333, H=1000, residual="bf16", gate="token"),
        # the gradient in a training step, a gate for each token, residual stream in 32 bits
        dict(name="between_backward_fp32", op="block_norm_backward", N=16384, H=4096, residual="fp32", gate="token"),
        # the gradient at the widest hidden size, a gate for each element
        dict(name="between_backward_wide", op="block_norm_backward", N=8192, H=7168, residual="bf16", gate="full"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["layer", "layer", "block_norm", "block_norm_backward"])
        if op == "layer":
            bits = rng.choice([16, 16, 8])
            scoring = rng.choice(["softmax", "sigmoid"])
            E = rng.choice([4, 8, 16, 32, 60, 64, 128, 256])
            case = dict(op=op, N=_log_int(rng, 1, 64), E=E, K=min(rng.choice([1, 2, 4, 6, 8]), E),
                        H=_log_int(rng, 128, 7168, 16 if bits == 8 else 8), I=_log_int(rng, 64, 4096, 8), bits=bits,
                        scoring=scoring, groups=1, renormalize=rng.random() < 0.7)
            if scoring == "sigmoid" and E >= 64 and E % 8 == 0 and rng.random() < 0.5:
                case["groups"] = 8
            if E * case["H"] * case["I"] > 256 * 7168 * 1024:
                continue
        else:
            case = dict(op=op, N=_log_int(rng, 1, 32768), H=_log_int(rng, 128, 8192, 8),
                        residual=rng.choice(["bf16", "fp32"]), gate=rng.choice(["none", "token", "full"]))
            if op == "block_norm":
                case["quantize"] = rng.random() < 0.6
            if case["N"] * case["H"] > 16384 * 4096:
                continue
        if work(case)["bytes"] <= most:
            return case


def work(case):
    N, H, op = case["N"], case["H"], case["op"]
    if op == "layer":
        E, K, I = case["E"], case["K"], case["I"]  # noqa: E741
        b = case["bits"] // 8
        # experts that at least one token reaches, for evenly spread tokens
        used = E * (1 - (1 - K / E) ** N)
        return {"bytes": used * H * I * (2 * b + 2) + N * (H * (b + 2) + 4 * E), "flops": 6 * N * K * H * I}
    res = 2 if case["residual"] == "bf16" else 4
    full = 2 if case["gate"] == "full" else 0
    if op == "block_norm":
        row = 2 + res + full + res + 2 + (1 if case["quantize"] else 0)
        return {"bytes": N * (H * row + 12) + 4 * H, "flops": 12 * N * H}
    # dy, x, the stored sum and its gradient come in, the gradients of x, the residual and the gate go out
    row = 2 + 2 + 2 * res + full + 2 + res + full
    return {"bytes": N * (H * row + 16) + 12 * H, "flops": 24 * N * H}


# ---------------------------------------------------------------- inputs
def _quantised(v):
    """e4m3 values and a scale for each last-axis row."""
    scale = v.abs().amax(-1).clamp_min(1e-12) / E4M3_MAX
    return (v / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    N, H, op = case["N"], case["H"], case["op"]
    bf16 = torch.bfloat16

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std

    s = {"case": case}
    if op == "layer":
        E, I = case["E"], case["I"]  # noqa: E741
        s["logits"] = normal(N, E)
        s["bias"] = (torch.rand(E, generator=gen, device=dev) - 0.5) * 0.2 if case["scoring"] == "sigmoid" else None
        x = normal(N, H)
        s["w_down"] = torch.empty(E, H, I, dtype=bf16, device=dev)
        if case["bits"] == 8:
            s["x"], s["x_scale"] = _quantised(x)
            s["w_gate_up"] = torch.empty(E, 2, I, H, dtype=torch.float8_e4m3fn, device=dev)
            s["w_scale"] = torch.empty(E, 2, I, device=dev)
        else:
            s["x"] = x.to(bf16)
            s["w_gate_up"] = torch.empty(E, 2, I, H, dtype=bf16, device=dev)
        for e in range(E):
            w = normal(2, I, H, std=H ** -0.5)
            if case["bits"] == 8:
                q, s["w_scale"][e] = _quantised(w)
                s["w_gate_up"][e].view(torch.uint8).copy_(q.view(torch.uint8))
            else:
                s["w_gate_up"][e] = w
            s["w_down"][e] = normal(H, I, std=I ** -0.5)
        return s

    kind = bf16 if case["residual"] == "bf16" else torch.float32
    size = torch.exp(normal(N, 1))       # rows of very different size
    s["post_weight"] = (1 + normal(H, std=0.1)).to(bf16)
    s["weight"] = (1 + normal(H, std=0.1)).to(bf16)
    s["x"] = (normal(N, H) * torch.exp(normal(N, 1))).to(bf16)
    s["scale"] = 0.75
    gate = case["gate"]
    s["gate"] = None if gate == "none" else torch.sigmoid(normal(N) if gate == "token" else normal(N, H))
    if gate == "full":
        s["gate"] = s["gate"].to(bf16)
    if op == "block_norm":
        s["residual"] = (normal(N, H) * size).to(kind)
    else:
        s["s"] = (normal(N, H) * size).to(kind)      # the forward pass kept the sum and the two roots
        s["rstd"] = torch.rsqrt(s["s"].float().square().mean(-1) + EPS)
        s["post_rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
        s["dy"] = normal(N, H).to(bf16)
        s["ds"] = normal(N, H).to(kind)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _routing(case):
    grouped = case["groups"] > 1
    return dict(scoring=case["scoring"], renormalize=case.get("renormalize", True), n_group=case["groups"],
                topk_group=case["groups"] // 2 if grouped else 1,
                routed_scaling=SCALING if case["scoring"] == "sigmoid" else 1.0)


def _run_own(s):
    import expert_dispatch_planning_gb300 as m
    case = s["case"]
    if case["op"] == "layer":
        return {"out": m.layer(s["x"], s["logits"], s["w_gate_up"], s["w_down"], case["K"], bias=s["bias"],
                               x_scale=s.get("x_scale"), w_scale=s.get("w_scale"), **_routing(case))}
    if case["op"] == "block_norm":
        o = m.block_norm(s["x"], s["residual"], s["post_weight"], s["weight"], gate=s["gate"],
                         residual_scale=s["scale"], eps=EPS, quantize=case["quantize"])
        return {"y": o.y, "residual": o.residual, "post_rstd": o.post_rstd, "rstd": o.rstd, "q": o.q,
                "q_scale": o.q_scale}
    dx, dres, dgate, dpost, dweight = m.block_norm_backward(
        s["dy"], s["x"], s["s"], s["post_weight"], s["weight"], s["post_rstd"], s["rstd"], gate=s["gate"],
        residual_scale=s["scale"], ds=s["ds"])
    return {"dx": dx, "dres": dres, "dgate": dgate, "dpost_weight": dpost, "dweight": dweight}


def _choice(case, logits, bias):
    """The router's choice (ties to the lower index) and its weights.  Selection is next to a border: 64 bits."""
    r = _routing(case)
    K = case["K"]
    v = logits.double()
    score = 1 / (1 + torch.exp(-v)) if r["scoring"] == "sigmoid" else v
    key = score if bias is None else score + bias.double()
    if r["n_group"] > 1:
        N, E = key.shape
        by_group = key.reshape(N, r["n_group"], -1)
        best = by_group.sort(dim=-1, descending=True).values[..., :2].sum(-1)
        kept = best.sort(dim=-1, descending=True, stable=True).indices[:, :r["topk_group"]]
        allowed = (kept[:, :, None] == torch.arange(r["n_group"], device=key.device)).any(1)
        key = torch.where(allowed[..., None], by_group, -math.inf).reshape(N, E)
    idx = key.sort(dim=-1, descending=True, stable=True).indices[:, :K]
    if r["scoring"] == "sigmoid":
        w = score.gather(1, idx)
        if r["renormalize"]:
            w = w / w.sum(-1, keepdim=True)
    else:
        top = torch.exp(score - score.amax(-1, keepdim=True))
        w = top.gather(1, idx)
        w = w / (w if r["renormalize"] else top).sum(-1, keepdim=True)
    return idx, (w * r["routed_scaling"]).float()


def _run_plain(s):
    case = s["case"]
    bf16 = torch.bfloat16
    if case["op"] == "layer":
        idx, w = _choice(case, s["logits"], s["bias"])
        N, K = idx.shape
        E, _, I, H = s["w_gate_up"].shape  # noqa: E741

        def taken(v, at):                   # the experts' weights in 32 bits
            if at is not None:
                v = v.view(torch.uint8)[at].view(v.dtype) if v.element_size() == 1 else v[at]
            return v.float()

        x = s["x"].float()
        if "x_scale" in s:
            x = x * s["x_scale"][:, None]
        # few pairs: each with its expert's weights; many: every expert with all tokens
        at = idx.reshape(-1) if N * K <= E else None
        xs = x[:, None, :].expand(N, K, H).reshape(N * K, 1, H) if at is not None else x.expand(E, N, H)
        wgu = taken(s["w_gate_up"], at)
        if "w_scale" in s:
            wgu = wgu * taken(s["w_scale"], at)[..., None]
        g, u = torch.bmm(xs, wgu.reshape(-1, 2 * I, H).transpose(1, 2)).split(I, dim=-1)
        h = g / (1 + torch.exp(-g)) * u
        y = torch.bmm(h, taken(s["w_down"], at).transpose(1, 2))
        if at is not None:
            return {"out": (y.reshape(N, K, H) * w[..., None]).sum(1).to(bf16)}
        y = y[idx, torch.arange(N, device=idx.device)[:, None]]
        return {"out": (y * w[..., None]).sum(1).to(bf16)}

    wp, w = s["post_weight"].float(), s["weight"].float()
    gate = None if s["gate"] is None else s["gate"].float()
    c = 1.0 if gate is None else gate[:, None] if gate.dim() == 1 else gate
    x = s["x"].float()
    if case["op"] == "block_norm":
        r = s["residual"]
        post_rstd = 1 / torch.sqrt(x.square().mean(-1) + EPS)
        v = s["scale"] * r.float() + c * (x * post_rstd[:, None] * wp)
        rstd = 1 / torch.sqrt(v.square().mean(-1) + EPS)
        out = v * rstd[:, None] * w
        q = q_scale = None
        if case["quantize"]:
            amax = out.abs().amax(-1)
            q_scale = torch.where(amax > 0, amax, 1.0) / E4M3_MAX
            q = (out / q_scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"y": out.to(bf16), "residual": v.to(r.dtype), "post_rstd": post_rstd, "rstd": rstd, "q": q,
                "q_scale": q_scale}
    v, dy = s["s"].float(), s["dy"].float()
    vhat, xhat = v * s["rstd"][:, None], x * s["post_rstd"][:, None]
    t = dy * w
    d = s["rstd"][:, None] * (t - vhat * (t * vhat).mean(-1, keepdim=True)) + s["ds"].float()
    e = d * c * wp
    dx = s["post_rstd"][:, None] * (e - xhat * (e * xhat).mean(-1, keepdim=True))
    dgate = None
    if gate is not None:
        dgate = d * (xhat * wp)
        dgate = dgate.sum(-1) if gate.dim() == 1 else dgate.to(bf16)
    return {"dx": dx.to(bf16), "dres": (s["scale"] * d).to(s["s"].dtype), "dgate": dgate,
            "dpost_weight": (d * c * xhat).sum(0), "dweight": (dy * vhat).sum(0)}


# ---------------------------------------------------------------- in 64 bits
def _exact_layer(case, s):
    """Token by token and expert by expert, from the definition."""
    N, E, K, H = case["N"], case["E"], case["K"], case["H"]
    r = _routing(case)
    out = torch.zeros(N, H, dtype=torch.float64, device="cuda")
    logits = s["logits"].double()
    bias = s["bias"].double().tolist() if s["bias"] is not None else [0.0] * E
    sigmoid = r["scoring"] == "sigmoid"
    score = torch.special.expit(logits) if sigmoid else torch.softmax(logits, dim=1)
    rank_by = (score if sigmoid else logits).tolist()
    score = score.tolist()
    chosen = {}
    for n in range(N):
        key = [v + b for v, b in zip(rank_by[n], bias)]
        open_to = range(E)
        if r["n_group"] > 1:
            size = E // r["n_group"]
            value = [sum(sorted(key[g * size:(g + 1) * size])[-2:]) for g in range(r["n_group"])]
            kept = sorted(range(r["n_group"]), key=lambda g: (-value[g], g))[:r["topk_group"]]
            open_to = [e for g in kept for e in range(g * size, (g + 1) * size)]
        top = sorted(open_to, key=lambda e: (-key[e], e))[:K]
        total = math.fsum(score[n][e] for e in top) if r["renormalize"] else 1.0
        for e in top:
            chosen.setdefault(e, []).append((n, r["routed_scaling"] * score[n][e] / total))
    for e, pairs in chosen.items():
        rows = torch.tensor([n for n, _ in pairs], device="cuda")
        x = s["x"].view(torch.uint8 if case["bits"] == 8 else torch.int16)[rows].view(s["x"].dtype).double()
        w = s["w_gate_up"][e].double()
        if case["bits"] == 8:
            x, w = x * s["x_scale"][rows].double()[:, None], w * s["w_scale"][e].double()[..., None]
        a = x @ w[0].T
        h = a * torch.special.expit(a) * (x @ w[1].T)
        share = torch.tensor([v for _, v in pairs], dtype=torch.float64, device="cuda")
        out[rows] += share[:, None] * (h @ s["w_down"][e].double().T)
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "layer":
        return _exact_layer(case, s)
    H = case["H"]
    x, wp, w, a = s["x"].double(), s["post_weight"].double(), s["weight"].double(), s["scale"]
    gate = torch.ones_like(x) if s["gate"] is None else s["gate"].double().reshape(x.shape[0], -1).expand_as(x)
    if case["op"] == "block_norm":
        post = (torch.linalg.vector_norm(x, dim=1).pow(2) / H + EPS).pow(-0.5)
        v = torch.einsum("nh,n,h,nh->nh", x, post, wp, gate) + a * s["residual"].double()
        rstd = (torch.linalg.vector_norm(v, dim=1).pow(2) / H + EPS).pow(-0.5)
        y = torch.einsum("nh,n,h->nh", v, rstd, w)
        q = scale = None
        if case["quantize"]:
            top = y.abs().max(dim=1).values
            scale = torch.where(top > 0, top, torch.ones_like(top)) / E4M3_MAX
            q = y / scale[:, None]
        return {"y": y, "residual": v, "post_rstd": post, "rstd": rstd, "q": q, "q_scale": scale}
    v, dy, r, p = s["s"].double(), s["dy"].double(), s["rstd"].double(), s["post_rstd"].double()
    along = torch.einsum("nh,h,nh->n", dy, w, v) * r.pow(3) / H
    d = torch.einsum("n,nh,h->nh", r, dy, w) - along[:, None] * v + s["ds"].double()
    down = d * gate
    along = torch.einsum("nh,h,nh->n", down, wp, x) * p.pow(3) / H
    dx = torch.einsum("n,nh,h->nh", p, down, wp) - along[:, None] * x
    dgate = None
    if case["gate"] == "token":
        dgate = torch.einsum("nh,nh,n,h->n", d, x, p, wp)
    elif case["gate"] == "full":
        dgate = torch.einsum("nh,nh,n,h->nh", d, x, p, wp)
    return {"dx": dx, "dres": a * d, "dgate": dgate, "dpost_weight": torch.einsum("nh,nh,n->h", down, x, p),
            "dweight": torch.einsum("nh,nh,n->h", dy, v, r)}

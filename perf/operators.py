"""Workloads of the operators around the routed experts, each in two forms.

* ``residual_norm`` and its gradient: root-mean-square norm with the residual's addition, with an
  8-bit output (e4m3, one scale a row) for the dispatch.
* ``expert_ffn`` and its gradient: the experts' gated feed-forward over the rows of a dispatch plan,
  in bf16 or with 8-bit rows and gate/up weights.
* ``combine_backward``: the gradient of the weighted combine.

With ``own`` false ``run`` computes the plain form from elementary torch operations in 32 bits; with
``own`` true it calls the package.  ``exact`` evaluates the definitions in 64 bits.
"""
import math
from types import SimpleNamespace

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step of a handful of sequences: latency
        dict(name="norm_decode_8bit", op="norm", N=4, H=2048, residual="bf16", quantize=True),
        # a long prompt at the widest hidden size: router reads bf16, the dispatch 8 bits
        dict(name="norm_prompt_8bit", op="norm", N=8192, H=7168, residual="bf16", quantize=True),
        # the norm's gradient in a training step, residual stream kept in 32 bits
        dict(name="norm_backward_fp32", op="norm_backward", N=16384, H=4096, residual="fp32"),
        # one new token through 8 of 128 experts: reads 8 experts' weights
        dict(name="ffn_token", op="ffn", N=1, E=128, K=8, H=2048, I=768, align=8, bits=16, skew=0.0),
        # a decoding batch whose tokens reach nearly every expert, 8-bit rows and weights
        dict(name="ffn_decode_8bit", op="ffn", N=61, E=64, K=6, H=4096, I=1280, align=16, bits=8, skew=0.0),
        # an odd-length prompt chunk, popular and rare experts: ragged groups
        dict(name="ffn_prompt", op="ffn", N=1777, E=128, K=8, H=2048, I=768, align=16, bits=16, skew=1.1),
        # a large prefill over few wide experts, 8-bit rows and weights
        dict(name="ffn_prefill_8bit", op="ffn", N=16384, E=8, K=2, H=4096, I=4096, align=16, bits=8, skew=0.0),
        # a small model's training step, sizes that fill no tile
        dict(name="train_tiny", op="ffn_train", N=256, E=8, K=2, H=128, I=72, align=8, skew=0.0),
        # a training step over many narrow experts with uneven popularity
        dict(name="train_many_experts", op="ffn_train", N=8192, E=128, K=8, H=2048, I=768, align=128, skew=1.1),
        # a training step over few wide experts: the largest case
        dict(name="train_wide_experts", op="ffn_train", N=16384, E=8, K=2, H=4096, I=4096, align=16, skew=0.0),
        # the combine's gradient of a small batch
        dict(name="combine_backward_small", op="combine_backward", N=333, E=8, K=2, H=4096, align=16, skew=0.0),
        # the combine's gradient of a training batch at the widest hidden size
        dict(name="combine_backward_large", op="combine_backward", N=16384, E=256, K=8, H=7168, align=128, skew=0.0),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    n = min(hi, max(lo, int(round(v / step)) * step))
    return n + step if n in (1536, 3072) else n


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm", "norm_backward", "ffn", "ffn", "ffn_train", "combine_backward"])
        if op in ("norm", "norm_backward"):
            case = dict(op=op, N=_log_int(rng, 1, 32768), H=_log_int(rng, 128, 8192, 8),
                        residual=rng.choice(["none", "bf16", "fp32"]))
            if op == "norm":
                case["quantize"] = rng.random() < 0.6
            if case["N"] * case["H"] > 8192 * 16384:
                continue
        else:
            E = rng.choice([4, 8, 16, 32, 60, 64, 128])
            case = dict(op=op, N=_log_int(rng, 1, 16384), E=E, K=min(rng.choice([1, 2, 4, 6, 8]), E),
                        H=_log_int(rng, 128, 7168, 16), align=rng.choice([1, 8, 16, 128]),
                        skew=rng.choice([0.0, 0.0, 1.1]))
            if op != "combine_backward":
                case["I"] = _log_int(rng, 64, 4096, 8)
                if case["E"] * case["H"] * case["I"] > 8 * 4096 * 4096 * 4:
                    continue
                tiles = case["N"] * case["K"] // _tile_rows(case) + case["E"]
                if tiles * case["H"] * case["I"] > 80 * 4096 * 4096:
                    continue
            if op == "ffn":
                case["bits"] = rng.choice([16, 16, 8])
        if _cost(case) <= most:
            return case


def work(case):
    N, H, op = case["N"], case["H"], case["op"]
    res = {"none": 0, "bf16": 2, "fp32": 4}[case.get("residual", "none")]
    if op == "norm":
        row = 2 + 2 * res + 2 + (1 if case["quantize"] else 0)
        return {"bytes": N * (H * row + 8) + 2 * H, "flops": 6 * N * H}
    if op == "norm_backward":
        # dy, the stored sum and its gradient come in, the gradients of x and of the residual go out
        s = max(2, res)
        row = 2 + s + s + 2 + (4 if res == 4 else 0)
        return {"bytes": N * (H * row + 4) + 6 * H, "flops": 10 * N * H}
    E, K = case["E"], case["K"]
    P = N * K
    if op == "combine_backward":
        return {"bytes": 2 * N * H + 4 * P * H + 12 * P, "flops": 3 * P * H}
    I = case["I"]  # noqa: E741
    # experts that at least one token reaches, for evenly spread tokens
    used = E * (1 - (1 - K / E) ** N)
    if op == "ffn":
        b = case["bits"] // 8
        return {"bytes": used * H * I * (2 * b + 2) + P * H * (b + 2), "flops": 6 * P * H * I}
    return {"bytes": used * 6 * H * I + E * 6 * H * I + P * H * 8, "flops": 18 * P * H * I}


# ---------------------------------------------------------------- inputs
def _tile_rows(case):
    """Rows of one product of the plain form: about a group's, so that the padding stays small."""
    mean = case["N"] * case["K"] / case["E"]
    return max(8, min(512, 1 << int(math.ceil(math.log2(max(1.0, mean / 4))))))


def _groups(case, gen):
    """A router's choice and its dispatch plan: groups in expert order, padded to the alignment."""
    N, E, K, a = case["N"], case["E"], case["K"], case["align"]
    dev = gen.device
    logits = torch.randn(N, E, generator=gen, device=dev)
    if case["skew"]:
        rank = torch.randperm(E, generator=gen, device=dev) + 1
        logits = logits - case["skew"] * torch.log(rank.float())
    val, idx = torch.topk(logits, K, dim=1)
    topk_w = torch.softmax(val, dim=1)
    count = torch.bincount(idx.reshape(-1), minlength=E)
    padded = (count + a - 1) // a * a
    cu = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.cumsum(padded, 0)
    order = torch.argsort(idx.reshape(-1), stable=True)      # pairs by expert, then by token
    first = torch.cumsum(count, 0) - count
    expert = idx.reshape(-1)[order]
    slot = torch.empty(N * K, dtype=torch.int64, device=dev)
    slot[order] = cu[expert] + torch.arange(N * K, device=dev) - first[expert]
    pad = padded - count
    zero = torch.where((pad > 0)[:, None], torch.stack([cu[:-1] + count, pad], 1), torch.zeros_like(pad)[:, None])
    i32 = torch.int32
    return SimpleNamespace(cu_seqlens=cu.to(i32), tokens_per_expert=count.to(i32), dst=slot.reshape(N, K).to(i32),
                           zero_fill_ranges=zero.to(i32).contiguous(),
                           status=torch.zeros(4, dtype=i32, device=dev), N=N, K=K, E=E, rows=N * K + E * (a - 1),
                           topk_w=topk_w)


def _tiles(case, p):
    """Tiles of the groups for the plain form: expert, row indices and which of them are live."""
    t = _tile_rows(case)
    dev = p.dst.device
    count = p.tokens_per_expert.long()
    n = (count + t - 1) // t
    expert = torch.repeat_interleave(torch.arange(p.E, device=dev), n)
    j = torch.arange(expert.numel(), device=dev) - (torch.cumsum(n, 0) - n)[expert]
    at = j[:, None] * t + torch.arange(t, device=dev)
    live = at < count[expert][:, None]
    rows = torch.where(live, p.cu_seqlens.long()[expert][:, None] + at, p.rows)
    return expert, rows


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
    if op in ("norm", "norm_backward"):
        s["weight"] = (1 + normal(H, std=0.1)).to(bf16)
        kind = {"none": None, "bf16": bf16, "fp32": torch.float32}[case["residual"]]
        size = torch.exp(normal(N, 1))       # rows of very different size
        if op == "norm":
            s["x"] = normal(N, H).to(bf16)
            s["residual"] = None if kind is None else (normal(N, H) * size).to(kind)
        else:
            stream = (normal(N, H) * size).to(kind or bf16)
            s["s"] = stream
            s["rstd"] = torch.rsqrt(stream.float().square().mean(-1) + EPS)
            s["dy"] = normal(N, H).to(bf16)
            s["ds"] = None if kind is None else normal(N, H).to(kind)
        return s

    p = s["p"] = _groups(case, gen)
    live = torch.zeros(p.rows, dtype=torch.bool, device=dev)
    live[p.dst.long().reshape(-1)] = True

    def rows_of(n):                         # rows of the permuted buffer, zero where it is padding
        return torch.where(live[:, None], normal(p.rows, n), 0.0)

    if op == "combine_backward":
        s["dout"] = normal(N, H).to(bf16)
        s["y"] = rows_of(H).to(bf16)
        s["out"] = torch.zeros(p.rows, H, dtype=bf16, device=dev)
        return s
    E, I = case["E"], case["I"]  # noqa: E741
    s["tiles"] = _tiles(case, p)
    x, wgu, wd = rows_of(H), normal(E, 2, I, H, std=H ** -0.5), normal(E, H, I, std=I ** -0.5)
    s["w_down"] = wd.to(bf16)
    # the caller's own row buffers, of the plan's capacity; the rows past the last group stay as they are
    s["out"] = torch.zeros(p.rows, H, dtype=bf16, device=dev)
    if case.get("bits") == 8:
        s["x"], s["x_scale"] = _quantised(x)
        s["w_gate_up"], s["w_scale"] = _quantised(wgu)
    else:
        s["x"], s["w_gate_up"] = x.to(bf16), wgu.to(bf16)
        if op == "ffn_train":
            s["dy"] = rows_of(H).to(bf16)
            s["dx"] = torch.zeros(p.rows, H, dtype=bf16, device=dev)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import expert_dispatch_planning_gb300 as m
    op = s["case"]["op"]
    if op == "norm":
        o = m.residual_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantize=s["case"]["quantize"])
        return {"y": o.y, "residual": o.residual, "rstd": o.rstd, "q": o.q, "q_scale": o.q_scale}
    if op == "norm_backward":
        dx, dres, dweight = m.residual_norm_backward(s["dy"], s["s"], s["weight"], s["rstd"], ds=s["ds"])
        return {"dx": dx, "dres": dres, "dweight": dweight}
    p = s["p"]
    if op == "combine_backward":
        dy, dw = m.combine_backward(s["dout"], s["y"], p.topk_w, p, dy=s["out"])
        return {"dy": dy, "dw": dw}
    if op == "ffn":
        return {"y": m.expert_ffn(s["x"], s["w_gate_up"], s["w_down"], p, x_scale=s.get("x_scale"),
                                  w_scale=s.get("w_scale"), out=s["out"])}
    M, I = s["x"].shape[0], s["case"]["I"]  # noqa: E741
    dev = s["x"].device
    h = torch.empty((M, I), dtype=torch.bfloat16, device=dev)
    preact = torch.empty((M, 2, I), dtype=torch.float32, device=dev)
    y = m.expert_ffn(s["x"], s["w_gate_up"], s["w_down"], p, h=h, preact=preact, out=s["out"])
    dx, dwgu, dwd = m.expert_ffn_backward(s["dy"], s["x"], h, preact, s["w_gate_up"], s["w_down"], p,
                                          dx=s["dx"])
    return {"y": y, "dx": dx, "dw_gate_up": dwgu, "dw_down": dwd}


def _run_plain(s):
    op = s["case"]["op"]
    bf16 = torch.bfloat16
    if op == "norm":
        v = s["x"].float()
        r = s["residual"]
        if r is not None:
            v = v + r.float()
        rstd = 1 / torch.sqrt(v.square().mean(-1) + EPS)
        out = v * rstd[:, None] * s["weight"].float()
        q = q_scale = None
        if s["case"]["quantize"]:
            amax = out.abs().amax(-1)
            q_scale = torch.where(amax > 0, amax, 1.0) / E4M3_MAX
            q = (out / q_scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"y": out.to(bf16), "residual": None if r is None else v.to(r.dtype), "rstd": rstd, "q": q,
                "q_scale": q_scale}
    if op == "norm_backward":
        v, dy, rstd = s["s"].float(), s["dy"].float(), s["rstd"][:, None]
        xhat = v * rstd
        t = dy * s["weight"].float()
        d = rstd * (t - xhat * (t * xhat).mean(-1, keepdim=True))
        if s["ds"] is not None:
            d = d + s["ds"].float()
        return {"dx": d.to(bf16), "dres": d if s["s"].dtype == torch.float32 else None,
                "dweight": (dy * xhat).sum(0)}
    p = s["p"]
    if op == "combine_backward":
        N, K = p.dst.shape
        H = s["dout"].shape[1]
        slot = p.dst.long().reshape(-1)
        dout = s["dout"].float()
        dy = torch.zeros(p.rows, H, dtype=bf16, device=dout.device)
        dy[slot] = (p.topk_w[:, :, None] * dout[:, None, :]).reshape(N * K, H).to(bf16)
        dw = (s["y"][slot].float().reshape(N, K, H) * dout[:, None, :]).sum(-1)
        return {"dy": dy, "dw": dw}

    expert, rows = s["tiles"]
    T, t = rows.shape
    E, _, I, H = s["w_gate_up"].shape  # noqa: E741

    def taken(v, at):                       # entries of the first axis in 32 bits
        return v.view(torch.uint8)[at].view(v.dtype).float() if v.element_size() == 1 else v[at].float()

    def tiles_of(v, scale=None):            # [T, t, n] in 32 bits; rows past a group's end are zero
        at = rows.clamp(max=max(0, p.rows - 1))
        r = taken(v, at.reshape(-1)).reshape(T, t, -1)
        if scale is not None:
            r = r * scale[at][..., None]
        return torch.where((rows < p.rows)[..., None], r, 0.0)

    def scattered(v):                       # [rows, n] from tiles; padding rows are zero
        o = torch.zeros(p.rows + 1, v.shape[-1], device=v.device)
        o[rows.reshape(-1)] = v.reshape(T * t, -1)
        return o[:-1].to(bf16)

    def by_expert(v):                       # the sum of an expert's tiles
        o = torch.zeros(E, *v.shape[1:], device=v.device)
        return o.index_add_(0, expert, v).to(bf16)

    x = tiles_of(s["x"], s.get("x_scale"))
    wgu = taken(s["w_gate_up"], expert)
    if "w_scale" in s:
        wgu = wgu * s["w_scale"][expert][..., None]
    wgu = wgu.reshape(T, 2 * I, H)
    wd = s["w_down"][expert].float()
    g, u = torch.bmm(x, wgu.transpose(1, 2)).split(I, dim=-1)
    sig = 1 / (1 + torch.exp(-g))
    h = g * sig * u
    y = scattered(torch.bmm(h, wd.transpose(1, 2)))
    if op == "ffn":
        return {"y": y}
    dy = tiles_of(s["dy"])
    dh = torch.bmm(dy, wd)
    dwd = by_expert(torch.bmm(dy.transpose(1, 2), h))
    dgu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=-1)
    dx = scattered(torch.bmm(dgu, wgu))
    dwgu = by_expert(torch.bmm(dgu.transpose(1, 2), x)).reshape(E, 2, I, H)
    return {"y": y, "dx": dx, "dw_gate_up": dwgu, "dw_down": dwd}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = s["x"].double()
        if s["residual"] is not None:
            v = v + s["residual"].double()
        rstd = (torch.linalg.vector_norm(v, dim=1).pow(2) / case["H"] + EPS).pow(-0.5)
        y = torch.einsum("nh,n,h->nh", v, rstd, s["weight"].double())
        q = scale = None
        if case["quantize"]:
            top = y.abs().max(dim=1).values
            scale = torch.where(top > 0, top, torch.ones_like(top)) / E4M3_MAX
            q = y / scale[:, None]
        return {"y": y, "residual": v if s["residual"] is not None else None, "rstd": rstd, "q": q, "q_scale": scale}
    if op == "norm_backward":
        v, dy, w, r = s["s"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
        proj = torch.einsum("nh,h,nh->n", dy, w, v) * r.pow(3) / case["H"]
        d = torch.einsum("n,nh,h->nh", r, dy, w) - proj[:, None] * v
        if s["ds"] is not None:
            d = d + s["ds"].double()
        return {"dx": d, "dres": d if case["residual"] == "fp32" else None,
                "dweight": torch.einsum("nh,nh,n->h", dy, v, r)}
    p = s["p"]
    if op == "combine_backward":
        H = case["H"]
        dy = torch.zeros(p.rows, H, dtype=torch.float64, device="cuda")
        dw = torch.empty(p.topk_w.shape, dtype=torch.float64, device="cuda")
        dout = s["dout"].double()
        for k in range(case["K"]):
            slot = p.dst[:, k].long()
            dy[slot] = p.topk_w[:, k].double()[:, None] * dout
            dw[:, k] = torch.einsum("nh,nh->n", dout, s["y"][slot].double())
        return {"dy": dy, "dw": dw}
    E, I, H = case["E"], case["I"], case["H"]  # noqa: E741
    y = torch.zeros(p.rows, H, dtype=torch.float64, device="cuda")
    out = {"y": y}
    if op == "ffn_train":
        out["dx"] = torch.zeros_like(y)
        out["dw_gate_up"] = torch.zeros(E, 2, I, H, dtype=torch.float64, device="cuda")
        out["dw_down"] = torch.zeros(E, H, I, dtype=torch.float64, device="cuda")
    begins, counts = p.cu_seqlens.tolist(), p.tokens_per_expert.tolist()
    for e in range(E):
        if counts[e] == 0:
            continue
        at = slice(begins[e], begins[e] + counts[e])
        x, w, wd = s["x"][at].double(), s["w_gate_up"][e].double(), s["w_down"][e].double()
        if "x_scale" in s:
            x, w = x * s["x_scale"][at].double()[:, None], w * s["w_scale"][e].double()[..., None]
        g, u = x @ w[0].T, x @ w[1].T
        sg = torch.special.expit(g)
        h = g * sg * u
        y[at] = h @ wd.T
        if op == "ffn_train":
            dy = s["dy"][at].double()
            dh = dy @ wd
            dg, du = dh * u * (sg + g * sg * torch.special.expit(-g)), dh * g * sg
            out["dx"][at] = dg @ w[0] + du @ w[1]
            out["dw_gate_up"][e, 0], out["dw_gate_up"][e, 1] = dg.T @ x, du.T @ x
            out["dw_down"][e] = dy.T @ h
    return out

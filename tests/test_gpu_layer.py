"""A whole layer for a few tokens against its definition in 64 bits, with the router's choice from route_topk.

Bounds: block_checks' error model (bf16 rounding U, F for every step of a sum of
products, S for functions in fp32).  h is rounded once to bf16, its error goes
through the down product; the weighted sum over the chosen experts is taken in
fp32 and rounded once.
"""
import pytest
import torch

from block_checks import F, S, U, assert_within

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def quantised(v):
    scale = v.abs().amax(-1).clamp_min(1e-12) / 448
    return (v / scale[..., None]).clamp(-448, 448).to(E4M3), scale


def inputs(N, E, H, I, bits=16, seed=0):  # noqa: E741
    g = gen(seed)

    def normal(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda") * std
    a = dict(logits=normal(N, E), w_down=normal(E, H, I, std=I ** -0.5).to(BF16))
    x, w = normal(N, H), normal(E, 2, I, H, std=H ** -0.5)
    if bits == 8:
        a["x"], a["x_scale"] = quantised(x)
        a["w_gate_up"], a["w_scale"] = quantised(w)
    else:
        a["x"], a["w_gate_up"] = x.to(BF16), w.to(BF16)
    return a


def wanted(m, a, K, routing):
    """out in 64 bits, its bound, and the router's choice."""
    idx, w = m.route_topk(a["logits"], K, **routing)
    x, wgu, wd = a["x"].double(), a["w_gate_up"], a["w_down"]
    if "x_scale" in a:
        x = x * a["x_scale"].double()[:, None]
    N, H = x.shape
    E, _, I, _ = wgu.shape  # noqa: E741
    out, tol, mag = (torch.zeros(N, H, dtype=torch.float64, device="cuda") for _ in range(3))
    for e in idx.unique().tolist():
        at, k = (idx == e).nonzero(as_tuple=True)
        W, D, share = wgu[e].double(), wd[e].double(), w[at, k].double()[:, None]
        if "w_scale" in a:
            W = W * a["w_scale"][e].double()[..., None]
        xs = x[at]
        g, u = xs @ W[0].T, xs @ W[1].T
        # the tensor core's sum, its parts' sum over the warps, and the scales' products
        dg, du = ((H + 16) * F * (xs.abs() @ W[i].abs().T) for i in (0, 1))
        h = g * torch.sigmoid(g) * u
        silu = (g * torch.sigmoid(g)).abs()
        fp32 = 1.1 * dg * (u.abs() + du) + silu * du + S * h.abs()
        eh = fp32 + U * (h.abs() + fp32)
        y_abs = h.abs() @ D.abs().T
        ey = eh @ D.abs().T
        out[at] += share * (h @ D.T)
        tol[at] += share.abs() * (ey + (I + 16) * F * (y_abs + ey))
        mag[at] += share.abs() * (y_abs + ey)
    tol = tol + (K + 8) * F * mag       # the weighted sum over the experts and over the warps
    return out, tol + U * (out.abs() + tol), idx, w


def check(m, a, K, **routing):
    N, E = a["logits"].shape
    out, tol, idx, w = wanted(m, a, K, routing)
    gi, gw = torch.full((N, K), -7, dtype=torch.int32, device="cuda"), torch.full((N, K), -7.0, device="cuda")
    got = m.layer(K=K, topk_idx=gi, topk_w=gw, **a, **routing)
    assert torch.equal(gi, idx) and torch.equal(gw, w)
    assert_within(got, out, tol, "out")
    assert torch.equal(m.layer(K=K, **a, **routing), got)       # the same bits again, without the optional outputs
    return got


SIZES = [(1, 1, 1, 8, 8), (1, 8, 2, 128, 72), (3, 4, 4, 24, 8), (2, 5, 3, 72, 200), (8, 16, 2, 264, 136), (9, 8, 8, 256, 64),
         (1, 128, 8, 2048, 768), (17, 60, 4, 1000, 712), (33, 128, 8, 512, 192), (64, 8, 2, 640, 328), (64, 3, 1, 128, 64),
         (5, 1024, 32, 64, 16), (64, 1024, 32, 64, 24), (7, 4, 2, 4880, 40), (64, 6, 3, 4888, 72), (20, 33, 5, 96, 1032),
         # many tiles a block; more tokens an expert than a pass takes
         (8, 128, 8, 1024, 456), (24, 60, 4, 1032, 712), (33, 64, 4, 1032, 1048), (64, 48, 12, 1040, 1024)]


@pytest.mark.parametrize("N,E,K,H,I", SIZES)
def test_bf16(m, N, E, K, H, I):  # noqa: E741
    check(m, inputs(N, E, H, I), K)


@pytest.mark.parametrize("N,E,K,H,I", [(1, 2, 1, 16, 8), (3, 8, 2, 272, 72), (1, 128, 8, 2048, 768), (12, 16, 4, 1040, 200),
                                       (31, 60, 6, 512, 136), (64, 8, 2, 256, 264), (6, 4, 3, 4880, 24), (16, 64, 6, 2064, 440)])
def test_8bit(m, N, E, K, H, I):  # noqa: E741
    check(m, inputs(N, E, H, I, bits=8), K)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("N", [1, 8, 9, 16, 17, 24, 32, 33, 48, 64])
def test_all_tokens_choose_the_same_experts(m, N, bits):
    """One expert has every token: up to eight eights of rows."""
    a = inputs(N, 12, 144, 88, bits=bits)
    a["logits"][:, 3] += 50
    a["logits"][:, 11] += 40
    check(m, a, 2)
    check(m, a, 1)


@pytest.mark.parametrize("routing", [
    dict(renormalize=False), dict(scoring="sigmoid"), dict(scoring="sigmoid", renormalize=False, routed_scaling=2.5),
    dict(scoring="sigmoid", n_group=8, topk_group=4, routed_scaling=2.5), dict(scoring="sigmoid", n_group=4, topk_group=1)])
def test_routing(m, routing):
    a = inputs(21, 64, 128, 72)
    if routing.get("scoring") == "sigmoid":
        routing = dict(routing, bias=(torch.rand(64, generator=gen(3), device="cuda") - 0.5) * 0.2)
    check(m, a, 6, **routing)


def test_masked_experts(m):
    """Experts masked by the lowest logits, by minus infinity: chosen last, with weight zero or next to it."""
    a = inputs(10, 16, 128, 64)
    a["logits"][:, 4:] = -float("inf")
    check(m, a, 4)
    a["logits"][:, 4:] = torch.finfo(F32).min
    check(m, a, 4)
    check(m, a, 7)              # more than are open: the masked ones come in, with weight zero


@pytest.mark.parametrize("bits", [16, 8])
def test_what_is_not_chosen_is_not_read(m, bits):
    """NaN and infinities in experts that no token chose, and in other tokens' rows, reach nothing."""
    N, E, K = 11, 24, 2
    a = inputs(N, E, 160, 72, bits=bits)
    a["logits"][:, 12:] -= 100
    clean = check(m, a, K)
    idx = m.route_topk(a["logits"], K)[0]
    unused = [e for e in range(E) if not (idx == e).any()]
    assert len(unused) >= 12
    a["w_down"][unused] = float("nan")
    a["w_gate_up"].view(torch.uint8 if bits == 8 else torch.int16)[unused] = 0x7f if bits == 8 else 0x7f80   # NaN, infinity
    assert torch.equal(m.layer(K=K, **a), clean)
    if bits == 16:
        a["x"][4] = float("nan")
        a["x"][7, 3] = float("inf")
        got = m.layer(K=K, **a)
        rest = [i for i in range(N) if i not in (4, 7)]
        assert torch.equal(got[rest], clean[rest]) and got[4].isnan().all() and not got[7].isfinite().any()
    else:
        a["x_scale"][4] = float("nan")
        got = m.layer(K=K, **a)
        rest = [i for i in range(N) if i != 4]
        assert torch.equal(got[rest], clean[rest]) and got[4].isnan().all()


def test_gates_of_every_size(m):
    """silu from -infinity's side to large values: no overflow, and it keeps its value down to the smallest numbers."""
    H, I = 16, 8  # noqa: E741
    sizes = torch.tensor([-200.0, -104, -95, -88, -60, -20, -1, 0, 1, 20, 90, 300], device="cuda")
    N = len(sizes)
    x = torch.zeros(N, H, device="cuda")
    x[:, 0], x[:, 1] = sizes, 1.0
    wgu = torch.zeros(1, 2, I, H, device="cuda")
    wgu[0, 0, :, 0], wgu[0, 1, :, 1] = 1.0, 2.0 ** 40         # g = x[0], u = 2^40
    wd = torch.zeros(1, H, I, device="cuda")
    wd[0, :, 0] = 1.0
    got = m.layer(x.to(BF16), torch.zeros(N, 1, device="cuda"), wgu.to(BF16), wd.to(BF16), 1)
    g = sizes.to(BF16).double()
    want = (g * torch.sigmoid(g) * 2.0 ** 40)[:, None].expand(N, H)
    # e^-|g| keeps fp32's precision down to its smallest normal number, 2^-126, and half a 2^-149 below
    fp32 = S * want.abs() + g.abs()[:, None] * 2.0 ** -149 * 2.0 ** 40
    assert_within(got, want, fp32 + 2 * U * (want.abs() + fp32), "out")


def test_given_output_and_guard_zones(m):
    N, E, K, H, I = 13, 8, 2, 200, 72  # noqa: E741
    a = inputs(N, E, H, I)
    want = m.layer(K=K, **a)
    big = torch.full((N + 2, H), 7.0, device="cuda").to(BF16)
    idx, w = torch.full((N + 2, K), 7, dtype=torch.int32, device="cuda"), torch.full((N + 2, K), 7.0, device="cuda")
    out = big[1:N + 1]
    assert m.layer(K=K, out=out, topk_idx=idx[1:N + 1], topk_w=w[1:N + 1], **a) is out
    assert torch.equal(out, want)
    for t in (big, idx, w):
        assert (t[0] == 7).all() and (t[N + 1] == 7).all()


def test_empty_batch(m):
    a = inputs(2, 8, 64, 16)
    out = m.layer(a["x"][:0], a["logits"][:0], a["w_gate_up"], a["w_down"], 2)
    assert out.shape == (0, 64)


def test_refusals(m):
    N, E, K, H, I = 4, 8, 2, 64, 16  # noqa: E741
    ok = dict(inputs(N, E, H, I), K=K)
    q = dict(inputs(N, E, H, I, bits=8), K=K)
    many = inputs(65, E, H, I)
    for base, change in ((ok, dict(x=ok["x"].float())), (ok, dict(x=ok["x"][:, ::2])), (ok, dict(logits=ok["logits"][:3])),
                         (ok, dict(logits=ok["logits"].to(BF16))), (ok, dict(w_gate_up=ok["w_gate_up"][:, :1])),
                         (ok, dict(w_down=ok["w_down"][:7])), (ok, dict(w_down=None)), (ok, dict(x_scale=q["x_scale"])),
                         (q, dict(w_scale=None)), (q, dict(w_gate_up=ok["w_gate_up"])), (ok, dict(out=ok["x"].float())),
                         (ok, dict(topk_idx=torch.zeros(N, K + 1, dtype=torch.int32, device="cuda"))), (ok, dict(x=ok["x"].cpu())),
                         (ok, dict(bias=torch.zeros(E - 1, device="cuda"), scoring="sigmoid")), (ok, dict(K="2")),
                         (ok, dict(x=many["x"], logits=many["logits"]))):
        with pytest.raises((ValueError, TypeError)):
            m.layer(**{**base, **change})
    for change in (dict(K=0), dict(K=9), dict(K=33), dict(bias=torch.zeros(E, device="cuda")), dict(n_group=2),
                   dict(scoring="sigmoid", n_group=3), dict(routed_scaling=float("nan"))):
        with pytest.raises(m.MoeError):
            m.layer(**{**ok, **change})
    odd = torch.empty(N * H + 1, dtype=BF16, device="cuda")[1:].view(N, H)
    with pytest.raises(m.MoeError):
        m.layer(**{**ok, "x": odd})
    with pytest.raises(m.MoeError):         # H is no multiple of 16 in 8 bits
        m.layer(**dict(inputs(N, E, 72, I, bits=8), K=K))


def test_two_calls_at_once(m):
    """Calls on two streams, each with its own workspace."""
    a, b = inputs(8, 32, 512, 200, seed=1), inputs(30, 64, 1024, 1040, seed=2)
    wa, wb = m.layer(K=4, **a), m.layer(K=6, **b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(m.layer(K=4, stream=s, **a), m.layer(K=6, stream=t, **b)) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in outs:
        assert torch.equal(x, wa) and torch.equal(y, wb)


@pytest.mark.parametrize("N,E,H,I", [(6, 16, 256, 136), (20, 64, 1024, 1024)])
def test_graph(m, N, E, H, I):  # noqa: E741
    """Two captured layers in a row, the second on the first one's output; replayed with new inputs."""
    a, b = inputs(N, E, H, I, seed=1), inputs(N, 16, H, 72, seed=2)
    del b["x"]

    def both(stream=None):
        y = m.layer(K=2, stream=stream, **a)
        return y, m.layer(x=y, K=3, stream=stream, **b)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = both()
    for seed in (5, 6):
        new = inputs(N, E, H, I, seed=seed)
        a["x"].copy_(new["x"])
        a["logits"].copy_(new["logits"])
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        y2, z2 = both()
        assert torch.equal(y, y2) and torch.equal(z, z2)


@pytest.mark.parametrize("bits", [16, 8])
def test_large_offsets(m, bits):
    """Weights past 2^31 elements and 2^32 bytes."""
    E, K, H, I = 160, 2, 7168, 1024  # noqa: E741
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    small = inputs(3, 4, H, I, bits=bits)
    small["logits"] = torch.tensor([[3.0, 2, 1, 0], [0, 1, 2, 3], [1, 3, 0, 2]], device="cuda")
    want = check(m, small, K)
    big = dict(small)
    for k in ("w_gate_up", "w_down") + (("w_scale",) if bits == 8 else ()):
        t = small[k]
        big[k] = torch.zeros((E,) + t.shape[1:], dtype=t.dtype, device="cuda")
        big[k].view(torch.uint8)[-4:] = t.view(torch.uint8)
    big["logits"] = torch.full((3, E), -100.0, device="cuda")
    big["logits"][:, -4:] = small["logits"]
    got = m.layer(K=K, **big)
    assert torch.equal(got, want)


def test_against_the_plan_path(m):
    """The same tokens through route_plan, permute, expert_ffn and combine: h, y and out are rounded there, so that the
    two differ by the roundings of y (U each, weighted) on top of both bounds."""
    for bits in (16, 8):
        N, E, K, H, I = 37, 32, 4, 512, 264  # noqa: E741
        a = inputs(N, E, H, I, bits=bits)
        out, tol, idx, w = wanted(m, a, K, {})
        idx, w, p = m.route_plan(a["logits"], K, 1, 8)
        src = (p.src_of_slot.clamp(min=0) // K).long()
        xp = a["x"].view(torch.int8 if bits == 8 else torch.int16)[src].view(a["x"].dtype)
        scales = {} if bits == 16 else dict(x_scale=a["x_scale"][src].contiguous(), w_scale=a["w_scale"])
        y = m.expert_ffn(xp, a["w_gate_up"], a["w_down"], p, **scales)
        ref = m.combine(y, w, p).double()
        slot = torch.where(p.dst < 0, -p.dst - 1, p.dst).long()
        rounding = U * (w.double()[..., None] * y[slot].double().abs()).sum(1)
        assert_within(m.layer(K=K, **a), ref, 2 * tol + 2 * rounding, "out")


def test_a_decoding_step(m):
    """block_norm -> logits -> layer -> block_norm, in a graph, 8 bits: each part against its own call."""
    N, E, K, H, I = 5, 16, 2, 256, 136  # noqa: E741
    a = inputs(N, E, H, I, bits=8)
    g = gen(7)
    x, r = torch.randn(N, H, generator=g, device="cuda").to(BF16), torch.randn(N, H, generator=g, device="cuda")
    w, router = torch.ones(H, device="cuda"), torch.randn(H, E, generator=g, device="cuda")
    gate = torch.rand(N, generator=g, device="cuda")

    def step(r):
        n = m.block_norm(x, r, w, w, quantize=True)
        out = m.layer(n.q, n.y.float() @ router, a["w_gate_up"], a["w_down"], K, x_scale=n.q_scale, w_scale=a["w_scale"])
        return n, out, m.block_norm(out, n.residual, w, w, gate=gate, residual_out=n.residual)
    n, out, o = step(r)
    keep = [t.clone() for t in (out, o.y, o.residual)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n, out, o = step(r)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got, want in zip((out, o.y, o.residual), keep):
        assert torch.equal(got, want)
    b = dict(a, x=n.q, x_scale=n.q_scale, logits=n.y.float() @ router)
    want, tol, _, _ = wanted(m, b, K, {})
    assert_within(out, want, tol, "out")

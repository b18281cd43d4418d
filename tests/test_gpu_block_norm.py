"""The norms between two blocks and their gradient against the formulas in 64 bits.

Error model.  FP is one fp32 rounding.  A sum over a row takes at most H/8 + 12
steps one after the other in a thread and in the trees; with the root, its
products and conversions the row's root is off by at most B = (H/8 + 30) FP
relative.  Everything after that is carried through the formulas: an error of
each value, through each product and sum it enters.
"""
from types import SimpleNamespace

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8          # bf16 rounding, relative
FP = 2.0 ** -24        # one fp32 rounding
EPS = 1e-5
ALPHA = 0.8125


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def rand(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


# a row in one warp (up to 512), in a block with 1, 2 or 4 chunks a thread, the bounds between them, and many rows
SIZES = [(1, 8), (3, 128), (7, 256), (5, 264), (129, 512), (2, 520), (1, 2048), (33, 2056), (4, 4096), (9, 7168),
         (3, 8200), (2, 16384), (1, 32768), (1000, 136), (5003, 520), (1300, 1000), (4900, 1000), (9800, 2048), (19500, 1032),
         (650, 2056), (1300, 4104), (1400, 4096), (1111, 7168), (700, 8192)]
KINDS = [(BF16, None, BF16, BF16), (F32, "token", F32, BF16), (BF16, "full", BF16, F32), (F32, "full", F32, F32),
         (F32, None, BF16, BF16), (BF16, "token", BF16, BF16)]


def bound(H):
    return (H / 8 + 30) * FP


def inputs(N, H, res, gate, post_type, weight_type, seed=0):
    x = (rand(N, H, seed=seed) * torch.exp(rand(N, 1, seed=seed + 1))).to(BF16)
    r = (rand(N, H, seed=seed + 2) * torch.exp(2 * rand(N, 1, seed=seed + 3))).to(res)
    wp, w = (1 + 0.2 * rand(H, seed=seed + 4)).to(post_type), (1 + 0.2 * rand(H, seed=seed + 5)).to(weight_type)
    c = None if gate is None else torch.sigmoid(rand(N, seed=seed + 6)) if gate == "token" else \
        torch.sigmoid(rand(N, H, seed=seed + 6)).to(BF16)
    return x, r, wp, w, c


def gate64(c, x):
    return torch.ones_like(x) if c is None else c.double().reshape(x.shape[0], -1).expand_as(x)


def forward64(x, r, wp, w, c, alpha=ALPHA, eps=EPS):
    """The outputs in 64 bits, and bounds of what the kernel may be off by before its last rounding."""
    x, r, wp, w = x.double(), r.double(), wp.double(), w.double()
    c = gate64(c, x)
    b = bound(x.shape[1])
    o = SimpleNamespace()
    o.post = (x.square().mean(1) + eps).rsqrt()
    n = c * x * o.post[:, None] * wp
    o.s = alpha * r + n
    # n: its root, two or three products; the fused sum rounds once
    o.s_err = (b + 4 * FP) * n.abs() + FP * (o.s.abs() + (b + 4 * FP) * n.abs())
    o.rstd = (o.s.square().mean(1) + eps).rsqrt()
    # the errors of s move its root by at most their own root mean square
    moved = o.s_err.square().mean(1).sqrt() * o.rstd
    o.rstd_err = (b + 1.1 * moved) * o.rstd
    o.y = o.s * o.rstd[:, None] * w
    o.y_err = o.s_err * (o.rstd[:, None] * w.abs()) * (1 + b) + o.y.abs() * ((o.rstd_err / o.rstd)[:, None] + 3 * FP)
    return o


def check_forward(o, e, res, H):
    b = bound(H)
    assert ((o.post_rstd.double() - e.post).abs() <= b * e.post).all()
    assert ((o.rstd.double() - e.rstd).abs() <= e.rstd_err).all()
    rounding = FP if res == F32 else U
    assert ((o.residual.double() - e.s).abs() <= e.s_err + rounding * (e.s.abs() + e.s_err) + 1e-38).all()
    assert ((o.y.double() - e.y).abs() <= e.y_err + U * (e.y.abs() + e.y_err) + 1e-38).all()
    if o.q is not None:
        amax = e.y.abs().amax(1)
        scale_err = e.y_err.amax(1) / 448 + 4 * FP * amax / 448
        assert ((o.q_scale.double() - amax / 448).abs() <= scale_err).all()
        q, v = o.q.float().double(), e.y / o.q_scale.double()[:, None]
        v_err = e.y_err / o.q_scale.double()[:, None] + 6 * FP * v.abs()
        assert (q.abs() <= 448).all()
        # e4m3: 3 mantissa bits, relative 2^-4 of the value, 2^-10 absolute below the normal range; saturates at 448
        assert ((q - v).abs() <= v_err + 2.0 ** -4 * (v.abs() + v_err) + 2.0 ** -10).all()


@pytest.mark.parametrize("N,H", SIZES)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_forward(m, N, H, kind):
    res, gate, pt, wt = KINDS[kind]
    x, r, wp, w, c = inputs(N, H, res, gate, pt, wt)
    o = m.block_norm(x, r, wp, w, gate=c, residual_scale=ALPHA, eps=EPS, quantize=True)
    check_forward(o, forward64(x, r, wp, w, c), res, H)
    # without the 8-bit output: the same bits
    p = m.block_norm(x, r, wp, w, gate=c, residual_scale=ALPHA, eps=EPS)
    assert torch.equal(p.y, o.y) and torch.equal(p.residual, o.residual) and p.q is None and p.q_scale is None
    assert torch.equal(p.rstd, o.rstd) and torch.equal(p.post_rstd, o.post_rstd)


@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("N,H", [(50, 2056), (1500, 2056), (1501, 256)])
def test_in_place_and_given_outputs(m, res, N, H):
    x, r, wp, w, c = inputs(N, H, res, "full", BF16, BF16)
    o = m.block_norm(x, r, wp, w, gate=c, quantize=True)
    r2, out = r.clone(), torch.empty_like(x)
    q, qs = torch.empty(N, H, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(N, device="cuda")
    o2 = m.block_norm(x, r2, wp, w, gate=c, residual_out=r2, out=out, quantize=True, q=q, q_scale=qs)
    assert o2.residual is r2 and o2.y is out and o2.q is q and o2.q_scale is qs
    assert torch.equal(r2, o.residual) and torch.equal(out, o.y) and torch.equal(qs, o.q_scale)
    assert torch.equal(q.view(torch.uint8), o.q.view(torch.uint8))


@pytest.mark.parametrize("N,H", [(12, 640), (1300, 2568)])
@pytest.mark.parametrize("gate", [None, "token", "full"])
def test_special_rows(m, N, H, gate):
    """Rows of zeros, of tiny and of huge values; NaN and infinities stay in their own rows; a closed gate."""
    x, r, wp, w, c = inputs(N, H, F32, gate, BF16, BF16)
    if c is not None:
        c = c.clone()
        c[0] = 0                                # nothing of the block's output
    x[1] = 0
    r[1] = 0                                    # a row of zeros
    x[2], r[2] = 0, r[2] * 1e-25                # the residual's squares vanish; eps covers them
    x[3] = (x[3].float() * 1e30).to(BF16)       # squares past fp32's range
    clean = m.block_norm(x, r, wp, w, gate=c, eps=EPS, quantize=True)
    e = forward64(x, r, wp, w, c, alpha=1.0)
    finite = torch.ones(N, dtype=torch.bool, device="cuda")
    finite[3] = False                           # its mean square, 1e60, counts as infinity
    for got, want, err in ((clean.y, e.y, e.y_err), (clean.residual, e.s, e.s_err)):
        rounding = U if got.dtype == BF16 else FP
        assert ((got.double() - want).abs() <= err + rounding * (want.abs() + err) + 1e-38)[finite].all()
    assert float(clean.post_rstd[3]) == 0 and torch.equal(clean.residual[3], r[3])
    assert (clean.y[1] == 0).all() and float(clean.q_scale[1]) == pytest.approx(1 / 448) and (clean.q[1].float() == 0).all()
    bad = x.clone()
    bad[5, 7], bad[6, 0] = float("nan"), float("inf")
    r2 = r.clone()
    r2[7, 639], r2[8, 1] = float("nan"), -float("inf")
    o = m.block_norm(bad, r2, wp, w, gate=c, eps=EPS, quantize=True)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[5:9] = False
    for f in ("y", "residual", "post_rstd", "rstd", "q_scale"):
        assert torch.equal(getattr(o, f)[rest], getattr(clean, f)[rest]), f
    assert torch.equal(o.q.view(torch.uint8)[rest], clean.q.view(torch.uint8)[rest])
    assert o.y[5].isnan().all() and o.y[7].isnan().all()


@pytest.mark.parametrize("N,H", [(3, 256), (2, 2048), (1, 16384), (2000, 1024)])
def test_rows_whose_squares_vanish_without_eps(m, N, H):
    """eps = 0: both roots are exact to fp32's precision however small the rows are."""
    for size in (1e-20, 1e-30, 1e-36):
        x, r = (rand(N, H) * size).to(BF16), rand(N, H, seed=1) * size
        wp = torch.ones(H, dtype=BF16, device="cuda")
        closed = torch.zeros(N, device="cuda")   # s = r, as small as it is
        o = m.block_norm(x, r, wp, wp, gate=closed, eps=0.0)
        post, rstd = x.double().square().mean(1).rsqrt(), r.double().square().mean(1).rsqrt()
        assert ((o.post_rstd.double() - post).abs() <= bound(H) * post).all()
        assert ((o.rstd.double() - rstd).abs() <= bound(H) * rstd).all()
        y = r.double() * rstd[:, None]
        assert ((o.y.double() - y).abs() <= (U + 2 * bound(H)) * y.abs()).all()


def backward64(dy, ds, s, x, rstd, post, wp, w, c, alpha=ALPHA):
    """Gradients in 64 bits from the stored s and roots, with their bounds before the last rounding."""
    H, N = x.shape[1], x.shape[0]
    shape_gate = None if c is None else c.dim()
    dy, s, x, wp, w = dy.double(), s.double(), x.double(), wp.double(), w.double()
    ds = torch.zeros_like(s) if ds is None else ds.double()
    rstd, post, c = rstd.double()[:, None], post.double()[:, None], gate64(c, x)
    steps = bound(H)
    o = SimpleNamespace()
    sh, xh, t = s * rstd, x * post, dy * w
    m1 = (t * sh).mean(1, keepdim=True)
    m1_err = (steps + 2 * FP) * (t * sh).abs().mean(1, keepdim=True)
    d = rstd * (t - sh * m1) + ds
    d_err = rstd * sh.abs() * m1_err + 6 * FP * (rstd * (t.abs() + (sh * m1).abs()) + ds.abs())
    o.dres, o.dres_err = alpha * d, abs(alpha) * d_err + FP * (alpha * d).abs()
    n = xh * wp
    if shape_gate == 2:
        o.dgate, o.dgate_err = d * n, n.abs() * d_err + 4 * FP * (d * n).abs()
    elif shape_gate == 1:
        o.dgate = (d * n).sum(1)
        o.dgate_err = (n.abs() * d_err).sum(1) + (steps + 4 * FP) * (d * n).abs().sum(1)
    e = d * c * wp
    e_err = (c * wp).abs() * d_err + 4 * FP * e.abs()
    m2 = (e * xh).mean(1, keepdim=True)
    m2_err = (e_err * xh.abs()).mean(1, keepdim=True) + (steps + 6 * FP) * (e * xh).abs().mean(1, keepdim=True)
    o.dx = post * (e - xh * m2)
    o.dx_err = post * (e_err + xh.abs() * m2_err) + 6 * FP * post * (e.abs() + (xh * m2).abs())
    rows = (N + 64) * FP                        # a column's sum over the rows, in any order
    o.dweight, o.dweight_err = (dy * sh).sum(0), rows * (dy * sh).abs().sum(0)
    o.dpost = (d * c * xh).sum(0)
    o.dpost_err = (d_err * (c * xh).abs()).sum(0) + rows * (d * c * xh).abs().sum(0)
    return o


def within(got, want, err, what):
    rounding = U if got.dtype == BF16 else FP
    bad = ~((got.double() - want).abs() <= err + rounding * (want.abs() + err) + 1e-38)
    assert not bad.any(), "%s: %d of %d outside" % (what, int(bad.sum()), bad.numel())


def check_backward(got, o, gate):
    dx, dres, dgate, dpost, dweight = got
    within(dx, o.dx, o.dx_err, "dx")
    within(dres, o.dres, o.dres_err, "dres")
    if gate is None:
        assert dgate is None
    else:
        within(dgate, o.dgate, o.dgate_err, "dgate")
    within(dpost, o.dpost, o.dpost_err, "dpost_weight")
    within(dweight, o.dweight, o.dweight_err, "dweight")


@pytest.mark.parametrize("N,H", SIZES)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_backward(m, N, H, kind):
    res, gate, pt, wt = KINDS[kind]
    x, r, wp, w, c = inputs(N, H, res, gate, pt, wt)
    f = m.block_norm(x, r, wp, w, gate=c, residual_scale=ALPHA, eps=EPS)
    dy, ds = rand(N, H, seed=8).to(BF16), rand(N, H, seed=9).to(res)
    for given in (ds, None):
        got = m.block_norm_backward(dy, x, f.residual, wp, w, f.post_rstd, f.rstd, gate=c, residual_scale=ALPHA, ds=given)
        assert got[1].dtype == res and (gate is None or got[2].shape == c.shape and got[2].dtype == c.dtype)
        check_backward(got, backward64(dy, given, f.residual, x, f.rstd, f.post_rstd, wp, w, c), gate)
        again = m.block_norm_backward(dy, x, f.residual, wp, w, f.post_rstd, f.rstd, gate=c, residual_scale=ALPHA, ds=given)
        for a, b in zip(got, again):            # sums in a fixed order: the same bits
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("gate", [None, "token", "full"])
def test_backward_against_differences(m, gate):
    """The formulas of backward64 against central differences of forward64's y and s."""
    N, H, eps = 3, 40, 1e-3
    x, r, wp, w, c = inputs(N, H, F32, gate, F32, F32)
    x, r, wp, w = [t.double() for t in (x, r, wp, w)]
    c = None if c is None else c.double()
    dy, ds = rand(N, H, seed=8).double(), rand(N, H, seed=9).double()

    def loss(x, r, wp, w, c):
        o = forward64(x, r, wp, w, c, eps=eps)
        return (o.y * dy + o.s * ds).sum()
    o = forward64(x, r, wp, w, c, eps=eps)
    g = backward64(dy, ds, o.s, x, o.rstd, o.post, wp, w, c)
    args = [x, r, wp, w] + ([] if c is None else [c])
    grads = [g.dx, g.dres, g.dpost, g.dweight] + ([] if c is None else [g.dgate])
    for i, (a, grad) in enumerate(zip(args, grads)):
        way = rand(*a.shape, seed=20 + i).double()
        h = 1e-5
        up, down = list(args), list(args)
        up[i], down[i] = a + h * way, a - h * way
        pad = [] if c is not None else [None]
        diff = (loss(*up, *pad) - loss(*down, *pad)) / (2 * h)
        # third derivatives of order ten and more: h^2 of them, and the rounding of the losses over h
        assert abs(float(diff - (grad * way).sum())) <= 1e-6 * float((grad * way).abs().sum())


@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("N,H", [(40, 640), (1300, 2568)])
def test_quantised_rows_of_every_size(m, N, H, res):
    """The 8-bit output's scale and values of rows from the smallest numbers to large ones, few rows and many."""
    size = 10.0 ** torch.linspace(-42 if res == F32 else -39, 18, N, device="cuda")[:, None]
    x, r = torch.zeros(N, H, dtype=BF16, device="cuda"), (rand(N, H) * size).to(res)
    w = torch.full((H,), 0.5, device="cuda")
    eps = 2.0 ** -80
    o = m.block_norm(x, r, w, w, eps=eps, quantize=True)
    e = forward64(x, r, w, w, None, alpha=1.0, eps=eps)
    check_forward(o, e, res, H)


def test_empty_batch(m):
    H = 256
    x, r, w = torch.empty(0, H, dtype=BF16, device="cuda"), torch.empty(0, H, device="cuda"), torch.ones(H, device="cuda")
    o = m.block_norm(x, r, w, w, quantize=True)
    assert o.y.shape == (0, H) and o.q.shape == (0, H) and o.rstd.shape == (0,)
    g = m.block_norm_backward(x, x, r, w, w, o.post_rstd, o.rstd, gate=torch.empty(0, device="cuda"))
    assert (g[3] == 0).all() and (g[4] == 0).all() and g[2].shape == (0,)


@pytest.mark.parametrize("N,H", [(5, 512), (7, 1000), (2500, 2568), (1400, 7168)])
def test_guard_zones(m, N, H):
    """Nothing is written outside the outputs."""
    x, r, wp, w, c = inputs(N, H, F32, "full", BF16, BF16)
    big = {k: torch.full((N + 2, H), 7.0, device="cuda").to(t) for k, t in
           (("out", BF16), ("residual_out", F32), ("q", torch.float8_e4m3fn))}
    qs = torch.full((N + 8,), 7.0, device="cuda")
    m.block_norm(x, r, wp, w, gate=c, quantize=True, q_scale=qs[4:N + 4], **{k: v[1:N + 1] for k, v in big.items()})
    for v in big.values():
        assert (v[0].float() == 7).all() and (v[N + 1].float() == 7).all()
    assert (qs[:4] == 7).all() and (qs[N + 4:] == 7).all()


def test_refusals(m):
    N, H = 4, 64
    x, r, wp, w, c = inputs(N, H, F32, "token", BF16, BF16)
    ok = dict(x=x, residual=r, post_weight=wp, weight=w)
    for change in (dict(x=x.float()), dict(x=x[:, ::2]), dict(x=x[0]), dict(residual=r.half()), dict(residual=r[:3]),
                   dict(residual=None), dict(post_weight=wp[:8]), dict(post_weight=None), dict(weight=w.half()),
                   dict(gate=c.to(BF16)), dict(gate=c[:3]), dict(gate=torch.ones(N, H, device="cuda")), dict(gate=c[None]),
                   dict(out=x.float()), dict(residual_out=x), dict(q=x), dict(quantize=True, q=x), dict(x=x.cpu())):
        with pytest.raises((ValueError, TypeError)):
            m.block_norm(**{**ok, **change})
    for change in (dict(eps=-1.0), dict(eps=float("nan")), dict(residual_scale=float("inf"))):
        with pytest.raises(m.MoeError):
            m.block_norm(**{**ok, **change})
    o = m.block_norm(**ok, gate=c)
    back = dict(dy=x, x=x, s=o.residual, post_weight=wp, weight=w, post_rstd=o.post_rstd, rstd=o.rstd, gate=c)
    for change in (dict(dy=x.float()), dict(x=x[:3]), dict(s=r.half()), dict(ds=x), dict(rstd=o.rstd[:3]), dict(gate=c[:3]),
                   dict(post_rstd=o.post_rstd.half()), dict(gate=x.float()), dict(weight=None)):
        with pytest.raises((ValueError, TypeError)):
            m.block_norm_backward(**{**back, **change})
    odd = torch.empty(N * H + 1, dtype=BF16, device="cuda")[1:].view(N, H)      # contiguous, 2 bytes off
    with pytest.raises(m.MoeError):
        m.block_norm(**{**ok, "x": odd})


def test_streams_and_graphs(m):
    """A captured forward and backward pass on other streams, replayed with new inputs."""
    N, H = 300, 2056
    x, r, wp, w, c = inputs(N, H, F32, "token", BF16, BF16)
    dy, ds = rand(N, H, seed=8).to(BF16), rand(N, H, seed=9)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()

    def both(stream=None):
        f = m.block_norm(x, r, wp, w, gate=c, quantize=True, stream=stream)
        return f, m.block_norm_backward(dy, x, f.residual, wp, w, f.post_rstd, f.rstd, gate=c, ds=ds, stream=stream)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        both(other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, g = both()
    for seed in (30, 40):
        new = inputs(N, H, F32, "token", BF16, BF16, seed=seed)
        for a, b in zip((x, r, wp, w, c), new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        f2, g2 = both(side)
        torch.cuda.synchronize()
        for a, b in zip((f.y, f.residual, f.rstd, f.post_rstd, f.q_scale) + tuple(g),
                        (f2.y, f2.residual, f2.rstd, f2.post_rstd, f2.q_scale) + tuple(g2)):
            assert torch.equal(a, b)


def test_large_offsets(m):
    """Rows past 2^31 elements."""
    H = 8192
    N = 2 ** 31 // H + 9
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    x, r = torch.zeros(N, H, dtype=BF16, device="cuda"), torch.zeros(N, H, dtype=BF16, device="cuda")
    gate = torch.ones(N, H, dtype=BF16, device="cuda")
    wp = w = torch.ones(H, dtype=BF16, device="cuda")
    last = inputs(9, H, BF16, "full", BF16, BF16)
    x[-9:], r[-9:], gate[-9:] = last[0], last[1], last[4]
    want = m.block_norm(x[-9:], r[-9:], wp, w, gate=gate[-9:], quantize=True, eps=EPS)
    got = m.block_norm(x, r, wp, w, gate=gate, quantize=True, eps=EPS)
    e = forward64(x[-9:], r[-9:], wp, w, gate[-9:], alpha=1.0)
    check_forward(want, e, BF16, H)
    tail = SimpleNamespace(**{f: getattr(got, f)[-9:] for f in ("y", "residual", "post_rstd", "rstd", "q", "q_scale")})
    check_forward(tail, e, BF16, H)
    del got.q
    dy = torch.zeros(N, H, dtype=BF16, device="cuda")
    dy[-9:] = rand(9, H, seed=8).to(BF16)
    back = m.block_norm_backward(dy, x, got.residual, wp, w, got.post_rstd, got.rstd, gate=gate)
    o = backward64(dy[-9:], None, got.residual[-9:], x[-9:], got.rstd[-9:], got.post_rstd[-9:], wp, w, gate[-9:], alpha=1.0)
    check_backward((back[0][-9:], back[1][-9:], back[2][-9:], back[3], back[4]), o, "full")

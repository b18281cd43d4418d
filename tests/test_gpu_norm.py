"""The residual norm and its gradient against the formulas in 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8          # bf16 rounding, relative
FP = 2.0 ** -24        # one fp32 rounding


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


# the row in one warp (up to 512), in a block with 1, 2 or 4 chunks a thread, and the bounds between them
SIZES = [(1, 8), (3, 128), (7, 256), (5, 264), (129, 512), (2, 520), (1, 2048), (33, 2056), (4, 4096), (9, 7168),
         (3, 8200), (2, 16384), (1, 32768), (1000, 136)]


def rel_bound(H):
    # sum of squares: H additions in a tree of at most H/8 + 12 sequential steps a thread, then the square root,
    # the division and two products
    return (H / 8 + 30) * FP


@pytest.mark.parametrize("N,H", SIZES)
@pytest.mark.parametrize("res,wt", [(None, BF16), (BF16, F32), (F32, BF16)])
def test_forward(m, N, H, res, wt):
    x = rand(N, H).to(BF16)
    w = (1 + 0.2 * rand(H, seed=1)).to(wt)
    r = None if res is None else (rand(N, H, seed=2) * torch.exp(2 * rand(N, 1, seed=3))).to(res)
    o = m.residual_norm(x, w, residual=r, eps=1e-5, quantize=True)
    s = x.double() + (0 if r is None else r.double())
    rstd = (s.square().mean(1) + 1e-5).rsqrt()
    y = s * rstd[:, None] * w.double()
    b = rel_bound(H)
    # s is rounded once to fp32; rows with cancellation keep an absolute error of the addends' size
    s_err = 0 if r is None else FP * s.abs()
    assert ((o.rstd.double() - rstd).abs() <= b * rstd).all()
    y_fp32 = b * y.abs() + 2 * s_err * rstd[:, None] * w.double().abs()
    assert ((o.y.double() - y).abs() <= y_fp32 + U * (y.abs() + y_fp32) + 1e-38).all()
    if r is None:
        assert o.residual is None
    else:
        assert ((o.residual.double() - s).abs() <= (FP if res == F32 else U + FP) * s.abs() + 1e-38).all()
    amax = y.abs().amax(1)
    assert ((o.q_scale.double() - amax / 448).abs() <= (2 * b + 4 * FP) * amax / 448).all()
    # e4m3: 3 mantissa bits, relative 2^-4 of the value, 2^-10 absolute below the normal range
    q = o.q.float().double()
    v = y / o.q_scale.double()[:, None]
    assert (q.abs() <= 448).all()
    assert ((q - v).abs() <= (2.0 ** -4 + 4 * b) * v.abs() + 2.0 ** -10).all()
    # without the 8-bit output: the same bits
    p = m.residual_norm(x, w, residual=r, eps=1e-5)
    assert torch.equal(p.y, o.y) and torch.equal(p.rstd, o.rstd) and p.q is None and p.q_scale is None


@pytest.mark.parametrize("res", [BF16, F32])
def test_residual_in_place(m, res):
    x, r, w = rand(50, 2056).to(BF16), rand(50, 2056, seed=1).to(res), torch.ones(2056, dtype=BF16, device="cuda")
    o = m.residual_norm(x, w, residual=r)
    r2 = r.clone()
    o2 = m.residual_norm(x, w, residual=r2, residual_out=r2)
    assert o2.residual is r2 and torch.equal(r2, o.residual) and torch.equal(o2.y, o.y)


def test_special_rows(m):
    """Rows of zeros, of tiny and of huge values; a NaN or an infinity stays in its own row."""
    H = 640
    x = rand(8, H).to(BF16)
    x[0] = 0
    x[1] *= 1e-30
    x[2] = 1e18
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    w = torch.ones(H, dtype=BF16, device="cuda")
    o = m.residual_norm(x, w, eps=1e-6, quantize=True)
    assert (o.y[0] == 0).all() and (o.q[0].float() == 0).all() and float(o.q_scale[0]) == pytest.approx(1 / 448)
    assert float(o.rstd[0]) == pytest.approx(1e3, rel=1e-6)
    want = x[1].double() * 1e3
    assert ((o.y[1].double() - want).abs() <= 2 * U * want.abs()).all()
    back = o.q[1].float() * o.q_scale[1]
    assert ((back.double() - want).abs() <= (2.0 ** -4 + 1e-4) * want.abs() + 2.0 ** -9 * want.abs().max()).all()
    assert ((o.y[2].float() - 1).abs() <= 2 * U).all()
    assert torch.isnan(o.y[3]).any() and not torch.isfinite(o.y[4]).all()
    ref = m.residual_norm(x[5:].contiguous(), w, eps=1e-6, quantize=True)
    assert torch.equal(o.y[5:], ref.y) and torch.equal(o.q[5:].view(torch.uint8), ref.q.view(torch.uint8))


def test_tiny_scale(m):
    """A weight so small that the scale's reciprocal would overflow."""
    H = 256
    x = rand(2, H).to(BF16)
    w = torch.full((H,), 1e-38, dtype=F32, device="cuda")
    o = m.residual_norm(x, w, quantize=True)
    v = x.double() * (x.double().square().mean(1, keepdim=True) + 1e-6).rsqrt() * 1e-38
    back = o.q.float().double() * o.q_scale.double()[:, None]
    # the scale (2^-134 or so) has about 14 bits, e4m3 4
    assert torch.isfinite(o.q.float()).all()
    assert ((back - v).abs() <= 2.0 ** -4 * v.abs() + 2.0 ** -8 * v.abs().amax(1, keepdim=True)).all()


@pytest.mark.parametrize("N,H", SIZES + [(5000, 256), (3000, 1024)])
@pytest.mark.parametrize("st,wt,with_ds", [(BF16, BF16, True), (F32, F32, True), (F32, BF16, False), (BF16, F32, False)])
def test_backward(m, N, H, st, wt, with_ds):
    s = (rand(N, H) * torch.exp(rand(N, 1, seed=4))).to(st)
    dy = rand(N, H, seed=1).to(BF16)
    w = (1 + 0.2 * rand(H, seed=2)).to(wt)
    ds = rand(N, H, seed=3).to(st) if with_ds else None
    rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
    dx, dres, dwt = m.residual_norm_backward(dy, s, w, rstd, ds=ds)
    S, D, R = s.double(), dy.double(), rstd.double()[:, None]
    xhat, t = S * R, D * w.double()
    mean = (t * xhat).mean(1, keepdim=True)
    d = R * (t - xhat * mean) + (0 if ds is None else ds.double())
    b = rel_bound(H)
    tol = R * (8 * FP * t.abs() + xhat.abs() * (b * (t * xhat).abs().mean(1, keepdim=True) + 8 * FP * mean.abs()))
    tol = tol + 4 * FP * ((R * t).abs() + (0 if ds is None else ds.double().abs()) + d.abs())
    assert ((dx.double() - d).abs() <= tol + U * (d.abs() + tol) + 1e-38).all()
    if st == F32:
        assert ((dres.double() - d).abs() <= tol + 1e-38).all()
    else:
        assert dres is None
    # at most N additions in sequence
    wt_tol = (N + 8) * FP * (D * xhat).abs().sum(0)
    assert ((dwt.double() - (D * xhat).sum(0)).abs() <= wt_tol).all()
    again = m.residual_norm_backward(dy, s, w, rstd, ds=ds)
    assert torch.equal(again[0], dx) and torch.equal(again[2], dwt)


def test_gradient_against_differences(m):
    """The formula's gradient (held to the kernel above) is that of the forward pass."""
    N, H, eps = 3, 40, 1e-3
    x, w, dy = rand(N, H).double(), rand(H, seed=1).double(), rand(N, H, seed=2).double()
    f = lambda x, w: ((x * (x.square().mean(1, keepdim=True) + eps).rsqrt() * w) * dy).sum()  # noqa: E731
    rstd = (x.square().mean(1, keepdim=True) + eps).rsqrt()
    xhat, t = x * rstd, dy * w
    dx, dw = rstd * (t - xhat * (t * xhat).mean(1, keepdim=True)), (dy * xhat).sum(0)
    for i, (g, ref) in enumerate(((dx, x), (dw, w))):
        d = rand(*ref.shape, seed=5 + i).double()
        h = 1e-6
        num = (f(x + h * d, w) - f(x - h * d, w)) / (2 * h) if i == 0 else (f(x, w + h * d) - f(x, w - h * d)) / (2 * h)
        assert abs(float(num - (g * d).sum())) <= 1e-6 * float((g * d).abs().sum())


def test_empty_batch_and_refusals(m):
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    o = m.residual_norm(z(0, 64), z(64), quantize=True)
    assert o.y.shape == (0, 64) and o.q.shape == (0, 64)
    dx, dres, dw = m.residual_norm_backward(z(0, 64), z(0, 64), z(64), z(0, t=F32))
    assert dx.shape == (0, 64) and (dw == 0).all()
    with pytest.raises(ValueError):
        m.residual_norm(z(4, 64, t=torch.float16), z(64))
    with pytest.raises(ValueError):
        m.residual_norm(z(4, 64), z(64), residual=z(4, 65))
    with pytest.raises(ValueError):
        m.residual_norm(z(4, 64), z(64), residual_out=z(4, 64))
    with pytest.raises(ValueError):
        m.residual_norm(z(4, 128)[:, ::2], z(64))            # not contiguous
    with pytest.raises(m.MoeError):
        m.residual_norm(z(4, 60), z(60))                     # H % 8
    with pytest.raises(m.MoeError):
        m.residual_norm(z(1, 40000), z(40000))               # wider than a block's registers
    with pytest.raises(m.MoeError):
        m.residual_norm(z(1, 64), z(64), eps=float("nan"))


def test_other_stream(m):
    x, r, w = rand(64, 1024).to(BF16), rand(64, 1024, seed=1), torch.ones(1024, dtype=BF16, device="cuda")
    want = m.residual_norm(x, w, residual=r, quantize=True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = m.residual_norm(x, w, residual=r, quantize=True, stream=st)
    st.synchronize()
    assert torch.equal(got.y, want.y) and torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8))

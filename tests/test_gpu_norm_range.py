"""The residual norm of rows whose squares are large, small or vanish in fp32, against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8          # bf16 rounding, relative
FP = 2.0 ** -24        # one fp32 rounding

SCALES = [1e-36, 1e-33, 1e-30, 1e-25, 1e-22, 1e-21, 1e-20, 1e-19, 1e-18, 1e-10, 1.0, 1e10, 1e15, 1e18]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


# a row in a warp, in a block (1, 2 and 4 chunks a thread), and many rows (the ring, where eps covers small squares)
@pytest.mark.parametrize("N,H", [(14, 136), (14, 512), (14, 520), (14, 4096), (14, 8200), (2800, 1032), (2800, 4096)])
@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-6])
def test_row_sizes(m, N, H, res, eps):
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    size = torch.tensor(SCALES, device="cuda").repeat(N // len(SCALES))[:, None]
    draw = lambda: torch.randn(N, H, generator=g, device="cuda").clamp(-3, 3) * size  # noqa: E731
    x = draw().to(BF16)
    r = None if res is None else draw().to(res)
    w = torch.ones(H, dtype=BF16, device="cuda")
    o = m.residual_norm(x, w, residual=r, eps=eps, quantize=True)
    s = x.double() + (0 if r is None else r.double())
    e = float(torch.tensor(eps, dtype=F32))               # what a float argument holds
    rstd = (s.square().mean(1) + e).rsqrt()
    y = s * rstd[:, None]
    # the sum's steps, the square root and the products; s is rounded once to fp32
    b = (H / 8 + 30) * FP + 4 * FP
    assert ((o.rstd.double() - rstd).abs() <= b * rstd).all()
    fp32 = (b + 2 * FP) * y.abs() + 2.0 ** -149 * rstd[:, None]
    assert ((o.y.double() - y).abs() <= fp32 + U * (y.abs() + fp32) + 1e-38).all()
    amax = y.abs().amax(1)
    assert ((o.q_scale.double() - amax / 448).abs() <= (2 * b + 4 * FP) * amax / 448).all()
    q, v = o.q.float().double(), y / o.q_scale.double()[:, None]
    assert ((q - v).abs() <= (2.0 ** -4 + 4 * b) * v.abs() + 2.0 ** -10).all()


def test_mean_square_beyond_fp32(m):
    """A mean square above fp32's largest number counts as infinity, in few rows and in many."""
    for N in (4, 2800):
        x = torch.full((N, 1032), 1e25, dtype=BF16, device="cuda")
        o = m.residual_norm(x, torch.ones(1032, dtype=BF16, device="cuda"), quantize=True)
        assert (o.rstd == 0).all() and (o.y == 0).all() and (o.q.float() == 0).all()


@pytest.mark.parametrize("N", [2, 5000])
def test_scale_at_the_end_of_fp32(m, N):
    """Outputs so small that max|v| / 448 is no number of fp32: the scale stays above 0 and zeros stay zeros."""
    H = 640
    x = torch.randn(N, H, device="cuda").to(BF16)
    x[:, ::3] = 0
    w = torch.full((H,), 4e-44, dtype=F32, device="cuda")
    o = m.residual_norm(x, w, quantize=True)
    assert (o.q_scale == 2.0 ** -149).all()
    assert torch.isfinite(o.q.float()).all() and (o.q.float()[:, ::3] == 0).all()
    v = x.double() * (x.double().square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.double()
    back = o.q.float().double() * o.q_scale.double()[:, None]
    # v itself is known to a unit of 2^-149, and q to 2^-4 of it
    assert ((back - v).abs() <= 2.0 ** -4 * v.abs() + 2 * 2.0 ** -149).all()

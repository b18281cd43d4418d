"""The 8-bit output of the norms between blocks with weights and rows from the smallest to the largest numbers.

The row's scale is its largest |v| over 448 for every finite v, whether few rows run (a block a row) or many (the ring of
rows), and whatever the product of a value and its weight is before the row's root.  Bounds: those of the forward tests;
a scale below 2^-126 has half a step of 2^-149 on top.
"""
import pytest
import torch

from test_gpu_block_norm import BF16, F32, FP, U, forward64, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


# weights' exponent, the residual stream's exponent; values near 2^128 are where v itself would overflow
CASES = [(100, 0), (118, 0), (40, 57), (26, 60), (110, 40), (60, -40), (-20, 30), (-100, -30), (-126, -40), (-120, 50), (0, 0)]


@pytest.mark.parametrize("N,H", [(12, 640), (12, 2568), (1300, 2568), (20001, 1024), (1300, 7168)])
@pytest.mark.parametrize("wide", [F32, BF16])
def test_scales(m, N, H, wide):
    for up, size in CASES:
        x = torch.zeros(N, H, dtype=BF16, device="cuda")
        r = (rand(N, H, seed=1) * 2.0 ** size).to(F32 if N < 5000 else BF16)    # (the ring takes fp32 rows from 2056 columns on)
        w = ((1 + 0.2 * rand(H, seed=2)) * 2.0 ** up).to(wide)
        wp = torch.ones(H, device="cuda")
        eps = 2.0 ** -95
        o = m.block_norm(x, r, wp, w, eps=eps, quantize=True)
        e = forward64(x, r, wp, w, None, alpha=1.0, eps=eps)
        assert e.y.abs().max() < 2.0 ** 128
        amax = e.y.abs().amax(1)
        step = 2.0 ** -149
        scale_err = e.y_err.amax(1) / 448 + 4 * FP * amax / 448 + step
        scale = o.q_scale.double()
        assert ((scale - amax / 448).abs() <= scale_err).all(), (up, size)
        q, v = o.q.float().double(), e.y / scale[:, None]
        v_err = (e.y_err + step) / scale[:, None] + 6 * FP * v.abs()
        assert ((q - v).abs() <= v_err + 2.0 ** -4 * (v.abs() + v_err) + 2.0 ** -10).all(), (up, size)
        assert ((o.y.double() - e.y).abs() <= e.y_err + U * (e.y.abs() + e.y_err) + 1e-38).all(), (up, size)


@pytest.mark.parametrize("N,H", [(12, 2568), (1300, 2568)])
def test_one_large_weight(m, N, H):
    """A weight that overflows by itself when scaled, at places where the row is zero and where it is not."""
    x, r, wp = torch.zeros(N, H, dtype=BF16, device="cuda"), rand(N, H, seed=1), torch.ones(H, device="cuda")
    w = torch.ones(H, device="cuda")
    w[7], w[2000] = 2.0 ** 110, 2.0 ** 127
    r[:, 2000] = 0
    r[::2, 7] = 0
    o = m.block_norm(x, r, wp, w, quantize=True)
    e = forward64(x, r, wp, w, None, alpha=1.0, eps=1e-6)
    amax = e.y.abs().amax(1)
    assert ((o.q_scale.double() - amax / 448).abs() <= e.y_err.amax(1) / 448 + 4 * FP * amax / 448).all()
    top = e.y.abs().argmax(1, keepdim=True)
    assert (o.q.float().gather(1, top).abs() == 448).all()

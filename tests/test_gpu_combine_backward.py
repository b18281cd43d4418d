"""The combine's gradient against the formulas in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
U = 2.0 ** -8
FP = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def case(m, N, E, K, R, a, H, seed=0):
    g = np.random.default_rng(seed)
    idx = torch.from_numpy(np.argsort(g.random((N, E)), axis=1)[:, :K].astype(np.int32).copy()).cuda()
    p = m.plan(idx, E, R, a)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    y = r(p.P_cap, H).to(BF16)
    y[p.src_of_slot < 0] = float("nan")                      # rows of no pair are not read
    return p, r(N, H).to(BF16), y, torch.rand(N, K, generator=gen, device="cuda")


@pytest.mark.parametrize("N,E,K,R,a,H", [
    (1, 4, 1, 1, 1, 8), (1, 8, 8, 2, 8, 256), (5, 8, 2, 2, 16, 136), (64, 16, 3, 4, 1, 1000), (333, 8, 2, 4, 16, 4096),
    (257, 64, 8, 8, 128, 2048), (40, 64, 6, 8, 8, 520), (19, 32, 32, 4, 4, 264), (700, 8, 4, 2, 7, 72),
    (100, 256, 8, 8, 128, 7168)])
def test_formula(m, N, E, K, R, a, H):
    p, dout, y, w = case(m, N, E, K, R, a, H)
    out = torch.full_like(y, 7.0)
    dy, dw = m.combine_backward(dout, y, w, p, dy=out)
    slot = torch.where(p.dst >= 0, p.dst, -p.dst - 1).long()
    P = int(p.cu_seqlens[-1])
    want = w.double()[:, :, None] * dout.double()[:, None, :]
    # the product of two exact factors is rounded to fp32, then to bf16
    assert ((dy[slot.reshape(-1)].double().reshape(N, K, H) - want).abs() <= (U + 2 * FP) * want.abs() + 1e-38).all()
    prod = dout.double()[:, None, :] * y[slot.reshape(-1)].double().reshape(N, K, H)
    assert ((dw.double() - prod.sum(-1)).abs() <= (H / 8 + 30) * FP * prod.abs().sum(-1)).all()
    live = torch.zeros(p.P_cap, dtype=torch.bool, device="cuda")
    live[slot.reshape(-1)] = True
    pad = ~live & (torch.arange(p.P_cap, device="cuda") < P)
    assert (dy[pad] == 0).all() and (dy[P:] == 7).all()
    assert m.get_status(p) == 0
    again = m.combine_backward(dout, y, w, p, dy=torch.full_like(y, 7.0))
    assert torch.equal(again[0].view(torch.int16), dy.view(torch.int16)) and torch.equal(again[1], dw)


def test_is_the_combines_gradient(m):
    """<dout, combine(y + d) - combine(y)> = <dy, d>, and the same for the weights: the combine is linear in both."""
    N, E, K, H = 50, 8, 4, 128
    p, dout, y, w = case(m, N, E, K, 2, 8, H)
    y = torch.nan_to_num(y.float(), nan=0.0).to(BF16)
    dy, dw = m.combine_backward(dout, y, w, p, dy=torch.zeros_like(y))
    slot = torch.where(p.dst >= 0, p.dst, -p.dst - 1).long()

    def combine(y, w):
        return (w[:, :, None] * y[slot.reshape(-1)].reshape(N, K, H)).sum(1)
    d = torch.randn(y.shape, device="cuda", dtype=torch.float64)
    lhs = (dout.double() * (combine(y.double() + d, w.double()) - combine(y.double(), w.double()))).sum()
    terms = dy.double() * d
    assert abs(float(lhs - terms.sum())) <= 2 * U * float(terms.abs().sum())
    e = torch.randn(w.shape, device="cuda", dtype=torch.float64)
    lhs = (dout.double() * (combine(y.double(), w.double() + e) - combine(y.double(), w.double()))).sum()
    terms = dw.double() * e
    assert abs(float(lhs - terms.sum())) <= 1e-4 * float(terms.abs().sum())


def test_bad_slots_and_plan_errors(m):
    p, dout, y, w = case(m, 20, 8, 2, 2, 8, 64)
    p.dst[3, 1] = 1 << 30
    out = torch.full_like(y, 7.0)
    m.combine_backward(dout, y, w, p, dy=out)
    assert m.get_status(p) == 6
    p.status[0] = 6
    out = torch.full_like(y, 7.0)
    m.combine_backward(dout, y, w, p, dy=out)
    assert (out == 7).all() and m.get_status(p) == 6


def test_empty_batch_and_refusals(m):
    p, dout, y, w = case(m, 4, 8, 2, 2, 8, 64)
    with pytest.raises(ValueError):
        m.combine_backward(dout, y.float(), w, p)
    with pytest.raises(ValueError):
        m.combine_backward(dout, y, w[:, :1].contiguous(), p)
    with pytest.raises(ValueError):
        m.combine_backward(dout[:3].contiguous(), y, w, p)
    e = m.plan(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 8, 2, 8)
    dy, dw = m.combine_backward(dout[:0], y[:0], w[:0], e)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)

"""The operators around the experts where element offsets pass 2^31: sampled rows against 64 bits."""
import numpy as np
import pytest
import torch

import block_checks as bc

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    yield m
    torch.cuda.empty_cache()


def rows_of(n, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = torch.empty(n, H, dtype=BF16, device="cuda")
    for i in range(0, n, 1 << 17):
        out[i:i + (1 << 17)] = torch.randn(min(1 << 17, n - i), H, generator=g, device="cuda").to(BF16)
    return out


def test_expert_ffn(m):
    H, I = 2048, 64  # noqa: E741
    counts = [600_001, 0, 599_990]
    p = bc.groups(counts, 16, 3)
    assert p.rows * H > 1 << 31
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    wgu = (torch.randn(3, 2, I, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    wd = (torch.randn(3, H, I, generator=g, device="cuda") * I ** -0.5).to(BF16)
    x, dy = rows_of(p.rows, H, 1), rows_of(p.rows, H, 2)
    h = torch.empty(p.rows, I, dtype=BF16, device="cuda")
    pre = torch.empty(p.rows, 2, I, device="cuda")
    y = m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
    dx, dwgu, dwd = m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p)
    assert int(p.status[0]) == 0
    for e in (0, 2):
        first, n = p.begins[e], counts[e]
        pick = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda") + first
        sub = bc.groups([5], 1)
        W, D = wgu[e:e + 1].double(), wd[e:e + 1].double()
        o = bc.ffn_forward(x[pick].double(), W, D, sub)
        bc.assert_within(h[pick], o.h, bc.h_bound(o, H), "h")
        bc.assert_within(y[pick], o.y, bc.y_bound(o, D, sub, H), "y")
        b = bc.ffn_backward(dy[pick].double(), x[pick].double(), h[pick].double(), pre[pick, 0].double(),
                            pre[pick, 1].double(), W, D, sub)
        bc.assert_within(dx[pick], b.dx, b.dx_tol, "dx")
        # the weights' gradients, summed in 64 bits over slices of the group.  The bound takes the worst rounding of
        # every dg, du (U each) and the sum's; 600000 rows bring F * n near 0.15 of the magnitudes' sum, far above the
        # actual error, so the 2-norm is held to the independent-rounding estimate too
        want_d, mag = torch.zeros_like(dwd[e], dtype=torch.float64), torch.zeros_like(dwd[e], dtype=torch.float64)
        for i in range(first, first + n, 1 << 16):
            j = min(i + (1 << 16), first + n)
            want_d += dy[i:j].double().T @ h[i:j].double()
            mag += dy[i:j].double().abs().T @ h[i:j].double().abs()
        err = (dwd[e].double() - want_d).abs()
        assert (err <= n * bc.F * mag + bc.U * want_d.abs()).all()
        assert float(err.norm()) <= bc.U * float(want_d.norm())
    assert (dwgu[1] == 0).all() and (dwd[1] == 0).all()


def test_norm(m):
    N, H = 1_100_000, 2048
    assert N * H > 1 << 31
    x = rows_of(N, H, 3)
    w = torch.ones(H, dtype=BF16, device="cuda")
    o = m.residual_norm(x, w, eps=0.0, quantize=True)
    pick = torch.tensor([0, N // 2, N - 2, N - 1], device="cuda")
    want = x[pick].double()
    want = want * want.square().mean(1, keepdim=True).rsqrt()
    assert ((o.y[pick].double() - want).abs() <= (bc.U + 1e-4) * want.abs()).all()
    back = o.q.view(torch.uint8)[pick].view(torch.float8_e4m3fn).float() * o.q_scale[pick, None]
    assert ((back.double() - want).abs() <= (2.0 ** -4 + 1e-4) * want.abs() + 2.0 ** -9 * want.abs().amax(1, keepdim=True)).all()
    dx, _, _ = m.residual_norm_backward(o.y, x, w, o.rstd)
    xhat, t = want, o.y[pick].double()
    d = o.rstd[pick].double()[:, None] * (t - xhat * (t * xhat).mean(1, keepdim=True))
    # t nearly cancels against xhat: what is left is y's rounding, known to an ulp of t
    assert ((dx[pick].double() - d).abs() <= bc.U * d.abs() + 2.0 ** -12 * t.abs()).all()


def test_combine_backward(m):
    N, E, K, H = 300_000, 16, 8, 1024
    g = np.random.default_rng(0)
    idx = torch.from_numpy(np.argsort(g.random((N, E), dtype=np.float32), axis=1)[:, :K].astype(np.int32).copy()).cuda()
    p = m.plan(idx, E, 4, 16)
    assert p.P_cap * H > 1 << 31
    y, dout = rows_of(p.P_cap, H, 4), rows_of(N, H, 5)
    w = torch.rand(N, K, device="cuda")
    dy, dw = m.combine_backward(dout, y, w, p)
    assert m.get_status(p) == 0
    pick = torch.tensor([0, 1, N // 2, N - 1], device="cuda")
    slot = torch.where(p.dst >= 0, p.dst, -p.dst - 1).long()[pick]
    assert int(slot.max()) * H > 1 << 31
    want = w[pick].double()[:, :, None] * dout[pick].double()[:, None, :]
    assert ((dy[slot].double() - want).abs() <= (bc.U + 2.0 ** -22) * want.abs()).all()
    prod = dout[pick].double()[:, None, :] * y[slot].double()
    assert ((dw[pick].double() - prod.sum(-1)).abs() <= (H / 8 + 30) * 2.0 ** -24 * prod.abs().sum(-1)).all()

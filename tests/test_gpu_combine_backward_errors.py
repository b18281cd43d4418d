"""The combine's gradient where slots are bad: the error is reported, good tokens before it are unharmed, no block hangs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


@pytest.mark.parametrize("N", [3, 200, 700, 1500, 5000])   # 8, 8, 4, 2 and 1 warps a token
def test_error_recorded_while_blocks_start(m, N):
    """A bad slot in the first token: whatever the later blocks read of the status, the call ends, reports the error,
    and every weight gradient is either the sum or untouched."""
    E, K, H = 8, 2, 1024
    g = np.random.default_rng(0)
    idx = torch.from_numpy(np.argsort(g.random((N, E)), axis=1)[:, :K].astype(np.int32).copy()).cuda()
    p = m.plan(idx, E, 2, 8)
    y, dout = torch.randn(p.P_cap, H, device="cuda").to(BF16), torch.randn(N, H, device="cuda").to(BF16)
    w = torch.rand(N, K, device="cuda")
    _, want = m.combine_backward(dout, y, w, p)
    p.dst[0, 0] = 1 << 30
    for _ in range(50):
        dw = torch.full((N, K), 7.0, device="cuda")
        m.combine_backward(dout, y, w, p, dw=dw)
        assert m.get_status(p) == 6
        assert (dw[0] == 7).all()
        assert ((dw == want) | (dw == 7)).all()

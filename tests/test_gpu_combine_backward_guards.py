"""Guard zones around the outputs of the combine's gradient."""
import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
GUARD = 256


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


@pytest.mark.parametrize("N,E,K,H,align", [(1, 8, 8, 136, 1), (37, 8, 3, 1000, 16), (700, 16, 2, 520, 7),
                                           (3000, 64, 6, 264, 128)])
def test_nothing_is_written_beside_the_outputs(m, N, E, K, H, align):
    from expert_dispatch_planning_gb300 import _lib
    g = np.random.default_rng(0)
    idx = torch.from_numpy(np.argsort(g.random((N, E)), axis=1)[:, :K].astype(np.int32).copy()).cuda()
    p = m.plan(idx, E, 1, align)
    P = int(p.cu_seqlens[-1])                    # exactly the groups' rows
    y, dout = torch.randn(P, H, device="cuda").to(BF16), torch.randn(N, H, device="cuda").to(BF16)
    w = torch.rand(N, K, device="cuda")
    raw_dy = torch.full((P * H + 2 * GUARD,), 3.0, dtype=BF16, device="cuda")
    raw_dw = torch.full((N * K + 2 * GUARD,), 3.0, device="cuda")
    dy, dw = raw_dy[GUARD:GUARD + P * H].view(P, H), raw_dw[GUARD:GUARD + N * K].view(N, K)
    rc = _lib.load().moe_combine_backward(dout.data_ptr(), y.data_ptr(), w.data_ptr(), N, K, H, E, P,
                                          ctypes.byref(p.c_struct), dy.data_ptr(), dw.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and m.get_status(p) == 0
    for raw, t in ((raw_dy, dy), (raw_dw, dw)):
        assert (raw[:GUARD] == 3).all() and (raw[GUARD + t.numel():] == 3).all()
    want = m.combine_backward(dout, y, w, p)
    assert torch.equal(want[0], dy) and torch.equal(want[1], dw)

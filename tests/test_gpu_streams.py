"""Planning calls on a stream that is not the current one, with the buffers they allocate themselves."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000      # cycles of a kernel that only sleeps: about 0.1 s, far longer than the calls


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def choice(N, E, K, seed=0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(np.argsort(g.random((N, E)), axis=1)[:, :K].astype(np.int32).copy()).cuda()


def test_rank_layout_workspace_outlives_the_call(m):
    """The workspace is released as the call returns; the current stream's next tensors must not get it."""
    N, R, C = 200_000, 8, 10
    p = m.plan(choice(N, 16, 2), 16, R, 8)
    want = [t.clone() for t in m.rank_layout(p, C)]
    size = m.rank_layout_workspace(N, R).numel()
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(SLEEP)
        got = m.rank_layout(p, C, stream=st)
        others = [torch.full((size,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert all((t == 0x5a).all() for t in others)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del got, others


def test_plan_status_is_ready_on_the_calls_stream(m):
    """The plan's status is zeroed on the stream that plans, not behind the current stream's work."""
    idx = choice(300, 16, 2)
    want = m.plan(idx, 16, 4, 8)
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        dirty = [torch.full((4,), 6, dtype=torch.int32, device="cuda") for _ in range(64)]
        torch.cuda.synchronize()
        del dirty
        torch.cuda._sleep(SLEEP)
        p = m.plan(idx, 16, 4, 8, stream=st)
        st.synchronize()
        with torch.cuda.stream(st):
            got = [t.cpu() for t in (p.status, p.cu_seqlens, p.dst)]
        assert not got[0].any()
        assert torch.equal(got[1], want.cu_seqlens.cpu()) and torch.equal(got[2], want.dst.cpu())
        torch.cuda.synchronize()
        assert m.get_status(p) == 0

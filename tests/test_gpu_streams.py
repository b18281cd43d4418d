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


def stream_calls(m):
    """Calls that allocate their outputs: name -> (call(stream), what counts of its outputs)."""
    N, E, K, R, H = 4000, 16, 2, 4, 256
    logits = torch.randn(N, E, device="cuda")
    idx = choice(N, E, K)
    p = m.plan(idx, E, R, 8)
    x = torch.randn(N, H, device="cuda").to(torch.bfloat16)
    xp = m.permute(x, p)
    P = int(p.cu_seqlens[-1])
    w = torch.rand(N, K, device="cuda")

    tiles_n = int(m.tile_map(p)[2][0])
    return {
        "route_topk": (lambda st: m.route_topk(logits, K, stream=st), list),
        "route_plan": (lambda st: m.route_plan(logits, K, R, 8, stream=st),
                       lambda o: [o[0], o[1], o[2].cu_seqlens, o[2].dst, o[2].status]),
        "plan": (lambda st: m.plan(idx, E, R, 8, stream=st), lambda o: [o.cu_seqlens, o.dst, o.is_token_in_rank, o.status]),
        "plan_balanced": (lambda st: m.plan_balanced(idx, p, 8, 4 * N, 2, 1 << 20, stream=st),
                          lambda o: [getattr(o, k) for k in ("z", "alloc", "expert_offsets", "dst")]),
        "tile_map": (lambda st: m.tile_map(p, stream=st), lambda o: [o[0][:tiles_n], o[1][:tiles_n], o[2]]),
        "rank_layout": (lambda st: m.rank_layout(p, 10, stream=st), list),
        "permute": (lambda st: m.permute(x, p, stream=st), lambda o: [o[:P]]),
        "combine": (lambda st: m.combine(xp, w, p, stream=st), lambda o: [o]),
    }


@pytest.mark.parametrize("name", ["route_topk", "route_plan", "plan", "plan_balanced", "tile_map", "rank_layout", "permute",
                                  "combine"])
def test_outputs_are_not_waiting_to_be_written(m, name):
    """Memory that the current stream has released but will still write to does not become an output on another one."""
    call, pick = stream_calls(m)[name]
    first = call(None)
    want = [t.clone() for t in pick(first)]
    sizes = sorted({t.numel() * t.element_size() for t in pick(first)}) + [16, 64, 4 * (10 + 4000) * 8]
    del first
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        held = [torch.full((s,), 0x5a, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]
        del held                              # released; the writes are queued
        out = call(st)
        st.synchronize()
        torch.cuda.synchronize()
        got = pick(out)
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
        del out, got

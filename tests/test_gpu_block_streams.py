"""The operators around the experts on a stream that is not the current one, with the buffers they allocate themselves.

What a call allocates has to belong to the stream it runs on.  Two ways to see
that it does not: a workspace that is released as the call returns goes to the
current stream's next tensors while the kernels still use it; and memory that
work queued on the current stream will still write to becomes a workspace or an
output.  A kernel that only sleeps keeps the streams apart.
"""
from types import SimpleNamespace

import pytest
import torch

import block_checks as bc

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
SLEEP = 200_000_000      # cycles: about 0.1 s, far longer than the calls below
NAMES = ["ffn", "ffn_backward", "norm", "norm_backward", "combine_backward"]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def case(m, name):
    """A call that leaves every buffer it can to the binding: call(stream), what counts of its outputs, and the bytes
    of its workspaces and outputs (all above a megabyte, or small)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    if name.startswith("ffn"):
        H, I = 512, 384  # noqa: E741
        p = bc.groups([700, 3, 0, 900], 16)
        P, live = p.rows, p.kind < 2
        x, dy, wgu, wd = r(P, H), r(P, H), r(4, 2, I, H, std=H ** -0.5), r(4, H, I, std=I ** -0.5)
        if name == "ffn":
            return (lambda st: [m.expert_ffn(x, wgu, wd, p, stream=st)], lambda o: [o[0][live]], [P * I * 2, P * H * 2])
        h, pre = torch.empty(P, I, dtype=BF16, device="cuda"), torch.empty(P, 2, I, device="cuda")
        m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
        return (lambda st: m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, stream=st),
                lambda o: [o[0][live], o[1], o[2]], [P * I * 4, P * H * 2, wgu.numel() * 2, wd.numel() * 2])
    N, H = 1500, 1024
    s, dy, w = r(N, H), r(N, H), r(H)
    rstd = torch.rand(N, generator=g, device="cuda") + 0.5
    every = lambda o: list(o)  # noqa: E731
    if name == "norm":
        def norm(st):
            o = m.residual_norm(s, w, residual=dy, quantize=True, stream=st)
            return [o.y, o.residual, o.rstd, o.q.view(torch.uint8), o.q_scale]
        return norm, every, [N * H * 2, N * H, N * 4]
    if name == "norm_backward":
        blocks = [torch.cuda.get_device_properties(0).multi_processor_count * k for k in range(1, 7)]
        return (lambda st: [t for t in m.residual_norm_backward(dy, s, w, rstd, stream=st) if t is not None], every,
                [N * H * 2, H * 4, N * H * 4] + [b * H * 4 for b in blocks])
    i32 = dict(dtype=torch.int32, device="cuda")
    p = SimpleNamespace(dst=torch.arange(N, **i32).reshape(N, 1), zero_fill_ranges=torch.zeros(1, 2, **i32),
                        status=torch.zeros(4, **i32))
    ones = torch.ones(N, 1, device="cuda")
    return lambda st: m.combine_backward(dy, s, ones, p, stream=st), every, [N * H * 2, N * 4]


def fill(sizes):
    return [torch.full((s,), 0x5a, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(3)]


@pytest.mark.parametrize("name", NAMES)
def test_workspaces_outlive_the_call(m, name):
    """Tensors that the current stream makes after the call, while the call's stream has not begun it."""
    call, pick, sizes = case(m, name)
    want = [t.clone() for t in pick(call(None))]
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(SLEEP)
        out = call(st)
        others = fill(sizes)
        torch.cuda.synchronize()
        assert all((t == 0x5a).all() for t in others)
        got = pick(out)
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
        del out, got, others


@pytest.mark.parametrize("name", NAMES)
def test_buffers_are_not_waiting_to_be_written(m, name):
    """Memory that the current stream has released but will still write to, after the call's stream is done."""
    call, pick, sizes = case(m, name)
    want = [t.clone() for t in pick(call(None))]
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        fill(sizes)                       # released at once; the writes are queued
        out = call(st)
        st.synchronize()
        torch.cuda.synchronize()
        got = pick(out)
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))
        del out, got


def test_outputs_are_the_current_streams_to_use(m):
    """An output read on the current stream and released: its memory does not go to the call's stream meanwhile."""
    call, pick, sizes = case(m, "norm")
    want = [t.clone() for t in call(None)]
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        out = call(st)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda._sleep(SLEEP)
        kept = [t.clone() for t in out]   # read after the sleep
        del out
        with torch.cuda.stream(st):
            others = fill(sizes)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        del others


def test_default_stream_by_its_handle(m):
    """The default stream given while another one is current."""
    call, pick, _ = case(m, "ffn")
    want = pick(call(None))[0].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(pick(out)[0], want)

"""The experts' gated feed-forward and its gradients against the formulas in 64 bits."""
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
    return m


def make(counts, align, H, I, seed=0, extra=5, fp8=False):  # noqa: E741
    """Rows with NaN, infinities and large values wherever no group is."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    p = bc.groups(counts, align, extra)
    E = len(counts)
    x, wgu, wd = r(p.rows, H), r(E, 2, I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5).to(BF16)
    dead = p.kind > 0
    if fp8:
        xs, ws = x.abs().amax(-1) / 448, wgu.abs().amax(-1) / 448
        x8, w8 = (x / xs[:, None]).to(torch.float8_e4m3fn), (wgu / ws[..., None]).to(torch.float8_e4m3fn)
        x8.view(torch.uint8)[dead] = 0x7f                     # NaN
        xs[dead] = float("inf")
        return p, x8, xs, w8, ws, wd
    x = x.to(BF16)
    x[dead] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38], device="cuda").to(BF16).repeat(
        (int(dead.sum()) * H + 3) // 4)[:int(dead.sum()) * H].reshape(-1, H)
    return p, x, wgu.to(BF16), wd


SIZES = [
    # counts, alignment, H, I
    ([1], 1, 8, 8),                                  # the smallest of everything
    ([0, 0, 3, 0], 8, 64, 40),                       # empty experts around one
    ([0, 0, 0], 4, 64, 64),                          # no rows at all
    ([5, 1, 0, 130], 16, 72, 136),                   # sizes that fill no tile
    ([127, 128, 129, 1], 1, 256, 128),               # around the tile's rows, no alignment
    ([300, 2, 0, 77, 256], 128, 520, 264),           # long and short groups, wide alignment
    ([1] * 60, 8, 512, 192),                         # single tokens over many experts
    ([64, 1000, 17, 0, 33, 513], 32, 1000, 504),     # ragged
    ([40, 30], 1000, 128, 72),                       # padding far longer than a tile
    ([700, 900], 16, 2048, 768),                     # long contractions
]


@pytest.mark.parametrize("counts,align,H,I", SIZES)
def test_forward(m, counts, align, H, I):  # noqa: E741
    p, x, wgu, wd = make(counts, align, H, I)
    M = p.rows
    h = torch.full((M, I), 7.0, dtype=BF16, device="cuda")
    pre = torch.full((M, 2, I), 7.0, device="cuda")
    out = torch.full((M, H), 7.0, dtype=BF16, device="cuda")
    y = m.expert_ffn(x, wgu, wd, p, h=h, preact=pre, out=out)
    assert y is out
    o = bc.ffn_forward(torch.nan_to_num(x.double()), wgu.double(), wd.double(), p)
    live = p.kind == 0
    assert (y[p.kind == 1] == 0).all() and (y[p.kind == 2] == 7).all()
    bc.assert_within(pre[live][:, 0], o.g[live], (H * bc.F * o.g_abs)[live], "g")
    bc.assert_within(pre[live][:, 1], o.u[live], (H * bc.F * o.u_abs)[live], "u")
    bc.assert_within(h[live], o.h[live], bc.h_bound(o, H)[live], "h")
    bc.assert_within(y[live], o.y[live], bc.y_bound(o, wd.double(), p, H)[live], "y")
    assert int(p.status[0]) == 0
    # without the saved pre-activations: the same bits
    y2 = m.expert_ffn(x, wgu, wd, p, out=torch.full_like(out, 7.0))
    assert torch.equal(y2, y)


@pytest.mark.parametrize("counts,align,H,I", [s for s in SIZES if s[2] % 16 == 0])
def test_forward_8bit(m, counts, align, H, I):  # noqa: E741
    p, x8, xs, w8, ws, wd = make(counts, align, H, I, fp8=True)
    out = torch.full((p.rows, H), 7.0, dtype=BF16, device="cuda")
    h = torch.empty((p.rows, I), dtype=BF16, device="cuda")
    y = m.expert_ffn(x8, w8, wd, p, x_scale=xs, w_scale=ws, h=h, out=out)
    live = p.kind == 0
    x = torch.where(live[:, None], x8.float().double() * xs.double()[:, None], 0.0)
    w = w8.float().double() * ws.double()[..., None]
    o = bc.ffn_forward(x, w, wd.double(), p)
    assert (y[p.kind == 1] == 0).all() and (y[p.kind == 2] == 7).all()
    bc.assert_within(h[live], o.h[live], bc.h_bound(o, H)[live], "h")
    bc.assert_within(y[live], o.y[live], bc.y_bound(o, wd.double(), p, H)[live], "y")


@pytest.mark.parametrize("counts,align,H,I", SIZES)
def test_backward(m, counts, align, H, I):  # noqa: E741
    p, x, wgu, wd = make(counts, align, H, I)
    M = p.rows
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    live = p.kind == 0
    dy = torch.randn(M, H, generator=g, device="cuda").to(BF16)
    dy[~live] = float("nan")
    h = torch.full((M, I), float("nan"), dtype=BF16, device="cuda")
    pre = torch.full((M, 2, I), float("inf"), device="cuda")
    ws = torch.full((M, 2, I), float("nan"), dtype=BF16, device="cuda")
    m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
    dx = torch.full((M, H), 7.0, dtype=BF16, device="cuda")
    got = m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, dx=dx, dgate_up=ws)
    clean = lambda t: torch.nan_to_num(t.double(), posinf=0.0, neginf=0.0)  # noqa: E731
    o = bc.ffn_backward(clean(dy), clean(x), clean(h), clean(pre[:, 0]), clean(pre[:, 1]), wgu.double(), wd.double(), p)
    assert (dx[p.kind == 1] == 0).all() and (dx[p.kind == 2] == 7).all()
    bc.assert_within(dx[live], o.dx[live], o.dx_tol[live], "dx")
    bc.assert_within(got[1], o.dwgu, o.dwgu_tol, "dw_gate_up")
    bc.assert_within(got[2], o.dwd, o.dwd_tol, "dw_down")
    assert int(p.status[0]) == 0
    # one output at a time: the same bits, and None for the others
    a = m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, dx=torch.full_like(dx, 7.0), need_dw=False)
    b = m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, need_dx=False)
    assert torch.equal(a[0], dx) and a[1] is None and a[2] is None
    assert b[0] is None and torch.equal(b[1], got[1]) and torch.equal(b[2], got[2])


def test_gradient_against_differences(m):
    """Directional derivatives of the 64-bit forward agree with the formula's
    gradients, which the kernels' are held to above."""
    p, x, wgu, wd = make([9, 0, 21], 8, 48, 40)
    X, G, D = torch.nan_to_num(x.double(), posinf=0.0, neginf=0.0), wgu.double(), wd.double()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    dy = torch.randn(p.rows, 48, generator=gen, device="cuda", dtype=torch.float64) * (p.kind == 0)[:, None]
    o = bc.ffn_forward(X, G, D, p)
    b = bc.ffn_backward(dy, X, o.h, o.g, o.u, G, D, p)
    step = 1e-6
    for i, grad in ((0, b.dx), (1, b.dwgu), (2, b.dwd)):
        args = [X, G, D]
        d = torch.randn(args[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + step * d, args[i] - step * d
        num = ((bc.ffn_forward(*up, p).y - bc.ffn_forward(*down, p).y) * dy).sum() / (2 * step)
        # central differences in 64 bits: step^2 and 1e-16/step errors, both under 1e-8 of the sum's size
        assert abs(float(num - (grad * d).sum())) <= 1e-6 * float((grad * d).abs().sum())


def test_extreme_activations(m):
    """Gates so large that e^-g overflows or vanishes: silu is 0 or g, and no NaN appears."""
    p = bc.groups([4], 1)
    H = I = 64  # noqa: E741
    x = torch.zeros(4, H, dtype=BF16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = 1e4, -1e4, 1e30, -1e30
    wgu = torch.zeros(1, 2, I, H, dtype=BF16, device="cuda")
    wgu[0, :, :, 0] = 1.0
    wd = torch.zeros(1, H, I, dtype=BF16, device="cuda")
    wd[0].fill_diagonal_(1.0)
    h = torch.empty(4, I, dtype=BF16, device="cuda")
    pre = torch.empty(4, 2, I, device="cuda")
    y = m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
    v = x[:, 0].double()
    want = torch.where(v > 0, v * v, 0.0)
    fits = want < 3e38                                   # row 2's product is beyond fp32
    want = want[:, None].expand(4, H)
    bc.assert_within(y[fits], want[fits], 3 * bc.U * want[fits], "y")
    assert not torch.isfinite(y[2]).any()
    dx, dwgu, dwd = m.expert_ffn_backward(torch.ones(4, H, dtype=BF16, device="cuda"), x, h, pre, wgu, wd, p)
    assert torch.isfinite(dx[:2]).all()


def test_plan_object_and_device_errors(m):
    """A Plan goes in as it is; a group outside the rows and a plan error are reported and write nothing bad."""
    N, E, K, R, H, I = 37, 8, 2, 2, 64, 72  # noqa: E741
    gen = np.random.default_rng(0)
    idx = torch.from_numpy(np.argsort(gen.random((N, E)), axis=1)[:, :K].astype(np.int32).copy()).cuda()
    plan = m.plan(idx, E, R, 8)
    xt = torch.randn(N, H, device="cuda").to(BF16)
    wgu, wd = (torch.randn(*s, device="cuda").mul(0.1).to(BF16) for s in ((E, 2, I, H), (E, H, I)))
    xp = m.permute(xt, plan)
    y = m.expert_ffn(xp, wgu, wd, plan, out=torch.zeros_like(xp))
    counts = plan.tokens_per_expert.tolist()
    p = bc.groups(counts, 8, xp.shape[0] - int(plan.cu_seqlens[-1]))
    o = bc.ffn_forward(torch.where((p.kind == 0)[:, None], xp.double(), 0.0), wgu.double(), wd.double(), p)
    live = p.kind == 0
    bc.assert_within(y[live], o.y[live], bc.y_bound(o, wd.double(), p, H)[live], "y")
    assert m.get_status(plan) == 0
    # fewer rows than the groups need: reported, and nothing of the group that does not fit is written
    cut = int(plan.cu_seqlens[E - 1])
    out = torch.full((cut + 1, H), 7.0, dtype=BF16, device="cuda")
    m.expert_ffn(xp[:cut + 1].contiguous(), wgu, wd, plan, out=out)
    assert (out[cut:] == 7).all()
    assert m.get_status(plan) == 6                       # MOE_ERR_DEVICE_INDEX
    # an error in the status: nothing is written
    plan.status[0] = 6
    out = torch.full_like(xp, 7.0)
    m.expert_ffn(xp, wgu, wd, plan, out=out)
    assert (out == 7).all()
    assert m.get_status(plan) == 6


def test_other_stream_and_graph(m):
    """On a stream of the caller's, and replayed from a captured graph with new contents."""
    p, x, wgu, wd = make([33, 4, 0, 90], 8, 128, 136)
    want = m.expert_ffn(x, wgu, wd, p, out=torch.zeros(p.rows, 128, dtype=BF16, device="cuda"))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = torch.zeros_like(want)
    h = torch.empty(p.rows, 136, dtype=BF16, device="cuda")
    m.expert_ffn(x, wgu, wd, p, out=out, h=h, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(want)
    with torch.cuda.graph(graph):
        m.expert_ffn(x, wgu, wd, p, out=out2, h=h)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, want)
    x.mul_(2)
    want2 = m.expert_ffn(x, wgu, wd, p, out=torch.zeros_like(want))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, want2) and not torch.equal(want, want2)


def test_empty_batch(m):
    p = bc.groups([0, 0], 1)
    z = lambda *s, t=BF16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    wgu, wd = z(2, 2, 16, 32), z(2, 32, 16)
    assert m.expert_ffn(z(0, 32), wgu, wd, p).shape == (0, 32)
    dx, a, b = m.expert_ffn_backward(z(0, 32), z(0, 32), z(0, 16), z(0, 2, 16, t=torch.float32), wgu, wd, p)
    assert dx.shape == (0, 32) and (a == 0).all() and (b == 0).all()


def test_guard_zones(m):
    """Nothing is written beside the outputs: rows before and after them keep their pattern."""
    p, x, wgu, wd = make([129, 3, 0, 40], 8, 136, 72, extra=0)
    M, H, I = p.rows, 136, 72  # noqa: E741

    def guarded(*shape, dtype=BF16):
        n = int(np.prod(shape))
        raw = torch.full((n + 256,), 3.0, dtype=dtype, device="cuda")
        return raw, raw[128:128 + n].view(*shape)
    y, h, pre, ws, dx = guarded(M, H), guarded(M, I), guarded(M, 2, I, dtype=torch.float32), guarded(M, 2, I), guarded(M, H)
    m.expert_ffn(x, wgu, wd, p, h=h[1], preact=pre[1], out=y[1])
    dy = torch.randn(M, H, device="cuda").to(BF16)
    m.expert_ffn_backward(dy, x, h[1], pre[1], wgu, wd, p, dx=dx[1], dgate_up=ws[1])
    torch.cuda.synchronize()
    for raw, t in (y, h, pre, ws, dx):
        assert (raw[:128] == 3).all() and (raw[128 + t.numel():] == 3).all()


def step(m, case, bufs=None):
    """A forward and backward pass; its outputs."""
    p, x, wgu, wd, dy = case
    M, H, I = x.shape[0], x.shape[1], wd.shape[2]  # noqa: E741
    h = torch.empty(M, I, dtype=BF16, device="cuda")
    pre = torch.empty(M, 2, I, device="cuda")
    y = m.expert_ffn(x, wgu, wd, p, h=h, preact=pre, out=torch.zeros_like(x))
    return (y, *m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, dx=torch.zeros_like(x)))


def cases():
    out = []
    for i, (counts, align, H, I) in enumerate([([300, 2, 0, 77, 256, 900], 8, 520, 264), ([64] * 40, 16, 256, 512)]):  # noqa: E741
        p, x, wgu, wd = make(counts, align, H, I, seed=10 + i)
        out.append((p, x, wgu, wd, torch.randn(p.rows, H, device="cuda").to(BF16)))
    return out


def test_two_streams_at_once(m):
    """Steps of different sizes on two streams, overlapping: the bits of the steps alone."""
    cs = cases()
    want = [step(m, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        got = []
        for c, st in zip(cs, streams):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(step(m, c))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert all(int(c[0].status[0]) == 0 for c in cs)


def test_training_step_in_a_graph(m):
    """Forward and backward captured and replayed, four kernels that start before their predecessors end."""
    c = cases()[0]
    want = step(m, c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step(m, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(m, c)
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_without_programmatic_launches(m, tmp_path):
    """MOE_PDL=0, every kernel in plain stream order: the same bits."""
    import os
    import subprocess
    import sys

    from conftest import ROOT
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import torch, test_gpu_expert_ffn as t, expert_dispatch_planning_gb300 as m\n"
            "torch.manual_seed(0)\n"
            "torch.save([[v.cpu() for v in t.step(m, c)] for c in t.cases()], sys.argv[1])\n"
            % (ROOT, os.path.join(ROOT, "tests")))
    runs = []
    for pdl in ("1", "0"):
        path = str(tmp_path / ("out%s.pt" % pdl))
        res = subprocess.run([sys.executable, "-c", code, path], env=dict(os.environ, MOE_PDL=pdl), capture_output=True,
                             text=True, timeout=300)
        assert res.returncode == 0, res.stderr[-2000:]
        runs.append(torch.load(path))
    assert all(torch.equal(a, b) for s, t in zip(*runs) for a, b in zip(s, t))


def test_wait_that_runs_out(m):
    """With a limit far below what a long product takes, the kernel gives up, says so and leaves the GPU usable."""
    p, x, wgu, wd = make([40_000, 50], 16, 256, 256)
    dy = torch.randn(x.shape, device="cuda").to(BF16)
    want = step(m, (p, x, wgu, wd, dy))
    torch.cuda.synchronize()
    assert int(p.status[0]) == 0
    try:
        m.set_plan_fault(-1, 1000)          # 1 us a wait; a tile of dw here takes hundreds
        step(m, (p, x, wgu, wd, dy))
        torch.cuda.synchronize()
        assert int(p.status[0]) == 5        # MOE_ERR_DEVICE_TIMEOUT
    finally:
        m.set_plan_fault()
    out = torch.full_like(x, 7.0)
    m.expert_ffn(x, wgu, wd, p, out=out)    # the error stands: nothing is written
    assert (out == 7).all()
    p.status.zero_()
    got = step(m, (p, x, wgu, wd, dy))
    assert int(p.status[0]) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))

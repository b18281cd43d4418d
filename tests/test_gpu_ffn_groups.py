"""The experts' feed-forward over other layouts of groups than the planner's, and many experts, against 64 bits."""
from types import SimpleNamespace

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


def layout(counts, sizes, extra=3):
    """Groups of `counts` rows in places of `sizes` rows."""
    begins = [0]
    for s in sizes:
        begins.append(begins[-1] + s)
    rows = begins[-1] + extra
    kind = torch.full((rows,), 2, dtype=torch.int64)
    for b, n, s in zip(begins, counts, sizes):
        kind[b:b + n], kind[b + n:b + s] = 0, 1
    i32 = dict(dtype=torch.int32, device="cuda")
    return SimpleNamespace(cu_seqlens=torch.tensor(begins, **i32), tokens_per_expert=torch.tensor(counts, **i32),
                           status=torch.zeros(4, **i32), rows=rows, counts=list(counts), begins=begins, kind=kind.cuda())


def check_step(m, p, H, I, seed=0):  # noqa: E741
    """A forward and backward step with NaN and infinities in the rows of no group: every output against 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    E, M = len(p.counts), p.rows
    x, dy, wgu, wd = r(M, H), r(M, H), r(E, 2, I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5)
    live = p.kind == 0
    x[~live], dy[~live] = float("nan"), float("inf")
    full = lambda *s, t=BF16, v=7.0: torch.full(s, v, dtype=t, device="cuda")  # noqa: E731
    h, pre = full(M, I), full(M, 2, I, t=torch.float32)
    y = m.expert_ffn(x, wgu, wd, p, h=h, preact=pre, out=full(M, H))
    dx, dwgu, dwd = m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, dx=full(M, H))
    assert int(p.status[0]) == 0
    W, D = wgu.double(), wd.double()
    clean = lambda t: torch.where(live.reshape(-1, *[1] * (t.dim() - 1)), t.double(), 0.0)  # noqa: E731
    o = bc.ffn_forward(clean(x), W, D, p)
    bc.assert_within(h[live], o.h[live], bc.h_bound(o, H)[live], "h")
    bc.assert_within(y[live], o.y[live], bc.y_bound(o, D, p, H)[live], "y")
    pre = clean(pre)
    b = bc.ffn_backward(clean(dy), clean(x), clean(h), pre[:, 0], pre[:, 1], W, D, p)
    bc.assert_within(dx[live], b.dx[live], b.dx_tol[live], "dx")
    bc.assert_within(dwgu, b.dwgu, b.dwgu_tol, "dw_gate_up")
    bc.assert_within(dwd, b.dwd, b.dwd_tol, "dw_down")
    for out in (y, dx):
        assert (out[p.kind == 1] == 0).all() and (out[p.kind == 2] == 7).all()


@pytest.mark.parametrize("counts,sizes", [
    ([5, 0, 130, 0], [160, 160, 160, 160]),          # a place of fixed size for every expert, two of them empty
    ([0, 0, 0], [16, 300, 1]),                       # nothing but padding
    ([0, 257, 0, 0, 3], [40, 512, 0, 7, 3]),         # empty places first, in the middle and of no rows
])
def test_places_of_empty_experts(m, counts, sizes):
    """The padding of a group without rows is written as zeros too."""
    check_step(m, layout(counts, sizes), 136, 72)


def test_any_of_the_gradients_alone(m):
    """The C call with each choice of dx, dw_gate_up and dw_down: the bits of all three together."""
    import ctypes
    import itertools

    from expert_dispatch_planning_gb300 import _lib
    p, H, I = bc.groups([70, 0, 3, 300], 16), 136, 72  # noqa: E741
    E, M = len(p.counts), p.rows
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    x, dy, wgu, wd = r(M, H), r(M, H), r(E, 2, I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5)
    h, pre = torch.empty(M, I, dtype=BF16, device="cuda"), torch.empty(M, 2, I, device="cuda")
    m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
    plan = _lib.MoePlanOut()
    plan.cu_seqlens, plan.tokens_per_expert = p.cu_seqlens.data_ptr(), p.tokens_per_expert.data_ptr()
    plan.status = p.status.data_ptr()
    shapes, want = [(M, H), (E, 2, I, H), (E, H, I)], None
    for pick in sorted(itertools.product((True, False), repeat=3), reverse=True):
        out = [torch.full(s, 7.0, dtype=BF16, device="cuda") for s in shapes]
        dgu = torch.empty(M, 2, I, dtype=BF16, device="cuda")
        rc = _lib.load().moe_expert_ffn_backward(
            dy.data_ptr(), x.data_ptr(), h.data_ptr(), pre.data_ptr(), wgu.data_ptr(), wd.data_ptr(), M, E, H, I,
            ctypes.byref(plan), dgu.data_ptr(), *[t.data_ptr() if k else None for t, k in zip(out, pick)],
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and int(p.status[0]) == 0
        want = want or out
        for t, k, w in zip(out, pick, want):
            assert torch.equal(t, w) if k else (t == 7).all()


def many(E, seed=0):
    """Groups of no rows, single rows, a few, and (every 97th) more than a tile."""
    g = torch.Generator()
    g.manual_seed(seed)
    kind = torch.randint(0, 4, (E,), generator=g).tolist()
    few = torch.randint(2, 40, (E,), generator=g).tolist()
    return [300 + e % 7 if e % 97 == 5 else (0, 1, 0, few[e])[kind[e]] for e in range(E)]


# a thread of the groups' scan has one expert up to 352 (384 in the gradients' launch), then two, at most three; with 1024
# the groups' tables take 16 KB from the ring
@pytest.mark.parametrize("E", [352, 353, 384, 385, 705, 1024])
def test_many_experts(m, E):
    check_step(m, bc.groups(many(E), 8, 3), 72, 40, seed=E)


@pytest.mark.parametrize("E", [353, 1024])
def test_many_experts_8bit(m, E):
    H, I = 144, 40  # noqa: E741
    p = bc.groups(many(E), 16, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    x, wgu, wd = r(p.rows, H), r(E, 2, I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5).to(BF16)
    xs, ws = x.abs().amax(-1) / 448, wgu.abs().amax(-1) / 448
    x8, w8 = (x / xs[:, None]).to(torch.float8_e4m3fn), (wgu / ws[..., None]).to(torch.float8_e4m3fn)
    live = p.kind == 0
    x8.view(torch.uint8)[~live] = 0x7f                 # NaN
    y = m.expert_ffn(x8, w8, wd, p, x_scale=xs, w_scale=ws, out=torch.full((p.rows, H), 7.0, dtype=BF16, device="cuda"))
    xd = torch.where(live[:, None], x8.float().double() * xs.double()[:, None], 0.0)
    o = bc.ffn_forward(xd, w8.float().double() * ws.double()[..., None], wd.double(), p)
    bc.assert_within(y[live], o.y[live], bc.y_bound(o, wd.double(), p, H)[live], "y")
    assert (y[p.kind == 1] == 0).all() and (y[p.kind == 2] == 7).all() and int(p.status[0]) == 0


def test_gate_up_gradient_at_large_offsets(m):
    """dw_gate_up of groups whose rows pass 2^31 elements, from the stored dgate_up, against sums in 64 bits."""
    H, I = 2048, 64  # noqa: E741
    counts = [600_001, 0, 599_990]
    p = bc.groups(counts, 16, 3)
    assert p.rows * H > 1 << 31
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def rows(n, cols):
        out = torch.empty(n, cols, dtype=BF16, device="cuda")
        for i in range(0, n, 1 << 17):
            out[i:i + (1 << 17)] = torch.randn(min(1 << 17, n - i), cols, generator=g, device="cuda").to(BF16)
        return out
    wgu = (torch.randn(3, 2, I, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    wd = (torch.randn(3, H, I, generator=g, device="cuda") * I ** -0.5).to(BF16)
    x, dy = rows(p.rows, H), rows(p.rows, H)
    h, pre = torch.empty(p.rows, I, dtype=BF16, device="cuda"), torch.empty(p.rows, 2, I, device="cuda")
    m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
    dgu = torch.empty(p.rows, 2, I, dtype=BF16, device="cuda")
    dx, dwgu, _ = m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, dgate_up=dgu)
    assert int(p.status[0]) == 0 and (dwgu[1] == 0).all()
    for e in (0, 2):
        first, n = p.begins[e], counts[e]
        want, mag = (torch.zeros(2 * I, H, dtype=torch.float64, device="cuda") for _ in range(2))
        for i in range(first, first + n, 1 << 16):
            j = min(i + (1 << 16), first + n)
            a, b = dgu[i:j].reshape(j - i, 2 * I).double(), x[i:j].double()
            want += a.T @ b
            mag += a.abs().T @ b.abs()
        err = (dwgu[e].reshape(2 * I, H).double() - want).abs()
        # each addition as in the error model; and, far closer, the independent roundings' size in the 2-norm
        assert (err <= n * bc.F * mag + bc.U * want.abs()).all()
        assert float(err.norm()) <= bc.U * float(want.norm())

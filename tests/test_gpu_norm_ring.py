"""The residual norm and its gradient of many rows, in every form of the ring, all rows against 64 bits.

Rows go to blocks that stay, each with a ring of 8, 4 or (backward) 2 rows in shared memory; the number of slots follows from the
bytes of a row's slot, and the ring is taken from four rows a block on.  `blocks` restates that rule, so that the sizes
here lie just below, at and above it, and the rows are no multiple of the blocks."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8          # bf16 rounding, relative
FP = 2.0 ** -24        # one fp32 rounding


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def ring(H, slot):
    """(slots, blocks) for rows whose slot takes `slot` bytes."""
    smem = 220 * 1024
    slots = 8 if 8 * slot <= smem // 2 else 4 if 4 * slot <= smem else 2
    threads = (H + 255) // 256 * 32
    per_sm = max(1, min(smem // (slots * slot), 1536 // threads, 6))
    return slots, torch.cuda.get_device_properties(0).multi_processor_count * per_sm


def rand(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def rel_bound(H):
    # sum of squares: a tree of at most H/8 + 12 sequential steps a thread, then the root and two products
    return (H / 8 + 30) * FP


# widths that fill the block's columns and widths that leave threads idle
WIDTHS = [520, 1032, 2048, 2056, 4104, 7168, 7176, 8192]


def test_every_number_of_slots_is_met():
    forward = {ring(H, H * b)[0] for H in WIDTHS for b in (2, 4, 6)}
    backward = {ring(H, H * b)[0] for H in WIDTHS for b in (4, 6, 10)}
    assert forward == {8, 4} and backward == {8, 4, 2}


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("quantize", [True, False])
def test_forward(m, H, res, quantize):
    _, blocks = ring(H, H * {None: 2, BF16: 4, F32: 6}[res])
    for N, wt in ((4 * blocks - 1, BF16), (4 * blocks, F32), (4 * blocks + blocks // 2 + 1, BF16)):
        x = rand(N, H).to(BF16)
        w = (1 + 0.2 * rand(H, seed=1)).to(wt)
        r = None if res is None else (rand(N, H, seed=2) * torch.exp(2 * rand(N, 1, seed=3))).to(res)
        o = m.residual_norm(x, w, residual=r, eps=1e-5, quantize=quantize)
        s = x.double() + (0 if r is None else r.double())
        rstd = (s.square().mean(1) + 1e-5).rsqrt()
        y = s * rstd[:, None] * w.double()
        b = rel_bound(H)
        s_err = 0 if r is None else FP * s.abs()
        assert ((o.rstd.double() - rstd).abs() <= b * rstd).all()
        fp32 = b * y.abs() + 2 * s_err * rstd[:, None] * w.double().abs()
        assert ((o.y.double() - y).abs() <= fp32 + U * (y.abs() + fp32) + 1e-38).all()
        if r is not None:
            assert ((o.residual.double() - s).abs() <= (FP if res == F32 else U + FP) * s.abs() + 1e-38).all()
            into = r.clone()
            again = m.residual_norm(x, w, residual=into, eps=1e-5, quantize=quantize, residual_out=into)
            assert again.residual is into and torch.equal(into, o.residual) and torch.equal(again.y, o.y)
        if quantize:
            amax = y.abs().amax(1)
            assert ((o.q_scale.double() - amax / 448).abs() <= (2 * b + 4 * FP) * amax / 448).all()
            q, v = o.q.float().double(), y / o.q_scale.double()[:, None]
            assert ((q - v).abs() <= (2.0 ** -4 + 4 * b) * v.abs() + 2.0 ** -10).all()
        else:
            assert o.q is None and o.q_scale is None


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("st", [BF16, F32])
@pytest.mark.parametrize("with_ds", [True, False])
def test_backward(m, H, st, with_ds):
    _, blocks = ring(H, H * (2 + (2 if with_ds else 1) * (2 if st == BF16 else 4)))
    for N, wt in ((4 * blocks - 1, BF16), (4 * blocks, F32), (4 * blocks + blocks // 2 + 1, BF16)):
        s = (rand(N, H) * torch.exp(rand(N, 1, seed=4))).to(st)
        dy = rand(N, H, seed=1).to(BF16)
        w = (1 + 0.2 * rand(H, seed=2)).to(wt)
        ds = rand(N, H, seed=3).to(st) if with_ds else None
        rstd = (s.float().square().mean(1) + 1e-6).rsqrt()
        dx, dres, dwt = m.residual_norm_backward(dy, s, w, rstd, ds=ds)
        S, D, R = s.double(), dy.double(), rstd.double()[:, None]
        xhat, t = S * R, D * w.double()
        mean = (t * xhat).mean(1, keepdim=True)
        d = R * (t - xhat * mean) + (0 if ds is None else ds.double())
        b = rel_bound(H)
        tol = R * (8 * FP * t.abs() + xhat.abs() * (b * (t * xhat).abs().mean(1, keepdim=True) + 8 * FP * mean.abs()))
        tol = tol + 4 * FP * ((R * t).abs() + (0 if ds is None else ds.double().abs()) + d.abs())
        assert ((dx.double() - d).abs() <= tol + U * (d.abs() + tol) + 1e-38).all()
        if st == F32:
            assert ((dres.double() - d).abs() <= tol + 1e-38).all()
        else:
            assert dres is None
        # a block's rows in sequence, then the blocks in 32 runs of which each is a sequence
        steps = N // blocks + 2 + blocks // 32 + 32
        assert ((dwt.double() - (D * xhat).sum(0)).abs() <= (steps + 8) * FP * (D * xhat).abs().sum(0)).all()


@pytest.mark.parametrize("N,H", [(5, 136), (9, 2056), (3, 16384), (1900, 4104), (4000, 520)])
def test_guard_zones(m, N, H):
    """Nothing is written beside the outputs, in few rows and in many."""
    from expert_dispatch_planning_gb300 import _lib
    lib, guard = _lib.load(), 512

    def guarded(*shape, t=BF16):
        n = 1
        for k in shape:
            n *= k
        raw = torch.full((n + 2 * guard,), 3.0, dtype=torch.float32, device="cuda").to(t)
        return raw, raw[guard:guard + n].view(*shape)
    x, r, w = rand(N, H).to(BF16), rand(N, H, seed=1), torch.ones(H, dtype=BF16, device="cuda")
    y, ro, rstd, qs = guarded(N, H), guarded(N, H, t=F32), guarded(N, t=F32), guarded(N, t=F32)
    q = guarded(N, H, t=torch.float8_e4m3fn)
    st = torch.cuda.current_stream().cuda_stream
    a = lambda g: g[1].data_ptr()  # noqa: E731
    assert lib.moe_residual_norm(x.data_ptr(), r.data_ptr(), 1, w.data_ptr(), 0, N, H, 1e-6, a(y), a(ro), a(rstd), a(q),
                                 a(qs), st) == 0
    size = lib.moe_residual_norm_backward_workspace_size(N, H)
    dx, dres, dw, ws = guarded(N, H), guarded(N, H, t=F32), guarded(H, t=F32), guarded(size // 4, t=F32)
    assert lib.moe_residual_norm_backward(x.data_ptr(), a(ro), 1, w.data_ptr(), 0, a(rstd), r.data_ptr(), N, H, a(dx),
                                          a(dres), a(dw), a(ws), size, st) == 0
    torch.cuda.synchronize()
    for raw, t in (y, ro, rstd, q, qs, dx, dres, dw, ws):
        n = t.numel()
        assert (raw[:guard].float() == 3).all() and (raw[guard + n:].float() == 3).all()
    o = m.residual_norm(x, w, residual=r, quantize=True)
    assert torch.equal(o.y, y[1]) and torch.equal(o.q.view(torch.uint8), q[1].view(torch.uint8))

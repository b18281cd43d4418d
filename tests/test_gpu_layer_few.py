"""The layer for one to eight tokens, whose down product has a kernel of its own, and workspaces of exactly the stated size."""
import ctypes

import pytest
import torch

from block_checks import S, U, assert_within
from test_gpu_block_norm import backward64, check_backward
from test_gpu_block_norm import inputs as norm_inputs
from test_gpu_block_norm import rand
from test_gpu_layer import BF16, F32, check, gen, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


@pytest.mark.parametrize("N,E,K,H,I,bits", [(1, 4, 2, 9728, 40, 16), (1, 4, 2, 9736, 40, 16), (3, 8, 2, 9744, 72, 8), (8, 8, 3, 16384, 24, 16),
                                            (2, 4, 2, 19464, 64, 16), (8, 4, 1, 40000, 8, 16), (5, 16, 2, 9720, 200, 16)])
def test_wide_rows(m, N, E, K, H, I, bits):  # noqa: E741
    """More 32-row parts of the output than blocks run at once, and the sizes around that."""
    check(m, inputs(N, E, H, I, bits=bits), K)


@pytest.mark.parametrize("N", range(1, 9))
@pytest.mark.parametrize("bits", [16, 8])
def test_guard_zones(m, N, bits):
    E, K, H, I = 8, 2, 208, 72  # noqa: E741
    a = inputs(N, E, H, I, bits=bits)
    want = check(m, a, K)
    big = torch.full((N + 2, H), 7.0, device="cuda").to(BF16)
    idx, w = torch.full((N + 2, K), 7, dtype=torch.int32, device="cuda"), torch.full((N + 2, K), 7.0, device="cuda")
    out = big[1:N + 1]
    assert m.layer(K=K, out=out, topk_idx=idx[1:N + 1], topk_w=w[1:N + 1], **a) is out
    assert torch.equal(out, want)
    for t in (big, idx, w):
        assert (t[0] == 7).all() and (t[N + 1] == 7).all()


@pytest.mark.parametrize("N", [2, 8])
@pytest.mark.parametrize("bits", [16, 8])
def test_what_is_not_chosen_is_not_read(m, N, bits):
    """NaN and infinities in experts that no token chose, and in other tokens' rows, reach nothing."""
    E, K = 40, 2
    a = inputs(N, E, 160, 72, bits=bits)
    a["logits"][:, 20:] -= 100
    clean = check(m, a, K)
    idx = m.route_topk(a["logits"], K)[0]
    unused = [e for e in range(E) if not (idx == e).any()]
    a["w_down"][unused] = float("nan")
    a["w_gate_up"].view(torch.uint8 if bits == 8 else torch.int16)[unused] = 0x7f if bits == 8 else 0x7f80   # NaN, infinity
    assert torch.equal(m.layer(K=K, **a), clean)
    if bits == 16:
        a["x"][N - 1, 5] = float("nan")
    else:
        a["x_scale"][N - 1] = float("nan")
    got = m.layer(K=K, **a)
    assert torch.equal(got[:N - 1], clean[:N - 1]) and got[N - 1].isnan().all()


@pytest.mark.parametrize("N", [1, 3, 8])
def test_masked_experts(m, N):
    a = inputs(N, 16, 128, 64)
    a["logits"][:, 4:] = torch.finfo(F32).min
    check(m, a, 4)
    check(m, a, 7)


@pytest.mark.parametrize("N", [1, 4, 8])
@pytest.mark.parametrize("routing", [
    dict(renormalize=False), dict(scoring="sigmoid"), dict(scoring="sigmoid", renormalize=False, routed_scaling=2.5),
    dict(scoring="sigmoid", n_group=8, topk_group=4, routed_scaling=2.5), dict(scoring="sigmoid", n_group=4, topk_group=1)])
def test_routing(m, N, routing):
    a = inputs(N, 64, 128, 72)
    if routing.get("scoring") == "sigmoid":
        routing = dict(routing, bias=(torch.rand(64, generator=gen(3), device="cuda") - 0.5) * 0.2)
    check(m, a, 6, **routing)


def test_gates_of_every_size(m):
    """silu from -infinity's side to large values: no overflow, and it keeps its value down to the smallest numbers."""
    H, I = 16, 8  # noqa: E741
    sizes = torch.tensor([-200.0, -104, -95, -88, -20, 0, 20, 300], device="cuda")
    N = len(sizes)
    x = torch.zeros(N, H, device="cuda")
    x[:, 0], x[:, 1] = sizes, 1.0
    wgu = torch.zeros(1, 2, I, H, device="cuda")
    wgu[0, 0, :, 0], wgu[0, 1, :, 1] = 1.0, 2.0 ** 40         # g = x[0], u = 2^40
    wd = torch.zeros(1, H, I, device="cuda")
    wd[0, :, 0] = 1.0
    got = m.layer(x.to(BF16), torch.zeros(N, 1, device="cuda"), wgu.to(BF16), wd.to(BF16), 1)
    g = sizes.to(BF16).double()
    want = (g * torch.sigmoid(g) * 2.0 ** 40)[:, None].expand(N, H)
    # e^-|g| keeps fp32's precision down to its smallest normal number, 2^-126, and half a 2^-149 below
    fp32 = S * want.abs() + g.abs()[:, None] * 2.0 ** -149 * 2.0 ** 40
    assert_within(got, want, fp32 + 2 * U * (want.abs() + fp32), "out")


@pytest.mark.parametrize("N", [9, 16, 33, 64])
@pytest.mark.parametrize("bits", [16, 8])
def test_more_than_eight_tokens_are_independent(m, N, bits):
    """A token's output has the same bits whatever the other tokens hold and choose."""
    E, K, H, I = 24, 3, 272, 136  # noqa: E741
    a, b = inputs(N, E, H, I, bits=bits, seed=1), inputs(N, E, H, I, bits=bits, seed=2)
    a["w_gate_up"], a["w_down"] = b["w_gate_up"], b["w_down"]
    keep = N // 2
    b["logits"][keep] = a["logits"][keep]
    b["x"].view(torch.uint8)[keep] = a["x"].view(torch.uint8)[keep]
    if bits == 8:
        a["w_scale"] = b["w_scale"]
        b["x_scale"][keep] = a["x_scale"][keep]
    b["logits"][:keep, 5] += 30     # an expert with many tokens
    x, y = m.layer(K=K, **a), m.layer(K=K, **b)
    assert torch.equal(x[keep], y[keep]) and not torch.equal(x, y)


def guarded(nbytes, around=4096):
    """(buffer, address of `nbytes` in it); the rest holds 0xA5."""
    t = torch.full((nbytes + 2 * around,), 0xA5, dtype=torch.uint8, device="cuda")
    return t, t.data_ptr() + around


def untouched(t, nbytes, around=4096):
    return bool((t[:around] == 0xA5).all()) and bool((t[around + nbytes:] == 0xA5).all())


def P(t):
    return ctypes.c_void_p(t if isinstance(t, int) else t.data_ptr() if t is not None else None)


@pytest.mark.parametrize("N,E,K,H,I", [(1, 4, 1, 8, 8), (3, 8, 3, 264, 72), (8, 16, 5, 2056, 72), (9, 16, 5, 264, 72), (64, 40, 7, 200, 136)])
@pytest.mark.parametrize("outputs", [True, False])
def test_layer_stays_in_its_workspace(m, N, E, K, H, I, outputs):  # noqa: E741
    lib = m.load()
    a = inputs(N, E, H, I)
    want = m.layer(K=K, **a)
    nbytes = lib.moe_layer_workspace_size(N, K, H, I)
    ws, at = guarded(nbytes)
    out = torch.empty(N, H, dtype=BF16, device="cuda")
    idx = torch.empty(N, K, dtype=torch.int32, device="cuda") if outputs else None
    w = torch.empty(N, K, device="cuda") if outputs else None
    rc = lib.moe_layer(P(a["x"]), None, P(a["logits"]), None, P(a["w_gate_up"]), None, P(a["w_down"]), N, E, H, I, K, 0, 0, 1, 1,
                       1, 1.0, P(idx), P(w), P(out), P(at), nbytes, P(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want) and untouched(ws, nbytes)


@pytest.mark.parametrize("N,H", [(1, 8), (5, 512), (700, 256), (2, 520), (3000, 520), (1300, 1000), (9800, 1024), (700, 2056),
                                 (1300, 4104), (1111, 7168), (700, 8192), (2, 16384), (700, 8200)])
@pytest.mark.parametrize("res,gate,with_ds", [(BF16, None, False), (F32, "full", True), (BF16, "token", True)])
def test_norm_gradient_stays_in_its_workspace(m, N, H, res, gate, with_ds):
    lib = m.load()
    x, r, wp, w, c = norm_inputs(N, H, res, gate, BF16, F32)
    f = m.block_norm(x, r, wp, w, gate=c)
    dy, ds = rand(N, H, seed=8).to(BF16), rand(N, H, seed=9).to(res) if with_ds else None
    nbytes = lib.moe_block_norm_backward_workspace_size(N, H)
    ws, at = guarded(nbytes)
    dx, dres = torch.empty_like(x), torch.empty_like(r)
    dgate = None if c is None else torch.empty_like(c)
    dpost, dweight = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    rc = lib.moe_block_norm_backward(P(dy), P(x), P(f.residual), 1 if res == F32 else 0, P(ds), P(c), 1 if gate == "token" else 0,
                                     P(wp), 0, P(w), 1, P(f.post_rstd), P(f.rstd), N, H, 1.0, P(dx), P(dres), P(dgate), P(dpost),
                                     P(dweight), P(at), nbytes, P(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    torch.cuda.synchronize()
    assert untouched(ws, nbytes)
    check_backward((dx, dres, dgate, dpost, dweight), backward64(dy, ds, f.residual, x, f.rstd, f.post_rstd, wp, w, c, alpha=1.0),
                   gate)

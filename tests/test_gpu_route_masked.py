"""Masked experts: logits of minus infinity, or so far apart that their difference overflows.

An expert whose logit is minus infinity has score 0 (e^-inf under softmax, sigmoid(-inf)): it is chosen after all open
experts, in ascending index, with weight exactly 0, and adds nothing to a normaliser.  A softmax row without any open
expert has no weights: NaN, as 0/0.  The expected weights come from a softmax or sigmoid in 64 bits on the logits, the
choice from a stable sort of them.  Bound: the router's own, 1e-6 relative.
"""
import numpy as np
import pytest
import torch

import oracle
from block_checks import F, S, U, assert_within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LOWEST = float(torch.finfo(F32).min)


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import expert_dispatch_planning_gb300 as m
    return m


def logits_of(N, E, open_experts, masked=-float("inf"), seed=0):
    """Random logits; in row s only open_experts (or fewer, never none) stay, at places that change with the row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(N, E, generator=g, device="cuda")
    rank = torch.rand(N, E, generator=g, device="cuda").argsort(1).argsort(1)
    keep = torch.randint(1, open_experts + 1, (N, 1), generator=g, device="cuda")
    keep[0] = open_experts
    return torch.where(rank < keep, x, torch.full_like(x, masked))


def expected(logits, K, scoring="softmax", renormalize=True, routed_scaling=1.0):
    """(idx, weights in 64 bits); a NaN weight has no value."""
    v = logits.double()
    score = torch.sigmoid(v) if scoring == "sigmoid" else torch.softmax(v, 1)
    idx = v.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = score.gather(1, idx)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    return idx, w * routed_scaling


def check(got, logits, K, **kw):
    idx, w = got
    ei, ew = expected(logits, K, **kw)
    assert torch.equal(idx.long(), ei)
    none = ew.isnan()
    assert torch.equal(w.isnan(), none)
    assert (w[ew == 0] == 0).all()
    assert ((w.double() - ew).abs() <= 1e-6 * ew.abs())[~none].all()


# every width of the router's kernels, and K up to the most
SHAPES = [(4, 2), (8, 5), (12, 4), (16, 7), (32, 8), (60, 4), (64, 6), (97, 8), (128, 8), (128, 20), (200, 8), (256, 8),
          (300, 32), (512, 8), (1000, 10), (1021, 32)]


@pytest.mark.parametrize("E,K", SHAPES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_fewer_open_experts_than_k(m, E, K, renormalize):
    N = 37
    x = logits_of(N, E, K - 1)
    check(m.route_topk(x, K, renormalize=renormalize, routed_scaling=1.5), x, K, renormalize=renormalize, routed_scaling=1.5)
    o_idx, o_w = oracle.route_topk(x.cpu().numpy(), K, scoring=0, renormalize=renormalize, routed_scaling=1.5)
    ei, ew = expected(x, K, renormalize=renormalize, routed_scaling=1.5)
    assert np.array_equal(o_idx, ei.cpu().numpy()) and np.allclose(o_w, ew.cpu().numpy(), rtol=1e-12, atol=0)


@pytest.mark.parametrize("E,K", SHAPES)
def test_one_masked_expert_that_is_not_chosen(m, E, K):
    """It is in the whole row's normaliser."""
    x = logits_of(29, E, E)
    x[torch.arange(29), torch.arange(29) % E] = -float("inf")
    for renormalize in (True, False):
        check(m.route_topk(x, K, renormalize=renormalize), x, K, renormalize=renormalize)


@pytest.mark.parametrize("E,K", [(8, 5), (64, 6), (256, 8), (97, 8)])
def test_sigmoid(m, E, K):
    x = logits_of(41, E, K - 1)
    for renormalize in (True, False):
        check(m.route_topk(x, K, scoring="sigmoid", renormalize=renormalize), x, K, scoring="sigmoid", renormalize=renormalize)


@pytest.mark.parametrize("E,K", [(8, 3), (128, 8), (300, 6)])
@pytest.mark.parametrize("low,high", [(LOWEST, -LOWEST), (-2.5e38, 2.5e38), (LOWEST, 3.0), (-1e30, 1e30), (-104.5, 0.0), (-300.0, 40.0)])
def test_logits_whose_difference_overflows(m, E, K, low, high):
    x = torch.full((5, E), low, device="cuda")
    x[:, 1] = high
    x[3, E - 1] = high
    for renormalize in (True, False):
        idx, w = m.route_topk(x, K, renormalize=renormalize)
        ei, ew = expected(x, K, renormalize=renormalize)
        assert torch.equal(idx.long(), ei)
        # below the smallest normal number an fp32 weight has no relative precision
        assert ((w.double() - ew).abs() <= 1e-6 * ew.abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_rows_without_an_open_expert(m, renormalize):
    """No weights (NaN), the lowest indices; the rows beside them keep theirs."""
    for E, K in ((8, 2), (64, 6), (128, 8), (300, 12)):
        x = logits_of(33, E, E)
        x[4] = x[32] = -float("inf")
        got = m.route_topk(x, K, renormalize=renormalize)
        check(got, x, K, renormalize=renormalize)
        assert torch.equal(got[0][4].cpu(), torch.arange(K, dtype=torch.int32)) and got[1][4].isnan().all()
        check(m.route_topk(x, K, scoring="sigmoid", renormalize=renormalize), x, K, scoring="sigmoid", renormalize=renormalize)


@pytest.mark.parametrize("E,K", [(128, 8), (256, 5), (512, 8)])
def test_fast_router(m, E, K):
    """From 16384 tokens on the same, masked rows between ordinary ones."""
    N = 16384 + 77
    x = logits_of(N, E, E)
    few = logits_of(N, E, K - 1, seed=1)
    at = torch.arange(N, device="cuda") % 5 == 0
    x[at] = few[at]
    check(m.route_topk(x, K), x, K)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("N", [1, 50, 4000])
def test_routing_and_plan_in_one_call(m, N, renormalize):
    x = logits_of(N, 64, 5)
    idx, w, _ = m.route_plan(x, 6, 8, 16, renormalize=renormalize)
    check((idx, w), x, 6, renormalize=renormalize)


@pytest.mark.parametrize("N", [1, 5, 8, 9, 20, 64])
@pytest.mark.parametrize("routing", [dict(), dict(renormalize=False), dict(scoring="sigmoid")])
def test_layer(m, N, routing):
    """A layer's output is the sum over the open experts, with weights and choice taken in 64 bits here."""
    E, K, H, I = 16, 6, 128, 72  # noqa: E741
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = torch.randn(N, H, generator=g, device="cuda").to(BF16)
    wgu = (torch.randn(E, 2, I, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
    wd = (torch.randn(E, H, I, generator=g, device="cuda") * I ** -0.5).to(BF16)
    logits = logits_of(N, E, K - 2)
    idx, w = expected(logits, K, **routing)
    out, tol = (torch.zeros(N, H, dtype=torch.float64, device="cuda") for _ in range(2))
    for s in range(N):
        for e, share in zip(idx[s].tolist(), w[s].tolist()):
            if share == 0:
                continue
            G, Up, D = wgu[e, 0].double(), wgu[e, 1].double(), wd[e].double()
            xs = x[s].double()
            gate, up = G @ xs, Up @ xs
            dg, du = ((H + 16) * F * (v.abs() @ xs.abs()) for v in (G, Up))
            h = gate * torch.sigmoid(gate) * up
            fp32 = 1.1 * dg * (up.abs() + du) + (gate * torch.sigmoid(gate)).abs() * du + S * h.abs()
            eh = fp32 + U * (h.abs() + fp32)
            y_abs = D.abs() @ h.abs()
            ey = D.abs() @ eh + (I + 16) * F * (y_abs + D.abs() @ eh)
            out[s] += share * (D @ h)
            tol[s] += share * (ey + (1e-6 + (K + 8) * F) * (y_abs + ey))
    got = m.layer(x, logits, wgu, wd, K, **routing)
    assert got.isfinite().all()
    assert_within(got, out, tol + U * (out.abs() + tol), "out")

"""silu and its gradient in the experts' feed-forward over every size of the gate, against 64 bits."""
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


def test_gates_of_every_size(m):
    """Gates from -104 (whose sigmoid lies below the normal numbers) to 104, with up values that bring h back among them.

    The documented bounds, in units of 2^-23: the exponential 2 + floor(1.173 |g|), the division 2, and a rounding each
    for 1 + e, e * near and the product with g; below -87.3 the exponential is known to a unit of 2^-149."""
    H = I = 64  # noqa: E741
    g = torch.arange(-104, 104.5, 0.5, device="cuda").to(BF16)
    n = g.numel()
    p = bc.groups([n], 1)
    x = torch.zeros(n, H, dtype=BF16, device="cuda")
    up = 2.0 ** 60
    x[:, 0], x[:, 1] = g, up
    wgu = torch.zeros(1, 2, I, H, dtype=BF16, device="cuda")
    wgu[0, 0, :, 0] = 1.0
    wgu[0, 1, :, 1] = 1.0
    wd = torch.eye(H, dtype=BF16, device="cuda")[None].contiguous()
    h, pre = torch.empty(n, I, dtype=BF16, device="cuda"), torch.empty(n, 2, I, device="cuda")
    dgu = torch.empty(n, 2, I, dtype=BF16, device="cuda")
    m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
    m.expert_ffn_backward(torch.ones_like(x), x, h, pre, wgu, wd, p, dgate_up=dgu)
    G = g.double()[:, None].expand(n, I)
    assert (pre[:, 0].double() == G).all() and (pre[:, 1] == up).all()
    s, rest = torch.sigmoid(G), torch.sigmoid(-G)
    rel = (2 + 1.173 * G.abs() + 2 + 3) * 2.0 ** -23
    lost = 4 * 2.0 ** -149                    # of the sigmoid

    def within(got, want, err, what):
        bc.assert_within(got, want, err + bc.U * (want.abs() + err) + 2.0 ** -134, what)
    silu = G * s
    within(h, silu * up, (rel * silu.abs() + lost * G.abs()) * up, "h")
    within(dgu[:, 1], silu, rel * silu.abs() + lost * G.abs(), "du")
    slope = up * s * (1 + G * rest)
    # the factors' errors, of which 1 + g rest may cancel
    err = up * (s * rel + lost) * (1 + G.abs() * rest) + up * s * (G.abs() * rest * rel + 2.0 ** -23) + up * s * 2.0 ** -22
    within(dgu[:, 0], slope, err, "dg")
    assert int(p.status[0]) == 0

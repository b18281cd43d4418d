"""The example block end to end: its gradients against autograd in 64 bits, its training and its 8-bit step."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block
    return moe_block


def test_gradients_against_autograd(ex):
    """Every gradient of the block, with the routing held fixed, from a 64-bit restatement of it.

    The chain rounds to bf16 in about eight places (norm's output, h, y, out,
    dout, dy of the experts, dgate_up, dx, dy of the norm), each with a relative
    rms error of at most 2^-8 / sqrt(3); independent, they add up to under
    3 * 2^-8, and the bound is twice that in the 2-norm."""
    N = 96
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(N, ex.H, generator=g, device="cuda").to(torch.bfloat16)
    stream = torch.randn(N, ex.H, generator=g, device="cuda")
    dout = torch.randn(N, ex.H, generator=g, device="cuda").to(torch.bfloat16)
    block = ex.Block(seed=3)
    before = [t.clone() for t in (block.norm, block.router, block.w_gate_up, block.w_down)]
    out, saved = block.forward(x, stream)
    idx = saved[1].long()
    wgu16, wd16 = block.w_gate_up16.double(), block.w_down16.double()
    dx, dstream = block.backward(dout, saved, lr=1.0)
    step = [b - t for b, t in zip(before, (block.norm, block.router, block.w_gate_up, block.w_down))]

    leaf = [t.double().requires_grad_() for t in (x, stream, before[0], before[1])]
    X, S, norm, router = leaf
    wgu, wd = wgu16.requires_grad_(), wd16.requires_grad_()
    s = X + S
    y = s * (s.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm
    w = torch.softmax((y @ router.T).gather(1, idx), dim=1)
    ref = torch.zeros_like(y)
    for k in range(ex.K):
        for e in range(ex.E):
            rows = (idx[:, k] == e).nonzero()[:, 0]
            if rows.numel():
                gate, up = y[rows] @ wgu[e, 0].T, y[rows] @ wgu[e, 1].T
                ref = ref.index_add(0, rows, w[rows, k, None] * ((torch.nn.functional.silu(gate) * up) @ wd[e].T))
    ref.backward(dout.double())
    tol = 6 * 2.0 ** -8
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, X.grad), ("dstream", dstream, S.grad),
                            ("dnorm", step[0], norm.grad), ("drouter", step[1], router.grad),
                            ("dw_gate_up", step[2], wgu.grad), ("dw_down", step[3], wd.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= tol, (name, rel)


def test_training_and_decoding(ex):
    losses, rel = ex.main(tokens=512, steps=12, verbose=False)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    # e4m3 rounds rows and weights each by at most 2^-4 relative (about 0.026 rms)
    assert 0 < rel < 2 * 2.0 ** -4

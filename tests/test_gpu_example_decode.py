"""The example block's decoding step takes any number of tokens."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 64, 65, 200])
def test_decoding(N):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block as ex
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(N, ex.H, generator=g, device="cuda").to(torch.bfloat16)
    stream = torch.randn(N, ex.H, generator=g, device="cuda")
    block = ex.Block(seed=3)
    want, _ = block.forward(x, stream)
    got = block.decode(x, stream, *ex.quantize_channels(block.w_gate_up))
    rel = float((got.float() - want.float()).norm() / want.float().norm())
    # e4m3 rounds rows and weights each by at most 2^-4 relative (about 0.026 rms)
    assert 0 < rel < 2 * 2.0 ** -4

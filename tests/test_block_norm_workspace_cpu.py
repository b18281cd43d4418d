"""The workspace of block_norm's gradient: a pair of rows of sums for every block of the launch, no more (no GPU)."""
import os

import pytest


@pytest.fixture(scope="module")
def size():
    from expert_dispatch_planning_gb300 import _lib
    from expert_dispatch_planning_gb300 import build as b
    if not os.path.exists(_lib.LIB_PATH):
        b.build()
    return _lib.load().moe_block_norm_backward_workspace_size


def test_no_more_than_the_largest_launch(size):
    """152 SMs without a GPU to ask: four blocks an SM where a block takes a row, one for the widest rings."""
    for H, blocks in ((7168, 152), (32768, 4 * 152), (8200, 4 * 152), (512, 4 * 152)):
        assert size(1 << 20, H) == blocks * 2 * H * 4, H


@pytest.mark.parametrize("H", [8, 512, 520, 1024, 2040, 2048, 4096, 5120, 7168, 7936, 8192, 8200, 32768])
def test_enough_for_fewer_rows(size, H):
    """A workspace for many rows serves fewer."""
    last = 0
    for N in (0, 1, 3, 100, 151, 152, 153, 303, 304, 600, 608, 609, 1215, 1216, 2432, 4863, 4864, 4865, 10000, 1 << 20, 1 << 30):
        assert size(N, H) >= max(last, 2 * H * 4)
        last = size(N, H)

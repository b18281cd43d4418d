"""The experts' feed-forward when something is wrong: reported at once, and the next call is unharmed."""
import time

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


def buffers(p, H, I, seed=0):  # noqa: E741
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    E = len(p.counts)
    return r(p.rows, H), r(p.rows, H), r(E, 2, I, H, std=H ** -0.5), r(E, H, I, std=I ** -0.5)


def step(m, p, x, dy, wgu, wd):
    h = torch.empty(x.shape[0], wd.shape[2], dtype=BF16, device="cuda")
    pre = torch.empty(x.shape[0], 2, wd.shape[2], device="cuda")
    y = m.expert_ffn(x, wgu, wd, p, h=h, preact=pre, out=torch.zeros_like(x))
    return (y, *m.expert_ffn_backward(dy, x, h, pre, wgu, wd, p, dx=torch.zeros_like(x)))


@pytest.mark.parametrize("bad", [0, 7, 31])
def test_a_group_outside_the_rows_is_reported_at_once(m, bad):
    """However the blocks' reads of the status fall, none waits for a block that has stopped: the limit of a wait is a
    second, and 200 steps take a few milliseconds each at most."""
    H, I = 256, 128  # noqa: E741
    p = bc.groups([40] * 32, 8)
    args = buffers(p, H, I)
    want = step(m, p, *args)
    good = p.tokens_per_expert.clone()
    wrong = good.clone()
    wrong[bad] = 41 + p.rows
    torch.cuda.synchronize()
    longest = 0.0
    for _ in range(200):
        p.tokens_per_expert.copy_(wrong)
        p.status.zero_()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        step(m, p, *args)
        torch.cuda.synchronize()
        longest = max(longest, time.perf_counter() - t0)
        assert int(p.status[0]) == 6                  # MOE_ERR_DEVICE_INDEX
    assert longest < 0.5
    p.tokens_per_expert.copy_(good)
    p.status.zero_()
    got = step(m, p, *args)
    assert int(p.status[0]) == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_long_groups_are_not_taken_for_a_wait_that_ran_out(m):
    """One group whose weights' gradients are a single tile of 625001 slices: some 0.1 s and more, during all of which
    the output waits. With a limit of 60 ms a wait for one slice's steps has ages, and the tile's must not run out."""
    rows, H, I = 40_000_005, 16, 16  # noqa: E741
    p = bc.groups([rows], 1)
    x = torch.ones(rows, H, dtype=BF16, device="cuda")
    wgu, wd = torch.ones(1, 2, I, H, dtype=BF16, device="cuda"), torch.ones(1, H, I, dtype=BF16, device="cuda")
    try:
        m.set_plan_fault(-1, 60_000_000)
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        h, pre = torch.empty(rows, I, dtype=BF16, device="cuda"), torch.empty(rows, 2, I, device="cuda")
        m.expert_ffn(x, wgu, wd, p, h=h, preact=pre)
        torch.cuda.synchronize()
        t0.record()
        m.expert_ffn_backward(x, x, h, pre, wgu, wd, p)
        t1.record()
        torch.cuda.synchronize()
    finally:
        m.set_plan_fault()
    assert int(p.status[0]) == 0
    assert t0.elapsed_time(t1) > 60          # the case is one that takes longer than the limit

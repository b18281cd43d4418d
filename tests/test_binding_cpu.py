"""The compiled binding refuses tensors that are not on the GPU with a ValueError, also where there is none."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    from expert_dispatch_planning_gb300 import build as b
    b.build()
    import expert_dispatch_planning_gb300 as m
    return m


def test_host_tensors_are_refused(m):
    from types import SimpleNamespace
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    p = SimpleNamespace(cu_seqlens=z(3, t=i32), tokens_per_expert=z(2, t=i32), status=z(4, t=i32), dst=z(4, 1, t=i32),
                        zero_fill_ranges=z(2, 2, t=i32))
    calls = [
        ("x", lambda: m.residual_norm(z(4, 64), z(64))),
        ("dy", lambda: m.residual_norm_backward(z(4, 64), z(4, 64), z(64), z(4, t=f32))),
        ("x", lambda: m.expert_ffn(z(4, 64), z(2, 2, 32, 64), z(2, 64, 32), p)),
        ("x", lambda: m.expert_ffn_backward(z(4, 64), z(4, 64), z(4, 32), z(4, 2, 32, t=f32), z(2, 2, 32, 64), z(2, 64, 32),
                                            p)),
        ("dout", lambda: m.combine_backward(z(4, 64), z(4, 64), z(4, 1, t=f32), p)),
    ]
    for name, call in calls:
        with pytest.raises(ValueError, match="^%s must be a contiguous CUDA .* on the current device .*on cpu" % name):
            call()

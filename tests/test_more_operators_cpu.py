"""Host-side argument checks of the norms between blocks and of the whole layer (no GPU: invalid calls return before any
CUDA call), and the binding's refusals of host tensors."""
import ctypes
import os

import pytest
import torch

P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10008)


@pytest.fixture(scope="module")
def lib():
    from expert_dispatch_planning_gb300 import _lib
    from expert_dispatch_planning_gb300 import build as b
    if not os.path.exists(_lib.LIB_PATH):
        b.build()
    return _lib.load()


FORWARD = ("x", "r", "rt", "c", "ct", "wp", "wpt", "w", "wt", "N", "H", "alpha", "eps", "y", "ro", "pr", "rs", "q", "qs")


def test_block_norm(lib):
    ok = dict(x=FAKE, r=FAKE, rt=0, c=FAKE, ct=0, wp=FAKE, wpt=0, w=FAKE, wt=1, N=4, H=64, alpha=1.0, eps=1e-6, y=FAKE,
              ro=FAKE, pr=FAKE, rs=FAKE, q=FAKE, qs=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_block_norm(*[a[k] for k in FORWARD], None)
    assert call(H=60) == 1 and call(H=0) == 1 and call(N=-1) == 1
    for k in ("x", "r", "wp", "w", "y", "ro", "pr", "rs"):
        assert call(**{k: None}) == 1, k
    for k in ("x", "r", "c", "wp", "w", "y", "ro"):
        assert call(**{k: ODD}) == 1, k
    assert call(ct=1, c=P(0x10002)) == 1 and call(ct=2) == 1 and call(rt=2) == 1 and call(wpt=2) == 1 and call(wt=3) == 1
    assert call(q=None) == 1 and call(qs=None) == 1
    assert call(pr=P(0x10002)) == 1 and call(rs=P(0x10002)) == 1 and call(q=P(0x10004)) == 1
    for v in (float("nan"), float("inf"), -float("inf")):
        assert call(eps=v) == 1 and call(alpha=v) == 1
    assert call(eps=-1.0) == 1
    assert call(H=32776) == 2
    assert call(N=0) == 0 and call(N=0, x=None, r=None, c=None, y=None, ro=None, pr=None, rs=None, q=None, qs=None) == 0


BACKWARD = ("dy", "x", "s", "st", "ds", "c", "ct", "wp", "wpt", "w", "wt", "pr", "rs", "N", "H", "alpha", "dx", "dr", "dc",
            "dwp", "dw", "ws", "n")


def test_block_norm_backward(lib):
    size = lib.moe_block_norm_backward_workspace_size
    assert size(-1, 64) == 0 and size(4, 60) == 0 and size(4, 40000) == 0
    assert size(0, 64) > 0 and size(100000, 4096) >= 2 * 4096 * 4
    ok = dict(dy=FAKE, x=FAKE, s=FAKE, st=0, ds=FAKE, c=FAKE, ct=0, wp=FAKE, wpt=0, w=FAKE, wt=0, pr=FAKE, rs=FAKE, N=4, H=64,
              alpha=1.0, dx=FAKE, dr=FAKE, dc=FAKE, dwp=FAKE, dw=FAKE, ws=FAKE, n=1 << 30)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_block_norm_backward(*[a[k] for k in BACKWARD], None)
    for k in ("dy", "x", "s", "wp", "w", "pr", "rs", "dx", "dr", "dc", "dwp", "dw", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("dy", "x", "s", "ds", "c", "wp", "w", "dx", "dr", "dc", "ws"):
        assert call(**{k: ODD}) == 1, k
    assert call(c=None) == 1                                    # a gate's gradient without a gate
    assert call(st=2) == 1 and call(ct=2) == 1 and call(wpt=2) == 1 and call(wt=3) == 1
    assert call(N=-1) == 1 and call(H=12) == 1 and call(alpha=float("nan")) == 1
    assert call(n=16) == 3
    assert call(H=32776) == 2


LAYER = ("x", "xs", "lg", "b", "wgu", "ws", "wd", "N", "E", "H", "I", "K", "t", "sc", "rn", "ng", "tg", "rsc", "idx", "w", "out",
         "wk", "n")


def test_layer(lib):
    size = lib.moe_layer_workspace_size
    for bad in (dict(N=-1), dict(N=65), dict(K=0), dict(K=33), dict(H=60), dict(H=0), dict(H=1 << 20), dict(I=60), dict(I=0),
                dict(I=1 << 20)):
        assert size(*dict(N=4, K=2, H=64, I=64).values()) > 0 and size(*{**dict(N=4, K=2, H=64, I=64), **bad}.values()) == 0
    assert size(0, 2, 64, 64) > 0 and size(64, 32, 64, 4096) >= 64 * 32 * (4096 * 2 + 64 * 4 + 8)
    ok = dict(x=FAKE, xs=None, lg=FAKE, b=None, wgu=FAKE, ws=None, wd=FAKE, N=4, E=8, H=64, I=40, K=2, t=0, sc=0, rn=1, ng=1,
              tg=1, rsc=1.0, idx=FAKE, w=FAKE, out=FAKE, wk=FAKE, n=1 << 30)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_layer(*[a[k] for k in LAYER], None)
    for k in ("x", "lg", "wgu", "wd", "out", "wk"):
        assert call(**{k: None}) == 1, k
    for k in ("x", "lg", "wgu", "wd", "out", "wk"):
        assert call(**{k: ODD}) == 1, k
    assert call(N=-1) == 1 and call(N=65) == 2
    assert call(E=0) == 1 and call(E=1025) == 1 and call(K=0) == 1 and call(K=9) == 1 and call(K=33, E=64) == 1
    assert call(H=60) == 1 and call(H=0) == 1 and call(I=44) == 1 and call(I=0) == 1 and call(H=1 << 20) == 1
    assert call(I=1 << 20) == 1 and call(t=1) == 1 and call(t=3) == 1
    assert call(xs=FAKE) == 1 and call(ws=FAKE) == 1            # scales go with 8 bits
    assert call(t=2) == 1 and call(t=2, xs=FAKE) == 1 and call(t=2, ws=FAKE) == 1
    assert call(t=2, xs=FAKE, ws=FAKE, H=72) == 1               # H % 16
    assert call(sc=2) == 1 and call(ng=0) == 1 and call(ng=2) == 2 and call(b=FAKE) == 2
    assert call(sc=1, ng=3) == 1 and call(sc=1, ng=4, tg=5) == 1 and call(rsc=float("nan")) == 1
    assert call(n=16) == 3
    assert call(N=0) == 0 and call(N=0, x=None, lg=None, out=None, wk=None, n=0) == 0


def test_host_tensors_are_refused():
    from expert_dispatch_planning_gb300 import build as b
    b.build()
    import expert_dispatch_planning_gb300 as m
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    f32 = torch.float32
    calls = [
        ("x", lambda: m.block_norm(z(4, 64), z(4, 64), z(64), z(64))),
        ("dy", lambda: m.block_norm_backward(z(4, 64), z(4, 64), z(4, 64), z(64), z(64), z(4, t=f32), z(4, t=f32))),
        ("x", lambda: m.layer(z(4, 64), z(4, 2, t=f32), z(2, 2, 32, 64), z(2, 64, 32), 1)),
    ]
    for name, call in calls:
        with pytest.raises(ValueError, match="^%s must be a contiguous CUDA .* on the current device .*on cpu" % name):
            call()

"""Host-side argument checks of the operators around the experts (no GPU: invalid calls return before any CUDA call)."""
import ctypes
import os

import pytest

P = ctypes.c_void_p
FAKE, ODD = P(0x10000), P(0x10008)


@pytest.fixture(scope="module")
def lib():
    from expert_dispatch_planning_gb300 import _lib
    from expert_dispatch_planning_gb300 import build as b
    if not os.path.exists(_lib.LIB_PATH):
        b.build()
    return _lib.load()


def plan(**kw):
    from expert_dispatch_planning_gb300._lib import MoePlanOut
    s = MoePlanOut(*([FAKE.value] * 14))
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def test_norm(lib):
    ok = dict(x=FAKE, r=FAKE, rt=0, w=FAKE, wt=0, N=4, H=64, eps=1e-6, y=FAKE, ro=FAKE, rstd=FAKE, q=FAKE, qs=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_residual_norm(*[a[k] for k in ("x", "r", "rt", "w", "wt", "N", "H", "eps", "y", "ro", "rstd", "q",
                                                      "qs")], None)
    assert call(H=60) == 1 and call(H=0) == 1 and call(N=-1) == 1
    assert call(x=None) == 1 and call(w=None) == 1 and call(y=None, q=None, qs=None) == 1
    assert call(x=ODD) == 1 and call(r=ODD) == 1 and call(w=ODD) == 1 and call(y=ODD) == 1
    assert call(rt=2) == 1 and call(wt=2) == 1
    assert call(r=None) == 1                                   # residual_out needs a residual
    assert call(q=None) == 1 and call(qs=None) == 1            # both or neither
    assert call(eps=-1.0) == 1 and call(eps=float("nan")) == 1 and call(eps=float("inf")) == 1
    assert call(H=32776) == 2
    assert call(N=0) == 0 and call(N=0, x=None, y=None, q=None, qs=None) == 0


def test_norm_backward(lib):
    size = lib.moe_residual_norm_backward_workspace_size
    assert size(-1, 64) == 0 and size(4, 60) == 0 and size(4, 40000) == 0
    assert size(0, 64) > 0 and size(100000, 4096) >= 4096 * 4
    ok = dict(dy=FAKE, s=FAKE, st=0, w=FAKE, wt=0, rstd=FAKE, ds=FAKE, N=4, H=64, dx=FAKE, dres=None, dw=FAKE, ws=FAKE,
              n=1 << 30)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_residual_norm_backward(*[a[k] for k in ("dy", "s", "st", "w", "wt", "rstd", "ds", "N", "H", "dx",
                                                               "dres", "dw", "ws", "n")], None)
    for k in ("dy", "s", "w", "rstd", "dx", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("dy", "s", "w", "ds", "dx", "ws"):
        assert call(**{k: ODD}) == 1, k
    assert call(dres=FAKE) == 1                                # only with fp32 sums
    assert call(st=2) == 1 and call(wt=3) == 1 and call(N=-1) == 1 and call(H=12) == 1
    assert call(n=16) == 3
    assert call(H=32776) == 2


FFN = ("x", "xs", "wgu", "ws", "wd", "rows", "E", "H", "I", "t", "p", "h", "pre", "y")
BACK = ("dy", "x", "h", "pre", "wgu", "wd", "rows", "E", "H", "I", "p", "dgu", "dx", "dwgu", "dwd")


def test_expert_ffn(lib):
    ok = dict(x=FAKE, xs=None, wgu=FAKE, ws=None, wd=FAKE, rows=64, E=4, H=64, I=40, t=0, p=plan(), h=FAKE, pre=FAKE,
              y=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_expert_ffn(*[a[k] for k in FFN], None)
    for k in ("x", "wgu", "wd", "p", "h", "y"):
        assert call(**{k: None}) == 1, k
    for k in ("x", "wgu", "wd", "h", "pre", "y"):
        assert call(**{k: ODD}) == 1, k
    assert call(p=plan(cu_seqlens=None)) == 1 and call(p=plan(tokens_per_expert=None)) == 1
    assert call(p=plan(status=None)) == 1
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1
    assert call(E=0) == 1 and call(E=1025) == 1
    assert call(H=60) == 1 and call(H=0) == 1 and call(I=44) == 1 and call(I=0) == 1 and call(H=1 << 20) == 1
    assert call(t=1) == 1 and call(t=3) == 1
    assert call(xs=FAKE) == 1 and call(ws=FAKE) == 1            # scales go with 8 bits
    assert call(t=2) == 1 and call(t=2, xs=FAKE) == 1 and call(t=2, ws=FAKE) == 1
    assert call(t=2, xs=FAKE, ws=FAKE, H=72) == 1               # H % 16
    assert call(t=2, xs=FAKE, ws=FAKE) == 2                     # no saved pre-activations in 8 bits
    assert call(rows=0) == 0 and call(rows=0, x=None, h=None, y=None, pre=None) == 0


def test_expert_ffn_backward(lib):
    ok = dict(dy=FAKE, x=FAKE, h=FAKE, pre=FAKE, wgu=FAKE, wd=FAKE, rows=64, E=4, H=64, I=40, p=plan(), dgu=FAKE, dx=FAKE,
              dwgu=FAKE, dwd=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_expert_ffn_backward(*[a[k] for k in BACK], None)
    for k in ("dy", "x", "h", "pre", "wgu", "wd", "p", "dgu"):
        assert call(**{k: None}) == 1, k
    for k in ("dy", "x", "h", "pre", "wgu", "wd", "dgu", "dx", "dwgu", "dwd"):
        assert call(**{k: ODD}) == 1, k
    assert call(rows=-1) == 1 and call(E=0) == 1 and call(H=4) == 1 and call(I=4) == 1
    assert call(p=plan(status=None)) == 1


def test_combine_backward(lib):
    ok = dict(dout=FAKE, y=FAKE, w=FAKE, N=4, K=2, H=64, E=8, rows=64, p=plan(), dy=FAKE, dw=FAKE)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.moe_combine_backward(*[a[k] for k in ("dout", "y", "w", "N", "K", "H", "E", "rows", "p", "dy", "dw")],
                                        None)
    for k in ("dout", "y", "w", "p", "dy", "dw"):
        assert call(**{k: None}) == 1, k
    for k in ("dout", "y", "dy"):
        assert call(**{k: ODD}) == 1, k
    assert call(p=plan(dst=None)) == 1 and call(p=plan(zero_fill_ranges=None)) == 1 and call(p=plan(status=None)) == 1
    assert call(N=-1) == 1 and call(K=0) == 1 and call(K=33, E=64) == 1 and call(K=9) == 1 and call(H=12) == 1
    assert call(E=1025) == 1 and call(rows=-1) == 1 and call(rows=1 << 31) == 1
    assert call(N=0) == 0 and call(N=0, dout=None, y=None, w=None, dy=None, dw=None) == 0

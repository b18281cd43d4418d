"""Plain 64-bit forms of the operators around the experts, and the bounds
their tests use.

Error model.  A bf16 store rounds to nearest: relative error at most
U = 2^-8 (half of the 2^-7 spacing; 8 significant bits).  An fp32 sum of n
products of exactly represented factors is off by at most n * F times the sum
of the products' magnitudes, with F = 2^-22 per step: a tensor-core sum may
truncate, and aligns its addends to the largest one, which costs more than the
2^-24 of a rounded fp32 addition.  Functions evaluated in fp32 (division,
exponential) add a few units of 2^-23, taken as S = 2^-19.
"""
from types import SimpleNamespace

import torch

U = 2.0 ** -8
F = 2.0 ** -22
S = 2.0 ** -19


def groups(counts, align, extra_rows=0, device="cuda"):
    """The plan arrays of groups of the given sizes, padded to `align` rows."""
    count = torch.tensor(counts, dtype=torch.int64)
    padded = (count + align - 1) // align * align
    cu = torch.zeros(len(counts) + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(padded, 0)
    rows = int(cu[-1]) + extra_rows
    kind = torch.full((rows,), 2, dtype=torch.int64)      # 0 a group's row, 1 padding, 2 past the groups
    for e, n in enumerate(counts):
        kind[cu[e]:cu[e] + n] = 0
        kind[cu[e] + n:cu[e + 1]] = 1
    i32 = dict(dtype=torch.int32, device=device)
    return SimpleNamespace(cu_seqlens=cu.to(**i32), tokens_per_expert=count.to(**i32),
                           status=torch.zeros(4, **i32), rows=rows, counts=list(counts), begins=cu.tolist(),
                           kind=kind.to(device))


def ffn_forward(x, w_gate_up, w_down, p):
    """g, u, h, y in 64 bits, and sums of magnitudes for the bounds (x, w already in 64 bits)."""
    E, _, I, H = w_gate_up.shape  # noqa: E741
    z = lambda n: torch.zeros(p.rows, n, dtype=torch.float64, device=x.device)  # noqa: E731
    o = SimpleNamespace(g=z(I), u=z(I), h=z(I), y=z(H), g_abs=z(I), u_abs=z(I), y_abs=z(H))
    for e, n in enumerate(p.counts):
        at = slice(p.begins[e], p.begins[e] + n)
        o.g[at], o.u[at] = x[at] @ w_gate_up[e, 0].T, x[at] @ w_gate_up[e, 1].T
        o.g_abs[at], o.u_abs[at] = x[at].abs() @ w_gate_up[e, 0].abs().T, x[at].abs() @ w_gate_up[e, 1].abs().T
        o.h[at] = o.g[at] * torch.sigmoid(o.g[at]) * o.u[at]
        o.y[at] = o.h[at] @ w_down[e].T
        o.y_abs[at] = o.h[at].abs() @ w_down[e].abs().T
    return o


def h_bound(o, H):
    """Bound of |h - h exact|: the errors of g and u through silu (slope at most 1.1), then the rounding."""
    dg, du = H * F * o.g_abs, H * F * o.u_abs
    silu = (o.g * torch.sigmoid(o.g)).abs()
    fp32 = 1.1 * dg * (o.u.abs() + du) + silu * du + S * o.h.abs()
    return fp32 + U * (o.h.abs() + fp32)


def y_bound(o, w_down, p, H):
    """Bound of |y - y exact|: h's error through w_down, the sum's error, then the rounding."""
    eh = h_bound(o, H)
    I = o.h.shape[1]  # noqa: E741
    e = torch.zeros_like(o.y)
    for k, n in enumerate(p.counts):
        at = slice(p.begins[k], p.begins[k] + n)
        e[at] = eh[at] @ w_down[k].abs().T
    e = e + I * F * (o.y_abs + e)
    return e + U * (o.y.abs() + e)


def ffn_backward(dy, x, h, g, u, w_gate_up, w_down, p):
    """Gradients in 64 bits from the stored h, g, u, with their bounds."""
    E, _, I, H = w_gate_up.shape  # noqa: E741
    dev = x.device
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    o = SimpleNamespace(dx=z(p.rows, H), dwgu=z(E, 2, I, H), dwd=z(E, H, I), dx_tol=z(p.rows, H),
                        dwgu_tol=z(E, 2, I, H), dwd_tol=z(E, H, I))
    sig = torch.sigmoid(g)
    slope, act = u * sig * (1 + g * (1 - sig)), g * sig
    for e, n in enumerate(p.counts):
        at = slice(p.begins[e], p.begins[e] + n)
        dh, dh_abs = dy[at] @ w_down[e], dy[at].abs() @ w_down[e].abs()
        dgu, err = [], []
        for f in (slope[at], act[at]):
            d = dh * f
            # |1 + g (1 - sig)| and its factors cancel at most where they are of order one: S of |u| covers them
            t = H * F * dh_abs * f.abs() + S * (d.abs() + dh.abs() * (u[at].abs() if f is not act[at] else 0))
            dgu.append(d)
            err.append(t + U * (d.abs() + t))
        D, T = torch.cat(dgu, 1), torch.cat(err, 1)
        W = w_gate_up[e].reshape(2 * I, H)

        def out(v, first, mag, k):
            t = first + k * F * (mag + first)
            return t + U * (v.abs() + t)
        o.dx[at] = D @ W
        o.dx_tol[at] = out(o.dx[at], T @ W.abs(), D.abs() @ W.abs(), 2 * I)
        v = D.T @ x[at]
        o.dwgu[e] = v.reshape(2, I, H)
        o.dwgu_tol[e] = out(v, T.T @ x[at].abs(), D.abs().T @ x[at].abs(), n).reshape(2, I, H)
        v = dy[at].T @ h[at]
        o.dwd[e] = v
        o.dwd_tol[e] = out(v, torch.zeros_like(v), dy[at].abs().T @ h[at].abs(), n)
    return o


def assert_within(got, want, tol, what):
    """|got - want| <= tol everywhere (tiny absolute slack for values below bf16's normal range)."""
    err = (got.double() - want).abs()
    bad = ~(err <= tol + 1e-30)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g against %.3g" % (
        what, int(bad.sum()), bad.numel(), float((err - tol)[bad].max()), float(tol[bad].max()))

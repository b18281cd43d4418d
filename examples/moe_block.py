"""One MoE block, forwards and backwards, and a decoding step of it, on one GPU.

    python examples/moe_block.py [--tokens 4096] [--steps 20]

norm -> router -> plan -> permute -> experts -> combine, then the gradients of all
of it: the combine's, the experts', the permute's (the combine with weights of
one), the router's (a few torch operations on [tokens, K] values) and the norm's.
Plain gradient steps on random data bring the loss down.  The decoding step uses
the norm's 8-bit rows and 8-bit gate/up weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_dispatch_planning_gb300 as moe  # noqa: E402

E, K, R, ALIGN = 32, 4, 4, 16
H, I = 1024, 512  # noqa: E741
BF16 = torch.bfloat16


class Block:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std
        # fp32 copies take the gradient steps; the bf16 ones are what the kernels read
        self.norm = torch.ones(H, device="cuda")
        self.router = normal(E, H, std=H ** -0.5)
        self.w_gate_up = normal(E, 2, I, H, std=H ** -0.5)
        self.w_down = normal(E, H, I, std=I ** -0.5)
        self.cast()

    def cast(self):
        self.w_gate_up16, self.w_down16 = self.w_gate_up.to(BF16), self.w_down.to(BF16)

    def forward(self, x, stream):
        """x bf16[N,H] (the layer's input) added to the residual stream float32[N,H]: (out, saved)."""
        n = moe.residual_norm(x, self.norm, residual=stream)
        logits = n.y.float() @ self.router.T
        idx, w, plan = moe.route_plan(logits, K, R, ALIGN)
        xp = moe.permute(n.y, plan)
        rows = xp.shape[0]
        h = torch.empty((rows, I), dtype=BF16, device="cuda")
        preact = torch.empty((rows, 2, I), dtype=torch.float32, device="cuda")
        yp = moe.expert_ffn(xp, self.w_gate_up16, self.w_down16, plan, h=h, preact=preact)
        out = moe.combine(yp, w, plan)
        return out, (n, idx, w, plan, xp, h, preact, yp)

    def backward(self, dout, saved, lr):
        """Gradient step for d(loss)/d(out) = dout; returns the gradients of x and of the residual stream."""
        n, idx, w, plan, xp, h, preact, yp = saved
        dyp, dw = moe.combine_backward(dout, yp, w, plan)
        dxp, dwgu, dwd = moe.expert_ffn_backward(dyp, xp, h, preact, self.w_gate_up16, self.w_down16, plan)
        dy = moe.combine(dxp, torch.ones_like(w), plan).float()
        # softmax over the chosen logits
        dlogit = w * (dw - (w * dw).sum(1, keepdim=True))
        dlogits = torch.zeros((idx.shape[0], E), device="cuda").scatter_(1, idx.long(), dlogit)
        drouter = dlogits.T @ n.y.float()
        dy = (dy + dlogits @ self.router).to(BF16)
        dx, dstream, dnorm = moe.residual_norm_backward(dy, n.residual, self.norm, n.rstd)
        self.norm -= lr * dnorm
        self.router -= lr * drouter
        self.w_gate_up -= lr * dwgu.float()
        self.w_down -= lr * dwd.float()
        self.cast()
        return dx, dstream

    def decode(self, x, stream, w8, w8_scale):
        """The forward pass with 8-bit rows and gate/up weights (w8 e4m3[E,2,I,H], w8_scale float32[E,2,I])."""
        n = moe.residual_norm(x, self.norm, residual=stream, quantize=True)
        idx, w, plan = moe.route_plan(n.y.float() @ self.router.T, K, R, ALIGN)
        # two 8-bit values are one 16-bit element to the permute; the scales follow by the plan's indexes
        qp = moe.permute(n.q.view(BF16), plan).view(torch.float8_e4m3fn)
        scale = n.q_scale[(plan.src_of_slot.clamp(min=0) // K).long()].contiguous()
        yp = moe.expert_ffn(qp, w8, self.w_down16, plan, x_scale=scale, w_scale=w8_scale)
        return moe.combine(yp, w, plan)


def quantize_channels(w):
    scale = w.float().abs().amax(-1).clamp_min(1e-12) / 448
    return (w.float() / scale[..., None]).to(torch.float8_e4m3fn), scale


def main(tokens=4096, steps=20, lr=0.3, decode_tokens=8, verbose=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(tokens, H, generator=g, device="cuda").to(BF16)
    stream = torch.randn(tokens, H, generator=g, device="cuda")
    target = torch.tanh(torch.randn(tokens, H, generator=g, device="cuda"))
    block = Block()
    losses = []
    for _ in range(steps):
        out, saved = block.forward(x, stream)
        err = out.float() - target
        losses.append(float(err.square().mean()))
        dout = (2 * err / tokens).to(BF16)      # of the sum over H of the mean over the tokens
        block.backward(dout, saved, lr)
    if verbose:
        print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], steps))

    xs, ss = x[:decode_tokens].contiguous(), stream[:decode_tokens].contiguous()
    want, _ = block.forward(xs, ss)
    got = block.decode(xs, ss, *quantize_channels(block.w_gate_up))
    rel = float((got.float() - want.float()).norm() / want.float().norm())
    if verbose:
        print("8-bit decoding step: %.3f from the bf16 one" % rel)
    return losses, rel


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    main(a.tokens, a.steps)

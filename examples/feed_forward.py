"""A gated feed-forward block with frozen int8 weights behind an RMS norm, as a decoder
layer has it, served and trained through.

Serving: four calls from the residual stream to the residual stream.

    q, s, h = rms_norm_quantize(x, gain, residual=r)
    y       = qgemm_a8w8_gated(q, W_gate, W_up, s, ...)          act(gate) * up
    b, t    = int8_quantize(y)
    out     = qgemm_a8w8_linear(b, W_down, t, ..., residual=h)

Training the gain and what lies below: the gated call leaves its two products in 8 bits (a
byte and an eighth a value, where bf16 products would take four together), and the
gradient reads them.  The backward pass takes three calls.

    python examples/feed_forward.py [--tokens 512] [--hidden 4096] [--inner 14336]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_int8_gemm_amd as q  # noqa: E402

EPS = 1e-6


class FeedForward(torch.nn.Module):
    """gate, up: [inner, hidden]; down: [hidden, inner]; gain: [hidden].  The weights are kept
    in int8 with a scale per output row; the gain is trained."""

    def __init__(self, gate, up, down, gain, activation="silu"):
        super().__init__()
        self.gain, self.activation = torch.nn.Parameter(gain), activation
        for name, w in (("gate", gate), ("up", up), ("down", down)):
            codes, scale = q.int8_quantize(w)
            self.register_buffer(name, codes)
            self.register_buffer(name + "_scale", scale)

    def forward(self, x, residual):
        """(output, h): h = x + residual is the stream that the block adds to.  x: bf16 or fp16,
        which the gradients take; serve takes fp32 too."""
        if x.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"x has dtype {x.dtype}; training through the block takes torch.bfloat16 or torch.float16")
        return _Step.apply(x, residual, self.gain, self)

    def serve(self, x, residual):
        a, s, h = q.rms_norm_quantize(x, self.gain, EPS, residual=residual)
        y = q.qgemm_a8w8_gated(a, self.gate, self.up, s, self.gate_scale, self.up_scale, self.activation, x.dtype, b_trans=True)
        return self._down(y, h), h

    def _down(self, y, h):
        b, t = q.int8_quantize(y)
        return q.qgemm_a8w8_linear(b, self.down, t, self.down_scale, residual=h, out_dtype=h.dtype, b_trans=True)


class _Step(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, gain, block):
        a, s, h = q.rms_norm_quantize(x, gain, EPS, residual=residual)
        y, saved = q.qgemm_a8w8_gated(a, block.gate, block.up, s, block.gate_scale, block.up_scale, block.activation, x.dtype,
                                      b_trans=True, checkpoint=True)
        ctx.block = block
        ctx.save_for_backward(h, gain, *saved)
        return block._down(y, h), h

    @staticmethod
    def backward(ctx, d_out, d_h):
        h, gain, codes, scale = ctx.saved_tensors
        b = ctx.block
        dy = q.qgemm_a8w8_linear_grad(d_out.contiguous(), b.down, b.down_scale, b_trans=True)
        dn = q.qgemm_a8w8_gated_grad(dy, b.gate, b.up, b.gate_scale, b.up_scale, (codes, scale), b.activation, b_trans=True)
        rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
        dx, dgain = q.rms_norm_grad(dn, h, gain, rstd, dh=d_out + d_h)
        return dx, dx, dgain, None


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=14336)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()   # noqa: E731
    gate, up, down = rand(a.inner, a.hidden) * a.hidden ** -0.5, rand(a.inner, a.hidden) * a.hidden ** -0.5, rand(a.hidden, a.inner) * a.inner ** -0.5
    block = FeedForward(gate, up, down, 1 + 0.1 * rand(a.hidden))
    for tokens in (1, a.tokens):
        x, r = rand(tokens, a.hidden), rand(tokens, a.hidden)
        out, h = block.serve(x, r)
        n = (h.double() * torch.rsqrt(h.double().square().mean(1, keepdim=True) + EPS) * block.gain.detach().double()).float()
        exact = (torch.nn.functional.silu(n @ gate.float().t()) * (n @ up.float().t())) @ down.float().t()
        added = out.float() - h.float()
        x.requires_grad_()
        y, h = block(x, r)
        (y.float().square().mean() + h.float().square().mean()).backward()
        print(f"{tokens} tokens: what the block adds is off by {((added - exact).norm() / exact.norm()).item():.4f} of the unquantised "
              f"block's; gradient norms {x.grad.float().norm().item():.4f}, {block.gain.grad.float().norm().item():.4f}")
        block.gain.grad = None


if __name__ == "__main__":
    main()

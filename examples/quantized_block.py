"""A frozen quantised projection behind an RMS norm, as a decoder layer has it,
served and trained through.

Serving, in int8 or in MX: the residual's addition, the norm and the activations'
quantisation are one call, the product the next.

    q, s, h = rms_norm_quantize(x, gain, residual=r)          ->  qgemm_a8w8(q, W8, s, ...)
    c, b, rstd, h = rms_norm_quantize(..., format="mxfp8")    ->  mx_matmul(c, b, W4, W4_scale, rstd)

Training the gain and what lies below, with the weight frozen in MXFP4: the
incoming gradient is quantised along the weight's rows, multiplied with the
transposed weight and taken back through the norm, the residual stream's own
gradient joined on the way.

    python examples/quantized_block.py [--tokens 512] [--width 4096] [--out 4096]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_int8_gemm_amd as q  # noqa: E402

EPS = 1e-6


class QuantizedBlock:
    """weight: [out, width] on the GPU; gain: [width].  The weight is kept in int8
    with a scale per output row, in MXFP4, and in MXFP4 transposed for the gradient."""

    def __init__(self, weight, gain, activations="mxfp8"):
        self.gain, self.activations = gain, activations
        top = weight.abs().amax(1).clamp(min=1e-30).float()
        self.w8 = torch.round(weight.float() * (127 / top)[:, None]).to(torch.int8)
        self.w8_scale = top / 127
        self.w4 = q.mx_quantize(weight, "mxfp4")
        self.w4_t = q.mx_quantize(weight.t().contiguous(), "mxfp4")

    def serve_int8(self, x, residual):
        """(output, h): h is the new residual stream."""
        codes, scale, h = q.rms_norm_quantize(x, self.gain, EPS, residual=residual, format="int8")
        return q.qgemm_a8w8(codes, self.w8, scale, self.w8_scale, out_dtype=torch.bfloat16, b_trans=True), h

    def forward(self, x, residual):
        """(output, h, rstd): what the next layer reads and what the gradient needs."""
        codes, scale, rstd, h = q.rms_norm_quantize(x, self.gain, EPS, residual=residual, format=self.activations)
        return q.mx_matmul(codes, scale, *self.w4, act_scale=rstd, out_dtype=torch.bfloat16), h, rstd

    def backward(self, d_out, h, rstd, d_h=None):
        """(gradient of x and of the residual alike, gradient of the gain)."""
        dy = q.mx_matmul(*q.mx_quantize(d_out, "mxfp8"), *self.w4_t, out_dtype=h.dtype)
        return q.rms_norm_grad(dy, h, self.gain, rstd, dh=d_h)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--out", type=int, default=4096)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()   # noqa: E731
    block = QuantizedBlock(0.02 * rand(a.out, a.width), 1 + 0.1 * rand(a.width))
    for tokens in (1, a.tokens):
        x, r = rand(tokens, a.width), rand(tokens, a.width)
        y8, h = block.serve_int8(x, r)
        y, h2, rstd = block.forward(x, r)
        exact = h.double() * torch.rsqrt(h.double().square().mean(1, keepdim=True) + EPS) * block.gain.double()
        exact = exact @ q.mx_dequantize(*block.w4, torch.float32).double().t().contiguous()
        off = lambda t: ((t.double() - exact).norm() / exact.norm()).item()   # noqa: E731
        dx, dgain = block.backward(rand(tokens, a.out), h2, rstd, d_h=rand(tokens, a.width))
        print(f"{tokens} tokens: MX off by {off(y):.4f} of the MXFP4 weight's exact output, int8 by {off(y8):.4f}; "
              f"gradient norms {dx.float().norm().item():.1f}, {dgain.float().norm().item():.1f}")


if __name__ == "__main__":
    main()

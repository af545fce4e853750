"""The feed-forward example refuses to train in a type that its gradients do not take, before
anything runs."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float64])
def test_forward_refuses(dtype):
    from feed_forward import FeedForward
    x = torch.zeros(2, 16, dtype=dtype)
    with pytest.raises(TypeError, match="training"):
        FeedForward.forward(None, x, x)


@pytest.mark.gpu
def test_serving_in_fp32():
    """Against the block in 64 bits with the same int8 weights, up to the two 8-bit roundings of
    activations (each at most 1.2 % of its values' root mean square)."""
    from feed_forward import EPS, FeedForward
    from gpu_util import dev
    g = torch.Generator(device=dev()).manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev())   # noqa: E731
    tokens, hidden, inner = 33, 320, 800
    block = FeedForward(rand(inner, hidden) * hidden ** -0.5, rand(inner, hidden) * hidden ** -0.5, rand(hidden, inner) * inner ** -0.5,
                        1 + 0.1 * rand(hidden))
    x, r = rand(tokens, hidden), rand(tokens, hidden)
    out, h = block.serve(x, r)
    assert out.dtype == h.dtype == torch.float32 and torch.equal(h, x + r)
    w = [(c.double() * s.double()[:, None]).cpu() for c, s in ((block.gate, block.gate_scale), (block.up, block.up_scale),
                                                              (block.down, block.down_scale))]
    hd = h.double().cpu()
    n = hd * torch.rsqrt(hd.square().mean(1, keepdim=True) + EPS) * block.gain.detach().double().cpu()
    want = (torch.nn.functional.silu(n @ w[0].t()) * (n @ w[1].t())) @ w[2].t() + hd
    assert (out.double().cpu() - want).norm() <= 0.06 * want.norm()

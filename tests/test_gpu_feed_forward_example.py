"""The feed-forward example: it runs, serves what it trains through, and its gradients are
those of the same block by torch's autograd in 64 bits, up to the 8-bit roundings."""
import os
import subprocess
import sys

import pytest
import torch

from gpu_util import dev

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu


def test_gradients():
    from feed_forward import EPS, FeedForward
    g = torch.Generator(device=dev()).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev()).bfloat16()   # noqa: E731
    tokens, hidden, inner = 65, 320, 800
    block = FeedForward(rand(inner, hidden) * hidden ** -0.5, rand(inner, hidden) * hidden ** -0.5, rand(hidden, inner) * inner ** -0.5,
                        1 + 0.1 * rand(hidden))
    x, r, d = (rand(tokens, hidden) for _ in range(3))
    x.requires_grad_()
    out, h = block(x, r)
    assert torch.equal(out, block.serve(x.detach(), r)[0])
    out.backward(d)
    w = [(c.double() * s.double()[:, None]).cpu() for c, s in ((block.gate, block.gate_scale), (block.up, block.up_scale),
                                                              (block.down, block.down_scale))]
    xd, gain = x.detach().double().cpu().requires_grad_(), block.gain.detach().double().cpu().requires_grad_()
    hd = xd + r.double().cpu()
    n = hd * torch.rsqrt(hd.square().mean(1, keepdim=True) + EPS) * gain
    want = (torch.nn.functional.silu(n @ w[0].t()) * (n @ w[1].t())) @ w[2].t() + hd
    want.backward(d.double().cpu())
    # each 8-bit rounding is off by at most 1.2 % of its values' root mean square, as in the test of
    # the calls together
    for got, ref in ((out, want.detach()), (x.grad, xd.grad), (block.gain.grad, gain.grad)):
        assert (got.detach().double().cpu() - ref).norm() <= 0.06 * ref.norm()


def test_it_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "feed_forward.py"), "--tokens", "40", "--hidden", "512", "--inner", "1424"],
                       capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and r.stdout.count("tokens:") == 2, r.stderr

"""The gradient of the RMS norm for rows far larger or smaller than one, whose
forward is an ordinary number: against the 64-bit formula."""
import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def d64(t):
    return t.detach().cpu().double().numpy()


# a width of every way that rows pass through the registers
@pytest.mark.parametrize("n", [6, 100, 700, 4096, 6144, 12288, 20000, 40000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size,dsize", [(1e13, 1.0), (1e15, 1.0), (1e18, 1.0), (1e-13, 1.0), (1e-18, 1.0), (1e-13, 1e-28), (1e18, 1e15)])
def test_gradient_of_large_and_small_rows(n, dtype, size, dsize):
    case(f"rms_norm_grad rows of {size}, gradients of {dsize}, n={n} {dtype}")
    g = torch.Generator().manual_seed(n)
    base = torch.randn(3, n, generator=g)
    h = (base * size).to(dtype)
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(dtype)
    dy = (dsize * (base / w.float() + 0.2 * torch.randn(3, n, generator=g))).to(dtype)   # along h: the projection counts
    r = torch.from_numpy(R.rstd(d64(h), 0.0)).float()
    dx, dw = q.rms_norm_grad(*(t.to(dev()) for t in (dy, h, w, r)))
    wx, ww = R.grad(d64(dy), d64(h), d64(w), d64(r))
    rr = d64(r)[:, None]
    # a lane's 64 products of four factors and 21 sums, then 8 steps around each term
    part = np.abs(d64(h) * rr) * rr / n * np.abs(d64(dy) * d64(w) * d64(h) * rr).sum(1, keepdims=True)
    tol = U * (110 * part + 8 * np.abs(rr * d64(dy) * d64(w)) + 8 * np.abs(wx))
    assert np.all(np.abs(d64(dx) - wx) <= tol + HALF[dtype] * 1.01 * np.abs(wx))
    size = np.abs(d64(dy) * d64(h) * rr).sum(0)
    assert np.all(np.abs(d64(dw) - ww) <= 12 * U * size + HALF[dtype] * 1.01 * np.abs(ww))


@pytest.mark.parametrize("n", [6, 700, 4096, 40000])
def test_gradient_of_a_row_of_zeros(n):
    """dx = r * dy * w: h is zero, r = 1 / sqrt(eps) = 2^50."""
    case(f"rms_norm_grad of zeros, n={n}")
    h = torch.zeros(2, n, device=dev())
    w = torch.ones(n, device=dev())
    dy = torch.randn(2, n, generator=torch.Generator().manual_seed(n)).to(dev())
    y, r = q.rms_norm(h, w, 2.0 ** -100)
    assert not y.any() and (r == 2.0 ** 50).all()
    dx, dw = q.rms_norm_grad(dy, h, w, r)
    assert torch.equal(dx, dy * 2.0 ** 50) and not dw.any()

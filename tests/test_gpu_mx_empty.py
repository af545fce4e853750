"""Batches without rows, wherever the empty dimension stands."""
import pytest
import torch

import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 2), (2, 0, 3), (3, 2, 0), (0, 0)])
def test_no_rows(lead):
    case(f"norm and MX calls on {lead} rows of 40")
    d = dev()
    x, w = torch.zeros(*lead, 40, device=d), torch.ones(40, device=d)
    y, r, h = q.rms_norm(x, w, residual=x)
    assert y.shape == x.shape == h.shape and r.shape == lead
    c, s = q.rms_norm_quantize(x, w)
    assert c.shape == x.shape and s.shape == lead
    for fmt, per in (("mxfp8", 32), ("mxfp4", 16)):
        c, s, r = q.rms_norm_quantize(x, w, format=fmt)
        assert c.shape == lead + (2 * per,) and s.shape == lead + (2,) and r.shape == lead
        c, s = q.mx_quantize(x, fmt)
        assert c.shape == lead + (2 * per,) and s.shape == lead + (2,)
        assert q.mx_dequantize(c, s, columns=40).shape == x.shape
    dx, dw = q.rms_norm_grad(x, x, w, r, dh=x)
    assert dx.shape == x.shape and dw.shape == (40,) and not dw.any()

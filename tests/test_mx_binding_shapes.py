"""Shapes that the norm and MX calls take, on the CPU: a call whose only fault is
the device has passed every check of its shapes."""
import pytest
import torch

import quantized_int8_gemm_amd as q


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 2), (2, 0, 3), (3, 2, 0), (0, 0), (2, 1, 3), (1, 1)])
def test_batches_with_and_without_rows(lead):
    x, w, r = torch.zeros(*lead, 64), torch.ones(64), torch.ones(lead)
    u, s = torch.zeros(*lead, 32, dtype=torch.uint8), torch.zeros(*lead, 2, dtype=torch.uint8)
    for call in (lambda: q.rms_norm(x, w, residual=x, residual_out=x), lambda: q.rms_norm_quantize(x, w, format="mxfp4"),
                 lambda: q.rms_norm_grad(x, x, w, r, dh=x), lambda: q.mx_quantize(x), lambda: q.mx_dequantize(u, s)):
        with pytest.raises(ValueError, match="GPU device"):
            call()


def test_rows_at_several_strides_are_still_refused():
    x = torch.zeros(3, 4, 80)[:, :3, :64]
    with pytest.raises(ValueError, match="one stride"):
        q.mx_quantize(x)

"""The MX product's byte kernel with more rows than one launch takes."""
import pytest
import torch

import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_rows_past_one_launch(fmt):
    """Rows before, at and after the border of 65535 * 16, with scale rows of three bytes:
    each as in a product of few rows, bit for bit (every element is one wave's, in one order)."""
    case(f"mx_matmul bytes, 2^20 + 50 rows, {fmt}")
    d = dev()
    m, n, k, edge = (1 << 20) + 50, 20, 96, 65535 * 16
    g = torch.Generator(device=d).manual_seed(4)
    a = torch.randint(0, 256, (m, k // 2 if fmt == "mxfp4" else k), generator=g, dtype=torch.uint8, device=d)
    if fmt == "mxfp8":
        a = torch.where(a % 128 == 127, 0, a).to(torch.uint8).view(torch.float8_e4m3fn)
    sa = torch.randint(120, 130, (m, k // 32), generator=g, dtype=torch.uint8, device=d)
    w, sw = q.mx_quantize(torch.randn(n, k, generator=g, device=d))
    s = torch.rand(m, generator=g, device=d) + 0.5
    for t in (torch.float32, torch.bfloat16):
        out = torch.full((m, n + 3), 9.0, dtype=t, device=d)
        q.mx_matmul(a, sa, w, sw, act_scale=s, out_dtype=t, out=out[:, :n])
        assert q._binding.last_kernel() == "mx_matmul_bytes"
        assert (out[:, n:] == 9).all()
        for lo, hi in ((0, 40), (edge - 40, edge + 1), (edge, m)):
            few = q.mx_matmul(a[lo:hi], sa[lo:hi].contiguous(), w, sw.contiguous(), act_scale=s[lo:hi], out_dtype=t)
            assert q._binding.last_kernel() == "mx_matmul_bytes"
            assert torch.equal(out[lo:hi, :n], few), (lo, hi)

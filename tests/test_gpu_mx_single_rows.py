"""MX products with one row of scales whose last word ends with its allocation:
nothing past it is asked for, and the values are those of padded rows."""
import pytest
import torch

import quantized_int8_gemm_amd as q
from gpu_util import case, dev, env

pytestmark = pytest.mark.gpu


def at_the_end(scale):
    """The same row in the last whole words of an allocation of its own."""
    n = scale.shape[1]
    buf = torch.empty(32 << 20, dtype=torch.uint8, device=scale.device)
    words = buf[-(-(-n // 4) * 4):]
    words[:n] = scale[0]
    return words[:n].view(1, n)


@pytest.mark.parametrize("K", [32, 64, 96, 160, 1056])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_one_row(K, fmt):
    case(f"mx_matmul one row of scales, K={K} {fmt}")
    g = torch.Generator(device=dev()).manual_seed(K)
    one, many = (torch.randn(m, K, generator=g, device=dev()) for m in (1, 70))
    for tile in (None, 0, 1, 2, 3, 4, 5):
        with env(**({} if tile is None else {"QGEMM_MX_TILE": tile})):
            a, sa = q.mx_quantize(one, fmt)
            w, sw = q.mx_quantize(many)
            want = q.mx_matmul(a, sa, w, sw)
            assert torch.equal(q.mx_matmul(a, at_the_end(sa), w, sw), want)
            assert q._binding.last_kernel() == "mx_decode" if tile is None else q._binding.last_kernel().startswith("mx_tiled")
            a, sa = q.mx_quantize(many, fmt)
            w, sw = q.mx_quantize(one)
            want = q.mx_matmul(a, sa, w, sw)
            assert torch.equal(q.mx_matmul(a, sa, w, at_the_end(sw)), want)
            assert q._binding.last_kernel().startswith("mx_tiled")

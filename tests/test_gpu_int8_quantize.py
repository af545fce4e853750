"""The int8 quantiser and back, against the definition's fp32 steps, bit for bit."""
import numpy as np
import pytest
import torch

import fused_reference as ref
import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
WIDTHS = [1, 5, 7, 8, 31, 32, 33, 100, 128, 129, 511, 513, 2048, 2050, 4096, 5000, 8192, 8200, 16384, 16400, 40000, 65536]


def check(x, block):
    codes, scale = q.int8_quantize(x, block)
    want, ws = ref.int8_form(x.float().cpu().numpy().reshape(-1, x.shape[-1]), block)
    assert np.array_equal(codes.cpu().numpy().reshape(want.shape), want)
    assert np.array_equal(scale.cpu().numpy().reshape(ws.shape), ws, equal_nan=True)
    for d in TYPES:
        back = q.int8_dequantize(codes, scale, d)
        s = ws[:, None] if block is None else np.repeat(ws, 32, 1)[:, :x.shape[-1]]
        v = torch.from_numpy(want.astype(np.float32) * s).to(d)
        got = back.cpu().reshape(v.shape)
        assert torch.equal(got.isnan(), v.isnan()) and torch.equal(got.nan_to_num(), v.nan_to_num())


@pytest.mark.parametrize("block", [None, 32])
@pytest.mark.parametrize("n", WIDTHS)
def test_widths(n, block):
    for i, d in enumerate(TYPES):
        m = (1, 3, 17)[(i + n) % 3] if n > 1000 else (1, 70, 301)[(i + n) % 3]
        case(f"int8 {m} x {n} {d} block={block}")
        g = torch.Generator(device=dev()).manual_seed(n)
        x = torch.randn(m, n, generator=g, device=dev())
        x[m // 2] = 0
        check(x.to(d), block)


@pytest.mark.parametrize("block", [None, 32])
@pytest.mark.parametrize("d", TYPES)
def test_values_at_the_ends(d, block):
    big, least = torch.finfo(d).max, torch.finfo(d).smallest_normal
    x = torch.randn(9, 96, device=dev())
    x[0, 3], x[1, 40], x[2, 95] = float("nan"), float("inf"), -float("inf")
    x[3] *= big / 8
    x[4] = big
    x[5] *= least
    x[6] = least / 2
    x[7] = -0.0
    x[8, 33:] = 0
    check(x.to(d), block)


@pytest.mark.parametrize("block", [None, 32])
def test_ties_go_to_the_even_code(block):
    x = torch.arange(-127, 128, dtype=torch.float32, device=dev()) / 2
    x = torch.cat([x, torch.tensor([127.0], device=dev())])[None].repeat(2, 1)
    x[:, 0::32] = 127.0   # every block's largest: one step is 1
    check(x, block)


def test_more_dimensions_and_strides():
    x = torch.randn(3, 5, 130, device=dev()).bfloat16()
    for block in (None, 32):
        codes, scale = q.int8_quantize(x, block)
        assert codes.shape == x.shape and scale.shape == ((3, 5) if block is None else (3, 5, 5))
        check(x, block)
        check(x[:, :, :77][1], block)
        check(x[0, 0], block)
        wide = torch.full((15, 200), 7, dtype=torch.int8, device=dev())
        wide[:, :130] = codes.view(15, 130)
        out = torch.full((15, 140), 3.0, device=dev())
        got = q.int8_dequantize(wide[:, :130], scale.view(15, *scale.shape[2:]), torch.float32, out=out[:, :130])
        assert torch.equal(got, q.int8_dequantize(codes, scale, torch.float32).view(15, 130)) and (out[:, 130:] == 3).all()
    e = q.int8_quantize(x[:, :0], 32)
    assert e[0].shape == (3, 0, 130) and e[1].shape == (3, 0, 5) and q.int8_dequantize(*e).shape == (3, 0, 130)


def test_rows_of_more_columns_are_refused_with_one_scale_only():
    x = torch.randn(2, 65537, device=dev())
    with pytest.raises(NotImplementedError):
        q.int8_quantize(x)
    check(x, 32)


def test_offsets_past_32_bits():
    """Rows behind 2^31 elements: the last ones as a small call gives them."""
    m, n = 70000, 32768
    x = torch.zeros(m, n, dtype=torch.bfloat16, device=dev())
    x[-2:] = torch.randn(2, n, device=dev()).bfloat16()
    for block in (None, 32):
        codes, scale = q.int8_quantize(x, block)
        c2, s2 = q.int8_quantize(x[-2:].clone(), block)
        assert torch.equal(codes[-2:], c2) and torch.equal(scale[-2:], s2) and (codes[:-2] == 0).all()
        back = q.int8_dequantize(codes, scale)
        assert torch.equal(back[-2:], q.int8_dequantize(c2, s2)) and (back[:-2] == 0).all()


def test_every_mantissa():
    """The largest magnitude takes every mantissa, at several exponents: codes of it and of
    its half, and the scale, as the division gives them."""
    m = torch.arange(1 << 23, device=dev(), dtype=torch.int32)
    for e in (0, 27, 28, 90, 127, 128, 200, 247, 248, 254):
        top = (m | (e << 23)).view(torch.float32)
        x = torch.stack([top, -top * 0.5, top * 0.3, top * 0.77], 1).contiguous()
        codes, scale = q.int8_quantize(x)
        t, y = top.cpu().numpy(), x.cpu().numpy()
        up = np.where(t < np.float32(2.0 ** -100), np.float32(2.0 ** 60), np.float32(1))
        with np.errstate(divide="ignore"):
            inv = np.where(t > 0, np.float32(127) / (t * up), np.float32(0))
        assert np.array_equal(scale.cpu().numpy(), np.where(t > 0, t / np.float32(127), np.float32(1)))
        assert np.array_equal(codes.cpu().numpy(), np.rint((y * up[:, None]) * inv[:, None]).astype(np.int8))

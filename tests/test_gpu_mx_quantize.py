"""MX quantisation and reading back on the GPU: bit for bit what the 64-bit
reference gives."""
import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]
FORMATS = ["mxfp8", "mxfp4"]


def elements(codes, fmt):
    c = codes.view(torch.uint8).cpu().numpy()
    return R.unpack(c) if fmt == "mxfp4" else c


def same(got, want):
    """Equal values, NaN (the values of a block with an infinity) included."""
    return np.array_equal(got.cpu().float().numpy(), want.float().numpy(), equal_nan=True)


@pytest.mark.parametrize("rows,n", [(1, 1), (3, 31), (2, 32), (5, 33), (16, 8192), (7, 1000), (257, 130), (1, 70001), (0, 64)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_and_back(rows, n, dtype, fmt):
    case(f"mx_quantize {rows}x{n} {dtype} {fmt}")
    x = torch.randn(rows, n, generator=torch.Generator().manual_seed(n)) * torch.exp(4 * torch.randn(rows, 1, generator=torch.Generator().manual_seed(1)))
    x = x.to(dtype)
    codes, scale = q.mx_quantize(x.to(dev()), fmt)
    c, s = R.mx_quantize(x.double().numpy(), fmt)
    assert codes.dtype == (torch.uint8 if fmt == "mxfp4" else torch.float8_e4m3fn)
    assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(elements(codes, fmt), c)
    assert rows < 2 or scale.stride(0) % 16 == 0
    v = R.mx_values(c, s, fmt)
    for out in TYPES:
        got = q.mx_dequantize(codes, scale, out, columns=n)
        assert got.shape == (rows, n) and same(got, torch.from_numpy(v[:, :n]).to(out))
    assert same(q.mx_dequantize(codes, scale, torch.float32), torch.from_numpy(v))


# rows of one group of eight, and of about as many as a workgroup moves (1024)
@pytest.mark.parametrize("rows,n", [(5000, 3), (2100, 9), (1030, 17), (900, 33), (11, 8160), (11, 8184), (11, 8192), (11, 8200), (9, 8225), (5, 16385), (3, 40000)])
@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_between_workgroups(rows, n, fmt):
    test_quantize_and_back(rows, n, torch.bfloat16, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_rounding_border(fmt):
    """Each value, each midpoint and both its neighbours, under three scales."""
    case(f"mx_quantize borders {fmt}")
    g = R.GRID[fmt]
    mid = (g[1:] + g[:-1]) / 2
    pts = np.concatenate([g, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                          np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    pts = np.concatenate([pts, -pts])
    top = g[-1]
    rows = []
    for e in (-100, 0, 90):
        for p in range(0, len(pts), 31):
            b = np.zeros(32)
            part = pts[p:p + 31]
            b[:len(part)], b[31] = part, top        # the block's maximum fixes the scale
            rows.append(np.ldexp(b, e))
    x = torch.from_numpy(np.array(rows)).float()
    codes, scale = q.mx_quantize(x.to(dev()), fmt)
    c, s = R.mx_quantize(x.double().numpy(), fmt)
    assert np.array_equal(scale.cpu().numpy(), s) and np.array_equal(elements(codes, fmt), c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_blocks(fmt):
    case(f"mx_quantize special blocks {fmt}")
    x = torch.randn(10, 64, generator=torch.Generator().manual_seed(3))
    x[0, :32] = 0
    x[1, 5], x[2, 40], x[3, 63] = float("nan"), float("inf"), float("-inf")
    x[4] = torch.randn(64) * 2.0 ** -126
    x[5] = 2.0 ** -149
    x[6] = torch.finfo(torch.float32).max
    x[7] = -0.0
    x[8] *= 2.0 ** -118
    x[9] *= 2.0 ** 120
    codes, scale = q.mx_quantize(x.to(dev()), fmt)
    c, s = R.mx_quantize(x.double().numpy(), fmt)
    assert np.array_equal(scale.cpu().numpy(), s)
    assert np.array_equal(elements(codes, fmt), c)
    assert s[1].tolist()[0] == 255 and s[2].tolist()[1] == 255 and s[0, 0] == 0
    got = q.mx_dequantize(codes, scale, torch.float32).cpu().double().numpy()
    assert np.array_equal(got, R.mx_values(c, s, fmt), equal_nan=True)


def test_every_code_and_scale_reads_back():
    case("mx_dequantize all codes")
    d = dev()
    for fmt, count, per in (("mxfp8", 256, 8), ("mxfp4", 16, 1)):
        elems = (np.arange(max(count, 32)) % count).astype(np.uint8)
        c = np.tile(elems, (256, 1))
        s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], per, 1)
        codes = torch.from_numpy(R.pack(c) if fmt == "mxfp4" else c).to(d)
        codes = codes if fmt == "mxfp4" else codes.view(torch.float8_e4m3fn)
        got = q.mx_dequantize(codes, torch.from_numpy(s).to(d), torch.float32).cpu()
        with np.errstate(over="ignore"):
            want = R.mx_values(c, s, fmt).astype(np.float32)
        assert np.array_equal(got.numpy(), want, equal_nan=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_strides_and_rank(fmt):
    case(f"mx_quantize strides {fmt}")
    d = dev()
    x = torch.randn(6, 77, device=d).half()
    wide = torch.full((6, 90), 9.0, device=d, dtype=torch.float16)
    wide[:, 3:80] = x
    a, b = q.mx_quantize(x, fmt), q.mx_quantize(wide[:, 3:80], fmt)
    assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])
    c = q.mx_quantize(x.view(2, 3, 77), fmt)
    assert torch.equal(c[0].view(torch.uint8).flatten(0, 1), a[0].view(torch.uint8)) and torch.equal(c[1].flatten(0, 1), a[1])
    one = q.mx_quantize(x[0], fmt)
    assert torch.equal(one[1], a[1][0])
    out = torch.full((6, 81), 4.0, device=d)
    got = q.mx_dequantize(*b, torch.float32, columns=77, out=out[:, 2:79])
    assert torch.equal(got, q.mx_dequantize(*a, torch.float32, columns=77)) and (out[:, :2] == 4).all() and (out[:, 79:] == 4).all()
    assert q.mx_dequantize(*c, columns=77).shape == (2, 3, 77)

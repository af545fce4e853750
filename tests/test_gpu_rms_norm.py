"""The RMS norm, its quantised outputs and its gradient on the GPU against
64-bit references.  Codes are compared bit for bit; floating results within
the roundings their sums can make (u = 2^-24 a step), counted below."""
import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
# a lane adds at most 64 squares, then at most 6 + 15 sums: half of that reaches 1/sqrt, which adds 4 steps
R_STEPS = 48
SHAPES = [(1, 1), (3, 7), (35, 5), (5, 32), (33, 127), (17, 128), (40, 129), (19, 250), (7, 256), (11, 257), (2, 12290), (1, 4096), (4, 100), (9, 512), (7, 513), (6, 1024), (3, 1025), (2, 2048), (3, 4095),
          (2, 5000), (2, 8192), (2, 8193), (1, 16384), (1, 20001), (1, 65536), (300, 256), (0, 64)]


def make(rows, n, dtype, seed, residual=True, wdtype=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n, generator=g).to(dtype)
    x[:, :: max(1, n // 3)] *= 9
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(wdtype or dtype)
    res = torch.randn(rows, n, generator=g).to(dtype) if residual else None
    return x, w, res


def hidden(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def up(*ts):
    return [None if t is None else t.to(dev()) for t in ts]


def d64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(rows, n, dtype):
    case(f"rms_norm {rows}x{n} {dtype}")
    for residual, wdtype, odtype in ((True, dtype, dtype), (False, torch.float32, torch.float32)):
        x, w, res = make(rows, n, dtype, rows + n, residual, wdtype)
        got = q.rms_norm(*up(x, w), 1e-5, residual=up(res)[0], out_dtype=odtype)
        h = hidden(x, res)
        if residual:
            assert torch.equal(got[2].cpu(), h)
        r = R.rstd(d64(h), 1e-5)
        assert np.all(np.abs(d64(got[1]) - r) <= R_STEPS * U * r)
        y = d64(h) * r[:, None] * d64(w)
        tiny = 2.0 ** -25 if odtype == torch.float16 else 0    # fp16 subnormals: half a step of 2^-24
        assert got[0].dtype == odtype and np.all(np.abs(d64(got[0]) - y) <= ((R_STEPS + 4) * U + HALF[odtype]) * 1.01 * np.abs(y) + tiny)


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_int8(rows, n, dtype):
    case(f"rms_norm_quantize int8 {rows}x{n} {dtype}")
    x, w, res = make(rows, n, dtype, rows + 3 * n)
    codes, scale, h = q.rms_norm_quantize(*up(x, w), 1e-6, residual=up(res)[0])
    assert torch.equal(h.cpu(), hidden(x, res))
    want, a = R.int8_codes(hidden(x, res).float().numpy(), w.float().numpy())
    assert np.array_equal(codes.cpu().numpy(), want)
    s = a.astype(np.float64) * R.rstd(d64(h), 1e-6) / 127
    assert np.all(np.abs(d64(scale) - s) <= (R_STEPS + 4) * U * s)


@pytest.mark.parametrize("rows,n", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_mx(rows, n, dtype, fmt):
    case(f"rms_norm_quantize {fmt} {rows}x{n} {dtype}")
    x, w, _ = make(rows, n, dtype, rows + 5 * n, False, torch.float32)
    codes, scale, r = q.rms_norm_quantize(*up(x, w), 1e-6, format=fmt)
    t = x.float().numpy() * w.numpy()          # fp32, as the definition has it
    c, s = R.mx_quantize(t, fmt)
    got = codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(R.unpack(got) if fmt == "mxfp4" else got, c)
    assert np.array_equal(scale.cpu().numpy(), s)
    want = R.rstd(d64(x), 1e-6)
    assert np.all(np.abs(d64(r) - want) <= R_STEPS * U * want)


def test_rows_of_zeros_nan_infinity_and_tiny_values():
    case("rms_norm_quantize special rows")
    n = 96
    x = torch.randn(9, n, generator=torch.Generator().manual_seed(2))
    x[0] = 0
    x[1, 40] = float("nan")
    x[2, 95] = float("inf")
    x[3] *= 2.0 ** -130
    x[4] = 2.0 ** -149
    x[5] = -0.0
    x[6] *= 1e25                                # the sum of squares passes fp32: r = 0
    w = torch.ones(n)
    codes, scale = q.rms_norm_quantize(*up(x, w), 1e-6)
    codes, scale = codes.cpu().numpy(), scale.cpu().numpy()
    assert not codes[[0, 1, 2, 5]].any() and scale[[0, 5]].tolist() == [1, 1] and np.isnan(scale[[1, 2]]).all()
    want, _ = R.int8_codes(x.numpy(), w.numpy())
    assert np.array_equal(codes[[3, 4, 6, 7]], want[[3, 4, 6, 7]]) and np.abs(want[3]).max() == 127 and scale[6] == 0
    for fmt in ("mxfp8", "mxfp4"):
        c, s, r = q.rms_norm_quantize(*up(x, w), 1e-6, format=fmt)
        wc, ws = R.mx_quantize(x.numpy(), fmt)
        got = c.view(torch.uint8).cpu().numpy()
        assert np.array_equal(s.cpu().numpy(), ws) and ws[1].tolist()[1] == 255 and ws[2].tolist()[2] == 255
        assert np.array_equal(R.unpack(got) if fmt == "mxfp4" else got, wc)
        assert r[0].item() == np.float32(1 / np.sqrt(np.float32(1e-6))) and r[6].item() == 0
    y, r = q.rms_norm(*up(x, w), 1e-6)
    assert not y[0].any() and torch.isnan(y[1]).all() and not torch.isnan(y[7:]).any()
    # infinity: r = 0, so 0 everywhere but inf * 0
    assert torch.isnan(y[2, 95]) and not y[2, :95].any()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_in_place_and_rank(dtype):
    case(f"rms_norm strides {dtype}")
    d = dev()
    rows, n = 6, 161
    x, w, res = make(rows, n, dtype, 77)
    h = hidden(x, res)
    xb = torch.full((rows, n + 13), 5.0, dtype=dtype, device=d)
    xb[:, 1:n + 1] = x.to(d)
    rb = torch.full((rows, n + 3), 5.0, dtype=dtype, device=d)
    rb[:, :n] = res.to(d)
    ob = torch.full((rows, n + 9), 7.0, dtype=dtype, device=d)
    ref = q.rms_norm(*up(x, w), residual=res.to(d))
    got = q.rms_norm(xb[:, 1:n + 1], w.to(d), residual=rb[:, :n], out=ob[:, 2:n + 2], residual_out=rb[:, :n])
    assert torch.equal(got[0], ref[0]) and torch.equal(rb[:, :n].cpu(), h)            # h over the residual
    assert (ob[:, :2] == 7).all() and (ob[:, n + 2:] == 7).all() and (rb[:, n:] == 5).all() and (xb[:, n + 1:] == 5).all()
    x3, r3 = x.to(d).view(2, 3, n), res.to(d).view(2, 3, n)
    y3, s3, h3 = q.rms_norm(x3, w.to(d), residual=r3, residual_out=x3)                # h over x
    assert y3.shape == (2, 3, n) and s3.shape == (2, 3) and torch.equal(y3.view(rows, n), ref[0]) and torch.equal(h3.view(rows, n).cpu(), h)
    y1, s1 = q.rms_norm(h.to(d)[0], w.to(d))
    assert y1.shape == (n,) and s1.shape == () and torch.equal(y1, ref[0][0])
    c, s, r = q.rms_norm_quantize(h.to(d).view(2, 3, n), w.to(d), format="mxfp4")
    assert c.shape == (2, 3, 96) and s.shape == (2, 3, 6) and r.shape == (2, 3)


GRAD_SHAPES = [(1, 1), (5, 7), (9000, 6), (35, 128), (8300, 65), (19, 200), (5000, 256), (4, 257), (6, 12288), (5, 12289), (1, 4096), (37, 100), (9, 512), (700, 96), (65, 1000), (33, 1025), (700, 2048), (17, 4095),
               (1100, 4096), (40, 8192), (9, 8200), (5, 16384), (3, 20000), (2, 65536)]


@pytest.mark.parametrize("rows,n", GRAD_SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_grad(rows, n, dtype):
    case(f"rms_norm_grad {rows}x{n} {dtype}")
    for with_dh, wdtype in ((True, dtype), (False, torch.float32)):
        h, w, dh = make(rows, n, dtype, rows + 7 * n, with_dh, wdtype)
        dy = torch.randn(rows, n, generator=torch.Generator().manual_seed(n)).to(dtype)
        r = torch.from_numpy(R.rstd(d64(h), 1e-5)).float()
        args = up(dy, h, w, r, dh)
        dx, dw = q.rms_norm_grad(*args)
        assert dx.dtype == dtype and dw.dtype == wdtype and dw.shape == (n,)
        wx, ww = R.grad(d64(dy), d64(h), d64(w), d64(r), None if dh is None else d64(dh))
        # dx: a lane's 64 products of three factors, 21 sums, then 8 steps around each of the terms
        rr = d64(r)[:, None]
        size = np.abs(d64(h)) * rr ** 3 / n * np.abs(d64(dy) * d64(w) * d64(h)).sum(1, keepdims=True)
        tol = U * (100 * size + 8 * np.abs(rr * d64(dy) * d64(w)) + 8 * np.abs(wx))
        if dh is not None:
            tol = tol + U * 2 * np.abs(d64(dh))
        tiny = 2.0 ** -25 if dtype == torch.float16 else 0
        assert np.all(np.abs(d64(dx) - wx) <= tol + HALF[dtype] * 1.01 * np.abs(wx) + tiny)
        # dw: at most ceil(rows / 256) rows in a lane, 15 groups, 16 partial rows, 7 + 3 sums, 2 steps a term
        steps = -(-rows // 256) + 15 + 16 + 10 + 4
        tiny = 2.0 ** -25 if wdtype == torch.float16 else 0
        size = np.abs(d64(dy) * d64(h) * rr).sum(0)
        assert np.all(np.abs(d64(dw) - ww) <= steps * U * size + HALF[wdtype] * 1.01 * np.abs(ww) + tiny)
        again = q.rms_norm_grad(*args)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("rows,n", [(513, 2049), (513, 4095), (260, 4100), (600, 6144), (600, 6145), (600, 8192), (513, 8200), (513, 12290)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_of_few_and_many_rows(rows, n, dtype):
    # the lanes of a row depend on how many rows there are; a row's codes and scale do not
    case(f"rms_norm_quantize {rows}x{n} {dtype} whole and in parts")
    x, w, res = up(*make(rows, n, dtype, n))
    whole = q.rms_norm_quantize(x, w, 1e-6, residual=res)
    part = [torch.cat(t) for t in zip(*[q.rms_norm_quantize(x[i:i + 250], w, 1e-6, residual=res[i:i + 250]) for i in range(0, rows, 250)])]
    assert torch.equal(whole[0], part[0]) and torch.equal(whole[2], part[2])
    assert torch.allclose(whole[1], part[1], rtol=2 * R_STEPS * U, atol=0)


@pytest.mark.parametrize("rows,n", [(8193, 100), (4100, 200), (2049, 300), (5000, 511), (2049, 512), (2049, 513), (513, 4090), (300, 5000), (600, 8192), (769, 2050)])
def test_grad_of_many_rows(rows, n):
    # more rows than the workgroups have in hand at once; the bounds of test_grad
    test_grad(rows, n, torch.bfloat16)


def test_grad_without_rows_and_strided():
    case("rms_norm_grad no rows, strides")
    d = dev()
    dx, dw = q.rms_norm_grad(torch.zeros(0, 64, device=d), torch.zeros(0, 64, device=d), torch.ones(64, device=d), torch.zeros(0, device=d))
    assert dx.shape == (0, 64) and not dw.any() and dw.shape == (64,)
    h, w, dh = up(*make(8, 200, torch.bfloat16, 4))
    dy = torch.randn(8, 200, device=d).bfloat16()
    _, r = q.rms_norm(h, w)
    ref = q.rms_norm_grad(dy, h, w, r, dh)
    wide = [torch.full((8, 211), 3.0, dtype=torch.bfloat16, device=d) for _ in range(3)]
    for b, t in zip(wide, (dy, h, dh)):
        b[:, 5:205] = t
    got = q.rms_norm_grad(wide[0][:, 5:205], wide[1][:, 5:205], w, r, wide[2][:, 5:205])
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    got = q.rms_norm_grad(dy.view(2, 4, 200), h.view(2, 4, 200), w, r.view(2, 4))
    assert got[0].shape == (2, 4, 200)


def test_gradient_of_the_forward_by_differences():
    """The forward's own outputs move as its gradient says."""
    case("rms_norm differences")
    d = dev()
    h, w, _ = up(*make(4, 33, torch.float32, 9))
    dy = torch.randn(4, 33, device=d)
    _, r = q.rms_norm(h, w, 1e-3)
    dx, dw = q.rms_norm_grad(dy, h, w, r)
    step, u = 2.0 ** -7, torch.randn(4, 33, device=d)
    v = torch.randn(33, device=d)
    f = lambda a, b: (q.rms_norm(a, b, 1e-3)[0].double() * dy.double()).sum().item()   # noqa: E731
    # the forward rounds each of 132 outputs by 52 steps at most; the third derivative adds step^2
    noise = 52 * U * (q.rms_norm(h, w, 1e-3)[0] * dy).abs().sum().item() / step
    along = (f(h + step * u, w) - f(h - step * u, w)) / (2 * step)
    assert abs(along - (dx.double() * u).sum().item()) <= noise + 100 * step ** 2
    along = (f(h, w + step * v) - f(h, w - step * v)) / (2 * step)
    assert abs(along - (dw.double() * v).sum().item()) <= noise + 1e-3


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_every_16_bit_value_passes_unchanged(dtype):
    # h = x + (-0) is x itself, the sign of a zero too; NaN stays some NaN
    case(f"every {dtype}")
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype).reshape(256, 256)
    h = q.rms_norm(*up(x, torch.ones(256, dtype=dtype)), residual=up(torch.full_like(x, -0.0))[0])[2].cpu()
    nan = x.isnan()
    assert torch.equal(h.isnan(), nan)
    assert torch.equal(h.view(torch.int16)[~nan], x.view(torch.int16)[~nan])

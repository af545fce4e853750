"""The MX product on the GPU against the 64-bit product of the values its
operands stand for."""
import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from gpu_util import case, dev, env

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def operand(rows, K, fmt, seed, spread=0.0, std=1.0):
    """(codes, scale) on the GPU and the values in 64 bits."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, K)) * std * np.exp2(spread * rng.normal(size=(rows, K // 32))).repeat(32, 1)
    x[:, rng.integers(0, K, 1 + K // 200)] *= 10
    c, s = R.mx_quantize(x, fmt)
    return place(c, s, fmt) + (R.mx_values(c, s, fmt),)


def place(c, s, fmt, pad=16):
    d = dev()
    buf = torch.full((s.shape[0], -(-s.shape[1] // pad) * pad), 255, dtype=torch.uint8, device=d)   # NaN past the row
    buf[:, :s.shape[1]] = torch.from_numpy(s).to(d)
    codes = torch.from_numpy(R.pack(c) if fmt == "mxfp4" else c).to(d)
    return codes if fmt == "mxfp4" else codes.view(torch.float8_e4m3fn), buf[:, :s.shape[1]]


def bound(va, vw, a8, out, scale):
    """How far an output may be off: each of the K / 16 sums of 16 products and
    their additions to the accumulator makes a step of 2^-23 (the hardware may
    truncate) of the sum of magnitudes; with e4m3 operands and a 16-bit output
    each of 16 products loses up to 2^-13 of its group's largest; then the
    row scale and the output's rounding."""
    size = np.abs(va) @ np.abs(vw).T
    tol = (va.shape[1] / 16 + 24) * 2 * U * size
    if a8 and out != torch.float32:
        m, k = va.shape
        ga = np.abs(va).reshape(m, k // 16, 16).max(-1)
        gw = np.abs(vw).reshape(len(vw), k // 16, 16).max(-1)
        tol += 16 * 2.0 ** -13 * (ga @ gw.T)
    want = va @ vw.T
    if scale is not None:
        tol, want = tol * scale[:, None], want * scale[:, None]
    tiny = 2.0 ** -25 if out == torch.float16 else 0
    return want, tol + (HALF[out] * 1.01 + U) * np.abs(want) + tiny


def check(M, N, K, fmt, out, scaled, seed=0, spread=0.0, **kw):
    a, sa, va = operand(M, K, fmt, seed + 1, spread)
    w, sw, vw = operand(N, K, "mxfp4", seed + 2, spread, 0.05)
    scale = torch.rand(M, generator=torch.Generator().manual_seed(seed)) + 0.5 if scaled else None
    got = q.mx_matmul(a, sa, w, sw, act_scale=None if scale is None else scale.to(dev()), out_dtype=out, **kw)
    want, tol = bound(va, vw, fmt == "mxfp8", out, None if scale is None else scale.double().numpy())
    assert got.shape == (M, N) and got.dtype == out
    err = np.abs(got.cpu().double().numpy() - want)
    assert np.all(err <= tol), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4].tolist())
    return got


SHAPES = [(1, 16, 32), (1, 1, 32), (2, 33, 96), (1, 4096, 4096), (5, 100, 160), (16, 1000, 2048), (16, 17, 8192), (8, 100, 4096), (5, 3000, 1056), (17, 64, 512),
          (33, 129, 320), (64, 256, 256), (100, 300, 1120), (128, 128, 128), (130, 257, 544), (200, 520, 64), (256, 256, 2048),
          (300, 513, 4096), (513, 700, 992), (1000, 1111, 288)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_product(M, N, K, fmt):
    case(f"mx_matmul {M}x{N}x{K} {fmt}")
    check(M, N, K, fmt, torch.float32, True)
    check(M, N, K, fmt, torch.bfloat16, False, seed=5)
    check(M, N, K, fmt, torch.float16, True, seed=9)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_large_product(fmt):
    case(f"mx_matmul 2304x2560x1024 {fmt}")
    check(2304, 2560, 1024, fmt, torch.bfloat16, True)
    check(2304, 2560, 1024, fmt, torch.float32, False)


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_block_scales_far_apart(M, fmt):
    """Block scales over many powers of two: each must reach its own block."""
    case(f"mx_matmul spread scales M={M} {fmt}")
    check(M, 200, 1024, fmt, torch.float32, False, spread=6.0)


@pytest.mark.parametrize("M,N,K", [(3, 40, 256), (150, 140, 512), (600, 300, 768)])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_exact_integers(M, N, K, fmt):
    """Small whole values: every order of summing gives the same bits."""
    case(f"mx_matmul integers {M}x{N}x{K} {fmt}")
    rng = np.random.default_rng(M)
    va, vw = rng.integers(-4, 5, (M, K)).astype(float), rng.integers(-3, 4, (N, K)).astype(float)
    one_a, one_w = np.full((M, K // 32), 127, np.uint8), np.full((N, K // 32), 127, np.uint8)
    code = lambda v, fmt: (R.nearest(R.GRID[fmt], np.abs(v)) | np.where(v < 0, 8 if fmt == "mxfp4" else 128, 0)).astype(np.uint8)  # noqa: E731
    a, sa = place(code(va, fmt), one_a, fmt)
    w, sw = place(code(vw, "mxfp4"), one_w, "mxfp4")
    got = q.mx_matmul(a, sa, w, sw)
    assert np.array_equal(got.cpu().double().numpy(), va @ vw.T)


@pytest.mark.parametrize("M", [2, 40, 300])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_nan_blocks_stay_in_their_row(M, fmt):
    case(f"mx_matmul NaN blocks M={M} {fmt}")
    N, K = 150, 384
    a, sa, _ = operand(M, K, fmt, 3)
    w, sw, _ = operand(N, K, "mxfp4", 4)
    ref = q.mx_matmul(a, sa, w, sw)
    sa, sw = sa.clone(), sw.clone()
    sa[1, 5], sw[77, 11] = 255, 255
    got = q.mx_matmul(a, sa, w, sw)
    nan = torch.zeros(M, N, dtype=torch.bool, device=got.device)
    nan[1], nan[:, 77] = True, True
    assert torch.equal(torch.isnan(got), nan) and torch.equal(got[~nan], ref[~nan])
    s = torch.ones(M, device=got.device)
    s[0] = float("nan")
    assert torch.isnan(q.mx_matmul(a, sa, w, sw, act_scale=s)[0]).all()


@pytest.mark.parametrize("M,N,K", [(1, 70, 96), (9, 300, 1056), (140, 90, 480)])
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_strides_and_alignment(M, N, K, fmt):
    """Operands inside wider buffers, at odd bytes, scale rows at any stride,
    an output inside a wider one: the same values, nothing else written."""
    case(f"mx_matmul strides {M}x{N}x{K} {fmt}")
    d = dev()
    a, sa, va = operand(M, K, fmt, 3)
    w, sw, vw = operand(N, K, "mxfp4", 4)
    want, tol = bound(va, vw, fmt == "mxfp8", torch.float32, None)

    def inside(t, left, right):
        u = t.view(torch.uint8)
        b = torch.full((u.shape[0], u.shape[1] + left + right), 255, dtype=torch.uint8, device=d)
        b[:, left:left + u.shape[1]] = u
        return b[:, left:left + u.shape[1]].view(t.dtype)

    for la, lw, ls in ((16, 16, 4), (1, 3, 1), (16, 5, 4), (0, 0, 3)):
        got = torch.full((M, N + 5), 7.0, device=d)
        q.mx_matmul(inside(a, la, 16), inside(sa, ls, 5), inside(w, lw, 0), inside(sw, ls, 2), out=got[:, 2:N + 2])
        assert np.all(np.abs(got[:, 2:N + 2].cpu().double().numpy() - want) <= tol)
        assert (got[:, :2] == 7).all() and (got[:, N + 2:] == 7).all()
    # scale rows that end with their last byte, and that of the last row with the storage
    got = q.mx_matmul(a, sa.contiguous(), w, sw.contiguous())
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= tol)


def test_empty_and_scalar_scale():
    case("mx_matmul empty")
    d = dev()
    a, sa, _ = operand(3, 64, "mxfp4", 3)
    w, sw, _ = operand(40, 64, "mxfp4", 4)
    assert q.mx_matmul(a[:0], sa[:0], w, sw).shape == (0, 40) and q.mx_matmul(a, sa, w[:0], sw[:0]).shape == (3, 0)
    ref = q.mx_matmul(a, sa, w, sw)
    for s in (torch.tensor(2.0, device=d), torch.full((1,), 2.0, device=d), torch.full((3,), 2.0, device=d), torch.full((3, 1), 2.0, device=d)):
        assert torch.equal(q.mx_matmul(a, sa, w, sw, act_scale=s), ref * 2)


@pytest.mark.parametrize("M", [1, 16, 64, 200])
def test_results_repeat(M):
    case(f"mx_matmul repeats M={M}")
    N, K = 1500, 4096
    a, sa, _ = operand(M, K, "mxfp8", 3)
    w, sw, _ = operand(N, K, "mxfp4", 4)
    first = q.mx_matmul(a, sa, w, sw)
    for _ in range(3):
        assert torch.equal(q.mx_matmul(a, sa, w, sw), first)


TILES = ["mx_tiled_256x256", "mx_tiled_128x128", "mx_tiled_64x128", "mx_tiled_64x64", "mx_tiled_64x32", "mx_tiled_32x32"]


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (40, 300, 96), (257, 129, 512), (300, 700, 1120), (600, 515, 2080), (2100, 2111, 352),
                                   (65, 90, 4096), (33, 40, 5024)])
@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_every_tile(M, N, K, tile, fmt):
    """Each tile shape, whatever the plan would choose."""
    case(f"mx_matmul tile {tile} {M}x{N}x{K} {fmt}")
    with env(QGEMM_MX_TILE=tile):
        check(M, N, K, fmt, torch.float32, True)
        assert q._binding.last_kernel() == TILES[tile]
        check(M, N, K, fmt, torch.bfloat16, False, spread=3.0)
        check(M, N, K, fmt, torch.float16, True)


@pytest.mark.parametrize("M,N,K,kernel", [
    (1, 512, 512, "mx_decode"), (8, 512, 544, "mx_decode"), (9, 512, 544, "mx_tiled_32x32"), (16, 8192, 64, "mx_tiled_32x32"), (17, 512, 512, "mx_tiled_32x32"),
    (64, 8192, 256, "mx_tiled_64x32"), (128, 8192, 256, "mx_tiled_64x64"), (512, 4096, 256, "mx_tiled_64x128"),
    (2048, 2048, 512, "mx_tiled_128x128"), (1024, 6000, 96, "mx_tiled_128x128"), (1300, 6000, 96, "mx_tiled_256x256"), (2049, 8192, 96, "mx_tiled_128x128"), (4096, 4096, 256, "mx_tiled_256x256")])
def test_kernel_choice(M, N, K, kernel):
    case(f"mx_matmul kernel for {M}x{N}x{K}")
    check(M, N, K, "mxfp4", torch.bfloat16, True)
    assert q._binding.last_kernel() == kernel
    with env(QGEMM_MX_KERNEL="bytes"):
        check(M, N, K, "mxfp8", torch.bfloat16, True)
        assert q._binding.last_kernel() == "mx_matmul_bytes"

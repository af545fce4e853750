"""The MX product's sums where the largest products of a group cancel: what is
left has to be exact whatever type leaves."""
import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from gpu_util import case, dev, env

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def cancelling(M, N, K, seed):
    """Codes whose every group of 16 k holds 448 * 6 and -448 * 6, among products that are
    any element below 2 (odd groups: from 2 to 15) times one of at most 2.

    Every product is a multiple of 2^-10 and the sum of the magnitudes that do not cancel
    is below 256 * 15 * 2 = 7680 < 2^13, so every partial sum is held exactly in fp32's 24
    bits, whatever the order, as long as a group's own sum is."""
    assert K <= 256
    rng = np.random.default_rng(seed)
    low = np.flatnonzero((R.E4M3 > 0) & (R.E4M3 < 2))
    high = np.flatnonzero((R.E4M3 >= 2) & (R.E4M3 <= 15))
    odd = (np.arange(K) // 16 % 2 == 1)
    a = np.where(odd, rng.choice(high, (M, K)), rng.choice(low, (M, K)))
    w = rng.integers(1, 5, (N, K)) | 8 * rng.integers(0, 2, (N, K))
    for k in range(0, K, 16):
        i, j = rng.permutation(16)[:2] + k
        a[:, [i, j]], w[:, i], w[:, j] = 126, 7, 15
    one = lambda rows: np.full((rows, K // 32), 127, np.uint8)   # noqa: E731
    va, vw = R.mx_values(a, one(M), "mxfp8"), R.mx_values(w, one(N), "mxfp4")
    up = lambda x: torch.from_numpy(np.ascontiguousarray(x.astype(np.uint8))).to(dev())   # noqa: E731
    ops = [up(a).view(torch.float8_e4m3fn), up(one(M)), up(R.pack(w)), up(one(N))]
    return ops, torch.from_numpy(va @ vw.T)


def check(M, N, K, **kw):
    ops, want = cancelling(M, N, K, M + N)
    for t in TYPES:
        got = q.mx_matmul(*ops, out_dtype=t).cpu()
        assert torch.equal(got, want.to(t)), (t, (got.double() - want).abs().max().item())


@pytest.mark.parametrize("M,N,K", [(1, 100, 256), (8, 130, 128)])
def test_sums_of_few_rows(M, N, K):
    case(f"mx_matmul cancelling groups {M}x{N}x{K}")
    check(M, N, K)
    assert q._binding.last_kernel() == "mx_decode"


@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (70, 90, 256)])
def test_sums_of_the_byte_kernel(M, N, K):
    case(f"mx_matmul cancelling groups, bytes, {M}x{N}x{K}")
    with env(QGEMM_MX_KERNEL="bytes"):
        check(M, N, K)
        assert q._binding.last_kernel() == "mx_matmul_bytes"


@pytest.mark.parametrize("tile", range(6))
@pytest.mark.parametrize("M,N,K", [(40, 70, 128), (300, 290, 256), (2100, 2111, 128)])
def test_sums_of_every_tile(tile, M, N, K):
    case(f"mx_matmul cancelling groups, tile {tile}, {M}x{N}x{K}")
    with env(QGEMM_MX_TILE=tile):
        check(M, N, K)
        assert q._binding.last_kernel().startswith("mx_tiled_")


@pytest.mark.parametrize("M,N,kernel", [(1, 4096, "mx_decode"), (8, 4096, "mx_decode"), (1, 4097, "mx_tiled_32x32"), (9, 4096, "mx_tiled_32x32")])
def test_the_kernel_of_few_rows(M, N, kernel):
    """MXFP8 activations, whose products are split."""
    case(f"mx_matmul kernel for MXFP8 {M}x{N}")
    check(M, N, 128)
    assert q._binding.last_kernel() == kernel

"""The A8W8 product with bias, activation and residual, and the gated pair, against
64-bit references; their checkpoints against the definition's fp32 steps, bit for
bit."""
import numpy as np
import pytest
import torch

import fused_reference as ref
import quantized_int8_gemm_amd as q
from gpu_util import case, dev, env

pytestmark = pytest.mark.gpu

EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -9 * 2, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half a subnormal step


def inputs(m, n, k, seed, halves=1, extreme=False):
    r = np.random.default_rng(seed)
    a = r.integers(-128, 128, (m, k), dtype=np.int8)
    w = [r.integers(-128, 128, (n, k), dtype=np.int8) for _ in range(halves)]
    if extreme:
        a[:], w[0][:] = -128, -128
    sa = r.uniform(0.2, 1.0, m).astype(np.float32)
    sw = [(r.uniform(0.2, 1.0, n) * np.where(r.random(n) < 0.1, -1, 1) * 2e-4 / np.sqrt(k)).astype(np.float32) for _ in range(halves)]
    return a, w, sa, sw


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dev())


def laid(w, b_trans):
    return gpu(w if b_trans else w.T)


def padded(t, extra):
    """The same matrix with `extra` columns of other values behind each row."""
    big = torch.full((t.shape[0], t.shape[1] + extra), 77, dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


def check(got, want, before, d):
    """want: 64-bit; before: bound of what is off before the last rounding."""
    g = got.double().cpu().numpy()
    tol = before * (1 + 2.0 ** -8) + np.abs(want) * EPS[d] + TINY[d]
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], g[bad][:3], want[bad][:3], tol[bad][:3])


def z_bound(z0, z=None):
    """z after the product's conversion and two scales, and the bias."""
    return 3 * 2.0 ** -24 * np.abs(z0) + (0 if z is None else 2.0 ** -24 * np.abs(z))


SHAPES = [(1, 1, 1), (1, 16, 64), (2, 33, 48), (3, 5, 7), (5, 100, 128), (16, 64, 256), (17, 130, 80), (31, 257, 33), (64, 32, 1040),
          (65, 128, 64), (128, 256, 144), (130, 300, 272), (257, 129, 96), (300, 511, 2064), (513, 640, 512)]
FORMS = [(None, False, False), ("silu", True, True), ("gelu", True, False), ("gelu_tanh", False, True), ("relu", True, True)]


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(shape, b_trans):
    m, n, k = shape
    for i, (act, with_bias, with_res) in enumerate(FORMS):
        d = (torch.float32, torch.bfloat16, torch.float16)[(i + m) % 3]
        case(f"linear {shape} b_trans={b_trans} {act} bias={with_bias} residual={with_res} {d}")
        a, (w,), sa, (sw,) = inputs(m, n, k, 100 * m + i)
        r = np.random.default_rng(i)
        bias = r.normal(size=n).astype(np.float32) if with_bias else None
        res = torch.from_numpy(r.normal(size=(m, n))).to(d).to(dev()) if with_res else None
        out, (codes, scale) = q.qgemm_a8w8_linear(gpu(a), laid(w, b_trans), gpu(sa), gpu(sw), bias=None if bias is None else gpu(bias),
                                                  activation=act, residual=res, out_dtype=d, b_trans=b_trans, checkpoint=True)
        acc = ref.accumulate(a, w.T, False)
        z0 = acc.astype(np.float64) * sa.astype(np.float64)[:, None] * sw.astype(np.float64)
        z = z0 if bias is None else z0 + bias.astype(np.float64)
        want = ref.act(act, z)
        before = 1.13 * z_bound(z0, z) + ref.act_error(act, z)
        if res is not None:
            want = want + res.double().cpu().numpy()
            before = before + 2.0 ** -24 * np.abs(want)
        check(out, want, before, d)
        zc, zs = ref.int8_form(ref.z32(acc, sa, sw, bias), ref.BLOCK)
        assert np.array_equal(codes.cpu().numpy(), zc) and np.array_equal(scale.cpu().numpy(), zs)
        again = q.qgemm_a8w8_linear(gpu(a), laid(w, b_trans), gpu(sa), gpu(sw), bias=None if bias is None else gpu(bias),
                                    activation=act, residual=res, out_dtype=d, b_trans=b_trans)
        assert torch.equal(again, out)   # without the checkpoint: the same bits


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated(shape, b_trans):
    m, n, k = shape
    for i, act in enumerate(("silu", "gelu", "gelu_tanh", "relu", "none")):
        d = (torch.float32, torch.bfloat16, torch.float16)[(i + m) % 3]
        case(f"gated {shape} b_trans={b_trans} {act} {d}")
        a, (wg, wu), sa, (sg, su) = inputs(m, n, k, 100 * m + i, 2)
        args = (gpu(a), laid(wg, b_trans), laid(wu, b_trans), gpu(sa), gpu(sg), gpu(su))
        out, (codes, scale) = q.qgemm_a8w8_gated(*args, activation=act, out_dtype=d, b_trans=b_trans, checkpoint=True)
        acc = [ref.accumulate(a, w.T, False) for w in (wg, wu)]
        g, u = (x.astype(np.float64) * sa.astype(np.float64)[:, None] * s.astype(np.float64) for x, s in zip(acc, (sg, su)))
        f = ref.act(act, g)
        before = (1.13 * z_bound(g) + ref.act_error(act, g)) * np.abs(u) + np.abs(f) * (z_bound(u) + 2.0 ** -24 * np.abs(u))
        check(out, f * u, before, d)
        for h, s in enumerate((sg, su)):
            zc, zs = ref.int8_form(ref.z32(acc[h], sa, s), ref.BLOCK)
            assert np.array_equal(codes[h].cpu().numpy(), zc) and np.array_equal(scale[h].cpu().numpy(), zs)
        assert torch.equal(q.qgemm_a8w8_gated(*args, activation=act, out_dtype=d, b_trans=b_trans), out)


@pytest.mark.parametrize("b_trans", [True, False])
def test_strides_offsets_and_an_output_that_is_the_residual(b_trans):
    for m, n, k, extra in ((70, 144, 96, 16), (70, 143, 95, 3), (3, 80, 160, 32), (200, 272, 320, 1)):
        case(f"strides {m} {n} {k} {extra} b_trans={b_trans}")
        a, (wg, wu), sa, (sg, su) = inputs(m, n, k, m, 2)
        A, G, U = padded(gpu(a), extra), padded(laid(wg, b_trans), extra), padded(laid(wu, b_trans), extra + 5)
        res = padded(torch.randn(m, n, device=dev()).bfloat16(), 3)
        plain = (gpu(a), laid(wg, b_trans), gpu(sa), gpu(sg))
        want = q.qgemm_a8w8_linear(*plain, activation="silu", residual=res.contiguous(), out_dtype=torch.bfloat16, b_trans=b_trans)
        behind = res._base[:, n:].clone()
        got = q.qgemm_a8w8_linear(A, G, gpu(sa)[:, None], gpu(sg)[None], activation="silu", residual=res, out=res,
                                  out_dtype=torch.bfloat16, b_trans=b_trans)
        assert got is res and torch.equal(res, want) and torch.equal(res._base[:, n:], behind)
        out = padded(torch.zeros(m, n, device=dev()), 2)
        q.qgemm_a8w8_gated(A, G, U, gpu(sa), gpu(sg), gpu(su), b_trans=b_trans, out=out)
        assert torch.equal(out, q.qgemm_a8w8_gated(gpu(a), laid(wg, b_trans), laid(wu, b_trans), gpu(sa), gpu(sg), gpu(su), b_trans=b_trans))
        assert (out._base[:, n:] == 77).all()


def test_scalar_scales():
    a, (wg, wu), sa, (sg, su) = inputs(40, 72, 112, 5, 2)
    one = lambda s, n: np.full(n, s, np.float32)   # noqa: E731
    A, G, U = gpu(a), gpu(wg), gpu(wu)
    got = q.qgemm_a8w8_gated(A, G, U, torch.tensor(0.5, device=dev()), gpu(sg)[:1], gpu(su)[:1, None], b_trans=True)
    want = q.qgemm_a8w8_gated(A, G, U, gpu(one(0.5, 40)), gpu(one(sg[0], 72)), gpu(one(su[0], 72)), b_trans=True)
    assert torch.equal(got, want)


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("m", [2, 40, 200])
def test_extreme_sums(m, b_trans):
    """The largest sums that int32 holds: 2^14 K = 2^30 at K = 65536."""
    n, k = 48, 65536
    case(f"extreme {m} b_trans={b_trans}")
    a, (w,), sa, (sw,) = inputs(m, n, k, 3, extreme=True)
    out, (codes, scale) = q.qgemm_a8w8_linear(gpu(a), laid(w, b_trans), gpu(sa), gpu(sw), b_trans=b_trans, checkpoint=True)
    want = 2.0 ** 30 * sa.astype(np.float64)[:, None] * sw.astype(np.float64)
    check(out, want, z_bound(want), torch.float32)
    zc, zs = ref.int8_form(ref.z32(np.full((m, n), 2 ** 30), sa, sw), ref.BLOCK)
    assert np.array_equal(codes.cpu().numpy(), zc) and np.array_equal(scale.cpu().numpy(), zs)


@pytest.mark.parametrize("m", [4, 100, 300])
def test_rows_that_are_not_finite_or_zero(m):
    n, k = 96, 128
    a, (wg, wu), sa, (sg, su) = inputs(m, n, k, 9, 2)
    sa[0], sa[1], a[2] = np.nan, np.inf, 0
    clean = [x.copy() for x in (a, sa)]
    clean[1][:2] = 1
    out, (codes, scale) = q.qgemm_a8w8_gated(gpu(a), gpu(wg), gpu(wu), gpu(sa), gpu(sg), gpu(su), b_trans=True, checkpoint=True)
    good = q.qgemm_a8w8_gated(gpu(clean[0]), gpu(wg), gpu(wu), gpu(clean[1]), gpu(sg), gpu(su), b_trans=True, checkpoint=True)
    assert not torch.isfinite(out[0]).any() and torch.isnan(scale[:, :2]).all() and (codes[:, :2] == 0).all()
    assert (out[2] == 0).all() and (codes[:, 2] == 0).all() and (scale[:, 2] == 1).all()
    assert torch.equal(out[2:], good[0][2:]) and torch.equal(codes[:, 2:], good[1][0][:, 2:]) and torch.equal(scale[:, 2:], good[1][1][:, 2:])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "none"])
def test_activations_far_out(act):
    """z from 2^-126 to 2^100, both signs: K = 1, A = +-1, the scale carries the size."""
    e = np.concatenate([np.arange(-126, 101), np.log2([3, 5, 7, 9, 11, 13, 30, 45, 60, 80, 88, 95, 103])])
    sw = (2.0 ** e).astype(np.float32)
    a = np.array([[1], [-1]], np.int8)
    out = q.qgemm_a8w8_linear(gpu(a), gpu(np.ones((1, len(sw)), np.int8)), gpu(np.ones(2, np.float32)), gpu(sw), activation=act)
    z = a.astype(np.float64) * sw.astype(np.float64)
    # below 2^-126 the hardware's exponential and reciprocal may flush, and a product of them
    check(out, ref.act(act, z), ref.act_error(act, z) + 2.0 ** -126 * (1 + np.abs(z)), torch.float32)


def test_outputs_without_elements():
    a, (w,), sa, (sw,) = inputs(4, 16, 32, 1)
    out = q.qgemm_a8w8_linear(gpu(a)[:0], gpu(w), gpu(sa)[:0], gpu(sw), b_trans=True)
    assert out.shape == (0, 16)
    out, (codes, scale) = q.qgemm_a8w8_gated(gpu(a), gpu(w)[:0], gpu(w)[:0], gpu(sa), gpu(sw)[:0], gpu(sw)[:0], b_trans=True, checkpoint=True)
    assert out.shape == (4, 0) and codes.shape == (2, 4, 0) and scale.shape == (2, 4, 0)
    with pytest.raises(ValueError):
        q.qgemm_a8w8_linear(gpu(a)[:, :0], gpu(w)[:, :0], gpu(sa), gpu(sw), b_trans=True)


TILES = ("256x256", "128x128", "128x128_deep", "64x128_deep", "any_64x128", "direct_16x16", "direct_16x32", "direct_32x16",
         "direct_32x32", "direct_64x16", "direct_64x32", "direct_kn_16", "direct_kn_32")


def taken(tile, b_trans, checkpoint):
    """Whether a forced kind takes the call: the direct ones want [N,K], and 32 columns for a
    checkpoint's blocks, or [K,N]."""
    if "kn" in TILES[tile]:
        return not b_trans
    return not TILES[tile].startswith("direct") or (b_trans and not (checkpoint and TILES[tile].endswith("x16")))


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("tile", range(len(TILES)))
def test_every_kernel_gives_the_same_bits(tile, b_trans):
    """Sums are exact and the epilogue is one, so outputs and checkpoints depend neither on
    the kernel nor on how K is divided, nor on padding."""
    for i, (m, n, k) in enumerate(((1, 16, 16), (33, 48, 80), (64, 128, 128), (300, 272, 400), (515, 528, 1040), (20, 33, 47), (70, 129, 300),
                                   (130, 143, 1025))):
        a, (wg, wu), sa, (sg, su) = inputs(m, n, k, m + n, 2)
        args = (gpu(a), laid(wg, b_trans), laid(wu, b_trans), gpu(sa), gpu(sg), gpu(su))
        res = torch.randn(m, n, device=dev()).half()
        pieces = k % 16 == 0 and (b_trans or n % 16 == 0)

        def run(checkpoint):
            y = q.qgemm_a8w8_gated(*args, out_dtype=torch.bfloat16, b_trans=b_trans, checkpoint=checkpoint)
            first = q.last_kernel()
            z = q.qgemm_a8w8_linear(args[0], args[1], args[3], args[4], residual=res, activation="gelu", out_dtype=torch.float16,
                                    b_trans=b_trans, checkpoint=checkpoint)
            second = q.last_kernel()
            return (y[0], *y[1], z[0], *z[1]) if checkpoint else (y, z), first, second

        with env(QGEMM_FUSED="4/1/0"):
            want, first, _ = run(True)
            assert first == "fused_pair_any_64x128"
        for splits in (1, 2, 6):
            for checkpoint in (True, False):
                case(f"tile {tile} {m} {n} {k} b_trans={b_trans} splits={splits} checkpoint={checkpoint}")
                with env(QGEMM_FUSED=f"{tile}/{splits}"):
                    got, first, second = run(checkpoint)
                can = tile in (1, 2, 3, 4)
                if taken(tile, b_trans, checkpoint) and (not can or -(-k // 128) >= splits):
                    joined = can and splits > 1
                    assert first == "fused_pair_" + ("joined" if joined else TILES[tile])
                    assert second == "fused_one_" + ("joined" if joined else TILES[tile])
                for x, y in zip(got, want if checkpoint else (want[0], want[3])):
                    assert torch.equal(x, y)
        if not pieces:
            for pad in (0, 1):
                with env(QGEMM_FUSED=f"-1/-1/{pad}"):
                    got, _, _ = run(True)
                for x, y in zip(got, want):
                    assert torch.equal(x, y)


@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("tile", range(len(TILES)))
def test_what_lies_past_k_adds_nothing(tile, pad):
    """Rows longer than K, with other values behind K, and a K that ends inside a chunk or a
    16-byte piece."""
    m, n = 70, 144
    for k in (1, 16, 47, 48, 144, 272, 273):
        a, (w, _), sa, (sw, _) = inputs(m, n, 512, k, 2)
        A, W = gpu(a), gpu(w)
        with env(QGEMM_FUSED=f"{tile}/-1/{pad}"):
            got = q.qgemm_a8w8_linear(A[:, :k], W[:, :k], gpu(sa), gpu(sw), b_trans=True)
            also = q.qgemm_a8w8_linear(A[:, :k], W.t().contiguous()[:k], gpu(sa), gpu(sw))
        want = ref.z32(ref.accumulate(a[:, :k], w[:, :k], True), sa, sw)
        assert np.array_equal(got.cpu().numpy(), want) and torch.equal(got, also)

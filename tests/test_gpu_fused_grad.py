"""Gradients of the fused A8W8 products against the formula in 64 bits and against
differences of the forward pass in 64 bits."""
import numpy as np
import pytest
import torch

import fused_reference as ref
import quantized_int8_gemm_amd as q
from gpu_util import case, dev, env
from test_gpu_fused_linear import TILES, check, gpu, inputs, laid, padded

pytestmark = pytest.mark.gpu

ACTS = ("silu", "gelu", "gelu_tanh", "relu")
SHAPES = [(1, 1, 1), (1, 64, 16), (2, 48, 33), (3, 7, 5), (17, 100, 128), (64, 130, 80), (65, 512, 64), (128, 513, 144), (130, 300, 272),
          (257, 2049, 96), (40, 4100, 48), (24, 8200, 64), (9, 16400, 32), (5, 33000, 16)]


def saved(m, n, seed, halves=1):
    """A checkpoint of ordinary values, with blocks of zeros among them."""
    r = np.random.default_rng(seed)
    codes = r.integers(-127, 128, (halves, m, n), dtype=np.int8)
    scale = (r.uniform(0.2, 2, (halves, m, -(-n // 32))) / 127 * 2).astype(np.float32)
    codes[:, :, 32:64] = 0
    return codes, scale


def upstream(m, n, seed, d):
    y = torch.from_numpy(np.random.default_rng(seed).normal(size=(m, n)) * 0.1).to(d)
    return y.to(dev()), y.double().numpy()


def curve(dy, scale_of_other):
    """What a factor may be off by where its sum cancels: 2^-19 of dy and the other factor."""
    return np.abs(dy) * scale_of_other * 2.0 ** -19


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_grad(shape, b_trans):
    m, n, k = shape
    for i, act in enumerate(ACTS + (None,)):
        d = (torch.bfloat16, torch.float16)[(i + m) % 2]
        case(f"linear grad {shape} b_trans={b_trans} {act} {d}")
        _, (w,), _, (sw,) = inputs(m, n, k, 50 * m + i)
        sw = sw * np.float32(np.sqrt(k) * 100)
        codes, scale = saved(m, n, i)
        dy, dyd = upstream(m, n, i + 7, d)
        ck = None if act is None else (gpu(codes[0]), gpu(scale[0]))
        dx, db = q.qgemm_a8w8_linear_grad(dy, laid(w, b_trans), gpu(sw), ck, act, b_trans=b_trans, bias_grad=True)
        z = ref.values(codes[0], scale[0])
        p = dyd * ref.slope(act, z)
        want, off = ref.grad([p], [sw], [w], True)
        off = off + curve(dyd, np.abs(sw.astype(np.float64)) * (1 + np.abs(z))) @ np.abs(w.astype(np.float64))
        check(dx, want, off + 2.0 ** -22 * np.abs(want), d)
        # a sum of m terms in fp32, in any order
        check(db, p.sum(0), (np.abs(p) * ((m + 4) * 2.0 ** -24 + 2.0 ** -20) + curve(dyd, 1 + np.abs(z))).sum(0), torch.float32)
        again = q.qgemm_a8w8_linear_grad(dy, laid(w, b_trans), gpu(sw), ck, act, b_trans=b_trans)
        assert torch.equal(again, dx)


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_grad(shape, b_trans):
    m, n, k = shape
    for i, act in enumerate(ACTS + ("none",)):
        d = (torch.bfloat16, torch.float16)[(i + m) % 2]
        case(f"gated grad {shape} b_trans={b_trans} {act} {d}")
        _, ws, _, ss = inputs(m, n, k, 50 * m + i, 2)
        ss = [s * np.float32(np.sqrt(k) * 100) for s in ss]
        codes, scale = saved(m, n, i, 2)
        dy, dyd = upstream(m, n, i + 7, d)
        dx = q.qgemm_a8w8_gated_grad(dy, *(laid(w, b_trans) for w in ws), *map(gpu, ss), (gpu(codes), gpu(scale)), act, b_trans=b_trans)
        g, u = (ref.values(codes[h], scale[h]) for h in range(2))
        want, off = ref.grad([dyd * u * ref.slope(act, g), dyd * ref.act(act, g)], ss, ws, True)
        for w, s, o in zip(ws, ss, (np.abs(u) * (1 + np.abs(g)), 1 + np.abs(g))):
            off = off + curve(dyd, o * np.abs(s.astype(np.float64))) @ np.abs(w.astype(np.float64))
        check(dx, want, off + 2.0 ** -22 * np.abs(want), d)


@pytest.mark.parametrize("m,n", [(2600, 300), (700, 2000), (1300, 4001), (600, 8001), (600, 16003), (600, 17003), (530, 40001)])
def test_bias_over_more_rows_than_workgroups(m, n):
    """Each workgroup of the factors' pass adds up several rows, of every width it is built for."""
    k, d = 16, torch.bfloat16
    case(f"bias {m} {n}")
    _, (w,), _, (sw,) = inputs(m, n, k, m)
    codes, scale = saved(m, n, 5)
    dy, dyd = upstream(m, n, 6, d)
    dx, db = q.qgemm_a8w8_linear_grad(dy, gpu(w), gpu(sw), (gpu(codes[0]), gpu(scale[0])), "silu", b_trans=True, bias_grad=True)
    z = ref.values(codes[0], scale[0])
    p = dyd * ref.slope("silu", z)
    check(db, p.sum(0), (np.abs(p) * ((m + 4) * 2.0 ** -24 + 2.0 ** -20) + curve(dyd, 1 + np.abs(z))).sum(0), torch.float32)
    want, off = ref.grad([p], [sw], [w], True)
    off = off + curve(dyd, np.abs(sw.astype(np.float64)) * (1 + np.abs(z))) @ np.abs(w.astype(np.float64))
    check(dx, want, off + 2.0 ** -22 * np.abs(want), d)
    again = q.qgemm_a8w8_linear_grad(dy, gpu(w), gpu(sw), (gpu(codes[0]), gpu(scale[0])), "silu", b_trans=True, bias_grad=True)
    assert torch.equal(again[0], dx) and torch.equal(again[1], db)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_against_differences(act):
    """d/dt of sum(dy * out(x + t v)) at t = 0, from values of the forward pass in 64 bits.
    The checkpoint's z is off by half a step of its block, so act' by that times the
    largest |act''| (0.5, 0.8 and 0.8 for these), and act, u likewise."""
    m, n, k = 9, 70, 48
    a, ws, sa, ss = inputs(m, n, k, 11, 2)
    ss = [s * np.float32(2000) for s in ss]
    r = np.random.default_rng(2)
    dy, dyd = upstream(m, n, 3, torch.bfloat16)
    bias = r.normal(size=n).astype(np.float32)
    x = a.astype(np.float64) * sa.astype(np.float64)[:, None]
    v = r.normal(size=x.shape)
    rows = [w.astype(np.float64).T * s.astype(np.float64) for w, s in zip(ws, ss)]
    bend, h = 0.8, 1e-4

    def differences(f):
        return (f(x + h * v) - f(x - h * v)) / (2 * h)

    out, ck = q.qgemm_a8w8_linear(gpu(a), gpu(ws[0]), gpu(sa), gpu(ss[0]), bias=gpu(bias), activation=act, b_trans=True, checkpoint=True)
    dx, db = q.qgemm_a8w8_linear_grad(dy, gpu(ws[0]), gpu(ss[0]), ck, act, b_trans=True, bias_grad=True)
    want = differences(lambda t: (dyd * ref.act(act, t @ rows[0] + bias)).sum())
    half = np.repeat(ck[1].double().cpu().numpy(), 32, 1)[:, :n] * 0.5
    rounding = (np.abs(dx.double().cpu().numpy()) * 2.0 ** -8 * np.abs(v)).sum() + 1e-6 * (np.abs(dyd) @ np.abs(rows[0].T)).sum()
    slack = (np.abs(dyd) * bend * half * np.abs(v @ rows[0])).sum() + rounding
    assert abs((dx.double().cpu().numpy() * v).sum() - want) <= slack + 1e-4 * (np.abs(dyd) @ np.abs(rows[0].T)).sum()
    vb = r.normal(size=n)
    z = x @ rows[0] + bias
    want = ((dyd * ref.act(act, z + h * vb)).sum() - (dyd * ref.act(act, z - h * vb)).sum()) / (2 * h)
    assert abs((db.double().cpu().numpy() * vb).sum() - want) <= (np.abs(dyd) * (bend * half + 1e-5) * np.abs(vb)).sum()

    out, ck = q.qgemm_a8w8_gated(gpu(a), *map(gpu, ws), gpu(sa), *map(gpu, ss), activation=act, b_trans=True, checkpoint=True)
    dx = q.qgemm_a8w8_gated_grad(dy, *map(gpu, ws), *map(gpu, ss), ck, act, b_trans=True).double().cpu().numpy()
    want = differences(lambda t: (dyd * ref.act(act, t @ rows[0]) * (t @ rows[1])).sum())
    hg, hu = (np.repeat(ck[1][i].double().cpu().numpy(), 32, 1)[:, :n] * 0.5 for i in range(2))
    u = np.abs(x @ rows[1])
    slack = (np.abs(dyd) * ((u + hu) * bend * hg + 1.13 * hu) * np.abs(v @ rows[0])).sum()
    slack += (np.abs(dyd) * 1.13 * hg * np.abs(v @ rows[1])).sum()
    slack += (np.abs(dx) * 2.0 ** -8 * np.abs(v)).sum() + 1e-4 * sum((np.abs(dyd) * (1 + u)) @ np.abs(w.T) for w in rows).sum()
    assert abs((dx * v).sum() - want) <= slack


def test_rows_that_are_not_finite_or_zero():
    m, n, k = 70, 96, 64
    _, ws, _, ss = inputs(m, n, k, 5, 2)
    codes, scale = saved(m, n, 1, 2)
    dy, _ = upstream(m, n, 2, torch.bfloat16)
    dy[0, 3], dy[1, 5], dy[2] = float("nan"), float("inf"), 0
    scale[0, 3, 1] = np.nan
    args = (*map(gpu, ws), *map(gpu, ss))
    dx = q.qgemm_a8w8_gated_grad(dy, *args, (gpu(codes), gpu(scale)), b_trans=True)
    assert torch.isnan(dx[0]).all() and torch.isnan(dx[1]).all() and (dx[2] == 0).all() and torch.isnan(dx[3]).all()
    clean, cs = dy.clone(), scale.copy()
    clean[:2] = 1
    cs[0, 3, 1] = 1
    good = q.qgemm_a8w8_gated_grad(clean, *args, (gpu(codes), gpu(cs)), b_trans=True)
    assert torch.equal(dx[4:], good[4:]) and torch.isfinite(good).all()
    dx, db = q.qgemm_a8w8_linear_grad(dy, gpu(ws[0]), gpu(ss[0]), b_trans=True, bias_grad=True)
    assert torch.isnan(dx[:2]).all() and torch.isnan(db[3]) and torch.isinf(db[5]) and torch.isfinite(db[6:]).all()


def test_small_gradients():
    """Rows of values near fp16's smallest, and scales that take their products far below."""
    m, n, k = 20, 64, 48
    _, (w,), _, _ = inputs(m, n, k, 5)
    dy = torch.full((m, n), 2.0 ** -24, dtype=torch.float16, device=dev())
    for e in (-20, -60, -90):
        sw = np.full(n, 2.0 ** e, np.float32)
        big = q.qgemm_a8w8_linear_grad(dy, gpu(w), gpu(np.full(n, 2.0 ** 14, np.float32)), b_trans=True)
        bf = q.qgemm_a8w8_linear_grad(dy.bfloat16(), gpu(w), gpu(sw), b_trans=True)
        want = w.astype(np.float64).sum(0) * 2.0 ** -24
        check(big, np.broadcast_to(want * 2.0 ** 14, (m, k)), np.abs(want * 2.0 ** 14) * 2.0 ** -20, torch.float16)
        check(bf, np.broadcast_to(want * 2.0 ** e, (m, k)), np.abs(want * 2.0 ** e) * 2.0 ** -20, torch.bfloat16)


@pytest.mark.parametrize("b_trans", [True, False])
def test_strides(b_trans):
    m, n, k = 70, 144, 112
    _, ws, _, ss = inputs(m, n, k, 5, 2)
    codes, scale = saved(m, n, 1, 2)
    dy, _ = upstream(m, n, 2, torch.float16)
    for extra in (16, 3):
        G, U = padded(laid(ws[0], b_trans), extra), padded(laid(ws[1], b_trans), extra + 5)
        ck = (gpu(codes), gpu(scale))
        got = q.qgemm_a8w8_gated_grad(padded(dy, extra), G, U, *map(gpu, ss), ck, "gelu", b_trans=b_trans)
        want = q.qgemm_a8w8_gated_grad(dy, laid(ws[0], b_trans), laid(ws[1], b_trans), *map(gpu, ss), ck, "gelu", b_trans=b_trans)
        assert torch.equal(got, want)


def test_no_rows():
    _, (w,), _, (sw,) = inputs(4, 40, 32, 1)
    dy = torch.zeros(0, 40, dtype=torch.bfloat16, device=dev())
    dx, db = q.qgemm_a8w8_linear_grad(dy, gpu(w), gpu(sw), b_trans=True, bias_grad=True)
    assert dx.shape == (0, 32) and db.shape == (40,) and (db == 0).all()
    ck = (torch.zeros(2, 0, 40, dtype=torch.int8, device=dev()), torch.zeros(2, 0, 2, device=dev()))
    assert q.qgemm_a8w8_gated_grad(dy, gpu(w), gpu(w), gpu(sw), gpu(sw), ck, b_trans=True).shape == (0, 32)


def test_the_most_columns():
    """Sums over 2 x 65535 extreme products stay inside int32, and one column more is refused."""
    m, n, k = 3, 65535, 32
    w = torch.full((n, k), -128, dtype=torch.int8, device=dev())
    s = torch.ones((), device=dev())
    codes = torch.full((2, m, n), 127, dtype=torch.int8, device=dev())
    scale = torch.full((2, m, 2048), 1 / 127, device=dev())
    dy = torch.ones(m, n, dtype=torch.bfloat16, device=dev())
    dx = q.qgemm_a8w8_gated_grad(dy, w, w, s, s, (codes, scale), "none", b_trans=True)
    assert ((dx.double() + 2 * 128 * n).abs() <= 2 * 128 * n * 2.0 ** -8).all()
    dx = q.qgemm_a8w8_gated_grad(-dy, w, w, s, s, (codes, scale), "none", b_trans=True)
    assert ((dx.double() - 2 * 128 * n).abs() <= 2 * 128 * n * 2.0 ** -8).all()
    with pytest.raises(NotImplementedError):
        q.qgemm_a8w8_linear_grad(torch.ones(1, n + 1, dtype=torch.bfloat16, device=dev()), torch.ones(n + 1, k, dtype=torch.int8, device=dev()),
                                 s, b_trans=True)


@pytest.mark.parametrize("b_trans", [True, False])
@pytest.mark.parametrize("tile", range(len(TILES)))
def test_every_kernel_gives_the_same_bits(tile, b_trans):
    """The bias's gradient too, which is added up in the product's launch."""
    for m, n, k in ((1, 16, 16), (33, 80, 48), (64, 128, 128), (140, 400, 272), (257, 1040, 528), (20, 47, 33), (70, 300, 129), (130, 1025, 143)):
        _, ws, _, ss = inputs(m, n, k, m + n, 2)
        ss = [s * np.float32(np.sqrt(k) * 100) for s in ss]
        codes, scale = saved(m, n, 3, 2)
        dy, _ = upstream(m, n, 4, torch.float16)

        def run():
            d = q.qgemm_a8w8_gated_grad(dy, *(laid(w, b_trans) for w in ws), *map(gpu, ss), (gpu(codes), gpu(scale)), b_trans=b_trans)
            first = q.last_kernel()
            one = q.qgemm_a8w8_linear_grad(dy, laid(ws[0], b_trans), gpu(ss[0]), (gpu(codes[0]), gpu(scale[0])), "gelu", b_trans=b_trans,
                                           bias_grad=True)
            return d, torch.cat([one[0].flatten().float(), one[1]]), first, q.last_kernel()

        with env(QGEMM_FUSED="4/1/0"):
            want = run()
        for splits, pad in ((1, 0), (2, 1), (4, 0)):
            case(f"tile {tile} {m} {n} {k} b_trans={b_trans} splits={splits} pad={pad}")
            with env(QGEMM_FUSED=f"{tile}/{splits}/{pad}"):
                got = run()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            for name, branches in ((got[2], 2), (got[3], 1)):
                # the gradient reads the weight the other way, and 32 rows of [N,K] are no kind of its
                if tile > 4 and ("kn" in TILES[tile]) != b_trans or TILES[tile] == "direct_kn_32":
                    continue
                joined = splits > 1 and 0 < tile < 5
                assert (joined and -(-n // 128) * branches < splits) or name == "fused_grad_" + ("joined" if joined else TILES[tile])

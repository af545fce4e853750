"""The norm, the quantisers and the products together: as the example's block
uses them, captured in a graph, on other streams, in place, and where offsets
pass 32 bits."""
import importlib.util
import os
import threading

import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from quantized_int8_gemm_amd import _binding as b
from quantized_int8_gemm_amd import _mx
from gpu_util import case, dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def block(n, k, seed, activations="mxfp8"):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantized_block.py")
    spec = importlib.util.spec_from_file_location("quantized_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    g = torch.Generator(device=dev()).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev()).bfloat16()   # noqa: E731
    return mod.QuantizedBlock(0.05 * rand(n, k), 1 + 0.1 * rand(k), activations), rand


def d64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("tokens,k,n", [(1, 256, 96), (7, 1000, 300), (130, 2048, 257)])
@pytest.mark.parametrize("act", ["mxfp8", "mxfp4"])
def test_forward_and_backward_of_the_block(tokens, k, n, act):
    """Each step against the 64-bit form of what its inputs stand for."""
    case(f"block {tokens}x{k}x{n} {act}")
    blk, rand = block(n, k, tokens, act)
    x, r, dout, dh = rand(tokens, k), rand(tokens, k), rand(tokens, n), rand(tokens, k)
    y, h, rstd = blk.forward(x, r)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    c, s = R.mx_quantize((h.float() * blk.gain.float()).cpu().numpy(), act)     # the codes are exact
    w = d64(q.mx_dequantize(*blk.w4, torch.float32))
    t = R.mx_values(c, s, act)
    rr = R.rstd(d64(h), 1e-6)[:, None]
    want, size = (t @ w.T) * rr, (np.abs(t) @ np.abs(w).T) * rr
    # bf16 output; r within 48 steps; sums of K / 16 groups; e4m3 groups lose up to 16 * 2^-13 of their largest product
    lose = 16 * 2.0 ** -13 * (np.abs(t).reshape(tokens, -1, 16).max(-1) @ np.abs(w).reshape(n, -1, 16).max(-1).T) * rr if act == "mxfp8" else 0
    assert np.all(np.abs(d64(y) - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (t.shape[1] / 16 + 80) * 2 * U * size + lose)
    dx, dgain = blk.backward(dout, h, rstd, dh)
    # the gradient through the product, as the kernel left it, is checked by its own tests: here the chain's
    dy = q.mx_matmul(*q.mx_quantize(dout, "mxfp8"), *blk.w4_t, out_dtype=torch.bfloat16)
    wx, wg = R.grad(d64(dy), d64(h), d64(blk.gain), d64(rstd), d64(dh))
    size = np.abs(d64(h)) * d64(rstd)[:, None] ** 3 / k * np.abs(d64(dy) * d64(blk.gain) * d64(h)).sum(1, keepdims=True)
    tol = U * (100 * size + 8 * np.abs(d64(rstd)[:, None] * d64(dy) * d64(blk.gain)) + 8 * np.abs(wx) + 2 * np.abs(d64(dh)))
    assert np.all(np.abs(d64(dx) - wx) <= tol + 2.0 ** -8 * 1.01 * np.abs(wx))
    gsize = np.abs(d64(dy) * d64(h) * d64(rstd)[:, None]).sum(0)
    assert np.all(np.abs(d64(dgain) - wg) <= 80 * U * gsize + 2.0 ** -8 * 1.01 * np.abs(wg))


def test_int8_block_feeds_the_integer_product():
    case("int8 block 33x512x200")
    blk, rand = block(200, 512, 3)
    x, r = rand(33, 512), rand(33, 512)
    y, h = blk.serve_int8(x, r)
    codes, a = R.int8_codes(h.float().cpu().numpy(), blk.gain.float().cpu().numpy())
    acc = codes.astype(np.float64) @ d64(blk.w8).T
    scale = a.astype(np.float64) * R.rstd(d64(h), 1e-6) / 127
    want = acc * scale[:, None] * d64(blk.w8_scale)
    # the integer sum is exact; scale within 52 steps, three roundings more, then bf16
    assert np.all(np.abs(d64(y) - want) <= (56 * U + 2.0 ** -8 * 1.01) * np.abs(want))


@pytest.mark.parametrize("tokens", [1, 200])
def test_captured_in_a_graph(tokens):
    """Forward and backward in one graph: several replays with eager calls and other
    inputs between them, each equal to the eager results."""
    case(f"block in a graph, {tokens} tokens")
    blk, rand = block(520, 1024, 5)
    x, r, dout, dh = rand(tokens, 1024), rand(tokens, 1024), rand(tokens, 520), rand(tokens, 1024)

    def step():
        y, h, rstd = blk.forward(x, r)
        y8, _ = blk.serve_int8(x, r)
        return (y, y8, h) + tuple(blk.backward(dout, h, rstd, dh))

    eager = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(captured, eager)), i
        if i == 1:
            x.copy_(rand(tokens, 1024))        # the graph reads the buffers anew
            dh.copy_(rand(tokens, 1024))
            eager = [t.clone() for t in step()]
        torch.randn(1000, device=dev()).sum().item()


def test_two_streams_and_threads_at_once():
    case("block on two streams from two threads")
    blocks = [block(700, 1024, s) for s in (7, 8)]
    ins = [[rand(t, 1024), rand(t, 1024), rand(t, 700)] for (_, rand), t in zip(blocks, (3, 150))]
    ref = []
    for (blk, _), (x, r, d) in zip(blocks, ins):
        y, h, rstd = blk.forward(x, r)
        ref.append([y, h, *blk.backward(d, h, rstd)])
    torch.cuda.synchronize()
    got, names = [[], []], [set(), set()]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                y, h, rstd = blocks[i][0].forward(*ins[i][:2])
                names[i].add(q.last_kernel())
                got[i].append([y, h, *blocks[i][0].backward(ins[i][2], h, rstd)])
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for i in range(2):
        assert len(names[i]) == 1 and len(got[i]) == 10
        for one in got[i]:
            assert all(torch.equal(a, c) for a, c in zip(one, ref[i]))


@pytest.mark.parametrize("n", [300, 1001, 4096, 9001, 20001])
@pytest.mark.parametrize("over", ["dy", "dh"])
def test_gradient_in_place(n, over):
    """dx over dy or over dh, as the header allows, at widths that end inside a group."""
    case(f"rms_norm_grad in place over {over}, n={n}")
    g = torch.Generator(device=dev()).manual_seed(n)
    dy, h, dh = (torch.randn(9, n, generator=g, device=dev()).bfloat16() for _ in range(3))
    w = torch.ones(n, device=dev()).bfloat16()
    _, rstd = q.rms_norm(h, w)
    want = q.rms_norm_grad(dy, h, w, rstd, dh)
    dx, dw = dict(dy=dy, dh=dh)[over], torch.empty(n, device=dev(), dtype=torch.bfloat16)
    ws = torch.empty(b.lib.rms_norm_grad_workspace_bytes(9, n), dtype=torch.uint8, device=dev())
    st = b.lib.rms_norm_grad(9, n, dy.data_ptr(), b.QG_BF16, n, h.data_ptr(), n, w.data_ptr(), b.QG_BF16, rstd.data_ptr(),
                             dh.data_ptr(), n, dx.data_ptr(), n, dw.data_ptr(), ws.data_ptr(), ws.numel(),
                             torch.cuda.current_stream().cuda_stream)
    assert st == b.QG_OK and torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_nan_codes_of_e4m3_reach_their_row():
    case("mx_matmul NaN codes")
    for m in (2, 40, 300):
        x = torch.randn(m, 256, generator=torch.Generator().manual_seed(m)).to(dev())
        a, sa = q.mx_quantize(x, "mxfp8")
        w, sw = q.mx_quantize(torch.randn(90, 256, generator=torch.Generator().manual_seed(1)).to(dev()))
        ref = q.mx_matmul(a, sa, w, sw)
        bad = a.view(torch.uint8).clone()
        bad[1, 77] = 0x7f
        got = q.mx_matmul(bad.view(torch.float8_e4m3fn), sa, w, sw)
        assert torch.isnan(got[1]).all() and torch.equal(got[0], ref[0]) and torch.equal(got[2:], ref[2:])


def test_rows_past_one_launch():
    """More rows than one launch of the norm takes (2^21)."""
    case("rms_norm 2^21 + 5 rows")
    m = (1 << 21) + 5
    g = torch.Generator(device=dev()).manual_seed(1)
    x, r = (torch.randn(m, 40, generator=g, device=dev()).half() for _ in range(2))
    w = (1 + 0.2 * torch.randn(40, generator=g, device=dev())).half()
    h = (x.float() + r.float()).half()
    at = torch.tensor([0, 5, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, m - 1], device=dev())
    for fmt in ("int8", "mxfp8", "mxfp4"):
        whole, part = (q.rms_norm_quantize(a, w, residual=c, format=fmt) for a, c in ((x, r), (x[at], r[at])))
        assert torch.equal(whole[-1], h)
        for a, c in zip(whole, part):
            assert torch.equal(a[at].view(torch.uint8), c.contiguous().view(torch.uint8))
    for dt in (torch.float16, torch.float32):
        whole, part = q.rms_norm(x, w, residual=r, out_dtype=dt), q.rms_norm(x[at], w, residual=r[at], out_dtype=dt)
        assert all(torch.equal(a[at], c) for a, c in zip(whole, part))


def test_offsets_past_32_bits():
    """2.3e9 elements through the norm, its gradient and the quantiser, and products
    whose operand and output rows lie past 2^31 bytes."""
    case("offsets past 2^31: norm, gradient, quantiser 70000 x 32768")
    d = dev()
    rows, n = 70000, 32768
    x = torch.empty(rows, n, dtype=torch.bfloat16, device=d)
    g = torch.Generator(device=d).manual_seed(2)
    for i in range(0, rows, 10000):
        x[i:i + 10000].copy_(torch.randn(min(10000, rows - i), n, generator=g, device=d))
    w = torch.ones(n, device=d).bfloat16()
    at = torch.tensor([0, 40000, 65535, 65536, rows - 1], device=d)
    some = x[at].clone()
    for fmt in ("int8", "mxfp4"):
        whole, part = q.rms_norm_quantize(x, w, format=fmt), q.rms_norm_quantize(some, w, format=fmt)
        assert all(torch.equal(a[at], c) for a, c in zip(whole, part))
        del whole
    whole, part = q.mx_quantize(x, "mxfp8"), q.mx_quantize(some, "mxfp8")
    assert torch.equal(whole[0].view(torch.uint8)[at], part[0].view(torch.uint8)) and torch.equal(whole[1][at], part[1])
    back = q.mx_dequantize(*whole)
    assert torch.equal(back[at], q.mx_dequantize(*part))
    del whole, back
    rstd = q.rms_norm(x, w)[1]
    dx, dw = q.rms_norm_grad(x, x, w, rstd)
    px, _ = q.rms_norm_grad(some, some, w, rstd[at])
    assert torch.equal(dx[at], px) and bool(torch.isfinite(dw).all())
    # sum over rows of x * x * r ~ rows, each within the noise of 70000 terms
    assert (dw.float() / rows - 1).abs().max().item() < 0.05
    del dx, x
    case("offsets past 2^31: MX product 600000 x 40 x 8192, and a stride of 4000000")
    m, k = 600000, 8192
    a = torch.randint(0, 256, (m, k // 2), generator=g, dtype=torch.uint8, device=d)
    sa = torch.randint(120, 130, (m, k // 32), generator=g, dtype=torch.uint8, device=d)
    wc, ws = q.mx_quantize(torch.randn(40, k, generator=g, device=d))
    out = torch.full((m, 4096), 9.0, dtype=torch.float16, device=d)
    q.mx_matmul(a, sa, wc, ws, out_dtype=torch.float16, out=out[:, 16:56])
    at = torch.tensor([0, 300000, 524287, 524288, m - 1], device=d)
    # the same tile for the few rows: with another, sums are added in another order
    want = q.mx_dequantize(a[at], sa[at], torch.float32).double().cpu() @ q.mx_dequantize(wc, ws, torch.float32).double().t().cpu()
    size = q.mx_dequantize(a[at], sa[at], torch.float32).double().abs().cpu() @ q.mx_dequantize(wc, ws, torch.float32).double().abs().t().cpu()
    got = out[at].double().cpu()
    assert ((got[:, 16:56] - want).abs() <= (k / 16 + 24) * 2 * U * size + 2.0 ** -11 * 1.01 * want.abs() + 2.0 ** -25).all()
    assert (got[:, :16] == 9).all() and (got[:, 56:] == 9).all()
    del out, a
    stride, rows = 4000000, 700
    buf = torch.zeros(rows * stride, dtype=torch.uint8, device=d)
    far = buf.as_strided((rows, 512), (stride, 1))
    far.copy_(torch.randint(0, 256, (rows, 512), generator=g, dtype=torch.uint8, device=d))
    s = torch.full((rows, 32), 127, dtype=torch.uint8, device=d)
    wc, ws = q.mx_quantize(torch.randn(300, 1024, generator=g, device=d))
    assert torch.equal(q.mx_matmul(far, s, wc, ws), q.mx_matmul(far.contiguous(), s, wc, ws))
    assert torch.equal(q.mx_matmul(wc, ws, far, s), q.mx_matmul(wc, ws, far.contiguous(), s))
    with pytest.raises(NotImplementedError):
        q.mx_matmul(buf[:4200000 * 2].as_strided((2, 512), (4200000, 1)), s[:2], wc, ws)

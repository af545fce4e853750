"""The fused calls together, as a feed-forward block uses them: norm, gated pair with a
checkpoint, quantiser, projection with the residual, and back; captured, on other
streams, from two threads and at offsets past 32 bits."""
import threading

import numpy as np
import pytest
import torch

import fused_reference as ref
import quantized_int8_gemm_amd as q
from gpu_util import case, dev, env
from test_gpu_fused_linear import gpu, inputs

pytestmark = pytest.mark.gpu


def rand(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator(device=dev()).manual_seed(seed), device=dev()).to(dtype)


class Block:
    """hidden -> inner -> hidden with frozen int8 weights [N,K]."""

    def __init__(self, hidden, inner, act="silu"):
        self.act = act
        self.gate, self.up = (q.int8_quantize(rand(inner, hidden, seed=i) * hidden ** -0.5) for i in (1, 2))
        self.down = q.int8_quantize(rand(hidden, inner, seed=3) * inner ** -0.5)
        self.gain = 1 + 0.1 * rand(hidden, seed=4)

    def forward(self, x, r, checkpoint=True):
        a, s, h = q.rms_norm_quantize(x, self.gain, residual=r)
        y = q.qgemm_a8w8_gated(a, self.gate[0], self.up[0], s, self.gate[1], self.up[1], self.act, torch.bfloat16, b_trans=True,
                               checkpoint=checkpoint)
        y, saved = y if checkpoint else (y, None)
        b, t = q.int8_quantize(y)
        out = q.qgemm_a8w8_linear(b, self.down[0], t, self.down[1], residual=h, out_dtype=torch.bfloat16, b_trans=True)
        return out, h, saved

    def backward(self, d_out, h, saved):
        dy = q.qgemm_a8w8_linear_grad(d_out, self.down[0], self.down[1], b_trans=True)
        dn = q.qgemm_a8w8_gated_grad(dy, self.gate[0], self.up[0], self.gate[1], self.up[1], saved, self.act, b_trans=True)
        rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
        return q.rms_norm_grad(dn, h, self.gain, rstd, dh=d_out)


def exact(block, x, r, d_out):
    """The same block in 64 bits on the CPU, without the activations' and the checkpoint's
    rounding, by autograd."""
    double = lambda t: t.double().cpu()   # noqa: E731
    w = [double(c) * double(s)[:, None] for c, s in (block.gate, block.up, block.down)]
    x, gain = double(x), double(block.gain).requires_grad_()
    x.requires_grad_()
    h = x + double(r)
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * gain
    out = torch.nn.functional.linear(torch.nn.functional.silu(n @ w[0].t()) * (n @ w[1].t()), w[2]) + h
    out.backward(double(d_out))
    return out.detach(), x.grad, gain.grad


@pytest.mark.parametrize("tokens,hidden,inner", [(1, 256, 512), (37, 320, 800), (300, 512, 1424)])
def test_a_block_forward_and_back(tokens, hidden, inner):
    """Off from the exact block by the 8-bit roundings alone.  Of a value a step of 1 / 127 of
    its row's (block's) largest, whose ratio to the root mean square is below 5 (rows) for
    these sizes, uniform within half a step: 5 / 127 / sqrt(12) = 1.2 % a rounding, of A, of y and
    (0.7 % with blocks of 32) of the checkpoint, through factors that no more than double
    it; 16-bit roundings are far below.  Together under 6 %."""
    case(f"block {tokens} {hidden} {inner}")
    block = Block(hidden, inner)
    x, r, d = rand(tokens, hidden, seed=5), rand(tokens, hidden, seed=6), rand(tokens, hidden, seed=7)
    out, h, saved = block.forward(x, r)
    dx, dgain = block.backward(d, h, saved)
    want = exact(block, x, r, d)
    for got, w in zip((out, dx, dgain), want):
        assert (got.double().cpu() - w).norm() <= 0.06 * w.norm()
    assert torch.equal(block.forward(x, r, checkpoint=False)[0], out)


def test_captured_and_replayed():
    """A step in a graph gives the eager step's bits at every replay, with eager work
    between and an eager step of the same tensors alive."""
    block = Block(512, 1424)
    x, r, d = (rand(130, 512, seed=i) for i in (5, 6, 7))

    def step():
        out, h, saved = block.forward(x, r)
        a, s = q.int8_quantize(out)
        lin, kept = q.qgemm_a8w8_linear(a, block.gate[0], s, block.gate[1], bias=bias, activation="gelu", out_dtype=torch.bfloat16,
                                        b_trans=True, checkpoint=True)
        back = q.qgemm_a8w8_linear_grad(lin, block.gate[0], block.gate[1], kept, "gelu", b_trans=True, bias_grad=True)
        return (out, *block.backward(d, h, saved), lin, *back)

    bias = rand(1424, seed=9, dtype=torch.float32)
    with env(QGEMM_FUSED="3/3"):   # K divided: workspaces in the graph
        keep = step()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got = step()
            graphs.append((g, got))
        for i in range(4):
            for t in (x, r, d):
                t.copy_(rand(*t.shape, seed=20 + i))
            want = step()
            for g, got in graphs:
                for t in got:
                    t.zero_()
                g.replay()
                torch.cuda.synchronize()
                for a, b in zip(got, want):
                    assert torch.equal(a, b)
    assert len(keep) == 6


def test_streams_and_threads():
    """Calls on their own streams from two threads, with their own workspaces."""
    block = Block(512, 1424)
    want, got, wrong = {}, {}, []
    args = {i: (rand(90 + i, 512, seed=i), rand(90 + i, 512, seed=50 + i), rand(90 + i, 512, seed=90 + i)) for i in range(2)}

    def step(i):
        x, r, d = args[i]
        out, h, saved = block.forward(x, r)
        return (out, *block.backward(d, h, saved))

    with env(QGEMM_FUSED="3/2"):
        for i in range(2):
            want[i] = step(i)
        torch.cuda.synchronize()

        def work(i):
            try:
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(10):
                        got[i] = step(i)
                s.synchronize()
            except Exception as e:   # noqa: BLE001
                wrong.append(e)

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not wrong, wrong
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["0/1", "1/1", "2/1", "3/1", "4/1", "6/1"])
def test_outputs_past_32_bit_offsets(kind):
    """Rows behind 2^32 bytes (2^31 elements): the last ones as a small call gives them."""
    m, n, k = 66000, 33000, 16
    case(f"past 32 bits, kind {kind}")
    a, (wg, wu), sa, (sg, su) = inputs(70, n, k, 3, 2)
    A = torch.zeros(m, k, dtype=torch.int8, device=dev())
    A[-70:] = gpu(a)
    S = torch.ones(m, device=dev())
    S[-70:] = gpu(sa)
    W, U = gpu(wg), gpu(wu)
    small = q.qgemm_a8w8_gated(gpu(a), W, U, gpu(sa), gpu(sg), gpu(su), out_dtype=torch.bfloat16, b_trans=True, checkpoint=True)
    with env(QGEMM_FUSED=kind):
        out, (codes, scale) = q.qgemm_a8w8_gated(A, W, U, S, gpu(sg), gpu(su), out_dtype=torch.bfloat16, b_trans=True, checkpoint=True)
    assert torch.equal(out[-70:], small[0]) and torch.equal(codes[:, -70:], small[1][0]) and torch.equal(scale[:, -70:], small[1][1])
    assert (out[:-70:97] == 0).all() and (codes[:, :-70:97] == 0).all()
    del codes, scale
    res = out
    with env(QGEMM_FUSED=kind):
        q.qgemm_a8w8_linear(A, W, S, gpu(sg), residual=res, out=res, out_dtype=torch.bfloat16, b_trans=True)
    want = q.qgemm_a8w8_linear(gpu(a), W, gpu(sa), gpu(sg), residual=small[0], out_dtype=torch.bfloat16, b_trans=True)
    assert torch.equal(res[-70:], want)


def test_gradients_past_32_bit_offsets():
    """dy, the checkpoint and the factors of rows behind 2^31 elements."""
    m, n, k = 66000, 33000, 32
    _, (w,), _, (sw,) = inputs(1, n, k, 3)
    r = np.random.default_rng(1)
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device=dev())
    dy[-40:] = rand(40, n, seed=3)
    codes = torch.zeros(m, n, dtype=torch.int8, device=dev())
    codes[-40:] = gpu(r.integers(-127, 128, (40, n), dtype=np.int8))
    scale = torch.ones(m, 1032, device=dev())
    scale[-40:] = 0.02
    dx, db = q.qgemm_a8w8_linear_grad(dy, gpu(w), gpu(sw), (codes, scale), "silu", b_trans=True, bias_grad=True)
    tail = [t[-40:].clone() for t in (dy, codes, scale)]
    wx, wb = q.qgemm_a8w8_linear_grad(tail[0], gpu(w), gpu(sw), (tail[1], tail[2]), "silu", b_trans=True, bias_grad=True)
    assert torch.equal(dx[-40:], wx) and (dx[:-40] == 0).all()
    p = tail[0].double().cpu().numpy() * ref.slope("silu", ref.values(tail[1].cpu().numpy(), tail[2].cpu().numpy()))
    off = np.abs(p).sum(0) * 2.0 ** -18 + 40 * 2.0 ** -18
    for b in (db, wb):
        assert (np.abs(b.double().cpu().numpy() - p.sum(0)) <= off).all()

"""The fused products' entry points on the CPU: what the header declares is
exported, and bad arguments are refused before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import quantized_int8_gemm_amd as q
from quantized_int8_gemm_amd import _binding as b
from quantized_int8_gemm_amd import _fused as f
from quantized_int8_gemm_amd._mx import QG_FP16, QG_MXFP8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)   # never dereferenced
INV, UNS, WS, OK = b.QG_ERR_INVALID_ARGUMENT, b.QG_ERR_UNSUPPORTED, b.QG_ERR_WORKSPACE, b.QG_OK
F32, BF16, I8, F16 = b.QG_FP32, b.QG_BF16, b.QG_INT8, QG_FP16


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qgemm_fused.h")).read(), flags=re.S)
    names = re.findall(r"\b((?:qgemm|int8)_\w+)\s*\(", text)
    assert names == list(f.PROTOTYPES)   # in this order, which the extension module goes by
    for n in names:
        assert hasattr(ctypes.CDLL(b.LIB_PATH), n)


def call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(b.lib, fn)(*a.values())


LINEAR = dict(M=4, N=40, K=48, A=FAKE, lda=48, W=FAKE, ldw=40, trans=0, sa=FAKE, nsa=4, sw=FAKE, nsw=40, bias=None, act=1,
              res=None, ldr=0, out=FAKE, type=BF16, ldo=40, ck=None, ldc=0, cs=None, lds=0, ws=None, wsb=0, stream=None)
GATED = dict(M=4, N=40, K=48, A=FAKE, lda=48, W=FAKE, ldw=40, W2=FAKE, ldw2=48, trans=0, sa=FAKE, nsa=4, sw=FAKE, nsw=40,
             sw2=FAKE, nsw2=1, act=2, out=FAKE, type=BF16, ldo=40, ck=None, ldc=0, cs=None, lds=0, ws=None, wsb=0, stream=None)
BOTH = [
    (dict(M=0, A=None, out=None), OK), (dict(N=0, W=None, out=None), OK), (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=-1), INV),
    (dict(K=0), INV), (dict(M=0, act=9), INV), (dict(M=1 << 30), INV), (dict(A=None), INV), (dict(W=None), INV), (dict(out=None), INV),
    (dict(sa=None), INV), (dict(sw=None), INV), (dict(sa=ODD), INV), (dict(sw=ODD), INV), (dict(nsa=3), INV), (dict(nsw=39), INV),
    (dict(nsw=0), INV), (dict(lda=47), INV), (dict(ldw=39), INV), (dict(trans=1, ldw=47), INV), (dict(trans=2), INV), (dict(ldo=39), INV),
    (dict(type=I8), INV), (dict(type=QG_MXFP8), INV), (dict(out=ODD), INV), (dict(act=-1), INV), (dict(act=5), INV),
    (dict(ck=FAKE, ldc=40), INV), (dict(cs=FAKE, lds=2), INV), (dict(ck=FAKE, ldc=39, cs=FAKE, lds=2), INV),
    (dict(ck=FAKE, ldc=40, cs=FAKE, lds=1), INV), (dict(ck=FAKE, ldc=40, cs=ODD, lds=2), INV), (dict(ws=ODD, wsb=1 << 30), INV),
    (dict(lda=1 << 23), UNS), (dict(ldw=1 << 23), UNS), (dict(trans=1, ldw=1 << 23), UNS), (dict(ldo=1 << 22), UNS),
    (dict(ck=FAKE, ldc=1 << 22, cs=FAKE, lds=2), UNS), (dict(ck=FAKE, ldc=40, cs=FAKE, lds=1 << 22), UNS),
    (dict(M=(1 << 30) - 1, nsa=1), UNS),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(bias=ODD), INV), (dict(res=FAKE, ldr=39), INV), (dict(res=FAKE, ldr=1 << 22), UNS), (dict(res=ODD, ldr=40), INV)])
def test_linear_rejects(kw, code):
    assert call("qgemm_a8w8_linear", LINEAR, kw) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(W2=None), INV), (dict(ldw2=39), INV), (dict(sw2=None), INV), (dict(nsw2=2), INV), (dict(ldw2=1 << 23), UNS),
    (dict(trans=1, ldw=48, ldw2=47), INV)])
def test_gated_rejects(kw, code):
    assert call("qgemm_a8w8_gated", GATED, kw) == code


LINEAR_GRAD = dict(M=4, N=40, K=48, dy=FAKE, type=BF16, ldy=40, W=FAKE, ldw=40, trans=0, sw=FAKE, nsw=40, ck=FAKE, ldc=40, cs=FAKE,
                   lds=2, act=2, dx=FAKE, ldx=48, db=None, ws=FAKE, wsb=1 << 30, stream=None)
GATED_GRAD = dict(M=4, N=40, K=48, dy=FAKE, type=BF16, ldy=40, W=FAKE, ldw=40, W2=FAKE, ldw2=40, trans=0, sw=FAKE, nsw=40, sw2=FAKE,
                  nsw2=1, ck=FAKE, ldc=40, cs=FAKE, lds=2, act=2, dx=FAKE, ldx=48, ws=FAKE, wsb=1 << 30, stream=None)
BOTH_GRADS = [
    (dict(M=0, dy=None, dx=None), OK), (dict(M=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(N=65536, ldy=65536), UNS),
    (dict(M=0, N=65536), UNS), (dict(dy=None), INV), (dict(dx=None), INV), (dict(W=None), INV), (dict(sw=None), INV), (dict(sw=ODD), INV),
    (dict(nsw=39), INV), (dict(type=F32), INV), (dict(type=I8), INV), (dict(ldy=39), INV), (dict(ldx=47), INV), (dict(ldw=39), INV),
    (dict(trans=1, ldw=47), INV), (dict(trans=-1), INV), (dict(dy=ODD), INV), (dict(dx=ODD), INV), (dict(act=5), INV),
    (dict(ck=None), INV), (dict(cs=None), INV), (dict(ldc=39), INV), (dict(lds=1), INV), (dict(cs=ODD), INV),
    (dict(ck=None, cs=None), INV), (dict(ws=ODD), INV), (dict(ws=None), WS), (dict(wsb=0), WS), (dict(ldw=1 << 23), UNS), (dict(ldx=1 << 22), UNS),
    (dict(M=1 << 29), UNS),
]


@pytest.mark.parametrize("kw,code", BOTH_GRADS + [(dict(db=ODD), INV), (dict(ck=None, cs=None, act=0, wsb=0), WS),
                                                  (dict(ck=None, act=0), INV)])
def test_linear_grad_rejects(kw, code):
    assert call("qgemm_a8w8_linear_grad", LINEAR_GRAD, kw) == code


@pytest.mark.parametrize("kw,code", BOTH_GRADS + [(dict(W2=None), INV), (dict(ldw2=39), INV), (dict(nsw2=0), INV),
                                                  (dict(ck=None, cs=None, act=0), INV)])
def test_gated_grad_rejects(kw, code):
    assert call("qgemm_a8w8_gated_grad", GATED_GRAD, kw) == code


QUANT = dict(M=4, n=40, x=FAKE, type=BF16, ldx=40, block=0, codes=FAKE, ldc=40, scale=FAKE, lds=1, stream=None)
DEQUANT = dict(M=4, n=40, codes=FAKE, ldc=40, scale=FAKE, lds=1, block=0, out=FAKE, type=BF16, ldo=40, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0, codes=None, scale=None), OK), (dict(M=-1), INV), (dict(n=0), INV), (dict(codes=None), INV), (dict(scale=None), INV),
    (dict(ldc=39), INV), (dict(lds=0), INV), (dict(block=32), INV), (dict(block=16, lds=3), INV), (dict(block=-1), INV),
    (dict(type=I8), INV), (dict(scale=ODD), INV),
])
def test_quantisers_reject(kw, code):
    assert call("int8_quantize", QUANT, kw) == code
    assert call("int8_dequantize", DEQUANT, kw) == code


def test_quantisers_reject_their_own():
    for kw, code in ((dict(x=None), INV), (dict(x=ODD), INV), (dict(ldx=39), INV), (dict(n=65537, ldx=65537, ldc=65537), UNS)):
        assert call("int8_quantize", QUANT, kw) == code
    for kw, code in ((dict(out=None), INV), (dict(out=ODD), INV), (dict(ldo=39), INV)):
        assert call("int8_dequantize", DEQUANT, kw) == code


def test_a_short_workspace_is_refused(monkeypatch):
    """The sums of a divided K, and a gradient's factors."""
    monkeypatch.setenv("QGEMM_FUSED", "3/3")
    kw = dict(LINEAR, K=300, lda=300)
    need = b.lib.qgemm_a8w8_linear_workspace_bytes(4, 40, 300, FAKE, 300, FAKE, 40, 0, 0)
    assert need > 0
    assert call("qgemm_a8w8_linear", kw, dict(ws=FAKE, wsb=need - 1)) == WS
    need = b.lib.qgemm_a8w8_gated_workspace_bytes(4, 40, 300, FAKE, 300, FAKE, 40, FAKE, 40, 0, 0)
    assert need > 0
    assert call("qgemm_a8w8_gated", dict(GATED, K=300, lda=300), dict(ws=FAKE, wsb=need - 1)) == WS
    need = b.lib.qgemm_a8w8_linear_grad_workspace_bytes(4, 40, 48, FAKE, 40, 0, 0)
    assert call("qgemm_a8w8_linear_grad", LINEAR_GRAD, dict(wsb=need - 1)) == WS
    need = b.lib.qgemm_a8w8_gated_grad_workspace_bytes(4, 40, 48, FAKE, 40, FAKE, 40, 0)
    assert call("qgemm_a8w8_gated_grad", GATED_GRAD, dict(wsb=need - 1)) == WS
    for M, N, K in ((0, 40, 48), (4, 0, 48), (4, 40, 0), (-1, 40, 48), (1 << 30, 40, 48)):
        assert b.lib.qgemm_a8w8_linear_workspace_bytes(M, N, K, FAKE, 47, FAKE, 40, 0, 1) == 0
        assert b.lib.qgemm_a8w8_linear_grad_workspace_bytes(M, N, K, FAKE, 40, 0, 1) == 0


A, W, SA, SW = torch.zeros(4, 48, dtype=torch.int8), torch.zeros(48, 40, dtype=torch.int8), torch.ones(4), torch.ones(40)
DY = torch.zeros(4, 40, dtype=torch.bfloat16)
SAVED = (torch.zeros(4, 40, dtype=torch.int8), torch.ones(4, 2))
SAVED2 = (torch.zeros(2, 4, 40, dtype=torch.int8), torch.ones(2, 4, 2))


@pytest.mark.parametrize("bad", [
    lambda: q.qgemm_a8w8_linear(A.float(), W, SA, SW), lambda: q.qgemm_a8w8_linear(A, W.int(), SA, SW),
    lambda: q.qgemm_a8w8_linear(A, W, SA.double(), SW), lambda: q.qgemm_a8w8_linear(A, W, SA, SW.half()),
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW, bias=SW.bfloat16()), lambda: q.qgemm_a8w8_linear(A, W, SA, SW, out_dtype=torch.int32),
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW, out_dtype="bf16"), lambda: q.qgemm_a8w8_linear(A, W, SA, SW, residual=DY),
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW, out=DY), lambda: q.qgemm_a8w8_linear([1], W, SA, SW),
    lambda: q.qgemm_a8w8_gated(A, W, W.short(), SA, SW, SW), lambda: q.qgemm_a8w8_gated(A, W, W, SA, SW, SW.half()),
    lambda: q.qgemm_a8w8_linear_grad(DY.float(), W, SW), lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, SAVED[0], "silu"),
    lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, (SAVED[0].int(), SAVED[1]), "silu"),
    lambda: q.qgemm_a8w8_gated_grad(DY, W, W, SW, SW, None), lambda: q.qgemm_a8w8_gated_grad(DY, W, W, SW, SW, (1, 2)),
    lambda: q.int8_quantize(A), lambda: q.int8_dequantize(A.float(), SA), lambda: q.int8_dequantize(A, SA.half()),
    lambda: q.int8_dequantize(A, SA, torch.int8),
])
def test_binding_types(bad):
    with pytest.raises(TypeError):
        bad()


@pytest.mark.parametrize("bad", [
    lambda: q.qgemm_a8w8_linear(A, W[:47], SA, SW), lambda: q.qgemm_a8w8_linear(A, W, SA, SW, b_trans=True),
    lambda: q.qgemm_a8w8_linear(A, W, SA[:3], SW), lambda: q.qgemm_a8w8_linear(A, W, SA[None], SW),
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW[:, None]), lambda: q.qgemm_a8w8_linear(A, W, SA, SW, bias=SA),
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW, activation="tanh"), lambda: q.qgemm_a8w8_linear(A, W, SA, SW, activation=2),
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW, residual=torch.zeros(4, 39)), lambda: q.qgemm_a8w8_linear(A[None], W, SA, SW),
    lambda: q.qgemm_a8w8_linear(A, W.t().contiguous().t(), SA, SW), lambda: q.qgemm_a8w8_linear(A, W, SA, SW, out=torch.zeros(4, 41)),
    lambda: q.qgemm_a8w8_linear(A[:1].expand(4, 48), W, SA, SW),
    lambda: q.qgemm_a8w8_gated(A, W, W[:, :39], SA, SW, SW), lambda: q.qgemm_a8w8_gated(A, W[:47], W[:47], SA, SW, SW),
    lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, activation="silu"), lambda: q.qgemm_a8w8_linear_grad(DY[:, :39], W, SW),
    lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, (SAVED[0][:3], SAVED[1]), "silu"),
    lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, (SAVED[0], SAVED[1][:, :1]), "silu"),
    lambda: q.qgemm_a8w8_gated_grad(DY, W, W, SW, SW, SAVED), lambda: q.qgemm_a8w8_gated_grad(DY, W, W[:, :39], SW, SW, SAVED2),
    lambda: q.int8_quantize(SA, block=16), lambda: q.int8_quantize(SA, block="32"), lambda: q.int8_quantize(torch.zeros(3, 0)),
    lambda: q.int8_dequantize(A, SA[:3]), lambda: q.int8_dequantize(A, torch.ones(4, 3)),
    # the last ones: not on a GPU
    lambda: q.qgemm_a8w8_linear(A, W, SA, SW), lambda: q.qgemm_a8w8_gated(A, W, W, SA, SW, SW, checkpoint=True),
    lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, SAVED, "gelu"), lambda: q.qgemm_a8w8_gated_grad(DY, W, W, SW, SW, SAVED2),
    lambda: q.int8_quantize(SA), lambda: q.int8_dequantize(A, SA), lambda: q.int8_dequantize(A, torch.ones(4, 2)),
])
def test_binding_shapes(bad):
    with pytest.raises(ValueError):
        bad()


@pytest.mark.parametrize("call", [
    lambda: q.qgemm_a8w8_linear(A[:0], W, SA[:0], SW, activation="none"), lambda: q.qgemm_a8w8_linear(A, W, SA[0], SW[None]),
    lambda: q.qgemm_a8w8_gated(A, W, W, SA[:, None], SW, SW[:1]), lambda: q.qgemm_a8w8_linear_grad(DY, W, SW, bias_grad=True),
    lambda: q.int8_quantize(torch.zeros(2, 0, 33)), lambda: q.int8_quantize(torch.zeros(5), block=32),
    lambda: q.int8_dequantize(SAVED2[0], SAVED2[1]),
])
def test_shapes_that_are_taken(call):
    """A call whose only fault is the device has passed every check of its shapes."""
    with pytest.raises(ValueError, match="GPU device"):
        call()

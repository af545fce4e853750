"""The norm and MX entry points on the CPU: what the header declares is
exported, and bad arguments are refused before any HIP call."""
import ctypes
import os
import re

import pytest
import torch

import quantized_int8_gemm_amd as q
from quantized_int8_gemm_amd import _binding as b
from quantized_int8_gemm_amd import _mx as m

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4097)   # never dereferenced
INV, UNS, WS, OK = b.QG_ERR_INVALID_ARGUMENT, b.QG_ERR_UNSUPPORTED, b.QG_ERR_WORKSPACE, b.QG_OK
F32, BF16, I8, F16, M8, M4 = b.QG_FP32, b.QG_BF16, b.QG_INT8, m.QG_FP16, m.QG_MXFP8, m.QG_MXFP4


def test_every_declared_symbol_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qgemm_mx.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:rms|mx)_\w+)\s*\(", text))
    assert names == set(m.PROTOTYPES)
    for n in names:
        assert hasattr(ctypes.CDLL(b.LIB_PATH), n)


def call(fn, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(b.lib, fn)(*a.values())


NORM = dict(M=4, n=40, x=FAKE, type=BF16, ldx=40, res=None, ldr=0, w=FAKE, wt=BF16, eps=1e-6, h=None, ldh=0, out=FAKE,
            format=BF16, ldo=40, bs=None, lds=0, rs=None, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0, x=None, w=None, out=None), OK), (dict(M=-1), INV), (dict(n=0), INV), (dict(n=-4), INV),
    (dict(M=0, n=0), INV), (dict(n=65537, ldx=65537, ldo=65537), UNS),
    (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(ldx=39), INV), (dict(ldo=39), INV),
    (dict(type=I8), INV), (dict(wt=F16), INV), (dict(format=F16), INV), (dict(format=b.QG_INT32), INV),
    (dict(type=F32, wt=BF16, format=F32), INV), (dict(format=99), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV),
    (dict(x=ODD), INV), (dict(out=ODD), INV), (dict(w=ODD), INV), (dict(rs=ODD), INV),
    (dict(res=FAKE, ldr=40), INV), (dict(res=FAKE, ldr=39, h=FAKE, ldh=40), INV),
    (dict(res=FAKE, ldr=40, h=FAKE, ldh=39), INV), (dict(res=FAKE, ldr=40, h=ODD, ldh=40), INV),
    (dict(format=I8), INV), (dict(format=I8, rs=FAKE, ldo=39), INV),
    (dict(format=M8, rs=FAKE, bs=FAKE, lds=1, ldo=64), INV), (dict(format=M8, rs=FAKE, bs=FAKE, lds=2, ldo=63), INV),
    (dict(format=M8, rs=FAKE, lds=2, ldo=64), INV), (dict(format=M8, bs=FAKE, lds=2, ldo=64), INV),
    (dict(format=M4, rs=FAKE, bs=FAKE, lds=2, ldo=31), INV),
])
def test_rms_norm_rejects(kw, code):
    assert call("rms_norm", NORM, kw) == code


GRAD = dict(M=4, n=40, dy=FAKE, type=BF16, ldy=40, h=FAKE, ldh=40, w=FAKE, wt=BF16, rstd=FAKE, dh=None, lddh=0, dx=FAKE,
            lddx=40, dw=FAKE, ws=FAKE, wsb=1 << 20, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INV), (dict(n=0), INV), (dict(n=65537, ldy=65537, ldh=65537, lddx=65537), UNS), (dict(M=0, dw=None), INV),
    (dict(dy=None), INV), (dict(h=None), INV), (dict(w=None), INV), (dict(rstd=None), INV), (dict(dx=None), INV),
    (dict(dw=None), INV), (dict(ldy=39), INV), (dict(ldh=39), INV), (dict(lddx=39), INV), (dict(dh=FAKE, lddh=39), INV),
    (dict(type=I8), INV), (dict(wt=F16), INV), (dict(dy=ODD), INV), (dict(dw=ODD), INV), (dict(ws=None), INV),
    (dict(ws=ctypes.c_void_p(4104)), INV), (dict(wsb=159), WS),
])
def test_rms_norm_grad_rejects(kw, code):
    assert call("rms_norm_grad", GRAD, kw) == code


def test_grad_workspace():
    assert b.lib.rms_norm_grad_workspace_bytes(4, 40) == 160          # one workgroup of four rows
    assert b.lib.rms_norm_grad_workspace_bytes(8192, 4096) == 512 * 4096 * 4
    assert b.lib.rms_norm_grad_workspace_bytes(2049, 400) == 257 * 400 * 4   # eight rows each
    assert b.lib.rms_norm_grad_workspace_bytes(768, 4096) == 256 * 4096 * 4
    assert b.lib.rms_norm_grad_workspace_bytes(0, 40) == 0
    assert b.lib.rms_norm_grad_workspace_bytes(4, 65537) == 0


QUANT = dict(M=4, n=40, x=FAKE, type=BF16, ldx=40, codes=FAKE, format=M4, ldc=32, scale=FAKE, lds=2, stream=None)
DEQUANT = dict(M=4, n=40, codes=FAKE, format=M4, ldc=32, scale=FAKE, lds=2, out=FAKE, type=BF16, ldo=40, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0, codes=None, scale=None), OK), (dict(M=-1), INV), (dict(n=0), INV), (dict(codes=None), INV),
    (dict(scale=None), INV), (dict(ldc=31), INV), (dict(format=M8, ldc=63), INV), (dict(lds=1), INV), (dict(type=I8), INV),
    (dict(format=I8), INV), (dict(format=BF16), INV),
])
def test_quantisers_reject(kw, code):
    assert call("mx_quantize", QUANT, kw) == code
    assert call("mx_dequantize", DEQUANT, kw) == code


def test_quantisers_reject_their_own():
    assert call("mx_quantize", QUANT, dict(x=None)) == INV
    assert call("mx_quantize", QUANT, dict(x=ODD)) == INV
    assert call("mx_quantize", QUANT, dict(ldx=39)) == INV
    assert call("mx_dequantize", DEQUANT, dict(out=None)) == INV
    assert call("mx_dequantize", DEQUANT, dict(out=ODD)) == INV
    assert call("mx_dequantize", DEQUANT, dict(ldo=39)) == INV


MUL = dict(M=4, N=40, K=64, A=FAKE, af=M4, lda=32, as_=FAKE, ldas=2, W=FAKE, ldw=32, ws=FAKE, ldws=2, padded=1, s=None,
           out=FAKE, ot=BF16, ldo=40, stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0, A=None, out=None), OK), (dict(N=0, K=0), OK), (dict(M=-1), INV), (dict(N=-1), INV), (dict(K=0), INV),
    (dict(K=48), INV), (dict(K=-32), INV), (dict(A=None), INV), (dict(as_=None), INV), (dict(W=None), INV),
    (dict(ws=None), INV), (dict(out=None), INV), (dict(lda=31), INV), (dict(af=M8, lda=63), INV), (dict(ldw=31), INV),
    (dict(ldas=1), INV), (dict(ldws=1), INV), (dict(ldo=39), INV), (dict(af=I8), INV), (dict(ot=I8), INV),
    (dict(out=ODD), INV), (dict(s=ODD), INV), (dict(lda=1 << 22), UNS),
    (dict(ldw=1 << 22), UNS), (dict(ldas=1 << 22), UNS), (dict(ldws=1 << 22), UNS),
])
def test_mx_matmul_rejects(kw, code):
    assert call("mx_matmul", MUL, kw) == code


def test_binding_refusals():
    x, w = torch.zeros(4, 40), torch.ones(40)
    for bad in (lambda: q.rms_norm(x.int(), w), lambda: q.rms_norm(x, w.half()), lambda: q.rms_norm([1.0], w),
                lambda: q.rms_norm(x, w, out_dtype=torch.bfloat16), lambda: q.rms_norm(x, w, residual=x.half()),
                lambda: q.mx_quantize(x.int()), lambda: q.rms_norm_grad(x, x.half(), w, torch.ones(4)),
                lambda: q.rms_norm_grad(x, x, w, torch.ones(4).double()),
                lambda: q.mx_matmul(x, x, x, x), lambda: q.mx_dequantize(x, x)):
        with pytest.raises(TypeError):
            bad()
    u = torch.zeros(4, 16, dtype=torch.uint8)
    for bad in (lambda: q.rms_norm(x, w[:39]), lambda: q.rms_norm(x, w, residual=x[:3]),
                lambda: q.rms_norm(torch.zeros(4, 0), torch.zeros(0)), lambda: q.rms_norm(x.t(), torch.ones(4)),
                lambda: q.rms_norm(x[:1].expand(4, 40), w), lambda: q.rms_norm(x, w, residual_out=x),
                lambda: q.rms_norm_quantize(x, w, format="fp6"), lambda: q.mx_quantize(x, "int8"),
                lambda: q.rms_norm(torch.zeros(4, 2, 40).transpose(0, 1), w, residual=None),
                lambda: q.rms_norm_grad(x, x, w, torch.ones(3)), lambda: q.rms_norm_grad(x[:3], x, w, torch.ones(4)),
                lambda: q.mx_dequantize(u, u), lambda: q.mx_dequantize(u, u[:, :1], columns=33),
                lambda: q.mx_dequantize(u, u[:, :1], columns=0), lambda: q.mx_dequantize(u[:, :15], u[:, :1]),
                lambda: q.mx_matmul(u, u[:, :1], u.repeat(1, 2), u[:, :2]), lambda: q.mx_matmul(u, u[:, :2], u, u[:, :1]),
                lambda: q.mx_matmul(u, u[:, :1], u, u[:, :1], act_scale=torch.ones(3)),
                lambda: q.mx_matmul(u, u[:, :1], u, u[:, :1]), lambda: q.rms_norm(x, w), lambda: q.mx_quantize(x)):
        with pytest.raises(ValueError):   # the last three: not on a GPU
            bad()

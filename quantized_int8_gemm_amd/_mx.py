"""Binding of the calls of include/qgemm_mx.h: the RMS norm with its quantised
outputs and its gradient, the MX quantiser and the MX product.

As in the binding of the integer products, each function checks dtypes
(TypeError) and shapes (ValueError), allocates its outputs with torch and
calls the C entry point of the same name on torch's current stream; all
arithmetic runs in the HIP kernels.  The marshalling itself is the extension
module _mx_binding (csrc/mx_binding.cpp), since for one token it took longer
in Python than the kernels do; it calls libqgemm.so as ctypes loaded it.  Where
the module is missing, each call raises ImportError.
"""
import ctypes

import torch

from ._binding import _check, _f32, _i64, _int, _p, _sz, lib


class _Missing:
    """In the extension module's place where it is not built or does not load
    (another torch): the calls below raise, the integer products work."""

    def __init__(self, why, name="_mx_binding"):
        self._text = (f"quantized_int8_gemm_amd/{name}.so is not built for this torch ({why}); run "
                      "__graft_entry__.build() (python -c 'import __graft_entry__ as g; g.build()')")

    def __getattr__(self, name):
        raise ImportError(self._text)


try:
    from . import _mx_binding
except ImportError as e:
    _mx_binding = _Missing(e)

QG_FP16, QG_MXFP8, QG_MXFP4 = 5, 6, 7
MX_BLOCK = 32

# C prototypes, in the order of include/qgemm_mx.h.
PROTOTYPES = {
    "rms_norm": ([_i64, _i64, _p, _int, _i64, _p, _i64, _p, _int, _f32, _p, _i64, _p, _int, _i64, _p, _i64, _p, _p], _int),
    "rms_norm_grad_workspace_bytes": ([_i64, _i64], _sz),
    "rms_norm_grad": ([_i64, _i64, _p, _int, _i64, _p, _i64, _p, _int, _p, _p, _i64, _p, _i64, _p, _p, _sz, _p], _int),
    "mx_quantize": ([_i64, _i64, _p, _int, _i64, _p, _int, _i64, _p, _i64, _p], _int),
    "mx_dequantize": ([_i64, _i64, _p, _int, _i64, _p, _i64, _p, _int, _i64, _p], _int),
    "mx_matmul": ([_i64, _i64, _i64, _p, _int, _i64, _p, _i64, _p, _i64, _p, _i64, _int, _p, _p, _int, _i64, _p], _int),
}
for _name, (_args, _res) in PROTOTYPES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes, _fn.restype = _args, _res


def _bind(library):
    """Hands the extension module the entry points of `library`."""
    _mx_binding.bind(_check, *(ctypes.cast(getattr(library, name), ctypes.c_void_p).value for name in PROTOTYPES))


if not isinstance(_mx_binding, _Missing):
    _bind(lib)


def rms_norm(x, weight, eps=1e-6, residual=None, out_dtype=None, out=None, residual_out=None):
    """y = h / sqrt(mean(h^2) + eps) * weight along the last dimension, with
    h = x + residual (h = x without one).

    x: fp32, bf16 or fp16 [..., n] (unit column stride, rows at one stride);
    weight: [n] of x's dtype or fp32; residual: x's shape and dtype.
    out_dtype: x's dtype (default) or torch.float32.  Returns (y, rstd), and h
    as a third where a residual is given: rstd is fp32 [...], 1 / sqrt(...), as
    rms_norm_grad takes it.  residual_out: the tensor to write h to; it may be
    x or residual itself."""
    return _mx_binding.rms_norm(x, weight, eps, residual, out_dtype, out, residual_out)


def rms_norm_quantize(x, weight, eps=1e-6, residual=None, format="int8", residual_out=None):
    """The same norm with a quantised output, in one pass over x.

    format "int8": returns (q, scale[, h]): q int8 of x's shape, scale fp32
    [...], y ~ q * scale[..., None]: the A and act_scale of qgemm_a8w8.
    format "mxfp8" or "mxfp4": returns (codes, block_scale, act_scale[, h]):
    h * weight in MX form (as mx_quantize returns it) and fp32 act_scale
    [...] = 1 / sqrt(mean(h^2) + eps): the A, a_scale and act_scale of
    mx_matmul.  Other arguments as rms_norm."""
    return _mx_binding.rms_norm_quantize(x, weight, eps, residual, format, residual_out)


def rms_norm_grad(dy, h, weight, rstd, dh=None):
    """Gradient of rms_norm (and, straight through the rounding, of
    rms_norm_quantize): returns (dx, dweight).

    dy, h: fp32, bf16 or fp16 [..., n] of one dtype, h as the norm saw it (its
    third output, or x without a residual); weight: [n]; rstd: fp32 [...] from
    rms_norm; dh: the gradient that reaches h from elsewhere, added to dx.
    dx, of h's shape and dtype, is the gradient of x and of the residual alike;
    dweight has weight's dtype.  Results repeat bit for bit."""
    return _mx_binding.rms_norm_grad(dy, h, weight, rstd, dh)


def mx_quantize(x, format="mxfp4"):
    """x: fp32, bf16 or fp16 [..., n] -> (codes, scale) in MX form.

    Blocks of 32 along the last dimension (filled up with zeros to B whole
    blocks) share a power-of-two scale.  codes: float8_e4m3fn [..., 32 B]
    ("mxfp8"), or uint8 [..., 16 B] with two e2m1 values to a byte, the even
    column in the low half ("mxfp4").  scale: uint8 [..., B], 2^(scale - 127),
    255 for a block that holds a NaN or an infinity; its rows start at
    multiples of 16 bytes."""
    return _mx_binding.mx_quantize(x, format)


def mx_dequantize(codes, scale, out_dtype=torch.bfloat16, columns=None, out=None):
    """The values an MX tensor stands for: fp32, bf16 or fp16 [..., columns]
    (default: all 32 B of them).  codes, scale: as mx_quantize returns them."""
    return _mx_binding.mx_dequantize(codes, scale, out_dtype, columns, out)


def mx_matmul(A, a_scale, W, w_scale, act_scale=None, out_dtype=torch.float32, out=None):
    """out[m, n] = act_scale[m] * sum_k A[m, k] * W[n, k] over MX operands.

    A: float8_e4m3fn [M, K] or packed e2m1 uint8 [M, K/2] with a_scale uint8
    [M, K/32]; W: packed e2m1 uint8 [N, K/2] with w_scale uint8 [N, K/32] (both
    as mx_quantize returns them); act_scale: fp32 [M], [M, 1], a scalar, or
    None for 1.  out_dtype: torch.float32, bfloat16 or float16, rounded once from
    fp32 sums of exact products.  Fast kernels
    need code rows at multiples of 16 bytes and scale rows at multiples of 4,
    as mx_quantize and rms_norm_quantize lay them out; other layouts run a
    slower one."""
    return _mx_binding.mx_matmul(A, a_scale, W, w_scale, act_scale, out_dtype, out)

"""Binding of the calls of include/qgemm_fused.h: the A8W8 product with bias,
activation and residual, the gated pair of products, their gradients from 8-bit
checkpoints, and the int8 quantiser.

As in the binding of the norm and MX calls, each function checks dtypes
(TypeError) and shapes (ValueError), allocates its outputs and workspace with torch
and calls the C entry point on torch's current stream, in an extension module
(_fused_binding, csrc/fused_binding.cpp).  Where the module is missing, each call
raises ImportError.

As everywhere in this package, nothing is recorded for autograd: outputs do not require
grad, whatever the inputs do, and a program calls the gradients itself, as in a
torch.autograd.Function (examples/feed_forward.py).
"""
import ctypes

import torch

from ._binding import _check, _i64, _int, _p, _sz, lib
from ._mx import _Missing

try:
    from . import _fused_binding
except ImportError as e:
    _fused_binding = _Missing(e, "_fused_binding")

INT8_BLOCK = 32

# C prototypes, in the order of include/qgemm_fused.h.
PROTOTYPES = {
    "qgemm_a8w8_linear_workspace_bytes": ([_i64, _i64, _i64, _p, _i64, _p, _i64, _int, _int], _sz),
    "qgemm_a8w8_linear": ([_i64, _i64, _i64, _p, _i64, _p, _i64, _int, _p, _i64, _p, _i64, _p, _int, _p, _i64, _p, _int, _i64,
                           _p, _i64, _p, _i64, _p, _sz, _p], _int),
    "qgemm_a8w8_gated_workspace_bytes": ([_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _int, _int], _sz),
    "qgemm_a8w8_gated": ([_i64, _i64, _i64, _p, _i64, _p, _i64, _p, _i64, _int, _p, _i64, _p, _i64, _p, _i64, _int, _p, _int, _i64,
                          _p, _i64, _p, _i64, _p, _sz, _p], _int),
    "qgemm_a8w8_linear_grad_workspace_bytes": ([_i64, _i64, _i64, _p, _i64, _int, _int], _sz),
    "qgemm_a8w8_linear_grad": ([_i64, _i64, _i64, _p, _int, _i64, _p, _i64, _int, _p, _i64, _p, _i64, _p, _i64, _int, _p, _i64, _p,
                                _p, _sz, _p], _int),
    "qgemm_a8w8_gated_grad_workspace_bytes": ([_i64, _i64, _i64, _p, _i64, _p, _i64, _int], _sz),
    "qgemm_a8w8_gated_grad": ([_i64, _i64, _i64, _p, _int, _i64, _p, _i64, _p, _i64, _int, _p, _i64, _p, _i64, _p, _i64, _p, _i64,
                               _int, _p, _i64, _p, _sz, _p], _int),
    "int8_quantize": ([_i64, _i64, _p, _int, _i64, _int, _p, _i64, _p, _i64, _p], _int),
    "int8_dequantize": ([_i64, _i64, _p, _i64, _p, _i64, _int, _p, _int, _i64, _p], _int),
}
for _name, (_args, _res) in PROTOTYPES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes, _fn.restype = _args, _res


def _bind(library):
    """Hands the extension module the entry points of `library`."""
    _fused_binding.bind(_check, *(ctypes.cast(getattr(library, name), ctypes.c_void_p).value for name in PROTOTYPES))


if not isinstance(_fused_binding, _Missing):
    _bind(lib)


def qgemm_a8w8_linear(A, W, act_scale, weight_scale, bias=None, activation=None, residual=None, out_dtype=torch.float32,
                      b_trans=False, checkpoint=False, out=None):
    """out = act(z) + residual, rounded once, with z = ((float)(A @ W)_int32 *
    act_scale[m]) * weight_scale[n] + bias[n].

    A, W, act_scale, weight_scale, b_trans: as qgemm_a8w8.  bias: fp32 [N].
    activation: None (or "none"), "relu", "silu", "gelu" (with erf) or "gelu_tanh".
    residual: [M, N] of out_dtype; out may be the residual itself.  out_dtype:
    torch.float32, bfloat16 or float16.  With checkpoint=True returns (out, saved):
    saved = (codes int8 [M, N], scale fp32 [M, ceil(N / 32)]) holds z in int8 form by
    blocks of 32 columns, for qgemm_a8w8_linear_grad (which takes the upstream gradient in
    bf16 or fp16, whatever out_dtype was)."""
    return _fused_binding.linear(A, W, act_scale, weight_scale, bias, activation, residual, out_dtype, b_trans, checkpoint, out)


def qgemm_a8w8_gated(A, W_gate, W_up, act_scale, gate_scale, up_scale, activation="silu", out_dtype=torch.float32, b_trans=False,
                     checkpoint=False, out=None):
    """out = act(g) * u, rounded once, with g and u the A8W8 products of A with W_gate
    and W_up.

    A: int8 [M, K]; W_gate, W_up: int8 [K, N] (or [N, K] with b_trans=True);
    act_scale: fp32 [M], [M, 1] or scalar; gate_scale, up_scale: fp32 [N], [1, N] or
    scalar; activation, out_dtype: as qgemm_a8w8_linear.  With checkpoint=True
    returns (out, saved): saved = (codes int8 [2, M, N], scale fp32 [2, M,
    ceil(N / 32)]) holds g and u in int8 form by blocks of 32 columns, for
    qgemm_a8w8_gated_grad (which takes the upstream gradient in bf16 or fp16, whatever
    out_dtype was)."""
    return _fused_binding.gated(A, W_gate, W_up, act_scale, gate_scale, up_scale, activation, out_dtype, b_trans, checkpoint, out)


def qgemm_a8w8_linear_grad(dy, W, weight_scale, checkpoint=None, activation=None, b_trans=False, bias_grad=False):
    """Gradient of qgemm_a8w8_linear with respect to what A stands for, A * act_scale
    (straight through its rounding), the frozen weight in its forward layout:
    dx[m, k] = sum_n (dy act'(z) weight_scale)[m, n] W[k, n], z as the checkpoint holds it.

    dy: bf16 or fp16 [M, N]; checkpoint: the forward call's saved pair (not needed
    without an activation); activation: the forward call's, which the pair does not
    hold (None gives the gradient of the product alone).  Returns dx [M, K] of dy's dtype, or with bias_grad=True
    (dx, dbias): dbias fp32 [N].  The residual's gradient is dy itself.  The factors
    are held in 16-bit fixed point per row, sums over n are exact; results repeat bit
    for bit."""
    return _fused_binding.linear_grad(dy, W, weight_scale, checkpoint, activation, b_trans, bias_grad)


def qgemm_a8w8_gated_grad(dy, W_gate, W_up, gate_scale, up_scale, checkpoint, activation="silu", b_trans=False):
    """Gradient of qgemm_a8w8_gated, as qgemm_a8w8_linear_grad: dx[m, k] = sum_n (dy u
    act'(g) gate_scale)[m, n] W_gate[k, n] + (dy act(g) up_scale)[m, n] W_up[k, n], g and u as
    the checkpoint (the forward call's saved pair) holds them."""
    return _fused_binding.gated_grad(dy, W_gate, W_up, gate_scale, up_scale, checkpoint, activation, b_trans)


def int8_quantize(x, block=None):
    """x: fp32, bf16 or fp16 [..., n] -> (codes int8 of x's shape, scale fp32), x ~ codes *
    scale.  block None: one scale a row, [...]: the A and act_scale of the A8W8
    products.  block 32: one per 32 columns, [..., ceil(n / 32)].  A row (block) of zeros
    gives scale 1, one that holds a NaN or an infinity scale NaN and codes 0."""
    return _fused_binding.int8_quantize(x, block)


def int8_dequantize(codes, scale, out_dtype=torch.bfloat16, out=None):
    """The values that int8 codes stand for, codes * scale, rounded once to fp32, bf16 or
    fp16.  codes, scale: as int8_quantize returns them, or a checkpoint's."""
    return _fused_binding.int8_dequantize(codes, scale, out_dtype, out)

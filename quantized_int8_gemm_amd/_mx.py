"""ctypes binding of the calls of include/qgemm_mx.h: the RMS norm with its
quantised outputs and its gradient, the MX quantiser and the MX product.

As in the binding of the integer products, each function checks dtypes
(TypeError) and shapes (ValueError), allocates its outputs with torch and
calls the C entry point of the same name on torch's current stream; all
arithmetic runs in the HIP kernels.
"""
import ctypes

import torch

from ._binding import (QG_BF16, QG_FP32, QG_INT8, _check, _f32, _i64, _int, _need, _on_gpu, _p, _sz, lib)

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

_FLOATS = {torch.float32: QG_FP32, torch.bfloat16: QG_BF16, torch.float16: QG_FP16}
_FORMATS = {"mxfp8": QG_MXFP8, "mxfp4": QG_MXFP4}
# element types of the codes: e4m3 as torch has it, e2m1 packed in pairs
_CODES = {torch.float8_e4m3fn: QG_MXFP8, torch.uint8: QG_MXFP4}

# The smallest calls take a few microseconds on the GPU, so what they do here
# counts: tensors are looked at through few calls, new outputs are not looked
# at again, and the stream and the current device come from torch's C
# functions, which cost a tenth of torch.cuda's own.
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _kind(t, table, name):
    """The library's number for t's dtype, one of `table`."""
    try:
        return table[t.dtype]
    except (AttributeError, KeyError):
        _need(t, tuple(table), name)
        raise


def _matrix(t, name):
    """(rows, columns, row stride in elements) of t seen as a matrix of its
    last dimension; more than two dimensions have to lie like one matrix."""
    shape = t.shape
    if len(shape) == 2:
        rows, n = shape
        stride, step = t.stride()
        if (step == 1 or n <= 1) and (rows <= 1 or stride >= n):
            return rows, n, stride if rows > 1 else n
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    n = shape[-1]
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    rows, stride = 1, None
    for size, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * rows:
            raise ValueError(f"the rows of {name} must lie at one stride")
        rows *= size
    if stride is None:
        stride = n
    if rows > 1 and stride < n:
        raise ValueError(f"the rows of {name} overlap")
    return rows, n, stride


def _device(t, *others):
    """The GPU that all the tensors are on (None: no tensor)."""
    index = t.get_device()
    for o in others:
        if o is not None and o.get_device() != index:
            index = -1
    if index < 0:
        _on_gpu(t, *(o for o in others if o is not None))
    return t.device


def _at(t):
    return None if t is None else t.data_ptr()


def _like(t, name, shape, dtype):
    """`t` checked against what it has to be."""
    _need(t, (dtype,), name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    return t


def _weight(weight, n, dtype):
    if weight.__class__ is not torch.Tensor or weight.dtype is not dtype:
        _need(weight, (dtype, torch.float32), "weight")
    if tuple(weight.shape) != (n,):
        raise ValueError(f"weight has shape {tuple(weight.shape)}; expected ({n},)")
    return weight.contiguous()


def _launch(dev, fn, *args):
    """Calls a C entry point with the tensors' device current."""
    index = dev.index
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(index))
    if st:
        _check(st, fn.__name__)


def _norm_inputs(x, weight):
    """x's number of its dtype, rows, columns and row stride, and the weight."""
    kind = _kind(x, _FLOATS, "x")
    rows, n, ldx = _matrix(x, "x")
    if n == 0:
        raise ValueError("x must have at least one column")
    return kind, rows, n, ldx, _weight(weight, n, x.dtype)


def _norm(x, inputs, eps, residual, residual_out, format, out, ldo, block_scale, lds, row_scale, dev):
    kind, rows, n, ldx, weight = inputs
    h, ldr, ldh = None, 0, 0
    if residual is not None:
        if residual.dtype is not x.dtype or residual.shape != x.shape:
            raise ValueError(f"residual has shape {tuple(residual.shape)}; x has {tuple(x.shape)}")
        ldr = _matrix(residual, "residual")[2]
        if residual_out is None:
            h, ldh = torch.empty(x.shape, dtype=x.dtype, device=dev), n
        else:
            h = _like(residual_out, "residual_out", x.shape, x.dtype)
            ldh = _matrix(h, "residual_out")[2]
            _device(x, h)
    _launch(dev, lib.rms_norm, rows, n, x.data_ptr(), kind, ldx, _at(residual), ldr, weight.data_ptr(),
            _FLOATS[weight.dtype], float(eps), _at(h), ldh, out.data_ptr(), format, ldo, _at(block_scale), lds,
            row_scale.data_ptr())
    return h


def _norm_device(x, weight, residual, residual_out):
    """The device of a norm's inputs, the residual's dtype checked."""
    if residual is not None:
        _need(residual, (x.dtype,), "residual")
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    return _device(x, weight, residual)


def rms_norm(x, weight, eps=1e-6, residual=None, out_dtype=None, out=None, residual_out=None):
    """y = h / sqrt(mean(h^2) + eps) * weight along the last dimension, with
    h = x + residual (h = x without one).

    x: fp32, bf16 or fp16 [..., n] (unit column stride, rows at one stride);
    weight: [n] of x's dtype or fp32; residual: x's shape and dtype.
    out_dtype: x's dtype (default) or torch.float32.  Returns (y, rstd), and h
    as a third where a residual is given: rstd is fp32 [...], 1 / sqrt(...), as
    rms_norm_grad takes it.  residual_out: the tensor to write h to; it may be
    x or residual itself."""
    inputs = _norm_inputs(x, weight)
    if out_dtype is None:
        out_dtype = x.dtype
    elif out_dtype not in (x.dtype, torch.float32):
        raise TypeError("out_dtype must be x's dtype or torch.float32")
    dev = _norm_device(x, inputs[4], residual, residual_out)
    if out is None:
        y, ldo = torch.empty(x.shape, dtype=out_dtype, device=dev), inputs[2]
    else:
        y = _like(out, "out", x.shape, out_dtype)
        ldo = _matrix(y, "out")[2]
        _device(x, y)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    h = _norm(x, inputs, eps, residual, residual_out, _FLOATS[out_dtype], y, ldo, None, 0, rstd, dev)
    return (y, rstd) if h is None else (y, rstd, h)


def rms_norm_quantize(x, weight, eps=1e-6, residual=None, format="int8", residual_out=None):
    """The same norm with a quantised output, in one pass over x.

    format "int8": returns (q, scale[, h]): q int8 of x's shape, scale fp32
    [...], y ~ q * scale[..., None]: the A and act_scale of qgemm_a8w8.
    format "mxfp8" or "mxfp4": returns (codes, block_scale, act_scale[, h]):
    h * weight in MX form (as mx_quantize returns it) and fp32 act_scale
    [...] = 1 / sqrt(mean(h^2) + eps): the A, a_scale and act_scale of
    mx_matmul.  Other arguments as rms_norm."""
    inputs = _norm_inputs(x, weight)
    n, lead = inputs[2], x.shape[:-1]
    dev = _norm_device(x, inputs[4], residual, residual_out)
    row_scale = torch.empty(lead, dtype=torch.float32, device=dev)
    if format == "int8":
        q = torch.empty(x.shape, dtype=torch.int8, device=dev)
        h = _norm(x, inputs, eps, residual, residual_out, QG_INT8, q, n, None, 0, row_scale, dev)
        return (q, row_scale) if h is None else (q, row_scale, h)
    kind, codes, ldo, scale, lds = _mx_outputs(lead, n, format, dev)
    h = _norm(x, inputs, eps, residual, residual_out, kind, codes, ldo, scale, lds, row_scale, dev)
    return (codes, scale, row_scale) if h is None else (codes, scale, row_scale, h)


def rms_norm_grad(dy, h, weight, rstd, dh=None):
    """Gradient of rms_norm (and, straight through the rounding, of
    rms_norm_quantize): returns (dx, dweight).

    dy, h: fp32, bf16 or fp16 [..., n] of one dtype, h as the norm saw it (its
    third output, or x without a residual); weight: [n]; rstd: fp32 [...] from
    rms_norm; dh: the gradient that reaches h from elsewhere, added to dx.
    dx, of h's shape and dtype, is the gradient of x and of the residual alike;
    dweight has weight's dtype.  Results repeat bit for bit."""
    kind = _kind(h, _FLOATS, "h")
    _need(dy, (h.dtype,), "dy")
    rows, n, ldh = _matrix(h, "h")
    if n == 0:
        raise ValueError("h must have at least one column")
    if dy.shape != h.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}; h has {tuple(h.shape)}")
    ldy = _matrix(dy, "dy")[2]
    weight = _weight(weight, n, h.dtype)
    _need(rstd, (torch.float32,), "rstd")
    if rstd.shape != h.shape[:-1]:
        raise ValueError(f"rstd has shape {tuple(rstd.shape)}; expected {tuple(h.shape[:-1])}")
    rstd = rstd.contiguous()
    lddh = 0
    if dh is not None:
        _need(dh, (h.dtype,), "dh")
        if dh.shape != h.shape:
            raise ValueError(f"dh has shape {tuple(dh.shape)}; h has {tuple(h.shape)}")
        lddh = _matrix(dh, "dh")[2]
    dev = _device(h, dy, weight, rstd, dh)
    dx = torch.empty(h.shape, dtype=h.dtype, device=dev)
    dweight = torch.empty(n, dtype=weight.dtype, device=dev)
    need = lib.rms_norm_grad_workspace_bytes(rows, n)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _launch(dev, lib.rms_norm_grad, rows, n, dy.data_ptr(), kind, ldy, h.data_ptr(), ldh, weight.data_ptr(),
            _FLOATS[weight.dtype], rstd.data_ptr(), _at(dh), lddh, dx.data_ptr(), n, dweight.data_ptr(), _at(ws), need)
    return dx, dweight


def _mx_outputs(lead, n, format, dev):
    """The library's number for the format, codes, their row stride in bytes,
    scale bytes whose rows start at multiples of 16 bytes, and their stride."""
    kind = _FORMATS.get(format)
    if kind is None:
        raise ValueError(f"unknown format {format!r}; expected one of {sorted(_FORMATS)}")
    blocks = -(-n // MX_BLOCK)
    lds = (blocks + 15) // 16 * 16
    if kind == QG_MXFP8:
        width = blocks * 32
        codes = torch.empty((*lead, width), dtype=torch.float8_e4m3fn, device=dev)
    else:
        width = blocks * 16
        codes = torch.empty((*lead, width), dtype=torch.uint8, device=dev)
    scale = torch.empty((*lead, lds), dtype=torch.uint8, device=dev)
    return kind, codes, width, scale if lds == blocks else scale.narrow(-1, 0, blocks), lds


def mx_quantize(x, format="mxfp4"):
    """x: fp32, bf16 or fp16 [..., n] -> (codes, scale) in MX form.

    Blocks of 32 along the last dimension (filled up with zeros to B whole
    blocks) share a power-of-two scale.  codes: float8_e4m3fn [..., 32 B]
    ("mxfp8"), or uint8 [..., 16 B] with two e2m1 values to a byte, the even
    column in the low half ("mxfp4").  scale: uint8 [..., B], 2^(scale - 127),
    255 for a block that holds a NaN or an infinity; its rows start at
    multiples of 16 bytes."""
    dtype = _kind(x, _FLOATS, "x")
    rows, n, ldx = _matrix(x, "x")
    if n == 0:
        raise ValueError("x must have at least one column")
    dev = _device(x)
    kind, codes, ldc, scale, lds = _mx_outputs(x.shape[:-1], n, format, dev)
    _launch(dev, lib.mx_quantize, rows, n, x.data_ptr(), dtype, ldx, codes.data_ptr(), kind, ldc, scale.data_ptr(), lds)
    return codes, scale


def _mx_operand(codes, scale, name):
    """(format, rows, K, code stride in bytes, scale stride) of one MX operand."""
    kind = _kind(codes, _CODES, name)
    if scale.__class__ is not torch.Tensor or scale.dtype is not torch.uint8:
        _need(scale, (torch.uint8,), name + " scale")
    rows, width, ldc = _matrix(codes, name)
    srows, blocks, lds = _matrix(scale, name + " scale")
    per = 32 if kind == QG_MXFP8 else 16
    if width == 0 or width % per:
        raise ValueError(f"{name} has {width} code columns; expected whole blocks of {per}")
    if blocks * per != width or codes.shape[:-1] != scale.shape[:-1]:
        raise ValueError(f"the scale of {name} has shape {tuple(scale.shape)}; "
                         f"expected {(*codes.shape[:-1], width // per)}")
    return kind, rows, blocks * MX_BLOCK, ldc, lds


def mx_dequantize(codes, scale, out_dtype=torch.bfloat16, columns=None, out=None):
    """The values an MX tensor stands for: fp32, bf16 or fp16 [..., columns]
    (default: all 32 B of them).  codes, scale: as mx_quantize returns them."""
    kind, rows, K, ldc, lds = _mx_operand(codes, scale, "codes")
    dtype = _FLOATS.get(out_dtype)
    if dtype is None:
        raise TypeError(f"out_dtype must be one of {tuple(_FLOATS)}")
    n = K if columns is None else int(columns)
    if not K - MX_BLOCK < n <= K:
        raise ValueError(f"columns = {n} does not fill {K // MX_BLOCK} blocks")
    dev = _device(codes, scale)
    shape = (*codes.shape[:-1], n)
    if out is None:
        out, ldo = torch.empty(shape, dtype=out_dtype, device=dev), n
    else:
        ldo = _matrix(_like(out, "out", shape, out_dtype), "out")[2]
        _device(codes, out)
    _launch(dev, lib.mx_dequantize, rows, n, codes.data_ptr(), kind, ldc, scale.data_ptr(), lds, out.data_ptr(), dtype, ldo)
    return out


def _rows_readable(scale, rows, lds):
    """Whether every scale row can be read to the end of its last 4-byte word."""
    blocks = scale.shape[-1]
    if blocks % 4 == 0:
        return True
    last = scale.storage_offset() + (rows - 1) * lds
    return scale.untyped_storage().nbytes() - last >= (blocks + 3) // 4 * 4


def mx_matmul(A, a_scale, W, w_scale, act_scale=None, out_dtype=torch.float32, out=None):
    """out[m, n] = act_scale[m] * sum_k A[m, k] * W[n, k] over MX operands.

    A: float8_e4m3fn [M, K] or packed e2m1 uint8 [M, K/2] with a_scale uint8
    [M, K/32]; W: packed e2m1 uint8 [N, K/2] with w_scale uint8 [N, K/32] (both
    as mx_quantize returns them); act_scale: fp32 [M], [M, 1], a scalar, or
    None for 1.  out_dtype: torch.float32, bfloat16 or float16.  Fast kernels
    need code rows at multiples of 16 bytes and scale rows at multiples of 4,
    as mx_quantize and rms_norm_quantize lay them out; other layouts run a
    slower one."""
    for t, name in ((A, "A"), (W, "W")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 2:
            raise ValueError(f"{name} must be 2-D")
    if W.dtype is not torch.uint8:
        _need(W, (torch.uint8,), "W")
    dtype = _FLOATS.get(out_dtype)
    if dtype is None:
        raise TypeError(f"out_dtype must be one of {tuple(_FLOATS)}")
    kind, M, K, lda, ldas = _mx_operand(A, a_scale, "A")
    _, N, K2, ldw, ldws = _mx_operand(W, w_scale, "W")
    if K != K2:
        raise ValueError(f"inner dimensions differ: A has {K} columns, W has {K2}")
    if act_scale is not None:
        _need(act_scale, (torch.float32,), "act_scale")
        shape = tuple(act_scale.shape)
        if shape in ((), (1,), (1, 1)) and M != 1:
            act_scale = act_scale.reshape(1).expand(M)
        elif shape not in ((), (1,), (M,), (M, 1)):
            raise ValueError(f"act_scale of shape {shape} is not [M], [M,1] or scalar (M={M})")
        if not act_scale.is_contiguous():
            act_scale = act_scale.contiguous()
    dev = _device(A, a_scale, W, w_scale, act_scale)
    if out is None:
        out, ldo = torch.empty((M, N), dtype=out_dtype, device=dev), N
    else:
        ldo = _matrix(_like(out, "out", (M, N), out_dtype), "out")[2]
        _device(A, out)
    if M == 0 or N == 0:
        return out
    padded = _rows_readable(a_scale, M, ldas) and _rows_readable(w_scale, N, ldws)
    _launch(dev, lib.mx_matmul, M, N, K, A.data_ptr(), kind, lda, a_scale.data_ptr(), ldas, W.data_ptr(), ldw,
            w_scale.data_ptr(), ldws, padded, _at(act_scale), out.data_ptr(), dtype, ldo)
    return out

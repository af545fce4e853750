"""ctypes binding of the calls of include/qgemm_mx.h: the RMS norm with its
quantised outputs and its gradient, the MX quantiser and the MX product.

As in the binding of the integer products, each function checks dtypes
(TypeError) and shapes (ValueError), allocates its outputs with torch and
calls the C entry point of the same name on torch's current stream; all
arithmetic runs in the HIP kernels.
"""
import ctypes

import torch

from ._binding import (QG_BF16, QG_FP32, QG_INT8, _check, _f32, _i64, _int, _need, _on_gpu, _p, _ptr, _stream, _sz, lib)

QG_FP16, QG_MXFP8, QG_MXFP4 = 5, 6, 7
MX_BLOCK = 32

# C prototypes, in the order of include/qgemm_mx.h.
PROTOTYPES = {
    "rms_norm": ([_i64, _i64, _p, _int, _i64, _p, _i64, _p, _int, _f32, _p, _i64, _p, _int, _i64, _p, _i64, _p, _p], _int),
    "rms_norm_grad_workspace_bytes": ([_i64, _i64], _sz),
    "rms_norm_grad": ([_i64, _i64, _p, _int, _i64, _p, _i64, _p, _int, _p, _p, _i64, _p, _i64, _p, _p, _sz, _p], _int),
    "mx_quantize": ([_i64, _i64, _p, _int, _i64, _p, _int, _i64, _p, _i64, _p], _int),
    "mx_dequantize": ([_i64, _i64, _p, _int, _i64, _p, _i64, _p, _int, _i64, _p], _int),
    "mx_matmul_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "mx_matmul": ([_i64, _i64, _i64, _p, _int, _i64, _p, _i64, _p, _i64, _p, _i64, _int, _p, _p, _int, _i64, _p, _sz,
                   _p], _int),
}
for _name, (_args, _res) in PROTOTYPES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes, _fn.restype = _args, _res

_FLOATS = {torch.float32: QG_FP32, torch.bfloat16: QG_BF16, torch.float16: QG_FP16}
_FORMATS = {"mxfp8": QG_MXFP8, "mxfp4": QG_MXFP4}
# element types of the codes: e4m3 as torch has it, e2m1 packed in pairs
_CODES = {torch.float8_e4m3fn: QG_MXFP8, torch.uint8: QG_MXFP4}


def _matrix(t, name):
    """(rows, columns, row stride in elements) of t seen as a matrix of its
    last dimension; more than two dimensions have to lie like one matrix."""
    if t.dim() == 0:
        raise ValueError(f"{name} must have at least one dimension")
    n = t.shape[-1]
    if n > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    rows, stride = 1, None
    for size, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
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


def _like(t, name, shape, dtype, dev):
    """`t` checked against what it has to be, or a new tensor of that kind."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, (dtype,), name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    return t


def _scale_rows(lead, blocks, dev):
    """[*lead, blocks] scale bytes whose rows start at multiples of 16 bytes."""
    return torch.empty((*lead, (blocks + 15) // 16 * 16), dtype=torch.uint8, device=dev)[..., :blocks]


def _weight(weight, n, dtype):
    _need(weight, (dtype, torch.float32), "weight")
    if tuple(weight.shape) != (n,):
        raise ValueError(f"weight has shape {tuple(weight.shape)}; expected ({n},)")
    return weight.contiguous()


def _launch(dev, fn, *args):
    """Calls a C entry point with the tensors' device current."""
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    _check(st, fn.__name__)


def _norm(x, weight, eps, residual, residual_out, format, out, out_dtype, block_scale, row_scale):
    rows, n, ldx = _matrix(x, "x")
    ts = [x, weight] + ([residual] if residual is not None else [])
    h, ldr, ldh = None, 0, 0
    if residual is not None:
        _need(residual, (x.dtype,), "residual")
        if residual.shape != x.shape:
            raise ValueError(f"residual has shape {tuple(residual.shape)}; x has {tuple(x.shape)}")
        _, _, ldr = _matrix(residual, "residual")
        h = _like(residual_out, "residual_out", x.shape, x.dtype, x.device)
        _, _, ldh = _matrix(h, "residual_out")
        ts.append(h)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    dev = _on_gpu(*ts, out, row_scale)
    _, _, ldo = _matrix(out, "out")
    lds = _matrix(block_scale, "block_scale")[2] if block_scale is not None else 0
    _launch(dev, lib.rms_norm, rows, n, _ptr(x), _FLOATS[x.dtype], ldx, _ptr(residual), ldr, _ptr(weight),
            _FLOATS[weight.dtype], float(eps), _ptr(h), ldh, _ptr(out), format, ldo, _ptr(block_scale), lds,
            _ptr(row_scale))
    return h


def _norm_inputs(x, weight):
    _need(x, tuple(_FLOATS), "x")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise ValueError("x must have at least one column")
    return _weight(weight, x.shape[-1], x.dtype)


def rms_norm(x, weight, eps=1e-6, residual=None, out_dtype=None, out=None, residual_out=None):
    """y = h / sqrt(mean(h^2) + eps) * weight along the last dimension, with
    h = x + residual (h = x without one).

    x: fp32, bf16 or fp16 [..., n] (unit column stride, rows at one stride);
    weight: [n] of x's dtype or fp32; residual: x's shape and dtype.
    out_dtype: x's dtype (default) or torch.float32.  Returns (y, rstd), and h
    as a third where a residual is given: rstd is fp32 [...], 1 / sqrt(...), as
    rms_norm_grad takes it.  residual_out: the tensor to write h to; it may be
    x or residual itself."""
    weight = _norm_inputs(x, weight)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    if out_dtype not in (x.dtype, torch.float32):
        raise TypeError("out_dtype must be x's dtype or torch.float32")
    y = _like(out, "out", x.shape, out_dtype, x.device)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    h = _norm(x, weight, eps, residual, residual_out, _FLOATS[out_dtype], y, out_dtype, None, rstd)
    return (y, rstd) if h is None else (y, rstd, h)


def rms_norm_quantize(x, weight, eps=1e-6, residual=None, format="int8", residual_out=None):
    """The same norm with a quantised output, in one pass over x.

    format "int8": returns (q, scale[, h]): q int8 of x's shape, scale fp32
    [...], y ~ q * scale[..., None]: the A and act_scale of qgemm_a8w8.
    format "mxfp8" or "mxfp4": returns (codes, block_scale, act_scale[, h]):
    h * weight in MX form (as mx_quantize returns it) and fp32 act_scale
    [...] = 1 / sqrt(mean(h^2) + eps): the A, a_scale and act_scale of
    mx_matmul.  Other arguments as rms_norm."""
    weight = _norm_inputs(x, weight)
    n, lead, dev = x.shape[-1], x.shape[:-1], x.device
    row_scale = torch.empty(lead, dtype=torch.float32, device=dev)
    if format == "int8":
        q = torch.empty(x.shape, dtype=torch.int8, device=dev)
        h = _norm(x, weight, eps, residual, residual_out, QG_INT8, q, torch.int8, None, row_scale)
        return (q, row_scale) if h is None else (q, row_scale, h)
    codes, scale = _mx_outputs(lead, n, format, dev)
    h = _norm(x, weight, eps, residual, residual_out, _FORMATS[format], codes, codes.dtype, scale, row_scale)
    return (codes, scale, row_scale) if h is None else (codes, scale, row_scale, h)


def rms_norm_grad(dy, h, weight, rstd, dh=None):
    """Gradient of rms_norm (and, straight through the rounding, of
    rms_norm_quantize): returns (dx, dweight).

    dy, h: fp32, bf16 or fp16 [..., n] of one dtype, h as the norm saw it (its
    third output, or x without a residual); weight: [n]; rstd: fp32 [...] from
    rms_norm; dh: the gradient that reaches h from elsewhere, added to dx.
    dx, of h's shape and dtype, is the gradient of x and of the residual alike;
    dweight has weight's dtype.  Results repeat bit for bit."""
    _need(h, tuple(_FLOATS), "h")
    _need(dy, (h.dtype,), "dy")
    if h.dim() == 0 or h.shape[-1] == 0:
        raise ValueError("h must have at least one column")
    if dy.shape != h.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}; h has {tuple(h.shape)}")
    rows, n, ldh = _matrix(h, "h")
    _, _, ldy = _matrix(dy, "dy")
    weight = _weight(weight, n, h.dtype)
    _need(rstd, (torch.float32,), "rstd")
    if rstd.shape != h.shape[:-1]:
        raise ValueError(f"rstd has shape {tuple(rstd.shape)}; expected {tuple(h.shape[:-1])}")
    rstd = rstd.contiguous()
    ts, lddh = [dy, h, weight, rstd], 0
    if dh is not None:
        _need(dh, (h.dtype,), "dh")
        if dh.shape != h.shape:
            raise ValueError(f"dh has shape {tuple(dh.shape)}; h has {tuple(h.shape)}")
        _, _, lddh = _matrix(dh, "dh")
        ts.append(dh)
    dev = _on_gpu(*ts)
    dx = torch.empty(h.shape, dtype=h.dtype, device=dev)
    dweight = torch.empty(n, dtype=weight.dtype, device=dev)
    need = lib.rms_norm_grad_workspace_bytes(rows, n)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    _launch(dev, lib.rms_norm_grad, rows, n, _ptr(dy), _FLOATS[h.dtype], ldy, _ptr(h), ldh, _ptr(weight),
            _FLOATS[weight.dtype], _ptr(rstd), _ptr(dh), lddh, _ptr(dx), n, _ptr(dweight), _ptr(ws) if need else None,
            need)
    return dx, dweight


def _mx_outputs(lead, n, format, dev):
    if format not in _FORMATS:
        raise ValueError(f"unknown format {format!r}; expected one of {sorted(_FORMATS)}")
    blocks = -(-n // MX_BLOCK)
    if format == "mxfp8":
        codes = torch.empty((*lead, blocks * 32), dtype=torch.float8_e4m3fn, device=dev)
    else:
        codes = torch.empty((*lead, blocks * 16), dtype=torch.uint8, device=dev)
    return codes, _scale_rows(lead, blocks, dev)


def mx_quantize(x, format="mxfp4"):
    """x: fp32, bf16 or fp16 [..., n] -> (codes, scale) in MX form.

    Blocks of 32 along the last dimension (filled up with zeros to B whole
    blocks) share a power-of-two scale.  codes: float8_e4m3fn [..., 32 B]
    ("mxfp8"), or uint8 [..., 16 B] with two e2m1 values to a byte, the even
    column in the low half ("mxfp4").  scale: uint8 [..., B], 2^(scale - 127),
    255 for a block that holds a NaN or an infinity; its rows start at
    multiples of 16 bytes."""
    _need(x, tuple(_FLOATS), "x")
    rows, n, ldx = _matrix(x, "x")
    if n == 0:
        raise ValueError("x must have at least one column")
    dev = _on_gpu(x)
    codes, scale = _mx_outputs(x.shape[:-1], n, format, dev)
    _launch(dev, lib.mx_quantize, rows, n, _ptr(x), _FLOATS[x.dtype], ldx, _ptr(codes), _FORMATS[format],
            codes.shape[-1], _ptr(scale), _matrix(scale, "scale")[2])
    return codes, scale


def _mx_operand(codes, scale, name):
    """(rows, K, code stride in bytes, scale stride) of one MX operand."""
    _need(codes, tuple(_CODES), name)
    _need(scale, (torch.uint8,), name + " scale")
    rows, width, ldc = _matrix(codes, name)
    srows, blocks, lds = _matrix(scale, name + " scale")
    per = 32 if codes.dtype == torch.float8_e4m3fn else 16
    if width == 0 or width % per:
        raise ValueError(f"{name} has {width} code columns; expected whole blocks of {per}")
    if codes.shape[:-1] != scale.shape[:-1] or blocks != width // per:
        raise ValueError(f"the scale of {name} has shape {tuple(scale.shape)}; "
                         f"expected {(*codes.shape[:-1], width // per)}")
    return rows, blocks * MX_BLOCK, ldc, lds


def mx_dequantize(codes, scale, out_dtype=torch.bfloat16, columns=None, out=None):
    """The values an MX tensor stands for: fp32, bf16 or fp16 [..., columns]
    (default: all 32 B of them).  codes, scale: as mx_quantize returns them."""
    rows, K, ldc, lds = _mx_operand(codes, scale, "codes")
    if out_dtype not in _FLOATS:
        raise TypeError(f"out_dtype must be one of {tuple(_FLOATS)}")
    n = K if columns is None else int(columns)
    if not K - MX_BLOCK < n <= K:
        raise ValueError(f"columns = {n} does not fill {K // MX_BLOCK} blocks")
    dev = _on_gpu(codes, scale)
    out = _like(out, "out", (*codes.shape[:-1], n), out_dtype, dev)
    _on_gpu(codes, out)
    _launch(dev, lib.mx_dequantize, rows, n, _ptr(codes), _CODES[codes.dtype], ldc, _ptr(scale), lds, _ptr(out),
            _FLOATS[out_dtype], _matrix(out, "out")[2])
    return out


_workspaces = {}
_outgrown = []   # a captured graph may still use these


def _workspace(dev, nbytes):
    """A zero-filled workspace per (device, stream); the library leaves its
    tickets at zero.  While a graph is captured nothing new is kept: the fill
    would run with the graph's replays only."""
    if nbytes == 0:
        return None
    key = (dev, torch.cuda.current_stream(dev).cuda_stream)
    ws = _workspaces.get(key)
    if ws is not None and ws.numel() >= nbytes:
        return ws
    if torch.cuda.is_current_stream_capturing():
        return torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    if ws is not None:
        _outgrown.append(ws)
        nbytes = max(nbytes, 2 * ws.numel())
    _workspaces[key] = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    return _workspaces[key]


def mx_matmul_workspace_bytes(M, N, K):
    """Bytes of workspace with which mx_matmul divides K among workgroups."""
    return int(lib.mx_matmul_workspace_bytes(M, N, K))


def _rows_readable(scale, rows, lds):
    """Whether every scale row can be read to the end of its last 4-byte word."""
    last = scale.storage_offset() + (rows - 1) * lds
    return scale.untyped_storage().nbytes() - last >= (scale.shape[-1] + 3) // 4 * 4


def mx_matmul(A, a_scale, W, w_scale, act_scale=None, out_dtype=torch.float32, out=None, workspace=None):
    """out[m, n] = act_scale[m] * sum_k A[m, k] * W[n, k] over MX operands.

    A: float8_e4m3fn [M, K] or packed e2m1 uint8 [M, K/2] with a_scale uint8
    [M, K/32]; W: packed e2m1 uint8 [N, K/2] with w_scale uint8 [N, K/32] (both
    as mx_quantize returns them); act_scale: fp32 [M], [M, 1], a scalar, or
    None for 1.  out_dtype: torch.float32, bfloat16 or float16.  Fast kernels
    need code rows at multiples of 16 bytes and scale rows at multiples of 4,
    as mx_quantize and rms_norm_quantize lay them out; other layouts run a
    slower one.  workspace: None (a cached, zeroed buffer per device and
    stream) or a zero-filled uint8 tensor of at least
    mx_matmul_workspace_bytes(M, N, K) bytes."""
    for t, name in ((A, "A"), (W, "W")):
        _need(t, tuple(_CODES) if name == "A" else (torch.uint8,), name)
        if t.dim() != 2:
            raise ValueError(f"{name} must be 2-D")
    if out_dtype not in _FLOATS:
        raise TypeError(f"out_dtype must be one of {tuple(_FLOATS)}")
    M, K, lda, ldas = _mx_operand(A, a_scale, "A")
    N, K2, ldw, ldws = _mx_operand(W, w_scale, "W")
    if K != K2:
        raise ValueError(f"inner dimensions differ: A has {K} columns, W has {K2}")
    ts = [A, a_scale, W, w_scale]
    if act_scale is not None:
        _need(act_scale, (torch.float32,), "act_scale")
        if act_scale.dim() == 0 or tuple(act_scale.shape) in ((1,), (1, 1)):
            act_scale = act_scale.reshape(1).expand(M)
        elif tuple(act_scale.shape) not in ((M,), (M, 1)):
            raise ValueError(f"act_scale of shape {tuple(act_scale.shape)} is not [M], [M,1] or scalar (M={M})")
        act_scale = act_scale.reshape(-1).contiguous()
        ts.append(act_scale)
    dev = _on_gpu(*ts)
    out = _like(out, "out", (M, N), out_dtype, dev)
    _on_gpu(A, out)
    if M == 0 or N == 0:
        return out
    if workspace is None:
        workspace = _workspace(dev, mx_matmul_workspace_bytes(M, N, K))
    else:
        _need(workspace, (torch.uint8, torch.int8), "workspace")
        _on_gpu(A, workspace)
    padded = _rows_readable(a_scale, M, ldas) and _rows_readable(w_scale, N, ldws)
    _launch(dev, lib.mx_matmul, M, N, K, _ptr(A), _CODES[A.dtype], lda, _ptr(a_scale), ldas, _ptr(W), ldw,
            _ptr(w_scale), ldws, int(padded), _ptr(act_scale), _ptr(out), _FLOATS[out_dtype],
            _matrix(out, "out")[2], _ptr(workspace), 0 if workspace is None else workspace.numel())
    return out

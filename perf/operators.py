"""The operators measured beside the quantised products: the root-mean-square
norm with its residual addition and quantised outputs, its gradient, the
microscaled (MX) quantiser and the MX matrix product.

``run`` computes a case in plain torch operations, or, with ``own`` true,
through the library.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
FORMATS = ("int8", "mxfp8", "mxfp4", "same")


def listed():
    return [
        # the norm ahead of a quantised projection for one generated token
        {"name": "norm_int8_1x4096", "op": "norm", "rows": 1, "n": 4096, "type": "bf16", "residual": True, "format": "int8"},
        # the same over a long prompt's tokens
        {"name": "norm_int8_8192x8192", "op": "norm", "rows": 8192, "n": 8192, "type": "bf16", "residual": True, "format": "int8"},
        # a ragged batch with a width that ends inside a block, to MXFP8
        {"name": "norm_mxfp8_1537x5000", "op": "norm", "rows": 1537, "n": 5000, "type": "fp16", "residual": False, "format": "mxfp8"},
        # the backward pass of a training step, the residual branch's gradient joined
        {"name": "grad_8192x4096", "op": "grad", "rows": 8192, "n": 4096, "type": "bf16", "residual": True},
        # the same in fp32, as the W8A32 input gradient gives it, at a small odd size
        {"name": "grad_fp32_1000x1000", "op": "grad", "rows": 1000, "n": 1000, "type": "fp32", "residual": False},
        # a weight matrix through MXFP4 and back, as quantisation-aware training reads it
        {"name": "quantize_mxfp4_8192x8192", "op": "quantize", "rows": 8192, "n": 8192, "type": "bf16", "format": "mxfp4"},
        # the inner activations of a few decoded tokens, to MXFP8
        {"name": "quantize_mxfp8_16x8192", "op": "quantize", "rows": 16, "n": 8192, "type": "fp32", "format": "mxfp8"},
        # one generated token: MXFP8 activations, a streamed MXFP4 weight
        {"name": "matmul_a8_1x8192x8192", "op": "matmul", "m": 1, "n": 8192, "k": 8192, "a": "mxfp8", "scaled": True, "out": "bf16"},
        # a batch of decoding sequences, MXFP4 on both sides
        {"name": "matmul_a4_16x8192x8192", "op": "matmul", "m": 16, "n": 8192, "k": 8192, "a": "mxfp4", "scaled": True, "out": "bf16"},
        # a short prompt against a weight of odd height
        {"name": "matmul_a8_300x5001x4096", "op": "matmul", "m": 300, "n": 5001, "k": 4096, "a": "mxfp8", "scaled": False, "out": "fp32"},
        # a prompt, MXFP8 activations
        {"name": "matmul_a8_4096x4096x4096", "op": "matmul", "m": 4096, "n": 4096, "k": 4096, "a": "mxfp8", "scaled": True, "out": "bf16"},
        # the largest product, MXFP4 on both sides
        {"name": "matmul_a4_8192x8192x8192", "op": "matmul", "m": 8192, "n": 8192, "k": 8192, "a": "mxfp4", "scaled": True, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("norm", "grad", "quantize", "matmul", "matmul"))
    if op == "matmul":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 16, 8192), "k": -(-_log(rng, 32, 8192) // BLOCK) * BLOCK,
                "a": rng.choice(("mxfp4", "mxfp8")), "scaled": rng.random() < 0.5, "out": rng.choice(("bf16", "fp16", "fp32"))}
    rows, n = _log(rng, 1, 16384), _log(rng, 64, 16384)
    rows = max(1, min(rows, 8192 * 4096 // n))
    case = {"op": op, "rows": rows, "n": n, "type": rng.choice(tuple(TYPES))}
    if op == "norm":
        case.update(residual=rng.random() < 0.5, format=rng.choice(FORMATS))
    elif op == "grad":
        case.update(residual=rng.random() < 0.5)
    else:
        case.update(format=rng.choice(("mxfp8", "mxfp4")))
    return case


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(rows, n, dtype, g):
    """Hidden states: normal, with a few channels that are far larger, as trained models have them."""
    x = torch.randn(rows, n, generator=g, device=DEV)
    loud = torch.rand(n, generator=g, device=DEV) < 0.004
    return (x * torch.where(loud, 12.0, 1.0)).to(dtype)


def _aligned_rows(scales):
    """The same scale bytes with rows that start at multiples of 16 bytes, as the quantisers lay them out."""
    m, b = scales.shape
    buf = torch.zeros(m, -(-b // 16) * 16, dtype=torch.uint8, device=scales.device)
    buf[:, :b] = scales
    return buf[:, :b]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] in ("norm", "quantize"):
        dt = TYPES[case["type"]]
        s["x"] = _activations(case["rows"], case["n"], dt, g)
        if case["op"] == "norm":
            s["weight"] = (1 + 0.2 * torch.randn(case["n"], generator=g, device=DEV)).to(dt)
            s["res"] = _activations(case["rows"], case["n"], dt, g) if case["residual"] else None
        return s
    if case["op"] == "grad":
        dt = TYPES[case["type"]]
        s["h"] = _activations(case["rows"], case["n"], dt, g)
        s["weight"] = (1 + 0.2 * torch.randn(case["n"], generator=g, device=DEV)).to(dt)
        s["dy"] = (0.1 * torch.randn(case["rows"], case["n"], generator=g, device=DEV)).to(dt)
        s["dh"] = (0.1 * torch.randn(case["rows"], case["n"], generator=g, device=DEV)).to(dt) if case["residual"] else None
        s["rstd"] = (s["h"].double().square().mean(1) + EPS).rsqrt().float()
        return s
    a = _activations(case["m"], case["k"], torch.float32, g)
    w = 0.02 * torch.randn(case["n"], case["k"], generator=g, device=DEV)
    for name, x, fmt in (("a", a, case["a"]), ("w", w, "mxfp4")):
        values, e = _mx_round(x, fmt)
        s[name + "_codes"] = _pack(values) if fmt == "mxfp4" else values.to(torch.float8_e4m3fn)
        s[name + "_scale"] = _aligned_rows(e)
    s["act_scale"] = 0.5 + torch.rand(case["m"], generator=g, device=DEV) if case["scaled"] else None
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _power(e):
    """2^e in 64 bits, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _mx_round(t, fmt):
    """fp32 [M, n] -> (element values, scale bytes); n filled up to whole blocks with zeros."""
    m, n = t.shape
    t = torch.nn.functional.pad(t, (0, -n % BLOCK)).view(m, -1, BLOCK)
    top = t.abs().amax(-1)
    emax, most, man, low = (2, 6.0, 1, 0) if fmt == "mxfp4" else (8, 448.0, 3, -6)
    e = (torch.frexp(top)[1] - 1 - emax).clamp(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    v = t.double() * _power(-e)[..., None]
    step = _power((torch.frexp(v)[1] - 1).clamp(min=low) - man)
    v = (torch.round(v / step) * step).clamp(-most, most)
    return v.float().view(m, -1), (e + 127).to(torch.uint8)


def _pack(values):
    """e2m1 values -> two codes a byte, the even column in the low half."""
    code = torch.tensor([0, 1, 2, 3, 4, 0, 5, 0, 6, 0, 0, 0, 7], device=values.device, dtype=torch.uint8)
    c = code[(values.abs() * 2).int()] | (torch.signbit(values).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _unpack(codes):
    value = torch.tensor([0.0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    return torch.stack((value[(codes & 15).int()], value[(codes >> 4).int()]), -1).flatten(1)


def _decode(codes, scale):
    v = _unpack(codes) if codes.dtype == torch.uint8 else codes.float()
    m, k = v.shape
    return (v.view(m, -1, BLOCK) * _power(scale.int() - 127).float()[..., None]).view(m, k)


def _plain_norm(s):
    x, fmt = s["x"], s["format"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(x.dtype)
    more = [] if s["res"] is None else [h]
    hf = h.float()
    r = torch.rsqrt(hf.square().mean(1) + EPS)
    if fmt == "same":
        return [(hf * r[:, None] * s["weight"].float()).to(x.dtype), r] + more
    t = hf * s["weight"].float()
    if fmt == "int8":
        top = t.abs().amax(1)
        inv = (127.0 / top.double()).float()
        q = torch.round(t * inv[:, None]).to(torch.int8)
        return [q, top * r / 127.0] + more
    values, e = _mx_round(t, fmt)
    if fmt == "mxfp8":
        return [values.to(torch.float8_e4m3fn), e, r] + more
    whole = (values.view(len(values), -1, BLOCK) * _power(e.int() - 127).float()[..., None]).flatten(1)
    return [whole[:, :x.shape[1]].bfloat16(), e, r] + more


def _plain_grad(s):
    h, w, dy, r = s["h"].float(), s["weight"].float(), s["dy"].float(), s["rstd"][:, None]
    g = dy * w
    dx = r * g - h * (r * r * r * (g * h).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return [dx.to(s["h"].dtype), (dy * h * r).sum(0).to(s["weight"].dtype)]


def _plain_quantize(s):
    values, e = _mx_round(s["x"].float(), s["format"])
    if s["format"] == "mxfp8":
        return [values.to(torch.float8_e4m3fn), e]
    whole = (values.view(len(values), -1, BLOCK) * _power(e.int() - 127).float()[..., None]).flatten(1)
    return [whole[:, :s["x"].shape[1]].bfloat16(), e]


def _plain_matmul(s):
    out = _decode(s["a_codes"], s["a_scale"]) @ _decode(s["w_codes"], s["w_scale"]).t()
    if s["act_scale"] is not None:
        out = out * s["act_scale"][:, None]
    return out.to(TYPES[s["out"]])


def _own(s):
    import quantized_int8_gemm_amd as q
    if s["op"] == "norm":
        if s["format"] == "same":
            return q.rms_norm(s["x"], s["weight"], EPS, residual=s["res"])
        got = q.rms_norm_quantize(s["x"], s["weight"], EPS, residual=s["res"], format=s["format"])
        if s["format"] == "mxfp4":   # packed in pairs: read back as the values they stand for
            return [q.mx_dequantize(got[0], got[1], columns=s["n"])] + list(got[1:])
        return got
    if s["op"] == "grad":
        return q.rms_norm_grad(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh"])
    if s["op"] == "quantize":
        codes, scale = q.mx_quantize(s["x"], s["format"])
        if s["format"] == "mxfp4":
            return [q.mx_dequantize(codes, scale, columns=s["n"]), scale]
        return [codes, scale]
    return q.mx_matmul(s["a_codes"], s["a_scale"], s["w_codes"], s["w_scale"], act_scale=s["act_scale"],
                       out_dtype=TYPES[s["out"]])


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "grad": _plain_grad, "quantize": _plain_quantize, "matmul": _plain_matmul}[state["op"]](state)


def _code_bytes(fmt, rows, n, size):
    """Bytes of one quantised output with its scales."""
    blocks = -(-n // BLOCK)
    return rows * {"same": n * size + 4, "int8": n + 4, "mxfp8": 33 * blocks + 4, "mxfp4": 17 * blocks + 4}[fmt]


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a = 33 if case["a"] == "mxfp8" else 17
        return {"bytes": (m * a + n * 17) * k // BLOCK + m * n * SIZE[case["out"]] + (4 * m if case["scaled"] else 0),
                "flops": 2 * m * n * k}
    rows, n, size = case["rows"], case["n"], SIZE[case["type"]]
    if case["op"] == "norm":
        return {"bytes": rows * n * size * (3 if case["residual"] else 1) + n * size + _code_bytes(case["format"], rows, n, size),
                "flops": 4 * rows * n}
    if case["op"] == "grad":
        return {"bytes": rows * n * size * (4 if case["residual"] else 3) + 2 * n * size + 4 * rows, "flops": 9 * rows * n}
    # the MXFP4 form is read back to bf16 values
    back = 2 * rows * n if case["format"] == "mxfp4" else 0
    return {"bytes": rows * n * size + _code_bytes(case["format"], rows, n, size) - 4 * rows + back, "flops": 2 * rows * n}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _grid(fmt):
    """The format's magnitudes in ascending order, from its bits: a number's place in it is its code."""
    bias, man, count = (1, 1, 8) if fmt == "mxfp4" else (7, 3, 127)
    got = []
    for c in range(count):
        e, f = c >> man, c & ((1 << man) - 1)
        got.append(math.ldexp(f, 1 - bias - man) if e == 0 else math.ldexp((1 << man) + f, e - bias - man))
    return torch.tensor(got, dtype=torch.float64, device=DEV)


def _exact_mx(t, fmt):
    """64-bit [M, n] -> (element values [M, whole blocks], their block factors)."""
    grid = _grid(fmt)
    m, n = t.shape
    pad = torch.zeros(m, -n % BLOCK, dtype=torch.float64, device=DEV)
    b = torch.cat((t, pad), 1).reshape(m, -1, BLOCK)
    top = b.abs().max(-1).values
    e = torch.floor(torch.log2(top.clamp(min=1e-300)))
    e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double()
    factor = torch.exp2((e - (2 if fmt == "mxfp4" else 8)).clamp(-127, 127))
    v = b / factor[..., None]
    at = v.abs().reshape(-1)
    hi = torch.searchsorted(grid, at).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = at - grid[lo], grid[hi] - at
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.sign(v) * grid[pick].reshape(v.shape), factor


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        def values(codes, scale):
            if codes.dtype == torch.uint8:
                c = torch.stack((codes % 16, codes // 16), -1).flatten(1)
                v = _grid("mxfp4")[(c % 8).int()] * torch.where(c >= 8, -1.0, 1.0)
            else:
                c = codes.view(torch.uint8)
                v = _grid("mxfp8")[(c % 128).int()] * torch.where(c >= 128, -1.0, 1.0)
            return v * torch.exp2(scale.double() - 127).repeat_interleave(BLOCK, 1)
        out = values(s["a_codes"], s["a_scale"]) @ values(s["w_codes"], s["w_scale"]).t().contiguous()
        return out if s["act_scale"] is None else out * s["act_scale"].double()[:, None]
    if case["op"] == "quantize":
        v, f = _exact_mx(s["x"].double(), case["format"])
        if case["format"] == "mxfp8":
            return [v.flatten(1), None]
        return [(v * f[..., None]).flatten(1)[:, :case["n"]], None]
    w = s["weight"].double()
    if case["op"] == "grad":
        h, dy, n = s["h"].double(), s["dy"].double(), case["n"]
        r = s["rstd"].double()[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = r * (dy * w - h * r * r * dot / n)
        return [dx if s["dh"] is None else dx + s["dh"].double(), (dy * (h * r)).sum(0)]
    # the norm sees the hidden state as it is stored
    h = s["x"].double() if s["res"] is None else (s["x"].double() + s["res"].double()).to(s["x"].dtype).double()
    more = [] if s["res"] is None else [h]
    r = 1 / torch.sqrt((h * h).sum(1) / case["n"] + EPS)
    if case["format"] == "same":
        return [h * r[:, None] * w, r] + more
    t = h * w
    if case["format"] == "int8":
        return [None, t.abs().max(1).values * r / 127] + more
    v, f = _exact_mx(t, case["format"])
    if case["format"] == "mxfp8":
        return [v.flatten(1), None, r] + more
    return [(v * f[..., None]).flatten(1)[:, :case["n"]], None, r] + more

"""The operators measured around the A8W8 product of a feed-forward block: the
product with bias, activation and residual, the gated pair of products, both with
an 8-bit checkpoint and the backward pass that reads it, and the int8 quantiser.

``run`` computes a case in plain torch operations, or, with ``own`` true,
through the library.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ACTIVATIONS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # the projection back to the residual stream, for one generated token
        {"name": "linear_1x4096x14336", "op": "linear", "m": 1, "n": 4096, "k": 14336, "bias": False, "act": "none", "residual": True, "out": "bf16", "trans": True},
        # the first layer of an ungated block over a ragged batch, a weight of odd height
        {"name": "linear_300x5001x2048", "op": "linear", "m": 300, "n": 5001, "k": 2048, "bias": True, "act": "gelu", "residual": False, "out": "fp32", "trans": True},
        # a long prompt, the weight as the products keep it by default
        {"name": "linear_8192x8192x8192", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "bias": True, "act": "gelu_tanh", "residual": True, "out": "bf16", "trans": False},
        # one generated token through the gate and the up projection
        {"name": "gated_1x14336x4096", "op": "gated", "m": 1, "n": 14336, "k": 4096, "act": "silu", "out": "bf16", "trans": True},
        # a batch of chunks of prompts, weights as [K,N]
        {"name": "gated_777x8192x4096", "op": "gated", "m": 777, "n": 8192, "k": 4096, "act": "gelu_tanh", "out": "fp16", "trans": False},
        # a long prompt
        {"name": "gated_8192x14336x4096", "op": "gated", "m": 8192, "n": 14336, "k": 4096, "act": "silu", "out": "bf16", "trans": True},
        # forward with a checkpoint and backward of a training step, of a small block
        {"name": "gated_step_515x2816x1024", "op": "gated_step", "m": 515, "n": 2816, "k": 1024, "act": "gelu_tanh", "out": "fp16", "trans": True},
        # and of a large one
        {"name": "gated_step_4096x14336x4096", "op": "gated_step", "m": 4096, "n": 14336, "k": 4096, "act": "silu", "out": "bf16", "trans": True},
        # the same for the ungated block, the bias's gradient included
        {"name": "linear_step_130x1000x512", "op": "linear_step", "m": 130, "n": 1000, "k": 512, "act": "gelu", "out": "bf16", "trans": False},
        {"name": "linear_step_4096x8192x2048", "op": "linear_step", "m": 4096, "n": 8192, "k": 2048, "act": "gelu", "out": "bf16", "trans": True},
        # the inner activations of one token, as the next product's left operand
        {"name": "int8_rows_1x14336", "op": "quantize", "m": 1, "n": 14336, "block": None, "type": "bf16"},
        # a checkpoint of a training step's activations, written and read back
        {"name": "int8_blocks_8192x14336", "op": "quantize", "m": 8192, "n": 14336, "block": BLOCK, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("linear", "linear", "gated", "gated", "gated_step", "linear_step", "quantize"))
    if op == "quantize":
        m, n = _log(rng, 1, 16384), _log(rng, 64, 16384)
        return {"op": op, "m": max(1, min(m, 8192 * 14336 // n)), "n": n, "block": rng.choice((None, BLOCK)), "type": rng.choice(tuple(TYPES))}
    # weights mostly have rows of whole 16-byte pieces; some have not
    n, k = _log(rng, 64, 14336), _log(rng, 64, 14336)
    n, k = (n if rng.random() < 0.5 else -(-n // 16) * 16), (k if rng.random() < 0.2 else -(-k // 16) * 16)
    case = {"op": op, "m": _log(rng, 1, 8192), "n": n, "k": k, "act": rng.choice(ACTIVATIONS), "trans": rng.random() < 0.6}
    most = 4096 * 8192 * 2048 if op == "linear_step" else 4096 * 14336 * 4096 if op == "gated_step" else 8192 * 14336 * 4096
    case["m"] = max(1, min(case["m"], most // (n * k)))
    if op == "linear":
        case.update(bias=rng.random() < 0.5, residual=rng.random() < 0.5, act=rng.choice(("none",) + ACTIVATIONS))
    case["out"] = rng.choice(("bf16", "fp16") if op.endswith("step") else tuple(TYPES))
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


def _rows_to_int8(x):
    top = x.abs().amax(1).clamp(min=1e-20)
    return torch.round(x * (127 / top)[:, None]).to(torch.int8), top / 127


def _weight(case, g):
    """int8 [N,K] or [K,N], with a scale per output."""
    w, scale = _rows_to_int8(torch.randn(case["n"], case["k"], generator=g, device=DEV) * case["k"] ** -0.5)
    return (w if case["trans"] else w.t().contiguous()), scale


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "quantize":
        s["x"] = _activations(case["m"], case["n"], TYPES[case["type"]], g)
        return s
    m, n, dt = case["m"], case["n"], TYPES[case["out"]]
    s["a"], s["a_scale"] = _rows_to_int8(_activations(m, case["k"], torch.float32, g))
    s["w"], s["w_scale"] = _weight(case, g)
    if case["op"].startswith("gated"):
        s["w2"], s["w2_scale"] = _weight(case, g)
    else:
        s["bias"] = 0.5 * torch.randn(n, generator=g, device=DEV) if case.get("bias", True) else None
        s["res"] = torch.randn(m, n, generator=g, device=DEV).to(dt) if case.get("residual") else None
    if case["op"].endswith("step"):
        s["dy"] = (0.1 * torch.randn(m, n, generator=g, device=DEV)).to(dt)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _act(name, z):
    """The activation and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "silu":
        e = 1 / (1 + torch.exp(-z))
        return z * e, e * (1 + z * (1 - e))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return z * c, c + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    k, b = (2 / math.pi) ** 0.5, 0.044715
    t = torch.tanh(k * (z + b * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * b * z * z)


def _product(s, w, scale):
    w = s[w].float()
    acc = s["a"].float() @ (w.t() if s["trans"] else w)
    return acc * s["a_scale"][:, None] * s[scale]


def _quantize(x, block):
    """fp32 [M, n] -> (int8 codes, scale) per row, or per block of columns."""
    m, n = x.shape
    b = x[:, None] if block is None else torch.nn.functional.pad(x, (0, -n % block)).view(m, -1, block)
    top = b.abs().amax(-1)
    one = torch.where(top > 0, top, torch.ones_like(top)).double()
    codes = torch.round(b * (127.0 / one).float()[..., None]).to(torch.int8)
    scale = torch.where(top > 0, (top.double() / 127.0).float(), torch.ones_like(top))
    return codes, scale


def _values(codes, scale, n):
    return (codes.float() * scale[..., None]).flatten(1)[:, :n]


def _plain_quantize(s):
    codes, scale = _quantize(s["x"].float(), s["block"])
    return [_values(codes, scale, s["n"]).bfloat16(), scale.squeeze(1) if s["block"] is None else scale]


def _plain_linear(s):
    z = _product(s, "w", "w_scale")
    if s["bias"] is not None:
        z = z + s["bias"]
    y = _act(s["act"], z)[0]
    if s["res"] is not None:
        y = y + s["res"].float()
    return y.to(TYPES[s["out"]])


def _plain_gated(s):
    return (_act(s["act"], _product(s, "w", "w_scale"))[0] * _product(s, "w2", "w2_scale")).to(TYPES[s["out"]])


def _back(s, p, w):
    w = s[w].float()
    return p @ (w if s["trans"] else w.t())


def _plain_linear_step(s):
    z = _product(s, "w", "w_scale") + s["bias"]
    y = _act(s["act"], z)[0].to(TYPES[s["out"]])
    z = _values(*_quantize(z, BLOCK), s["n"])
    p = s["dy"].float() * _act(s["act"], z)[1]
    return [y, _back(s, p * s["w_scale"], "w").to(TYPES[s["out"]]), p.sum(0)]


def _plain_gated_step(s):
    g, u = _product(s, "w", "w_scale"), _product(s, "w2", "w2_scale")
    y = (_act(s["act"], g)[0] * u).to(TYPES[s["out"]])
    g, u = _values(*_quantize(g, BLOCK), s["n"]), _values(*_quantize(u, BLOCK), s["n"])
    f, slope = _act(s["act"], g)
    dy = s["dy"].float()
    return [y, (_back(s, dy * u * slope * s["w_scale"], "w") + _back(s, dy * f * s["w2_scale"], "w2")).to(TYPES[s["out"]])]


def _own(s):
    import quantized_int8_gemm_amd as q
    if s["op"] == "quantize":
        codes, scale = q.int8_quantize(s["x"], block=s["block"])
        return [q.int8_dequantize(codes, scale, torch.bfloat16), scale]
    kw = {"activation": s["act"], "b_trans": s["trans"]}
    out = {"out_dtype": TYPES[s["out"]]}
    if s["op"] == "linear":
        return q.qgemm_a8w8_linear(s["a"], s["w"], s["a_scale"], s["w_scale"], bias=s["bias"], residual=s["res"], **kw, **out)
    if s["op"] == "linear_step":
        y, saved = q.qgemm_a8w8_linear(s["a"], s["w"], s["a_scale"], s["w_scale"], bias=s["bias"], checkpoint=True, **kw, **out)
        return [y, *q.qgemm_a8w8_linear_grad(s["dy"], s["w"], s["w_scale"], saved, bias_grad=True, **kw)]
    weights = (s["w"], s["w2"])
    if s["op"] == "gated":
        return q.qgemm_a8w8_gated(s["a"], *weights, s["a_scale"], s["w_scale"], s["w2_scale"], **kw, **out)
    y, saved = q.qgemm_a8w8_gated(s["a"], *weights, s["a_scale"], s["w_scale"], s["w2_scale"], checkpoint=True, **kw, **out)
    return [y, q.qgemm_a8w8_gated_grad(s["dy"], *weights, s["w_scale"], s["w2_scale"], saved, **kw)]


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "gated": _plain_gated, "linear_step": _plain_linear_step, "gated_step": _plain_gated_step,
            "quantize": _plain_quantize}[state["op"]](state)


def work(case):
    m, n = case["m"], case["n"]
    if case["op"] == "quantize":
        # codes and scales written, and read again for the values
        held = m * n + 4 * m * (1 if case["block"] is None else -(-n // BLOCK))
        return {"bytes": m * n * (SIZE[case["type"]] + 2) + 2 * held, "flops": 4 * m * n}
    k, size = case["k"], SIZE[case["out"]]
    pair = 2 if case["op"].startswith("gated") else 1
    moved = m * k + 4 * m + pair * n * (k + 4) + m * n * size
    if case["op"] == "linear":
        moved += (4 * n if case["bias"] else 0) + (m * n * size if case["residual"] else 0)
    if case["op"].endswith("step"):
        return {"bytes": moved + m * n * size + m * k * size + (8 * n if pair == 1 else 0), "flops": 4 * pair * m * n * k}
    return {"bytes": moved, "flops": 2 * pair * m * n * k}


# ---------------------------------------------------------------------------
# From the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_act(name, z, slope=False):
    if name == "none":
        return torch.ones_like(z) if slope else z
    if name == "silu":
        e = torch.sigmoid(z)
        return e + z * e * torch.sigmoid(-z) if slope else z * e
    if name == "gelu":
        c = 0.5 * torch.erfc(-z / math.sqrt(2))
        return c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi) if slope else z * c
    # tanh(x) = 2 sigmoid(2 x) - 1
    inner = math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    e = torch.sigmoid(inner)
    return e + z * e * torch.sigmoid(-inner) * math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z) if slope else z * e


def _fl(t):
    """Rounded to 32 bits: codes are defined by such steps, and one that differs is a whole step off."""
    return t.float().double()


def _exact_blocks(z, width):
    """What 8-bit codes with a scale for `width` columns of a row stand for, and the scales."""
    rows, n = z.shape
    full = torch.zeros(rows, -(-n // width) * width, dtype=torch.float64, device=DEV)
    full[:, :n] = z
    full = full.reshape(rows, -1, width)
    top = full.abs().max(-1, keepdim=True).values
    step = torch.where(top == 0, 1.0, _fl(top / 127))
    return (torch.round(_fl(full * _fl(127 / torch.where(top == 0, 1.0, top)))) * step).flatten(1)[:, :n], step.squeeze(-1)


def _exact_saved(s, scale, w, bias):
    """The values of a checkpoint of the product with w, [K,N]."""
    z = _fl(_fl(_fl(s["a"].double() @ w) * s["a_scale"].double()[:, None]) * scale)
    return _exact_blocks(z if bias is None else _fl(z + bias), BLOCK)[0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        back, step = _exact_blocks(s["x"].double(), case["block"] or case["n"])
        return [back, step.squeeze(1) if case["block"] is None else step]

    def rows_of(w):   # [N, K] in 64 bits, scaled
        w, scale = s[w].double(), s[w + "_scale"].double()
        return (w if case["trans"] else w.t().contiguous()) * scale[:, None]

    def saved(w, bias=None):
        t = s[w].double()
        return _exact_saved(s, s[w + "_scale"].double(), t.t().contiguous() if case["trans"] else t, bias)

    x = s["a"].double() * s["a_scale"].double()[:, None]
    w = rows_of("w")
    z = x @ w.t().contiguous()
    if case["op"].startswith("gated"):
        w2 = rows_of("w2")
        u = x @ w2.t().contiguous()
        y = _exact_act(case["act"], z) * u
        if case["op"] == "gated":
            return y
        z, u, dy = saved("w"), saved("w2"), s["dy"].double()
        return [y, (dy * u * _exact_act(case["act"], z, True)) @ w + (dy * _exact_act(case["act"], z)) @ w2]
    if s["bias"] is not None:
        z = z + s["bias"].double()
    y = _exact_act(case["act"], z)
    if case["op"] == "linear":
        return y if s["res"] is None else y + s["res"].double()
    p = s["dy"].double() * _exact_act(case["act"], saved("w", s["bias"].double()), True)
    return [y, p @ w, p.sum(0)]

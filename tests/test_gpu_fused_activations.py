"""The fused products' activations in fp32 against 64 bits, relative to the value itself: far
on the negative side, where 1 + erf or 1 + tanh would cancel, and next to zero; and
GELU's slope.

Units are 2^-24; the hardware's exponential and reciprocal are within one unit in the last place (2
each, relative).
SiLU: the exponent is rounded once, its constant too (5/4 |z| of the exponential), then the
exponential, the sum, the reciprocal and the product: 5/4 |z| + 6, below 2 (|z| + 4).
GELU by tanh, z / (1 + exp(-y)): the factor of z and its constant, the square, its constant
and the sum, the product, and the exponent's two, at most 25/4 |y|, and 6 as above: below 8 (|y| + 2).
GELU by erf: Phi(-a) is the density times a polynomial's value.  The density's exponent is
rounded twice, its constant once (5/4 z^2), the exponential and the reciprocal take 2 each,
and the argument, the polynomial, two products and the fit (1/2) at most 2: with the
last product below 2 (z^2 + 5)."""
import math

import numpy as np
import pytest
import torch

import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def phi(z):
    return 0.5 * _erfc(-z / math.sqrt(2))


def forward(z, activation="gelu"):
    """act(z) in fp32: the products are zeros, the bias is z."""
    n = z.size
    out = q.qgemm_a8w8_linear(torch.zeros(1, 16, dtype=torch.int8, device=dev()), torch.ones(n, 16, dtype=torch.int8, device=dev()),
                              torch.ones(1, device=dev()), torch.ones(n, device=dev()), bias=torch.from_numpy(z).to(dev()),
                              activation=activation, b_trans=True)
    return out.double().cpu().numpy()[0]


def values(seed, n=40000):
    r = np.random.default_rng(seed)
    return np.concatenate([np.linspace(-12.9, 12.9, n), r.normal(size=n) * 0.1, r.normal(size=n // 4) * 1e-6]).astype(np.float32)


def sigmoid_of(kind, z):
    return z if kind == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)


@pytest.mark.parametrize("kind,least", [("silu", -80.0), ("gelu_tanh", -9.5), ("gelu", -12.9)])
def test_relative_to_the_value(kind, least):
    case(f"{kind} from {least} on")
    z = values(1) * np.float32(least / -12.9)
    got, zd = forward(z, kind), z.astype(np.float64)
    if kind == "gelu":
        want, tol = zd * phi(zd), 2 * (zd * zd + 5) * U
    else:
        y = sigmoid_of(kind, zd)
        want = zd / (1 + np.exp(-y))
        tol = 2 * (np.abs(y) + 4) * U if kind == "silu" else 8 * (np.abs(y) + 2) * U
    bad = ~(np.abs(got - want) <= tol * np.abs(want))
    assert not bad.any(), (int(bad.sum()), zd[bad][:3], got[bad][:3], want[bad][:3])


def test_gelu_next_to_zero():
    """|z| < 1/2, as max(z, 0) - |z| Phi(-|z|).  Of Phi(-|z|) <= 1/2 the argument, the reciprocal
    and the exponential take 2^-25 each, two products and the polynomial 2^-26 each, the exponent's
    roundings and the fit less than 2^-26 together; the difference's own rounding is at most 2^-24
    of Phi(z) < 0.7."""
    case("gelu next to zero")
    z = values(2)
    z = z[(np.abs(z) < 0.5) & (z != 0)]
    zd = z.astype(np.float64)
    off = np.abs(forward(z) / zd - phi(zd))
    assert off.max() <= 4 * U, (off.max() / U, zd[off.argmax()])


def test_gelu_at_the_ends():
    case("gelu at the ends")
    big = np.finfo(np.float32).max
    z = np.array([0.0, -0.0, 14.0, 40.0, 1e20, big, np.inf, -14.0, -40.0, -1e20, -big, np.nan, -np.inf, 1e-38, -1e-38, 2.0 ** -149], np.float32)
    got = forward(z)
    assert np.array_equal(got[:7], z[:7].astype(np.float64))
    assert (np.abs(got[7:11]) <= 1e-36).all() and np.isnan(got[11:13]).all()   # -infinity times 0, as the formula gives it
    assert np.abs(got[13:] - z[13:] * 0.5).max() <= 2.0 ** -149


def test_gelu_slope():
    """One row of dy = 1: dbias is the slope at the checkpoint's values, in fp32.  z density is
    rounded three times beside the density itself, the sum once."""
    case("gelu slope")
    n = 65504
    r = np.random.default_rng(3)
    codes = r.integers(-127, 128, (1, n), dtype=np.int8)
    scale = (np.exp(r.uniform(np.log(0.01), np.log(12.9), (1, n // 32))) / 127).astype(np.float32)
    dy = torch.ones(1, n, dtype=torch.bfloat16, device=dev())
    w = torch.ones(n, 16, dtype=torch.int8, device=dev())
    saved = (torch.from_numpy(codes).to(dev()), torch.from_numpy(scale).to(dev()))
    _, db = q.qgemm_a8w8_linear_grad(dy, w, torch.ones(n, device=dev()), saved, "gelu", b_trans=True, bias_grad=True)
    z = (codes.astype(np.float32) * np.repeat(scale, 32, 1))[0].astype(np.float64)
    density = np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    least = phi(-np.abs(z))
    want = phi(z) + z * density
    tol = least * (z * z + 5) * 2 * U + np.where(z > 0, U, 0) + np.abs(z) * density * (1.25 * z * z + 2 + 3) * U + U * np.abs(want)
    bad = ~(np.abs(db.double().cpu().numpy() - want) <= 1.01 * tol)
    assert not bad.any(), (int(bad.sum()), z[bad][:3], db.cpu().numpy()[bad][:3], want[bad][:3])

"""Plain restatements of the norm, the 16-bit products, the gated block and the
8-bit rows for the tests, in 64 bits, written from include/zero.h: no code of
the library.  Tensors of float64 on any device; beside a value, where it helps,
what an fp32 computation of it may be off by."""
from __future__ import annotations

import math

import torch

from tests.ops_ref import ROUND, TINY

ULP = 2.0 ** -23                       # an fp32 spacing, relative
NONE, RELU, GELU, GELU_TANH, SILU = range(5)


def argument(z, kind):
    """The magnitude of the exponential's argument in an activation: what its relative
    error grows with."""
    if kind == GELU_TANH:
        return 2 * math.sqrt(2 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3)
    if kind == GELU:
        return z * z
    return z.abs() if kind == SILU else torch.zeros_like(z)


def normal(z):
    """The normal distribution function.  (torch's ndtr loses the tail's digits.)"""
    return 0.5 * torch.special.erfc(-z * math.sqrt(0.5))


def activation(z, kind):
    """(value, slope)."""
    if kind == RELU:
        return torch.where(z > 0, z, 0.0), (z > 0).double()
    if kind == GELU:
        phi = normal(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if kind == GELU_TANH:
        c = math.sqrt(2 / math.pi)
        w = 2 * c * (z + 0.044715 * z ** 3)
        p, q = torch.sigmoid(w), torch.sigmoid(w) * torch.sigmoid(-w)
        return z * p, p + z * q * 2 * c * (1 + 3 * 0.044715 * z * z)
    if kind == SILU:
        p, q = torch.sigmoid(z), torch.sigmoid(z) * torch.sigmoid(-z)
        return z * p, p + z * q
    return z, torch.ones_like(z)


def value_error(z, dz, kind):
    """What an fp32 activation of z, itself off by dz, may be off by.

    The exponential's relative error is at most (2 + 1.2 |w|) spacings, w its
    argument, whose own relative error of a few roundings multiplies by |w| again;
    a logistic's is no larger, and the quotient and the product add a few.  So
    (8 + 4 |w|) spacings of the value, and dz times the largest slope, 1.13.  An
    exponential below 2^-126 is 0, which is off by less than that and comes to the value
    times |z|."""
    if kind == NONE:
        return dz
    if kind == RELU:
        return dz
    return (1.13 * dz + (8 + 4 * argument(z, kind)) * ULP * activation(z, kind)[0].abs()
            + 2.0 ** -126 * z.abs())


def slope_error(z, kind):
    """The same of its slope at an exact z: of both terms' magnitudes.  An
    exponential that is 0 for less than 2^-126 comes to the first term as it is and to the
    second times |z| and w's slope: at the tanh's, where w is 87 there, by 2^8 in all."""
    if kind in (NONE, RELU):
        return torch.zeros_like(z)
    y, slope = activation(z, kind)
    first = torch.sigmoid(z) if kind == SILU else activation(z, GELU_TANH)[0] / torch.where(
        z == 0, 1.0, z) if kind == GELU_TANH else normal(z)
    rise = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z) if kind == GELU_TANH else 1.0
    return ((12 + 4 * argument(z, kind)) * ULP * (first.abs() + (slope - first).abs())
            + 2.0 ** -126 * (1 + z.abs() * rise))


def product(a, b):
    """(sum of a b over the columns, what an fp32 sum of the exact products may be
    off by): k additions, each of which loses less than a spacing of a partial sum."""
    return a @ b.t(), (a.shape[1] + 1) * ULP * (a.abs() @ b.abs().t())


def power(e):
    """2^e for whole e by its bits: a GPU's pow() is not exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def pack(x):
    """(values, scale exponents + 127) of the rows of x."""
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, -C % 32)).reshape(R, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    bad = ~torch.isfinite(b).all(2, keepdim=True)
    frac, ex = torch.frexp(torch.where(bad, 1.0, top))
    e = torch.where(frac > 0, ex - 9 + (frac > 0.875).int(), -127).clamp(min=-127)
    unit = power(e)
    v = b / unit
    step = power((torch.frexp(v).exponent - 1).clamp(min=-6) - 3)
    out = torch.where(bad, math.nan, torch.round(v / step) * step * unit)
    return (out.reshape(R, -1)[:, :C],
            torch.where(bad, 255, e + 127).reshape(R, -1).to(torch.uint8))


def rounded(x, dtype):
    """x rounded once to the type, finite values saturating: what the 8-bit rows'
    values are given as."""
    f = torch.finfo(dtype)
    y = x.clamp(f.min, f.max) if dtype != torch.float32 else x.clamp(-f.max, f.max)
    return y.to(dtype)


def within(got, want, error, dtype=None):
    """|got - want| is at most `error` and the rounding to the type, of a value that is
    `error` off, and infinities and NaN are where they should be."""
    u, tiny = ROUND[dtype or got.dtype], TINY[dtype or got.dtype]
    g, w = got.double().cpu(), want.double().cpu()
    e = error.double().cpu() if isinstance(error, torch.Tensor) else torch.full_like(w, error)
    fine = torch.isfinite(w)
    assert torch.equal(torch.isnan(g), torch.isnan(w))
    assert torch.equal(g[~fine & ~torch.isnan(w)], w[~fine & ~torch.isnan(w)])
    bound = e + u * (w.abs() + e) + tiny
    off = ((g - w).abs() - bound)[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, (
        "off by %.3g more than the bound at %d of %d" % (float(off.max()), int((off > 0).sum()),
                                                         off.numel()))

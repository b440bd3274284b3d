"""Plain restatements of the training operators for the tests, in 64 bits,
written from include/zero.h: no code of the library."""
from __future__ import annotations

import math

import numpy as np
import torch

#: unit roundoff of each element type (half the spacing above 1)
ROUND = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
#: half of the smallest subnormal: what rounding to the type loses at most near 0
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def philox(counter, key):
    """Philox4x32-10: counter [n, 4] and key (2 words) of 32 bits in uint64;
    returns [n, 4]."""
    m = np.uint64(0xFFFFFFFF)
    c = np.array(counter, dtype=np.uint64).reshape(-1, 4).copy()
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        a, b = c[:, 0] * np.uint64(0xD2511F53), c[:, 2] * np.uint64(0xCD9E8D57)
        c = np.stack([(b >> np.uint64(32)) ^ c[:, 1] ^ np.uint64(k0), b & m,
                      (a >> np.uint64(32)) ^ c[:, 3] ^ np.uint64(k1), a & m], 1)
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def keep(n, p, seed, offset, first=0):
    """Which of elements first .. first + n are kept (first a multiple of 4)."""
    groups = first // 4 + np.arange(-(-n // 4), dtype=np.uint64)
    c = np.stack([groups & np.uint64(0xFFFFFFFF), groups >> np.uint64(32),
                  np.full_like(groups, offset & 0xFFFFFFFF),
                  np.full_like(groups, (offset >> 32) & 0xFFFFFFFF)], 1)
    words = philox(c, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)[:n]
    return words >= np.uint64(math.floor(p * 2.0 ** 32))


def quantize(x):
    """(codes [R, C], scale bytes [R, ceil(C / 32)]) of a float64 matrix, by
    looking the nearest grid value up: ties go to the even code."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    nb = -(-C // 32)
    full = np.zeros((R, nb * 32))
    full[:, :C] = x
    b = full.reshape(R, nb, 32)
    top = np.abs(b).max(2)
    bad = ~np.isfinite(b).all(2)
    with np.errstate(invalid="ignore"):
        e = np.where((top > 0) & ~bad, np.frexp(np.where(bad, 1.0, top))[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    v = np.abs(np.where(bad[:, :, None], 0.0, b)) / np.ldexp(1.0, e)[:, :, None]
    mid = (GRID[1:] + GRID[:-1]) / 2                      # 7 midpoints
    code = np.zeros(v.shape, dtype=np.uint8)
    for i, m in enumerate(mid):
        code += (v > m) | ((v == m) & (i % 2 == 1))       # the tie of codes i, i + 1
    code |= np.where(np.signbit(b), 8, 0).astype(np.uint8)
    scale = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(R, -1)[:, :C], scale


def values(codes, scales):
    """The float64 values codes and scale bytes stand for."""
    C = codes.shape[1]
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, 1)[:, :C]


def unpack(q, rows, cols):
    """(codes, scale bytes) of a matrix laid out as include/zero.h says, for
    all columns of its records (multiples of 256 and 8)."""
    rt, kt = -(-rows // 128), -(-cols // 256)
    q = np.asarray(q, dtype=np.uint8).reshape(rt, kt, 17408)
    codes = np.zeros((rt * 128, kt * 256), dtype=np.uint8)
    scales = np.zeros((rt * 128, kt * 8), dtype=np.uint8)
    r = np.arange(128)
    for i in range(rt):
        for t in range(kt):
            body = q[i, t, :16384].reshape(128, 8, 16)
            for p in range(8):
                piece = body[r, p ^ (r & 7)]               # [128, 16]
                c0 = t * 256 + p * 32
                codes[i * 128:(i + 1) * 128, c0:c0 + 32:2] = piece & 15
                codes[i * 128:(i + 1) * 128, c0 + 1:c0 + 32:2] = piece >> 4
            for b in range(8):
                at = 16384 + (b // 4) * 512 + (r % 32) * 16 + (r // 32) * 4 + b % 4
                scales[i * 128:(i + 1) * 128, t * 8 + b] = q[i, t, at]
    return codes[:rows], scales[:rows]


def host(t):
    return t.detach().double().cpu().numpy()


def within(got, want, bound):
    """|got - want| <= bound where want is finite; NaN and infinities equal."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    off = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)) - np.where(fine, bound, 0)
    assert (off <= 0).all(), "worst excess %g at %s" % (off.max(), np.unravel_index(
        np.argmax(off), off.shape))

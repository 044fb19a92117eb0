"""Plain references of the 8-bit-integer operators for the tests.

The codes are decided by single binary32 operations (numpy float32 arithmetic
is IEEE, one rounding per operation), so they have one right value; sums,
norms and products are taken in 64 bits.
"""
from __future__ import annotations

import numpy as np

F = np.float32
TINY = F(2.0 ** -100)


def bf16_round(v):
    """float32 -> the nearest BF16 value (ties to even), as float32; NaN stays NaN."""
    v = np.asarray(v, F)
    b = v.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(F)
    return np.where(np.isnan(v), v, r)


def codes_of(t):
    """(codes, T, zero, bad) of a float32 matrix, per row."""
    t = np.asarray(t, F)
    bad = ~np.isfinite(t).all(axis=1)
    mag = np.where(bad[:, None], F(0), np.abs(t))
    amax = mag.max(axis=1)
    top = np.maximum(amax, TINY)
    mult = F(127.0) / top
    codes = np.rint(np.where(bad[:, None], F(0), t) * mult[:, None]).astype(np.int8)
    return codes, top, amax == 0, bad


def quantize(x):
    """Codes and scales of float32 values: both have one right value."""
    codes, top, zero, bad = codes_of(x)
    scale = np.where(zero, F(1), top / F(127.0))
    return codes, np.where(bad, F(np.nan), scale).astype(F)


def add_rms_norm(x, residual, weight, offset, eps):
    """codes (exact), scale in 64 bits, v in 64 bits, r as BF16 values."""
    with np.errstate(all="ignore"):
        r = np.asarray(x, F) if residual is None else np.asarray(x, F) + np.asarray(residual, F)
        t = r * (np.asarray(weight, F) + F(offset))[None, :]
        codes, top, zero, bad = codes_of(np.where(np.isfinite(r), t, F(np.nan)))
        r64 = r.astype(np.float64)
        rstd = 1.0 / np.sqrt((r64 * r64).mean(axis=1) + float(F(eps)))
        scale = np.where(zero, 1.0, top.astype(np.float64) / 127.0 * rstd)
        v = r64 * (np.asarray(weight, np.float64) + offset)[None, :] * rstd[:, None]
        return codes, np.where(bad, np.nan, scale), v, bf16_round(r)


def scale_tolerance(cols):
    """Relative error the norm's scale may have: a binary32 sum of `cols`
    non-negative squares, added along a chain of at most cols/32 fused
    multiply-adds in a thread (32 threads at the least), 5 shuffle steps and 32
    warps, errs by at most (cols/32 + 37) 2^-24 relatively, the mean's factor
    1/cols and the addition of eps by two more half steps; the inverse square
    root halves that and rounds once (2^-24), T/127 and the product once each."""
    return ((cols / 32 + 37 + 2) / 2 + 3) * 2.0 ** -24 * 1.01


def gemm(a, sa, w, sw):
    """BF16 values (as float32): every sum below 2^31 is exact in float64, and
    the three roundings after it are numpy float32 operations."""
    acc = a.astype(np.float64) @ w.astype(np.float64).T
    with np.errstate(all="ignore"):
        v = (acc.astype(np.int64).astype(F) * np.asarray(sa, F)[:, None]) * np.asarray(sw, F)[None, :]
    return bf16_round(v)

"""fp64 definitions of the microscaled 4-bit path and of the expert layer for a few
tokens -- TEST INFRASTRUCTURE, like the package it is in.

Only the roundings that a definition names are done (the codes, the bf16 of a stored h);
everything else is exact or fp64.
"""
from __future__ import annotations

import numpy as np

from . import dequant_mxfp4

BLOCK = 32
SLAB = 512
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])   # E2M1 by code


def scale_bytes(d: int) -> int:
    return 16 * -(-d // SLAB)


def exponent(m, fit: bool) -> np.ndarray:
    """E8M0 of blocks whose largest magnitude is m; 255 where it is not finite."""
    m = np.asarray(m, np.float64)
    ok = np.isfinite(m) & (m > 0)
    f, e = np.frexp(np.where(ok, m, 1.0))           # f in [1/2, 1): m = 2f·2^(e-1)
    e = e - 1 - 2 + 127
    if fit:
        e = e + (f > 0.75)                          # over 1.5 in its binade: over 6·2^(E-127)
    e = np.where(m == 0, 0, np.clip(e, 0, 254))
    return np.where(np.isfinite(m), e, 255)


def round_code(a) -> np.ndarray:
    """Code of the nearest magnitude, a midpoint to the even code, 7 (6.0) from 5 on."""
    a = np.asarray(a, np.float64)
    hi = np.clip(np.searchsorted(MAGNITUDES, a), 1, 7)
    lo = hi - 1
    down, up = a - MAGNITUDES[lo], MAGNITUDES[hi] - a
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def pack_codes(c) -> np.ndarray:
    return (c[..., 0::2] | c[..., 1::2] << 4).astype(np.uint8)


def quant(x, fit: bool):
    """(codes uint8[t][d/2], scales uint8[t][scale_bytes(d)]) of rows."""
    x = np.asarray(x, np.float64)
    t, d = x.shape
    b = x.reshape(t, d // BLOCK, BLOCK)
    e = exponent(np.abs(b).max(2), fit)             # numpy's max keeps a NaN
    bad = (e == 255)[..., None]
    v = np.where(bad, 0.0, np.nan_to_num(b, posinf=0.0, neginf=0.0)) * 2.0 ** (127.0 - e)[..., None]
    c = round_code(np.abs(v)) | np.where(np.signbit(v) & ~bad, 8, 0)
    scales = np.zeros((t, scale_bytes(d)), np.uint8)
    scales[:, :d // BLOCK] = e
    return pack_codes(c.reshape(t, d)), scales


def dequant(codes, scales) -> np.ndarray:
    """Rows as their codes stand for them; a block with the exponent 255 is NaN."""
    blocks = codes.shape[1] * 2 // BLOCK
    s = np.asarray(scales)[:, :blocks]
    v = dequant_mxfp4(codes, np.where(s == 255, 0, s))
    return np.where(np.repeat(s == 255, BLOCK, axis=1), np.nan, v)


def gemm(x, w):
    """(Y, R) of dequantised rows and matrix: the product, and what the fp32 sum that the
    kernels form may be off by.  A term goes through at most 128 additions in the matrix
    instruction that reads it, one for each 128 codes after it, and 16 across waves; each
    loses at most 2^-23 of the sum of the magnitudes (products of two codes are exact)."""
    a = np.abs(x) @ np.abs(w).T
    return x @ w.T, (128 + x.shape[1] / 128 + 16) * 2.0 ** -23 * a


def gemm_tolerance(y, rest):
    """What |y_gpu - y| may be: `rest` before the rounding, half a bf16 ulp of the sum."""
    return 2.0 ** -8 * (np.abs(y) + rest) + rest + 2.0 ** -133


def silu(v):
    return v / (1.0 + np.exp(-v))


def swiglu(g, u, tol_g, tol_u):
    """(h, what its fp32 value may be off by): silu is 1.1-Lipschitz; the fp32 evaluation
    (exponential to 2^-19 relative for |g| < 40, a division, two products) on top."""
    h = silu(g) * u
    move = 1.1 * tol_g * np.abs(u) + np.abs(silu(g)) * tol_u + 1.1 * tol_g * tol_u
    return h, move + 2.0 ** -18 * (np.abs(h) + move) + 2.0 ** -140


def check_quantised(codes, scales, want, tol, fit: bool):
    """Whether codes and scales are those of some values within `tol` of `want`: the
    exponents between those of the smallest and largest maxima, and, rounding being
    monotone, every value between the roundings of its interval's ends at that exponent."""
    t, d = want.shape
    blocks = d // BLOCK
    scales = np.asarray(scales)
    if np.any(scales[:, blocks:] != 0):
        return False
    e = scales[:, :blocks].astype(np.int64)
    b, w = want.reshape(t, blocks, BLOCK), tol.reshape(t, blocks, BLOCK)
    lo = exponent(np.maximum(np.abs(b) - w, 0.0).max(2), fit)
    hi = exponent((np.abs(b) + w).max(2), fit)
    if not np.all((lo <= e) & (e <= hi)):
        return False
    s = 2.0 ** (127.0 - e)[..., None]

    def rounded(v):
        return np.copysign(MAGNITUDES[round_code(np.abs(v * s))], v)
    got = (dequant(codes, scales).reshape(t, blocks, BLOCK)) * s
    return bool(np.all((rounded(b - w) <= got) & (got <= rounded(b + w))))


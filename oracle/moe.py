"""A mixture-of-experts layer for given choices in fp64, with what fp32 sums and
intermediates of 16 bits may be off by."""
import numpy as np

from .mxfp4 import swiglu

STEP = 2.0 ** -23


def product(x, tol_x, w):
    """(x @ w.T, its error bound): x off by tol_x, and a sum in fp32 in which a term goes
    through at most 32 additions in the matrix instruction that reads it, one for each 32
    codes after it (two where x has two parts), and 16 in the joining of parts; each loses at most 2^-23 of the sum of the
    magnitudes (products of a weight's 2 and a bf16's 8 bits are exact)."""
    a = (np.abs(x) + tol_x) @ np.abs(w).T
    return x @ w.T, tol_x @ np.abs(w).T + (33 + x.shape[1] / 16 + 16) * STEP * a


def two_parts(h):
    """What h is off by that is kept in two bf16 parts."""
    return 2.0 ** -16 * h + 2.0 ** -132


def pairs(h):
    """Two neighbours as multiples of one unit: 2^-10 of the larger one's binade, or of the next
    where it rounds there (from 2 - 2^-11 on), at least 2^-126."""
    most = np.repeat(h.reshape(*h.shape[:-1], -1, 2).max(-1), 2, -1)
    return 2.0 ** -11 * (1 + 2.0 ** -11) * most + 2.0 ** -127


def layer(x, gate_up, down, ids, weights, shared, kept=two_parts):
    """(out, tolerance of the bf16 output): gate_up[e] and down[e] dequantised matrices, ids
    [t][k] (-1: none), weights [t][k]; kept: what h of given magnitudes is off by in the workspace."""
    t, d = x.shape
    out, tol, mag = np.zeros((t, d)), np.zeros((t, d)), np.zeros((t, d))
    for i in range(t):
        for j, e in enumerate(ids[i]):
            if e < 0:
                continue
            half = gate_up[e].shape[0] // 2
            s, ts = product(x[i:i + 1], np.zeros((1, d)), gate_up[e])
            h, th = swiglu(s[:, :half], s[:, half:], ts[:, :half], ts[:, half:])
            th = th + kept(np.abs(h) + th)
            y, ty = product(h, th, down[e])
            out[i] += weights[i, j] * y[0]
            tol[i] += abs(weights[i, j]) * ty[0]
            mag[i] += abs(weights[i, j]) * (np.abs(y[0]) + ty[0])
    if shared is not None:
        out, mag = out + shared, mag + np.abs(shared)
    # every expert's product with its weight, the sum over experts, parts, waves and shared
    tol = tol + (ids.shape[1] + 20) * STEP * mag
    return out, 2.0 ** -8 * (np.abs(out) + tol) + tol + 2.0 ** -133

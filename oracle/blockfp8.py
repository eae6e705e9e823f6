"""FP8 E4M3FN in blocks of 128: quantisation and the block-scaled product in float64 (oracle; test
infrastructure only).

scale = max(largest magnitude / 448, 2^-126) of a row's 128 columns; a code stands for its E4M3FN
value times its scale.  The product sums every block's dot product times both scales.

Pinned by: hand-worked blocks, and torch's float8_e4m3fn conversion on the grid of half steps.
"""

import numpy as np

from .fp8 import E4M3FN_TABLE

BLOCK = 128
SCALE_MIN = 2.0 ** -126


def block_scales(x):
    """float64 scales [rows, blocks] of a matrix."""
    x = np.abs(np.asarray(x, np.float64))
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    out = np.empty((rows, nb))
    for b in range(nb):
        out[:, b] = x[:, b * BLOCK:(b + 1) * BLOCK].max(1)
    return np.maximum(out / 448.0, SCALE_MIN)


def spread(scale, cols):
    """A scale per block as a scale per column."""
    return np.repeat(scale, BLOCK, axis=1)[:, :cols]


_FINITE = np.unique(E4M3FN_TABLE[np.isfinite(E4M3FN_TABLE)])


def nearest_distance(v):
    """Distance of each value from the E4M3FN number nearest to it."""
    v = np.asarray(v, np.float64)
    i = np.clip(np.searchsorted(_FINITE, v), 1, len(_FINITE) - 1)
    return np.minimum(np.abs(v - _FINITE[i - 1]), np.abs(v - _FINITE[i]))


def matmul(a, a_scale, b, b_scale):
    """(c, T) in float64: the product of two matrices of codes, and the sum of the magnitudes of
    its terms, which bounds the rounding of any order of summation."""
    k = a.shape[1]
    av = E4M3FN_TABLE[a] * spread(np.asarray(a_scale, np.float64), k)
    rows = np.repeat(np.asarray(b_scale, np.float64), BLOCK, axis=0)[:b.shape[0]]
    bv = E4M3FN_TABLE[b] * spread(rows, k)
    return av @ bv.T, np.abs(av) @ np.abs(bv).T


def group_maxima(a, a_scale, b, b_scale):
    """Sum over the groups of eight neighbouring products of the largest magnitude among them, for
    every output: what a matrix core that aligns the products of a group loses goes by it."""
    m, k = a.shape
    n = b.shape[0]
    out = np.zeros((m, n))
    av, bv = np.nan_to_num(np.abs(E4M3FN_TABLE[a])), np.nan_to_num(np.abs(E4M3FN_TABLE[b]))
    for p in range(0, k, 8):
        g = (av[:, None, p:p + 8] * bv[None, :, p:p + 8]).max(2)
        out += g * np.asarray(a_scale, np.float64)[:, p // BLOCK][:, None] \
            * np.repeat(np.asarray(b_scale, np.float64)[:, p // BLOCK], BLOCK)[:n][None, :]
    return out

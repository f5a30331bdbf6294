"""Oracle: rows as signed 8-bit integers and the scaled integer GEMM.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

One scale per output channel of a weight and one per token of an activation.  With
a = max|x| of a row:

    scale = a / 127   and   inv = 127 / a,   each rounded to fp32 once,
    q     = the integer nearest to x * inv, ties to even,

a row with a < 2^-100 counts as zero (scale 1, q 0), and a row that holds an infinity
or a NaN has q 0 and a NaN scale.  The sums of products are exact integers and the
result is multiplied by both scales.
"""

import numpy as np

TINY = 2.0 ** -100


def row_scales(x):
    """(scale, inv) of each row, float64 arrays of fp32 values."""
    x = np.asarray(x, np.float64)
    a = np.abs(x).max(axis=-1)
    a = np.where(np.isnan(x).any(axis=-1), np.nan, a)
    none = a < TINY
    bad = ~np.isfinite(a)
    safe = np.where(none | bad, 1.0, a)
    # a float64 quotient of fp32 numbers rounds to fp32 as the exact quotient does (53 >= 2 * 24 + 2 bits)
    scale = (safe / 127.0).astype(np.float32).astype(np.float64)
    inv = (127.0 / safe).astype(np.float32).astype(np.float64)
    scale = np.where(bad, np.nan, np.where(none, 1.0, scale))
    return scale, np.where(none | bad, 0.0, inv)


def quantize_rows(x):
    """(integers as float64, scales); exact for x of at most 29 significant bits."""
    x = np.asarray(x, np.float64)
    scale, inv = row_scales(x)
    keep = np.isfinite(scale)
    q = np.rint(np.where(keep[:, None], x, 0.0) * inv[:, None])
    return q, scale


def scaled_matmul(x, w):
    """x [n, K] @ w [m, K].T in 8-bit integers: per-token scales of x, per-channel scales of w."""
    qx, sx = quantize_rows(x)
    qw, sw = quantize_rows(w)
    return (qx @ qw.T) * sx[:, None] * sw[None, :]

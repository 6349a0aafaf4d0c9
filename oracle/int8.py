"""int8 rows and the int8 expert FFN, plainly (oracle; test infrastructure only).

rows     scale = amax / 127 (fp32; 1 where amax is 0), code = value / scale rounded to nearest even
product  sums of code products are whole numbers, exact in fp64; times the row's and the channel's scale
FFN      A = silu(X W13[0:I]^T) * (X W13[I:2I]^T), A as int8 rows, y = A W2^T
"""
from __future__ import annotations

import numpy as np

TINY = np.float32(2.0 ** -126)


def rows(x):
    """(codes int8, scales fp32) of fp32 rows, every step rounded to fp32 as the operator defines it."""
    x = np.asarray(x, np.float32)
    amax = np.abs(x).max(1)
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        scale = np.where(amax == 0, np.float32(1), np.maximum(amax / np.float32(127), TINY)).astype(np.float32)
        bad = ~np.isfinite(amax)
        scale[bad] = np.nan
        q = np.rint(x / scale[:, None])
    q[bad] = 0
    return q.astype(np.int8), scale


def product(a, a_scale, w, w_scale):
    """fp64 a [M,K] w [N,K]^T with scales per row of each."""
    return (a.astype(np.float64) @ w.astype(np.float64).T) * a_scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)


def gate_up(x, x_scale, w13, s13):
    """(A [M,I] before its rounding, the gate's pre-activation [M,I])."""
    h = product(x, x_scale, w13, s13)
    g, u = np.split(h, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u, g

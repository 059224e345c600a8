"""Plain fp64 restatement of the 8-bit block-scaled projection (numpy).

The e4m3 values are found by comparing with the list of all of them, not by a conversion.
"""
from __future__ import annotations

import numpy as np

__all__ = ["e4m3_values", "round_e4m3", "quantize", "matmul"]


def e4m3_values():
    """The 127 finite values >= 0 of e4m3 (4 exponent bits of bias 7, 3 mantissa bits; the code with
    all of them set is NaN), in order."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    norm = [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return np.array((sub + norm)[:127])


def round_e4m3(x):
    """Nearest e4m3 value, ties to the even code, saturated at 448."""
    x = np.asarray(x, dtype=np.float64)
    v = e4m3_values()
    a = np.minimum(np.abs(x), v[-1])
    hi = np.searchsorted(v, a, side="left")
    lo = np.maximum(hi - 1, 0)
    mid = (v[lo] + v[hi]) / 2
    pick = np.where(a > mid, hi, np.where(a < mid, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.copysign(v[pick], x)


def quantize(x, rows):
    """(values [R, C], fp32 scales): the scale is the fp32 number nearest to amax / 448 (at least
    2^-126); a value is rounded from the fp32 number nearest to x / scale."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    rb, cb = -(-R // rows), -(-C // 128)
    q = np.empty_like(x)
    scale = np.empty((rb, cb), dtype=np.float32)
    for i in range(rb):
        for j in range(cb):
            blk = np.s_[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]
            s = max(np.float32(np.abs(x[blk]).max() / 448.0), np.float32(2.0 ** -126))
            scale[i, j] = s
            q[blk] = round_e4m3((x[blk] / np.float64(s)).astype(np.float32))
    return q, scale


def matmul(a, sa, b, sb):
    K = a.shape[1]
    A = np.asarray(a, dtype=np.float64) * np.repeat(np.asarray(sa, dtype=np.float64), 128, axis=1)[:, :K]
    S = np.repeat(np.repeat(np.asarray(sb, dtype=np.float64), 128, axis=0), 128, axis=1)
    B = np.asarray(b, dtype=np.float64) * S[:b.shape[0], :K]
    return A @ B.T, np.abs(A) @ np.abs(B).T

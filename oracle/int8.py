"""CPU oracle for the products in 8-bit integers: codes and scales bit by bit, products in
whole numbers, the scaling in fp64.

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package).

  rows to 8 bits  s = fl32(max |x| / 127), c = round-half-even(fl32(x / s)) in [-127, 127];
                  s = 0, c = 0 for a row of zeros; s = NaN, c = 0 for a row that holds an
                  infinity or a NaN
  product         y[i, j] = s_i t_j sum_k c[i, k] d[j, k] (+ bias[j])
"""
from __future__ import annotations

import numpy as np


def rows_to_int8(x):
    """(codes int8, scale fp32) of the last dimension of x (values exact in fp32)."""
    x = np.asarray(x, np.float32)
    codes = np.zeros(x.shape, np.int8)
    if x.shape[-1] == 0:
        return codes, np.zeros(x.shape[:-1], np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        scale = (np.abs(x).max(axis=-1) / np.float32(127)).astype(np.float32)
        scale[~np.isfinite(x).all(axis=-1)] = np.nan
        c = np.rint((x / scale[..., None]).astype(np.float32))
    live = (scale > 0)[..., None] & np.ones(x.shape, bool)
    codes[live] = np.clip(c[live], -127, 127).astype(np.int8)
    return codes, scale


def product(x, codes, scale, bias=None):
    """(y in fp64, |scaled sum| in fp64) of tokens x with a weight's codes [n, k] and scales [n]."""
    c, s = rows_to_int8(x)
    acc = c.astype(np.int64) @ codes.astype(np.int64).T
    y = acc.astype(np.float64) * s.astype(np.float64)[:, None] * scale.astype(np.float64)[None, :]
    mag = np.abs(y)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)[None, :]
    return y, mag


def clean_offsets(offsets, m):
    """The rows each expert has: [0, m] limits, and an offset below an earlier one counts as it."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, m))

"""CPU oracle for the products in 8-bit floats (e4m3) with power-of-two block scales.

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package).

  block    s = 2^e, e the smallest integer >= -127 with max |x| <= 448 s; code = the e4m3 value
           nearest to x / s, ties to the even code; s = 1 and NaN codes where the block holds an
           infinity or a NaN.  Tokens: 128 columns of a row; weights: 128 rows by 128 columns.
  product  y[i, j] = sum_k xq[i, k] wq[j, k] (+ bias[j]) over the values the codes stand for
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def values():
    """The value of each of the 256 codes."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


_MAG = values()[:127]  # magnitudes, ascending


def encode(v):
    """Codes of v (fp64, |v| <= 448, or NaN): the nearest magnitude, ties to the even code."""
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_MAG, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _MAG[lo], _MAG[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(v), code + 128, code)
    return np.where(np.isnan(v), 127, code).astype(np.uint8)


def exponent(amax):
    """e of a block from its largest magnitude (fp64), by trying every exponent."""
    e = np.full(np.shape(amax), -127)
    for k in range(-127, 121):
        e = np.where(amax > 448.0 * 2.0 ** k, k + 1, e)
    return e


def to_fp8(x, tall):
    """(codes [rows, ld], exponent bytes [row blocks, column blocks]) of x by blocks of `tall` rows."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    rb, kb = -(-rows // tall), -(-cols // BLOCK)
    p = np.zeros((rb * tall, kb * BLOCK))
    p[:rows, :cols] = x
    b = p.reshape(rb, tall, kb, BLOCK)
    bad = ~np.isfinite(b).all(axis=(1, 3))
    e = np.where(bad, 0, exponent(np.where(np.isfinite(b), np.abs(b), 0).max(axis=(1, 3))))
    v = np.where(bad[:, None, :, None], np.nan, b) / 2.0 ** e[:, None, :, None]
    codes = encode(v).reshape(p.shape)
    codes[:, cols:] = 0
    return codes[:rows], (e + 127).astype(np.uint8)


def decode(codes, scale, tall, cols):
    """Values [rows, cols] of codes under their blocks' exponent bytes."""
    v = values()[codes]
    s = 2.0 ** (scale.astype(np.float64) - 127)
    s = np.repeat(np.repeat(s, tall, axis=0)[: v.shape[0]], BLOCK, axis=1)[:, : v.shape[1]]
    return (v * s)[:, :cols]


def product(x, w, bias=None):
    """(y, sum of the products' magnitudes) of tokens x [m, k] with a weight w [n, k], in fp64."""
    cols = x.shape[1]
    xq = decode(*to_fp8(x, 1), 1, cols)
    wq = decode(*to_fp8(w, BLOCK), BLOCK, cols)
    y = xq @ wq.T
    mag = np.abs(xq) @ np.abs(wq).T
    return (y if bias is None else y + np.asarray(bias, np.float64)[None, :]), mag

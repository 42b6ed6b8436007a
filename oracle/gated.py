"""CPU oracle for the gated feed-forward block, h = act(g) u, in fp64.

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package).
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def act(z, kind):
    """(act(z), act'(z)), from the textbook forms."""
    z = np.asarray(z, np.float64)
    if kind == "silu":
        with np.errstate(over="ignore"):
            q = 1 / (1 + np.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if kind == "gelu":
        phi = 0.5 * _erfc(-z / math.sqrt(2))
        return z * phi, phi + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def forward(g, u, kind):
    return act(g, kind)[0] * np.asarray(u, np.float64)


def backward(g, u, dh, kind):
    """(dg, du)."""
    value, slope = act(g, kind)
    dh = np.asarray(dh, np.float64)
    return dh * np.asarray(u, np.float64) * slope, dh * value

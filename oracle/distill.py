"""CPU oracle for the distillation loss against a teacher's top logits, in fp64, row by row.

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package).

  p = softmax(u / T) over the present slots, q = softmax(z / T) over the vocabulary,
  kl = T^2 sum_j p_j (log p_j - log q[idx_j]), loss = sum_i w_i kl_i, dz_i = w_i T (q - p).
A slot is absent when its index lies outside the vocabulary or its value is -inf; a row of
weight 0 or without a present slot has kl 0 and gradient 0.
"""
from __future__ import annotations

import numpy as np


def _log_softmax(v):
    m = v.max()
    with np.errstate(invalid="ignore", divide="ignore"):
        e = v - m
        return e - np.log(np.exp(e).sum())


def loss_grad(z, u, idx, temperature=1.0, weight=None):
    """Returns (loss, kl [n], dz [n, V], kl_mag [n]); kl_mag is the size of the numbers that
    cancel in kl (for rounding bounds)."""
    z, u, idx = np.asarray(z, np.float64), np.asarray(u, np.float64), np.asarray(idx, np.int64)
    n, V = z.shape
    w = np.full(n, 1.0 / n) if weight is None else np.asarray(weight, np.float64)
    T = float(temperature)
    kl, mag, dz = np.zeros(n), np.zeros(n), np.zeros((n, V))
    for i in range(n):
        here = (idx[i] >= 0) & (idx[i] < V) & ~(u[i] == -np.inf)
        if w[i] == 0 or not here.any():
            continue
        at = idx[i][here]
        lp = _log_softmax(u[i][here] / T)
        lq = _log_softmax(z[i] / T)
        p = np.exp(lp)
        with np.errstate(invalid="ignore"):
            terms = np.where(p == 0, 0.0, p * (lp - lq[at]))
            mags = np.where(p == 0, 0.0, p * (1.0 + np.abs(lp) + np.abs(lq[at]) + np.abs(z[i][at] - z[i].max()) / T
                                              + np.abs(u[i][here] - u[i][here].max()) / T))
        kl[i], mag[i] = T * T * terms.sum(), T * T * mags.sum()
        g = np.exp(lq)
        np.subtract.at(g, at, p)
        dz[i] = w[i] * T * g
    live = w != 0
    return float((w[live] * kl[live]).sum()), kl, dz, mag

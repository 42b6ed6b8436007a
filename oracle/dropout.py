"""CPU oracle for the QLoRA layer with LoRA dropout (p > 0).

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package).

Pages: rust_ai_core QLoraConfig docs, "Fields" (the LoRA configuration carries rank,
alpha and dropout); "LoRA and QLoRA, mathematically", "Tooling" (PEFT's LoraConfig
with its dropout field).  Reading (PEFT's LoRA dropout, the plainest one the pages
support): dropout acts on the input of the low-rank branch only, as inverted
dropout with a caller-drawn keep mask M (1 = kept) and rate p:

    x_d = x * M / (1 - p)
    y   = x W~^T + s (x_d A^T) B^T (+ bias)

and with W frozen:  dT = s dY B,  dX = dY W~ + (dT A) * M / (1 - p),
dA = dT^T x_d,  dB = s dY^T (x_d A^T).

Arithmetic is fp64 with plain matrix products; operands are the exact values the
kernels read (compute-dtype values as fp32 arrays, the mask as 0/1).
"""
from __future__ import annotations

import numpy as np


def _d(a):
    return np.asarray(a, np.float64)


def forward(x, W, A, B, s: float, mask, p: float, bias=None):
    x, W, A, B, M = _d(x), _d(W), _d(A), _d(B), _d(mask)
    xd = x * M / (1.0 - p)
    y = x @ W.T + s * (xd @ A.T) @ B.T
    return y if bias is None else y + _d(bias)[None, :]


def backward(x, W, A, B, dY, s: float, mask, p: float):
    x, W, A, B, dY, M = _d(x), _d(W), _d(A), _d(B), _d(dY), _d(mask)
    xd = x * M / (1.0 - p)
    dT = s * dY @ B
    dX = dY @ W + (dT @ A) * M / (1.0 - p)
    dA = dT.T @ xd
    dB = s * dY.T @ (xd @ A.T)
    return dX, dA, dB


def philox(counter, key):
    """The four words of Philox 4x32-10 (Salmon et al., SC 2011) for one counter (four words) and
    key (two), in Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def threshold(p: float) -> int:
    return min(65535, int(np.floor(float(np.float32(p)) * 65536 + 0.5)))


def drawn_mask(m: int, cols: int, seed: int, offset: int, p: float):
    """The keep mask [m, cols] (u8) the seeded dropout draws, word by word in numpy."""
    lo, t = np.uint64(0xFFFFFFFF), threshold(p)
    seed, offset = seed & ((1 << 64) - 1), offset & ((1 << 64) - 1)
    groups = -(-cols // 8)
    c = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (m, groups)),
         np.broadcast_to(np.arange(m, dtype=np.uint64)[:, None], (m, groups)),
         np.full((m, groups), offset & 0xFFFFFFFF, np.uint64), np.full((m, groups), offset >> 32, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & lo, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    halves = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], axis=2)
    return (halves.reshape(m, groups * 8)[:, :cols] >= t).astype(np.uint8)

"""The 4-bit row format and attention over it in 64 bits, from their definition
(include/qa.h): numpy and torch float64, none of the library's code."""
from __future__ import annotations

import numpy as np
import torch

GROUP = 32
NAN_BYTE = 0x7F
# The value of every scale byte up to the largest: 5 exponent and 2 mantissa bits.
SCALES = np.array([(b & 3) * 2.0 ** -16 if b < 4 else (4 + (b & 3)) * 2.0 ** ((b >> 2) - 17)
                   for b in range(0x54)])


def quantise(x: np.ndarray):
    """(codes [..., D/2] uint8, scale bytes [..., D/32] uint8) of rows x [..., D]."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    top = np.abs(g).max(-1)
    fine = np.isfinite(top)
    t = np.minimum(np.where(fine, top, 0.0) / 7, SCALES[-1])
    # 7 has no power of two but 1: a tie of two scales is a bf16 value times 1/7 that
    # float64's quotient reproduces exactly, and nothing else comes within 2^-9 of one.
    dist = np.abs(t[..., None] - SCALES)
    best = dist.min(-1, keepdims=True)
    byte = np.where(dist == best, np.arange(SCALES.size) + 1000 * (np.arange(SCALES.size) % 2),
                    10 ** 6).min(-1) % 1000
    s = SCALES[byte][..., None]
    q = np.where(np.isfinite(g) & (s > 0), g, 0.0) / np.where(s > 0, s, 1.0)
    n = np.clip(np.sign(q) * np.floor(np.abs(q) + 0.5), -8, 7) + 8
    n = np.where(fine[..., None], n, 8).astype(np.uint8).reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return n[..., 0] | n[..., 1] << 4, np.where(fine, byte, NAN_BYTE).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*scales.shape, GROUP).astype(np.float64) - 8
    table = np.concatenate((SCALES, np.full(256 - SCALES.size, np.nan)))
    return (n * table[scales][..., None]).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, start: int, window: int = 0):
    """q [n, Hq, D] at positions start.. over k, v [Hkv, start + n, D]: causal
    softmax attention and, per output, sum_j p_j |v_j| (what a relative error of
    the weights is scaled by).  All float64."""
    n, hq, d = q.shape
    group = hq // k.shape[0]
    pos = torch.arange(start, start + n, device=q.device)[:, None]
    key = torch.arange(start + n, device=q.device)[None]
    hidden = key > pos
    if window:
        hidden = hidden | (key <= pos - window)
    out, mag = torch.empty_like(q), torch.empty_like(q)
    for h in range(hq):
        t = (q[:, h] @ k[h // group].T / d ** 0.5).masked_fill(hidden, -torch.inf)
        p = torch.softmax(t, -1)
        out[:, h] = p @ v[h // group]
        mag[:, h] = p @ v[h // group].abs()
    return out, mag

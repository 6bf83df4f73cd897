"""The 8-bit block format, the choice of blocks and attention over them, from their
definition (include/qa.h): numpy and torch, none of the library's code.  The format's
own roundings are fp32's; everything else is in 64 bits."""
from __future__ import annotations

import numpy as np
import torch

BLOCK = 64
SMALL = 2.0 ** -64


def _codes(x: np.ndarray, axes):
    """Integers of x with one scale over `axes`, and the scales."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        a = np.abs(x).max(axes, keepdims=True)
        fine = np.isfinite(x).all(axes, keepdims=True)
        used = fine & (a >= np.float32(SMALL))
        by = np.float32(127) / np.where(used, a, np.float32(1))
        n = np.rint((np.where(used, x, np.float32(0)) * by).astype(np.float32))
        s = np.where(used, a / np.float32(127), np.float32(0))
    return n.astype(np.int32), np.where(fine, s, np.float32(np.nan)).astype(np.float32)


def quantise(x: np.ndarray):
    """(n [..., 64, D] int32, s [...] fp32) of blocks x [..., 64, D]."""
    n, s = _codes(x, (-2, -1))
    return n, s[..., 0, 0]


def values(n: np.ndarray, s: np.ndarray) -> np.ndarray:
    return n.astype(np.float64) * s[..., None, None].astype(np.float64)


def bf16(x: np.ndarray) -> np.ndarray:
    """float64 of x rounded to fp32 and then to bf16."""
    return torch.from_numpy(np.asarray(x, np.float64)).float().bfloat16().double().numpy()


def scores(q: np.ndarray, n: np.ndarray, s: np.ndarray) -> np.ndarray:
    """q [G, D] of one kv head, complete blocks n [full, 64, D], s [full]: their scores."""
    if np.isfinite(q).all():
        c, _ = _codes(q, (0, 1))
    else:
        c = np.zeros(q.shape, np.int32)
    lo, hi = n.min(1), n.max(1)
    got = np.array([np.maximum(c * lo[j], c * hi[j]).sum() for j in range(len(n))], np.float32) * s
    got[np.isnan(s)] = np.inf
    got[[0, -1]] = np.inf
    return got


def select(q, n, s, n_blocks):
    """The chosen blocks in rising order, then -1."""
    full = len(n)
    got = np.full(n_blocks, -1, np.int32)
    if full:
        x = scores(q, n, s)
        best = sorted(sorted(range(full), key=lambda j: (-x[j], j))[:n_blocks])
        got[: len(best)] = best
    return got


def attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, start: int):
    """q [n, Hq, D] at positions start .. over k, v [Hkv, start + n, D]: causal softmax
    attention; per output sum_j p_j |v_j| (what a relative error of the weights is scaled
    by) and sum_j |v_j| / sum_j e^(t_j - max t) (an absolute one).  All float64."""
    n, hq, d = q.shape
    group = hq // k.shape[0]
    keys = k.shape[1]
    hidden = torch.arange(keys, device=q.device)[None] > torch.arange(keys - n, keys, device=q.device)[:, None]
    out, mag, flat = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    for h in range(hq):
        t = (q[:, h] @ k[h // group].T / d ** 0.5).masked_fill(hidden, -torch.inf)
        w = torch.exp(t - t.amax(-1, keepdim=True))
        w = torch.where(hidden, 0.0, w)
        l = w.sum(-1, keepdim=True)
        out[:, h] = w @ v[h // group] / l
        mag[:, h] = w @ v[h // group].abs() / l
        flat[:, h] = (~hidden).double() @ v[h // group].abs() / l
    return out, mag, flat


class Rows:
    """What a layer of the cache holds: rows as they came and complete blocks.  k, v
    are float64 [T, Hkv, D]."""

    def __init__(self, batch, hkv, d, cap):
        self.hkv, self.d = hkv, d
        nblk = -(-cap // BLOCK)
        self.came = np.zeros((2, batch, hkv, nblk * BLOCK, d))
        self.n = np.zeros((2, batch, hkv, nblk, BLOCK, d), np.int32)
        self.s = np.zeros((2, batch, hkv, nblk), np.float32)

    def write(self, start, ntok, k, v):
        at = 0
        for b, (p, m) in enumerate(zip(start, ntok)):
            for i, x in enumerate((k, v)):
                self.came[i, b, :, p:p + m] = x[at:at + m].swapaxes(0, 1)
                for j in range(p // BLOCK, (p + m) // BLOCK):
                    self.n[i, b, :, j], self.s[i, b, :, j] = quantise(self.came[i, b, :, j * BLOCK:(j + 1) * BLOCK])
            at += m

    def held(self, i, b, end, blocks=None):
        """Rows below `end` of sequence b as attention sees them in a call that begins
        there, [Hkv, .., D]; blocks [Hkv, m]: of complete blocks these alone."""
        full = end // BLOCK
        got = []
        for h in range(self.hkv):
            pick = np.arange(full) if blocks is None else blocks[h][blocks[h] >= 0]
            x = values(self.n[i, b, h, pick], self.s[i, b, h, pick]).reshape(-1, self.d)
            got.append(np.concatenate((x, self.came[i, b, h, full * BLOCK:end])))
        return got

    def read(self, i, b, start, m, end):
        """What qa_q8_read gives of positions start .. start + m - 1 of a sequence of `end`."""
        full = end // BLOCK
        x = np.concatenate((bf16(values(self.n[i, b, :, :full], self.s[i, b, :, :full]).reshape(self.hkv, -1, self.d)),
                            self.came[i, b, :, full * BLOCK:end]), 1)
        return x[:, start:start + m].swapaxes(0, 1)

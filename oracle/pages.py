"""Oracle of the long-context operators: plain numpy, CPU only.

* ``rotate_axes``: pair i of a row turns by the row's position on axis[i]; otherwise kv4.rotate.
* ``summarize``: smallest and largest of a page's keys per channel, 8-bit codes under one scale.
* ``select``: the pages that each row of queries reads, in whole numbers and single fp32 products.
"""
from __future__ import annotations

import numpy as np

D = 128


def rotate_axes(x: np.ndarray, positions: np.ndarray, axis, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x fp32 [rows][heads][128], positions [rows][axes], cos / sin fp32 [positions][rot / 2]."""
    y = np.array(x, dtype=np.float32)
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[positions[:, axis[i]], i][:, None], sin[positions[:, axis[i]], i][:, None]
        xa, xb = np.float32(x[..., a]), np.float32(x[..., b])
        y[..., a] = xa * c - xb * s
        y[..., b] = xb * c + xa * s
    return y


def summarize(k: np.ndarray):
    """k fp32 [tokens][128], one page's cached values -> codes int8 [256] (largest, then smallest), scale fp32."""
    k = np.asarray(k, dtype=np.float32)
    hi, lo = k.max(0), k.min(0)
    s = np.maximum(np.abs(hi), np.abs(lo)).max() / np.float32(127)
    if s == 0:
        return np.zeros(2 * D, np.int8), np.float32(0)
    return np.concatenate([np.minimum(np.ceil(hi / s), 127), np.maximum(np.floor(lo / s), -127)]).astype(np.int8), s


def query_codes(q: np.ndarray):
    """q [...][128] (bf16 values) -> whole numbers [...][128], scales fp32 [...]."""
    q = np.asarray(q, dtype=np.float32)
    t = np.abs(q).max(-1) / np.float32(127)
    safe = np.where(t > 0, t, np.float32(1))[..., None]
    return np.where(t[..., None] > 0, np.clip(np.rint(q / safe), -127, 127), 0).astype(np.int64), t


def scores(q: np.ndarray, codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """q [heads][128] of one K/V head's group, codes int8 [blocks][256], scale fp32 [blocks] -> fp32 [blocks]."""
    qc, t = query_codes(q)
    hi, lo = codes[:, :D].astype(np.int64), codes[:, D:].astype(np.int64)
    best = None
    for c, th in zip(qc, t):
        z = th * np.maximum(c * hi, c * lo).sum(-1).astype(np.float32)
        best = z if best is None else np.maximum(best, z)
    return (best * scale).astype(np.float32)


def select(q, codes, scale, position: int, page: int, keep: int, first: int, last: int):
    """Blocks (ascending) and tokens that a row at `position` reads; codes and scale of its blocks 0, 1, ..."""
    n = position // page + 1
    if n <= keep:
        return np.arange(n), position + 1
    s = scores(q, codes[:n], scale[:n])
    s[:first] = s[n - last:] = np.inf
    return np.sort(np.lexsort((np.arange(n), -s))[:keep]), (keep - 1) * page + position % page + 1

"""Oracle of the rotated appends and of the 4-bit cache: plain numpy, CPU only, one token and one byte at
a time where the layout is concerned.  Test infrastructure, as the rest of this package.

* ``rotate``: a pair (a, b) of channels at position p becomes (a c - b s, b c + a s), every product
  and sum an IEEE fp32 operation of its own.
* ``quantize4``: groups of 32 channels, scale fp16(bf16(max|x| / 7)) <= 9344, code
  clamp(round_half_even(x / scale), -7, 7), codes 0 under a zero scale.
* ``write4`` / ``read4``: the page layout (see include/cai.h, cai_kv4_pool).
* ``attend_rows``: softmax attention in float64, with the weighted sum of |v| that error bounds need.
"""
from __future__ import annotations

import numpy as np

D, GROUP, BLOCK = 128, 32, 2304


def bf16_round(x: np.ndarray) -> np.ndarray:
    """fp32 -> nearest bf16 (ties to even), as fp32."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32).reshape(np.shape(x))


def rotate(x: np.ndarray, pos: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x fp32 [rows][heads][128], pos [rows], cos / sin fp32 [positions][rot / 2]."""
    half = cos.shape[1]
    y = np.array(x, dtype=np.float32)
    a, b = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved else (np.arange(half), np.arange(half) + half)
    c, s = cos[pos][:, None].astype(np.float32), sin[pos][:, None].astype(np.float32)
    xa, xb = np.float32(x[..., a]), np.float32(x[..., b])
    y[..., a] = xa * c - xb * s
    y[..., b] = xb * c + xa * s
    return y


def quantize4(x: np.ndarray):
    """x fp32 [..., 128] -> codes int8 [..., 128], scales fp16 [..., 4]."""
    g = np.ascontiguousarray(x, dtype=np.float32).reshape(*x.shape[:-1], D // GROUP, GROUP)
    s = np.minimum(bf16_round(np.abs(g).max(-1) / np.float32(7)), np.float32(9344)).astype(np.float16)
    sf = s.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(sf > 0, np.clip(np.rint(g / sf), -7, 7), 0)
    return c.astype(np.int8).reshape(x.shape), s


def dequantize4(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values, exact."""
    return codes.astype(np.float64) * np.repeat(scales.astype(np.float64), GROUP, -1)


def page_bytes4(page_size: int) -> int:
    return page_size // 16 * BLOCK


def pool4(num_pages: int, page_size: int, fill: int = 0xFF) -> np.ndarray:
    """An untouched pool; 0xFF bytes make every scale a NaN and every code 7."""
    return np.full(num_pages * page_bytes4(page_size), fill, dtype=np.uint8)


def _where(table_row, pos: int, page_size: int):
    """Byte offset of the block of position pos, and the token's slot in it."""
    slot = pos % page_size
    return int(table_row[pos // page_size]) * page_bytes4(page_size) + slot // 16 * BLOCK, slot % 16


_CH = np.arange(D)


def _k_at(r):
    """Byte (in the block) and bit of every channel's K code of token r."""
    bit = 4 * (_CH % 8 // 2) + 16 * (_CH % 2)
    return 64 * r + 16 * (_CH % 32 // 8) + 4 * (_CH // 32) + bit // 8, bit % 8


def _v_at(r):
    m, g, i0 = _CH // 16, _CH % 8, _CH % 16 // 8
    t, b, e = r % 8 // 2, r // 8, r % 2
    bit = 4 * (2 * b + i0) + 16 * e
    return 1024 + 4 * ((32 * (m // 4) + 4 * g + t) * 4 + m % 4) + bit // 8, bit % 8


def _ks_at(r):
    return 2048 + 8 * r + 2 * np.arange(4)


def _vs_at(r):
    return 2176 + 2 * (16 * (r % 8 // 2) + 8 * (r // 8) + 2 * np.arange(4) + r % 2)


def write4(pool, table_row, pos0, kc, ks, vc, vs, page_size) -> None:
    """Codes [n][128] and scales [n][4] of tokens pos0 .. pos0 + n - 1 into their pages."""
    for i in range(len(kc)):
        base, r = _where(table_row, pos0 + i, page_size)
        for at, codes in ((_k_at(r), kc[i]), (_v_at(r), vc[i])):
            for byte, bit, code in zip(base + at[0], at[1], codes):
                pool[byte] = (int(pool[byte]) & ~(15 << int(bit)) & 0xFF) | ((int(code) + 8) << int(bit))
        half = pool.view(np.float16)
        half[(base + _ks_at(r)) // 2] = ks[i]
        half[(base + _vs_at(r)) // 2] = vs[i]


def read4(pool, table_row, positions, page_size):
    """(K codes, K scales, V codes, V scales) of the given positions."""
    kc, ks, vc, vs = [], [], [], []
    half = pool.view(np.float16)
    for p in positions:
        base, r = _where(table_row, int(p), page_size)
        for at, to in ((_k_at(r), kc), (_v_at(r), vc)):
            to.append((pool[base + at[0]].astype(np.int32) >> at[1] & 15) - 8)
        ks.append(half[(base + _ks_at(r)) // 2])
        vs.append(half[(base + _vs_at(r)) // 2])
    return np.array(kc, np.int8), np.array(ks), np.array(vc, np.int8), np.array(vs)


def attend_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, seen: np.ndarray):
    """q [n][h][128], k, v [T][128] float64, seen bool [n][T] -> out [n][h][128], lse [n][h], and for error
    bounds sum p |v| [n][h][128] and max over seen keys of scale * sum |q k| [n][h]."""
    z = np.einsum("nhd,td->nht", q, k) * scale
    z = np.where(seen[:, None], z, -np.inf)
    m = z.max(-1, keepdims=True, initial=-np.inf)
    e = np.exp(z - np.where(np.isfinite(m), m, 0.0))
    s = e.sum(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(s > 0, np.where(np.isfinite(m), m, 0.0)[..., 0] + np.log(s), -np.inf)
    p = e / np.where(s > 0, s, 1.0)[..., None]
    big = np.where(seen[:, None], np.einsum("nhd,td->nht", np.abs(q), np.abs(k)) * abs(scale), 0.0).max(-1, initial=0.0)
    return np.einsum("nht,td->nhd", p, v), lse, np.einsum("nht,td->nhd", p, np.abs(v)), big

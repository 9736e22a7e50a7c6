"""Plain fp64 form of the serving step around a paged key/value cache.

Positions: token i (of n new ones) of a sequence of length kv (with them) is at
kv - n + i, in page table[pos // page], row pos % page.
"""

from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import numpy as np


def norm_rope(x: np.ndarray, weight: Optional[np.ndarray], eps: float, angles: np.ndarray,
              rot: int, interleaved: bool) -> np.ndarray:
    """x [..., heads, 128] fp64; angles [..., rot]: cosines then sines of the row's position."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * weight
    if rot == 0:
        return y
    out = y.copy()
    for m in range(rot // 2):
        i, j = (2 * m, 2 * m + 1) if interleaved else (m, m + rot // 2)
        c = angles[..., None, m]
        s = angles[..., None, rot // 2 + m]
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
    return out


def rope_table(rows: int, rot: int, base: float = 500000.0) -> np.ndarray:
    inv = base ** (-np.arange(0, rot, 2, dtype=np.float64) / max(rot, 1))
    ang = np.arange(rows, dtype=np.float64)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], axis=1).astype(np.float32)


def sequence_rows(cache: np.ndarray, table: Sequence[int], head: int, length: int) -> np.ndarray:
    """Rows 0..length-1 of one sequence and kv head from [pages, heads, page, 128]."""
    page = cache.shape[2]
    out = np.empty((length, cache.shape[3]), cache.dtype)
    for x in range(length):
        out[x] = cache[table[x // page], head, x % page]
    return out


def page_bounds(q: np.ndarray, lo: np.ndarray, hi: np.ndarray) -> np.ndarray:
    """fp32 score of every page: max over the heads q [group, 128] of
    sum_d max(q_d lo_d, q_d hi_d), lo / hi [pages, 128], summed in fp64."""
    u = np.maximum(q[:, None] * lo[None], q[:, None] * hi[None])
    total = np.array([[math.fsum(row) for row in head] for head in u], dtype=np.float64)
    return total.max(axis=0).astype(np.float32)


def select_pages(pos: int, page: int, sink: int, local: int, top: int, score) -> np.ndarray:
    """Ascending pages of a token at pos; score(first, last) gives the fp32
    scores of pages first..last-1.  Ties go to the lowest page."""
    if pos < 0:
        return np.zeros(0, np.int64)
    seen = pos // page + 1
    first, last = min(sink, seen), max(seen - local, 0)
    always = [p for p in range(seen) if p < sink or p >= seen - local]
    middle = list(range(first, last)) if last > first else []
    if len(middle) > top:
        u = score(first, last)
        ranked = sorted(range(len(middle)), key=lambda i: (-float(u[i]), i))
        middle = [middle[i] for i in ranked[:top]]
    return np.array(sorted(set(always) | set(middle)), np.int64)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float
           ) -> Tuple[np.ndarray, float, np.ndarray]:
    """Output, LSE and sum p|v| of one query over the keys given (none: 0, -inf)."""
    if k.shape[0] == 0:
        z = np.zeros(v.shape[1])
        return z, -math.inf, z
    s = (k @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    l = p.sum()
    return (p @ v) / l, float(m + math.log(l)), (p @ np.abs(v)) / l

"""Helpers of the paged-cache tests: a batch of sequences over a shuffled cache.

Everything that no sequence owns -- the unfilled ends of pages, free pages, the
gap between strided pages, token rows outside the sequences -- holds NaN, so a
read of it that reaches an output shows.
"""

from __future__ import annotations

import math

import numpy as np
import torch

import block_sparse_long_sm_b200 as spa
from oracle import paged as op
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

D = 128


def to_gpu(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def to_f64(t: torch.Tensor) -> np.ndarray:
    return t.float().cpu().numpy().astype(np.float64)


def bits_of(x: np.ndarray) -> np.ndarray:
    return f32_to_bf16_bits(np.ascontiguousarray(x, np.float32))


def f64(bits: np.ndarray) -> np.ndarray:
    return bf16_bits_to_f32(bits).astype(np.float64)


NAN_BITS = np.uint16(0x7FC0)


class Batch:
    """Sequences with (n, kv) each; K/V bits of every position, and the GPU's tensors.

    filled: "all" puts every position below kv into the cache, "old" only those
    before the new tokens (the state before an append)."""

    def __init__(self, hq, hkv, page, seqs, *, seed=0, filled="all", gap=0, joint=False,
                 free=2, extra_cols=1, lead_rows=0, pad_rows=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.page, self.group = hq, hkv, page, hq // hkv
        self.n = [a for a, _ in seqs]
        self.kv = [b for _, b in seqs]
        self.S = len(seqs)
        need = [max(0, (b + page - 1) // page) for b in self.kv]
        self.per_seq = max([1] + need) + extra_cols
        self.num_pages = sum(need) + free
        perm = rng.permutation(self.num_pages)
        self.table = rng.integers(0, self.num_pages, size=(max(self.S, 1), self.per_seq)).astype(np.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = perm[at:at + m]
            at += m
        self.cu = lead_rows + np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        self.T = int(self.cu[-1]) + pad_rows
        own = hkv * page * D
        self.stride = own * (2 if joint else 1) + gap * D
        # K/V bits of every position of every sequence
        self.k = [bits_of(rng.standard_normal((max(b, 0), hkv, D))) for b in self.kv]
        self.v = [bits_of(rng.standard_normal((max(b, 0), hkv, D))) for b in self.kv]
        raw = np.full((2 if not joint else 1, self.num_pages * self.stride), NAN_BITS, np.uint16)
        if joint:
            base = torch.from_numpy(raw.view(np.int16)).cuda().view(torch.bfloat16)[0]
            self.raw = [base]
            views = [base, base[own:]]
        else:
            self.raw = [to_gpu(raw[0]), to_gpu(raw[1])]
            views = self.raw
        size = (self.num_pages, hkv, page, D)
        st = (self.stride, page * D, D, 1)
        self.kc, self.vc = (x.as_strided(size, st, x.storage_offset()) for x in views)
        kh = np.full(size, NAN_BITS, np.uint16)
        vh = np.full(size, NAN_BITS, np.uint16)
        for s in range(self.S):
            hi = self.kv[s] if filled == "all" else max(0, self.kv[s] - self.n[s])
            for x in range(hi):
                kh[self.table[s, x // page], :, x % page] = self.k[s][x]
                vh[self.table[s, x // page], :, x % page] = self.v[s][x]
        self.kc.copy_(to_gpu(kh))
        self.vc.copy_(to_gpu(vh))
        # token rows: a fused projection, NaN outside the sequences
        self.qkv = np.full((self.T, hq + 2 * hkv, D), NAN_BITS, np.uint16)
        lo, hi = int(self.cu[0]), int(self.cu[-1])
        self.qkv[lo:hi] = bits_of(rng.standard_normal((hi - lo, hq + 2 * hkv, D)))
        self.qkv_gpu = to_gpu(self.qkv)
        self.q = self.qkv_gpu[:, :hq]
        self.cu_gpu = torch.from_numpy(self.cu).cuda()
        self.kv_gpu = torch.tensor(self.kv, dtype=torch.int32).cuda() if self.S else \
            torch.zeros(1, dtype=torch.int32).cuda()
        self.table_gpu = torch.from_numpy(self.table).cuda()
        self.error = torch.zeros(1, dtype=torch.int32, device="cuda")

    def params(self, **kw):
        return spa.make_paged_params(
            self.hq, self.hkv, page_size=self.page, num_pages=self.num_pages, seqs=self.S,
            tokens=self.T, pages_per_seq=self.per_seq,
            page_stride=0 if self.stride == self.hkv * self.page * D else self.stride, **kw)

    def tokens(self):
        """(row, sequence, position) of every new token."""
        for s in range(self.S):
            for i in range(self.n[s]):
                yield int(self.cu[s]) + i, s, self.kv[s] - self.n[s] + i

    def summary(self):
        """bf16 [num_pages, hkv, 2, 128] over the filled rows; NaN for pages without."""
        out = np.full((self.num_pages, self.hkv, 2, D), NAN_BITS, np.uint16)
        for s in range(self.S):
            for j in range((self.kv[s] + self.page - 1) // self.page):
                rows = f64(self.k[s][j * self.page:min(self.kv[s], (j + 1) * self.page)])
                out[self.table[s, j], :, 0] = bits_of(rows.min(0))
                out[self.table[s, j], :, 1] = bits_of(rows.max(0))
        return out

    def workspace(self, p):
        ws = torch.empty(spa.sparse_paged_workspace_bytes(p), dtype=torch.uint8, device="cuda")
        return ws.fill_(0xFF)

    def ok(self):
        spa.check(spa.sparse_paged_status(self.error), "status")


SENTINEL = 7.0


def attend(b: Batch, p=None, lists=None, counts=None, ws=None, q=None, stream=None):
    p = b.params() if p is None else p
    ws = b.workspace(p) if ws is None else ws
    o = torch.full((b.T, b.hq, D), SENTINEL, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((b.T, b.hq), SENTINEL, device="cuda")
    spa.check(spa.sparse_paged_attn(p, b.q if q is None else q, b.kc, b.vc, b.cu_gpu, b.kv_gpu,
                                    b.table_gpu, lists, counts, o, lse, ws, b.error,
                                    stream=stream), "attn")
    return o, lse


def check_attention(b: Batch, o, lse, pages_of=None, scale=1.0 / math.sqrt(D), rows=None):
    """Against fp64.  Bounds: the probabilities enter the second product rounded to bf16
    (half a step: 2^-8 of each), the output is rounded once to bf16 (2^-8 of it); the fp32
    arithmetic before stays below 2^-13 of sum p|v| (factor 1 + 2^-5 on the whole).  LSE: a
    score is a 128-term fp32 sum, off by at most 128 * 2^-23 of sum |q||k| scale, and the
    exponential and the sum add less than 2^-18."""
    oh, lh = to_f64(o), lse.cpu().numpy().astype(np.float64)
    seen_rows = set()
    cache = {}
    for t, s, pos in b.tokens():
        seen_rows.add(t)
        if rows is not None and t not in rows:
            continue
        for g in range(b.hkv):
            if pages_of is None:
                idx = np.arange(max(0, pos + 1))
            else:
                pg = pages_of(t, g)
                idx = (pg[:, None] * b.page + np.arange(b.page)).reshape(-1)
                idx = idx[idx <= pos]
            if (s, g) not in cache:
                cache[(s, g)] = (f64(b.k[s][:, g]), f64(b.v[s][:, g]))
            k, v = cache[(s, g)][0][idx], cache[(s, g)][1][idx]
            for h in range(g * b.group, (g + 1) * b.group):
                q = f64(b.qkv[t, h])
                ref, lref, w = op.attend(q, k, v, scale)
                lim = 2.0 ** -8 * (w + np.abs(ref)) * (1 + 2.0 ** -5)
                d = np.abs(oh[t, h] - ref)
                assert np.all(d <= lim), (t, s, pos, h, float(np.nanmax(d / np.maximum(lim, 1e-30))))
                if idx.size == 0:
                    assert lh[t, h] == -math.inf, (t, s, pos, h, lh[t, h])
                    assert np.all(oh[t, h] == 0)
                else:
                    big = float(np.max(np.abs(k) @ np.abs(q))) * scale
                    tol = 2.0 ** -16 * big + 2.0 ** -20 * abs(lref) + 2.0 ** -18
                    assert abs(lh[t, h] - lref) <= tol, (t, s, pos, h, lh[t, h], lref, tol)
    for t in range(b.T):
        if t not in seen_rows:
            assert np.all(oh[t] == SENTINEL) and np.all(lh[t] == SENTINEL), t

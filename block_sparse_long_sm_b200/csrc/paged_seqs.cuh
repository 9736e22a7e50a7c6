// paged_seqs.cuh -- the sequences of a paged call as its kernels see them: the
// checked reading of cu_q, kv_lens and the block table, and the search for the
// sequence that holds a flat work index.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace spa {

struct Seqs {
  const int32_t* cu_q;      // [S + 1]
  const int32_t* kv_lens;   // [S]
  const int32_t* table;     // [S][per_seq]
  int S, T;                 // sequences, token rows
  int per_seq, num_pages;
  int page, shift;          // page_size, its logarithm
  uint32_t* err;
};

struct Seq {
  int q0;      // first token row
  int n;       // new tokens (0: none, or out-of-range values)
  int kv;      // length with them
};

// A sequence whose values are out of range counts as one without new tokens.
__device__ __forceinline__ Seq seq_at(const Seqs& v, int s) {
  Seq q;
  const int c0 = v.cu_q[s], c1 = v.cu_q[s + 1];
  q.kv = v.kv_lens[s];
  q.q0 = c0;
  q.n = c1 - c0;
  if (c0 < 0 || c1 < c0 || c1 > v.T || q.kv < 0 ||
      q.kv > static_cast<long long>(v.per_seq) * v.page) {
    atomicOr(v.err, kErrBadIndex);
    q.n = 0;
    q.kv = 0;
    q.q0 = 0;
  }
  return q;
}

// The sequence s of token row t (n = 0 when no sequence has it).
__device__ __forceinline__ Seq seq_of_token(const Seqs& v, int t, int& s) {
  Seq q{0, 0, 0};
  s = 0;
  if (v.S == 0) return q;
  if (v.S == v.T && v.cu_q[t] == t && v.cu_q[t + 1] == t + 1) {   // one token each
    s = t;
  } else {
    int hi = v.S;                  // the last s with cu_q[s] <= t
    while (hi - s > 1) {
      const int m = (s + hi) >> 1;
      if (v.cu_q[m] <= t)
        s = m;
      else
        hi = m;
    }
  }
  q = seq_at(v, s);
  if (t < q.q0 || t >= q.q0 + q.n) q.n = 0;
  return q;
}

// Physical page of page j of sequence s; -1 (reported) when the table entry is
// outside the cache.  j < per_seq.
__device__ __forceinline__ int phys_page(const Seqs& v, int s, int j) {
  const int p = v.table[static_cast<long long>(s) * v.per_seq + j];
  if (p < 0 || p >= v.num_pages) {
    atomicOr(v.err, kErrBadIndex);
    return -1;
  }
  return p;
}

// ---------------------------------------------------------------------------
// Search over the sequences' costs by a whole block.
// ---------------------------------------------------------------------------
struct FindSmem {
  long long warp_sums[32];
  long long total, base, cost;
  int s;
};

struct Found {
  int s;             // -1: x is past the last sequence
  long long base;    // cost of the sequences before s
  long long total, x;
  long long cost;    // of s
};

// Quotients of non-negative numbers that mostly fit into 32 bits (a 64-bit
// division is some 150 cycles on the way to a kernel's first load).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ long long block_exclusive_sum(long long c, FindSmem& sm) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long incl = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sm.warp_sums[w] = incl;
  __syncthreads();
  if (w == 0) {
    const long long mine = lane < nw ? sm.warp_sums[lane] : 0;
    long long s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < nw) sm.warp_sums[lane] = s - mine;
    if (lane == 31) sm.total = s;
  }
  __syncthreads();
  return sm.warp_sums[w] + incl - c;
}

// Sums cost(s) over the sequences, asks target(total) for a flat index x, and
// finds the sequence that x lies in.  Every thread of the block calls it.
template <class Cost, class Target>
__device__ __forceinline__ Found block_find(int S, Cost cost, Target target, FindSmem& sm) {
  const int nt = blockDim.x;
  const int chunks = (S + nt - 1) / nt;
  long long total = 0, c = 0, excl = 0;
  for (int ch = 0; ch < chunks; ++ch) {
    const int s = ch * nt + threadIdx.x;
    c = s < S ? cost(s) : 0;
    excl = total + block_exclusive_sum(c, sm);
    total += sm.total;
    __syncthreads();
  }
  const long long x = target(total);
  if (threadIdx.x == 0) sm.s = -1;
  __syncthreads();
  if (chunks == 1) {
    if (excl <= x && x < excl + c) {
      sm.s = threadIdx.x;
      sm.base = excl;
      sm.cost = c;
    }
  } else {
    long long run = 0;
    for (int ch = 0; ch < chunks; ++ch) {
      const int s = ch * nt + threadIdx.x;
      c = s < S ? cost(s) : 0;
      excl = run + block_exclusive_sum(c, sm);
      run += sm.total;
      if (excl <= x && x < excl + c) {
        sm.s = s;
        sm.base = excl;
        sm.cost = c;
      }
      __syncthreads();
    }
  }
  __syncthreads();
  Found f;
  f.s = sm.s;
  f.base = sm.s >= 0 ? sm.base : 0;
  f.cost = sm.s >= 0 ? sm.cost : 0;
  f.total = total;
  f.x = x;
  return f;
}

// The same by one warp, for up to 32 * kWarpFind sequences: all lengths are
// read side by side, nothing waits for the block.
constexpr int kWarpFind = 4;
template <class Cost, class Target>
__device__ __forceinline__ Found warp_find(int S, Cost cost, Target target) {
  const int lane = threadIdx.x & 31;
  long long c[kWarpFind], mine = 0;
#pragma unroll
  for (int k = 0; k < kWarpFind; ++k) {
    const int s = kWarpFind * lane + k;
    c[k] = s < S ? cost(s) : 0;
    mine += c[k];
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  Found f;
  f.total = __shfl_sync(0xffffffffu, incl, 31);
  f.x = target(f.total);
  long long at = incl - mine;
  int hit = -1;
  long long base = 0, cost_hit = 0;
#pragma unroll
  for (int k = 0; k < kWarpFind; ++k) {
    if (at <= f.x && f.x < at + c[k]) {
      hit = kWarpFind * lane + k;
      base = at;
      cost_hit = c[k];
    }
    at += c[k];
  }
  const uint32_t who = __ballot_sync(0xffffffffu, hit >= 0);
  const int src = who ? __ffs(who) - 1 : 0;
  f.s = __shfl_sync(0xffffffffu, hit, src);
  f.base = __shfl_sync(0xffffffffu, base, src);
  f.cost = __shfl_sync(0xffffffffu, cost_hit, src);
  return f;
}

}  // namespace spa

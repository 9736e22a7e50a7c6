// paged_select.cuh -- the pages a new token attends to, by an upper bound of
// its logits.
//
// A page's summary holds, per kv head, the minimum and maximum of every key
// dimension over the page's rows.  For a query q,
//
//     sum_d max(q_d min_d, q_d max_d)  >=  q . k   for every key k of the page,
//
// and a kv head's score of a page is the largest bound over its q heads: no
// page that holds a large logit for any of them scores low.  512 bytes of
// summary stand for 512 * page_size bytes of keys and values.
//
// Exactness.  Which pages are kept is a whole-number output, so the scores are
// taken so that no order of summation can change them: a product of two bf16
// is exact in fp32, a sum of 128 of them in 64 bits is off by at most 2^-46 of
// the largest partial sum, and rounding that once to fp32 gives the same value
// whatever the order (but for sums within 2^-46 of a rounding border).
//
// page_score_kernel    a thread quad per page: each lane reads four 16-byte
//                      pieces of the minima and of the maxima (64 contiguous
//                      bytes per quad and load), then serves the q heads from
//                      shared memory.  max(q min, q max) is q times the
//                      maximum where q >= 0 and times the minimum elsewhere.
// page_top_kernel      one block per token and kv head: a radix search of the
//                      score with rank top_pages (four passes of eight bits
//                      over the order-preserving integer image), then one scan
//                      that writes the kept pages in ascending order.
#pragma once

#include "paged_seqs.cuh"
#include "rope.cuh"

namespace spa {

struct SelectArgs {
  Seqs q;
  Rows xq;
  const __nv_bfloat16* summary;   // [num_pages][Hkv][2][128]
  float* score;                   // [T][Hkv][per_seq]
  int32_t* lists;                 // [T][Hkv][width]
  int32_t* counts;                // [T][Hkv]
  int Hkv, group;
  int sink, local, top, width;
  int chunks;                     // score blocks per (token, kv head)
};

constexpr int kScoreThreads = 128;
constexpr int kScorePages = 64;          // pages per score block
constexpr int kScoreHeads = 8;           // q heads per pass
constexpr int kTopThreads = 256;

// Visible pages of a token and the candidates [sink, sink + n) among them.
struct Candidates {
  int seen, n;
};
__device__ __forceinline__ Candidates candidates(const SelectArgs& a, int pos) {
  Candidates c;
  c.seen = pos < 0 ? 0 : (pos >> a.q.shift) + 1;
  c.n = max(0, c.seen - a.local - a.sink);
  return c;
}

__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelectArgs a) {
  __shared__ double qs[kScoreHeads][128];
  const long long tg = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - tg * a.chunks);
  const int t = static_cast<int>(tg / a.Hkv), g = static_cast<int>(tg - (long long)t * a.Hkv);
  int s;
  const Seq q = seq_of_token(a.q, t, s);
  if (q.n == 0) return;
  const Candidates cd = candidates(a, q.kv - q.n + (t - q.q0));
  const int c0 = chunk * kScorePages;
  if (cd.n <= a.top || c0 >= cd.n) return;          // nothing to rank
  const int part = threadIdx.x & 3;
  constexpr int kPer = kScorePages * 4 / kScoreThreads;
  uint4 lo[kPer][4], hi[kPer][4];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = c0 + i * (kScoreThreads / 4) + (threadIdx.x >> 2);
    const int phys = c < cd.n ? phys_page(a.q, s, a.sink + c) : -1;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.summary + (static_cast<long long>(phys < 0 ? 0 : phys) * a.Hkv + g) * 256);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[i][j] = src[4 * j + part];
      hi[i][j] = src[16 + 4 * j + part];
    }
  }
  double best[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) best[i] = -INFINITY;
  for (int h0 = 0; h0 < a.group; h0 += kScoreHeads) {
    const int nh = min(kScoreHeads, a.group - h0);
    __syncthreads();
    for (int i = threadIdx.x; i < kScoreHeads * 128; i += kScoreThreads) {
      const int h = i >> 7;
      qs[h][i & 127] = h < nh ? static_cast<double>(__bfloat162float(
                                    a.xq.at(0, t, g * a.group + h0 + h)[i & 127]))
                              : 0.0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      double acc[kScoreHeads];
#pragma unroll
      for (int h = 0; h < kScoreHeads; ++h) acc[h] = 0.0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float l8[8], h8[8];
        unpack8(lo[i][j], l8);
        unpack8(hi[i][j], h8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double dl = l8[e], dh = h8[e];
          const int d = 8 * (4 * j + part) + e;
#pragma unroll
          for (int h = 0; h < kScoreHeads; ++h) {
            if (h < nh) {
              const double x = qs[h][d];
              acc[h] = fma(x, __double2hiint(x) >= 0 ? dh : dl, acc[h]);
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < kScoreHeads; ++h) {
        if (h < nh) {
          acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 1);
          acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 2);
          best[i] = fmax(best[i], acc[h]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = c0 + i * (kScoreThreads / 4) + (threadIdx.x >> 2);
    if (part == 0 && c < cd.n)
      a.score[tg * a.q.per_seq + c] = static_cast<float>(best[i]) + 0.0f;   // -0 becomes +0
  }
}

// Order-preserving image of a float: larger value, larger integer.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];                     // digit, rank left within it
  __shared__ unsigned long long sums[kTopThreads / 32];
  const long long tg = blockIdx.x;
  const int t = static_cast<int>(tg / a.Hkv);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int s;
  const Seq q = seq_of_token(a.q, t, s);
  if (q.n == 0) return;
  const Candidates cd = candidates(a, q.kv - q.n + (t - q.q0));
  int32_t* out = a.lists + tg * a.width;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int kept = min(cd.n, a.top);
  const int head = min(a.sink, cd.seen);            // sink pages
  const int tail = cd.seen - head - cd.n;           // recent pages
  const int count = head + kept + tail;
  if (tid == 0) a.counts[tg] = count;
  for (int i = tid; i < a.width; i += kTopThreads) {
    // everything but the chosen pages (all candidates when they fit)
    if (i < head)
      out[i] = i;
    else if (i >= count)
      out[i] = -1;
    else if (i >= head + kept)
      out[i] = cd.seen - (count - i);
    else if (cd.n <= a.top)
      out[i] = i;
  }
  if (cd.n <= a.top || a.top == 0) return;
  const float* score = a.score + tg * a.q.per_seq;
  // the score of rank top: its digits from the highest down
  uint32_t prefix = 0, rank = a.top;                // rank-th largest, from 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < cd.n; i += kTopThreads) {
      const uint32_t u = ordered(score[i]);
      if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(u >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits 255 - 8 l .. 248 - 8 l
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = hist[255 - 8 * lane - i];
        sum += n[i];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      uint32_t above = incl - sum;
      if (above < rank && rank <= incl) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (above < rank && rank <= above + n[i]) {
            found[0] = 255 - 8 * lane - i;
            found[1] = rank - above;
          }
          above += n[i];
        }
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    rank = found[1];
    __syncthreads();
  }
  // every score above `prefix`, and the first `rank` equal to it
  const int per = (cd.n + kTopThreads - 1) / kTopThreads;
  const int i0 = min(cd.n, tid * per), i1 = min(cd.n, i0 + per);
  unsigned long long mine = 0;                      // above in the high word, equal in the low
  for (int i = i0; i < i1; ++i) {
    const uint32_t u = ordered(score[i]);
    if (u > prefix) mine += 1ull << 32;
    if (u == prefix) mine += 1ull;
  }
  unsigned long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  unsigned long long excl = incl - mine;
  for (int w = 0; w < warp; ++w) excl += sums[w];
  uint32_t gt = static_cast<uint32_t>(excl >> 32), eq = static_cast<uint32_t>(excl);
  for (int i = i0; i < i1; ++i) {
    const uint32_t u = ordered(score[i]);
    if (u > prefix || (u == prefix && eq < rank)) out[head + gt + min(eq, rank)] = a.sink + i;
    gt += u > prefix;
    eq += u == prefix;
  }
}

}  // namespace spa

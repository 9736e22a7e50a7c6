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
// The sum is two products, max(q, 0) . max + min(q, 0) . min, so it runs on
// the tensor cores (mma.sync m16n8k16: sixteen rows of tokens x heads against
// eight pages; the call is bound by the bytes of the summaries, 512 for 16 x
// 512 multiply-adds, which this instruction's rate serves many times over).
//
// Exactness.  Which pages are kept is a whole-number output, defined by the
// sum taken in 64 bits and rounded once to fp32.  The tensor core's fp32 sum
// differs from it by at most
//
//     e = 2^-14 sum_d |q_d| max(|min_d|, |max_d|):
//
// the products of two bf16 are exact, and each of the 16 accumulating steps
// adds 16 of them with an error of at most 17 * 2^-23 of the sum of
// magnitudes, 2^-14.9 in all (the rounding to fp32 is 2^-24).  A third product
// gives that sum of magnitudes for every page.  With t the score of rank
// top_pages among the fp32 sums and e the largest bound of the token and head,
// a page above t + 2e is among the best whatever the errors, one below t - 2e
// is not, and only the pages between -- two or three of thousands -- are
// summed again in 64 bits and ranked exactly.
//
// page_score_kernel  a warp per 32 pages.  All four lanes that share a page
//                    read 16-byte pieces of it (the order of a dot product's
//                    terms is free, so the pieces are the matrix operand as
//                    they come).  Tokens of one sequence that fit into the
//                    sixteen rows share the loads.  16 sequences of up to 32K in
//                    pages of 16: 50 MB of summaries, 22 us (2.3 TB/s: three blocks
//                    per SM of 168 registers, 32 bytes spilled, have few loads under
//                    way); 250 tokens that share 6 MB: 32 us (loads from L2, three
//                    products a page).
// page_top_kernel    one block per token and kv head: the score of rank top_pages
//                    is found to within the error of the sums, by counting keys
//                    above three points of an interval (up to 2048 candidates,
//                    keys in registers) or by a radix search; then the exact sums
//                    between, and one scan that writes the kept pages in ascending
//                    order.  Bound by latency, the barriers and the loads between:
//                    8.4 us for one token among 2042 pages, 9.9 us for 16 (with a
//                    radix search there: 14 and 17 us).
//                    Radix search above 2048 candidates: scores and ranking for one
//                    token 15.9 us at 2054 candidates (11.0 us at 2048 with the points,
//                    14.6 us with a radix search), 22 us at 4090, 37 us at 8186.
// page_top_warp_kernel  the same by one warp, for up to 512 candidates and many
//                    selections: no barriers, and all of a chunk's tokens are under
//                    way at once: 20 us for 2000 selections among 506 pages.  A warp
//                    alone takes longer over its keys than a block does, so few
//                    selections are left to blocks.
#pragma once

#include "paged_seqs.cuh"
#include "rope.cuh"

namespace spa {

struct SelectArgs {
  Seqs q;
  Rows xq;
  const __nv_bfloat16* summary;   // [num_pages][Hkv][2][128]
  float2* score;                  // [T][Hkv][per_seq]: fp32 sum, sum of magnitudes
  int32_t* lists;                 // [T][Hkv][width]
  int32_t* counts;                // [T][Hkv]
  int Hkv, group;
  int sink, local, top, width;
  int chunks;                     // score blocks per (token, kv head)
  int tm;                         // tokens that share the sixteen rows
};

constexpr int kScoreThreads = 128;
constexpr int kWarpPages = 32;           // pages per warp
constexpr int kScorePages = kWarpPages * kScoreThreads / 32;
constexpr int kTopThreads = 256;
constexpr int kTopKeys = 16384;          // scores kept in shared memory
constexpr int kTopBand = 256;            // pages ranked exactly there
constexpr int kTopSteps = 8;             // keys of a thread, when they fit
constexpr int kTopHeld = kTopSteps * kTopThreads;

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

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Tokens t0 .. t0 + ntok - 1 of sequence s, one kv head, 32 pages of one warp.
__device__ __forceinline__ void score_pages(const SelectArgs& a, const Seq& q, int s, int t0,
                                            int ntok, int g, int chunk, float (*tile)[16][9]) {
  const int pos0 = q.kv - q.n + (t0 - q.q0);
  const Candidates cd = candidates(a, pos0 + ntok - 1);   // the last token sees most
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = chunk * kScorePages + warp * kWarpPages;
  if (cd.n <= a.top || c0 >= cd.n) return;                // nothing to rank
  const int part = lane & 3, r0 = lane >> 2;
  const int mtiles = (a.group + 15) / 16;                 // 1 unless the group fills the rows
  const int hrows = min(a.group, 16);
  // lane l looks up page l of the warp's 32
  const int cl = c0 + lane;
  int mine = cl < cd.n ? phys_page(a.q, s, a.sink + cl) : 0;
  if (mine < 0) mine = 0;
  float best[kWarpPages / 8][4], mag[kWarpPages / 8][4];  // running maxima over m-tiles
#pragma unroll
  for (int i = 0; i < kWarpPages / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) best[i][e] = mag[i][e] = -INFINITY;
  for (int mt = 0; mt < mtiles; ++mt) {
    // the lane's two rows of q: (token, head) of rows r0 and r0 + 8
    const uint4* src[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = r0 + 8 * i;
      const int ti = mtiles == 1 ? row / a.group : 0;
      const int h = mtiles == 1 ? row - ti * a.group : 16 * mt + row;
      live[i] = ti < ntok && h < a.group;
      src[i] = reinterpret_cast<const uint4*>(
          a.xq.at(0, live[i] ? t0 + ti : t0, g * a.group + (live[i] ? h : 0)));
    }
    uint4 qa[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        qa[i][j] = live[i] ? src[i][4 * j + part] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int n8 = 0; n8 < kWarpPages / 8; ++n8) {
      const int phys = __shfl_sync(0xffffffffu, mine, 8 * n8 + r0);
      const uint4* pg = reinterpret_cast<const uint4*>(
          a.summary + (static_cast<long long>(phys) * a.Hkv + g) * 256);
      uint4 lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = pg[4 * j + part];
        hi[j] = pg[16 + 4 * j + part];
      }
      float u[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // k16 step: words 2k, 2k + 1 of this piece; rows r0 and r0 + 8
          const uint32_t x[4] = {word(qa[0][j], 2 * k), word(qa[1][j], 2 * k),
                                 word(qa[0][j], 2 * k + 1), word(qa[1][j], 2 * k + 1)};
          uint32_t p[4], m[4], b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = max_bf16x2(x[e], 0u);
            m[e] = min_bf16x2(x[e], 0u);
            b[e] = x[e] & 0x7fff7fffu;
          }
          const uint32_t l0 = word(lo[j], 2 * k), l1 = word(lo[j], 2 * k + 1);
          const uint32_t h0 = word(hi[j], 2 * k), h1 = word(hi[j], 2 * k + 1);
          mma_16816(u, p, h0, h1);
          mma_16816(u, m, l0, l1);
          mma_16816(v, b, max_bf16x2(l0 & 0x7fff7fffu, h0 & 0x7fff7fffu),
                    max_bf16x2(l1 & 0x7fff7fffu, h1 & 0x7fff7fffu));
        }
      }
      // a row without a head must not win
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        best[n8][e] = live[e >> 1] ? fmaxf(best[n8][e], u[e]) : best[n8][e];
        mag[n8][e] = live[e >> 1] ? fmaxf(mag[n8][e], v[e]) : mag[n8][e];
      }
    }
  }
  // maxima over the heads of a token: element e of the lane is row r0 + 8 (e / 2),
  // page 2 part + e % 2 of its eight
#pragma unroll
  for (int n8 = 0; n8 < kWarpPages / 8; ++n8) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      tile[0][r0 + 8 * (e >> 1)][2 * part + (e & 1)] = best[n8][e];
      tile[1][r0 + 8 * (e >> 1)][2 * part + (e & 1)] = mag[n8][e];
    }
    __syncwarp();
    for (int i = lane; i < 8 * ntok; i += 32) {
      const int ti = i >> 3, page = i & 7;
      float x = -INFINITY, y = -INFINITY;
      for (int h = 0; h < hrows; ++h) {
        x = fmaxf(x, tile[0][ti * hrows + h][page]);
        y = fmaxf(y, tile[1][ti * hrows + h][page]);
      }
      const int c = c0 + 8 * n8 + page;
      if (c < cd.n)
        a.score[(static_cast<long long>(t0 + ti) * a.Hkv + g) * a.q.per_seq + c] =
            make_float2(x, y);
    }
  }
}

// Block: tm token rows, one kv head, kScorePages candidates.  Rows of several
// sequences are taken one sequence after the other.
__global__ void __launch_bounds__(kScoreThreads, 3) page_score_kernel(const SelectArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the ranking waits by itself
  // scores of one n8 group: [row][page], [row][page] of the magnitudes
  __shared__ float tile[kScoreThreads / 32][2][16][9];
  const long long bg = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - bg * a.chunks);
  const int block = static_cast<int>(bg / a.Hkv);
  const int g = static_cast<int>(bg - static_cast<long long>(block) * a.Hkv);
  const int end = min(a.q.T, (block + 1) * a.tm);
  for (int t = block * a.tm; t < end;) {
    int s;
    const Seq q = seq_of_token(a.q, t, s);
    const int next = q.n > 0 ? min(end, q.q0 + q.n) : t + 1;
    if (q.n > 0) score_pages(a, q, s, t, next - t, g, chunk, tile[threadIdx.x >> 5]);
    t = next;
  }
}

// Order-preserving image of a float: larger value, larger integer; -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

static_assert(kTopBand == kTopThreads && kTopThreads == 256, "a thread per page between, eight warps");
struct TopSmem {
  uint32_t band[kTopBand], exact[kTopBand], band_n;
  int phys[kTopBand];
  uint32_t hist[256];
  uint32_t red[3][kTopThreads / 32];
  uint32_t found[2];
  uint32_t count[2][2][kTopThreads / 32];
  unsigned long long sums[kTopThreads / 32];
  uint32_t keys[1];                      // [cap]: as many as pages_per_seq, up to kTopKeys
};
__host__ __device__ constexpr int top_keys(int per_seq) {
  return per_seq < kTopKeys ? per_seq : kTopKeys;
}
__host__ __device__ constexpr uint32_t top_smem_bytes(int per_seq) {
  return static_cast<uint32_t>(sizeof(TopSmem)) + 4u * top_keys(per_seq);
}

// The key of rank `rank` (from 1, largest first) among key(i), i < n, where
// use(i): eight bits at a time below the highest bit that the keys differ in.
// Returns the key, and in `rank` its rank among the equal ones.  Every thread
// of the block calls it.
template <class Key, class Use>
__device__ __forceinline__ uint32_t radix_rank(int n, Key key, Use use, uint32_t& rank,
                                               TopSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t lo = 0xffffffffu, hi = 0u;
  for (int i = tid; i < n; i += kTopThreads)
    if (use(i)) {
      lo = min(lo, key(i));
      hi = max(hi, key(i));
    }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    sm.red[0][warp] = lo;
    sm.red[1][warp] = hi;
  }
  __syncthreads();
  lo = sm.red[0][lane & (kTopThreads / 32 - 1)];
  hi = sm.red[1][lane & (kTopThreads / 32 - 1)];
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  uint32_t prefix = 0;                              // of key - lo
  int bits = 32 - __clz(hi - lo);                   // bits not yet decided
  while (bits > 0) {
    const int shift = max(0, bits - 8);
    const uint32_t mask = (1u << (bits - shift)) - 1u;
    sm.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kTopThreads) {
      if (!use(i)) continue;
      const uint32_t u = key(i) - lo;
      if (bits == 32 || (u >> bits) == (prefix >> bits))
        atomicAdd(&sm.hist[(u >> shift) & mask], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l: digits 255 - 8 l down to 248 - 8 l
      uint32_t c[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = sm.hist[255 - 8 * lane - i];
        sum += c[i];
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
          if (above < rank && rank <= above + c[i]) {
            sm.found[0] = 255 - 8 * lane - i;
            sm.found[1] = rank - above;
          }
          above += c[i];
        }
      }
    }
    __syncthreads();
    prefix |= sm.found[0] << shift;
    rank = sm.found[1];
    bits = shift;
  }
  __syncthreads();                                  // found and red are written again
  return prefix + lo;
}

// Score of the candidate in physical page `phys` in 64 bits, rounded once: by a
// warp, four heads side by side.
__device__ __forceinline__ float exact_score(const SelectArgs& a, int t, int g, int phys) {
  const int lane = threadIdx.x & 31;
  const uint2* pg = reinterpret_cast<const uint2*>(
      a.summary + (static_cast<long long>(max(phys, 0)) * a.Hkv + g) * 256);
  const uint2 l2 = pg[lane], h2 = pg[32 + lane];
  const float lo[4] = {__uint_as_float(l2.x << 16), __uint_as_float(l2.x & 0xffff0000u),
                       __uint_as_float(l2.y << 16), __uint_as_float(l2.y & 0xffff0000u)};
  const float hi[4] = {__uint_as_float(h2.x << 16), __uint_as_float(h2.x & 0xffff0000u),
                       __uint_as_float(h2.y << 16), __uint_as_float(h2.y & 0xffff0000u)};
  double best = -INFINITY;
#pragma unroll 1
  for (int h0 = 0; h0 < a.group; h0 += 4) {
    uint2 q2[4];
    double sum[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)                     // (past the group: its last head again)
      q2[k] = reinterpret_cast<const uint2*>(
          a.xq.at(0, t, g * a.group + min(h0 + k, a.group - 1)))[lane];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float qd[4] = {__uint_as_float(q2[k].x << 16), __uint_as_float(q2[k].x & 0xffff0000u),
                           __uint_as_float(q2[k].y << 16), __uint_as_float(q2[k].y & 0xffff0000u)};
      sum[k] = 0.0;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        sum[k] += static_cast<double>(qd[d]) * static_cast<double>(qd[d] >= 0.f ? hi[d] : lo[d]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
#pragma unroll
    for (int k = 0; k < 4; ++k) best = fmax(best, sum[k]);
  }
  return static_cast<float>(best);
}

__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the attention waits by itself
  extern __shared__ __align__(16) uint8_t top_smem[];
  TopSmem& sm = *reinterpret_cast<TopSmem*>(top_smem);
  const long long tg = blockIdx.x;
  const int t = static_cast<int>(tg / a.Hkv);
  const int g = static_cast<int>(tg - static_cast<long long>(t) * a.Hkv);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int s;
  const Seq q = seq_of_token(a.q, t, s);
  if (q.n == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // not done before the kernel before
    return;
  }
  const Candidates cd = candidates(a, q.kv - q.n + (t - q.q0));
  int32_t* out = a.lists + tg * a.width;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the scores
  if (cd.n <= a.top || a.top == 0) return;
  if (tid == 0) sm.band_n = 0;
  const int cap = top_keys(a.q.per_seq);
  float2* score = a.score + tg * a.q.per_seq;
  float big = 0.f;
  uint32_t least_key = 0xffffffffu, most_key = 0u;
  const bool few = cd.n <= kTopHeld;                // keys stay in registers
  uint32_t held[kTopSteps];
  auto note = [&](const float2& x) {
    const uint32_t u = ordered(x.x);
    big = fmaxf(big, x.y);
    least_key = min(least_key, u);
    most_key = max(most_key, u);
    return u;
  };
  if (few) {
    float2 x[kTopSteps];
#pragma unroll
    for (int k = 0; k < kTopSteps; ++k)
      if (tid + k * kTopThreads < cd.n) x[k] = score[tid + k * kTopThreads];
#pragma unroll
    for (int k = 0; k < kTopSteps; ++k) {
      held[k] = 0u;                                 // below every point of the search
      if (tid + k * kTopThreads < cd.n) {
        held[k] = note(x[k]);
        sm.keys[tid + k * kTopThreads] = held[k];
      }
    }
  } else {
#pragma unroll 4
    for (int i = tid; i < cd.n; i += kTopThreads) {
      const uint32_t u = note(score[i]);
      if (i < cap) sm.keys[i] = u;
    }
  }
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
  least_key = __reduce_min_sync(0xffffffffu, least_key);
  most_key = __reduce_max_sync(0xffffffffu, most_key);
  if (lane == 0) {
    sm.red[0][warp] = least_key;
    sm.red[1][warp] = most_key;
    sm.red[2][warp] = __float_as_uint(big);
  }
  __syncthreads();
  least_key = __reduce_min_sync(0xffffffffu, sm.red[0][lane & (kTopThreads / 32 - 1)]);
  most_key = __reduce_max_sync(0xffffffffu, sm.red[1][lane & (kTopThreads / 32 - 1)]);
  big = __uint_as_float(
      __reduce_max_sync(0xffffffffu, sm.red[2][lane & (kTopThreads / 32 - 1)]));
  auto key = [&](int i) { return i < cap ? sm.keys[i] : ordered(score[i].x); };
  // The key of rank `top` lies in [first, last].  That interval is cut until it is
  // no wider than the error of two sums; more would narrow the pages between only
  // a little (26.4 us for one token, 26.8 us with an interval of a sixteenth of that).
  const float e2 = big * (1.0f / 8192.0f);
  uint32_t rank = a.top;
  uint32_t first = least_key, last = most_key;
  if (few) {
    int turn = 0;
    while (first < last && !(unordered(last) - unordered(first) <= e2)) {
      // three points, all within it, cut the interval into four
      const uint32_t quarter = (last - first) >> 2;
      const uint32_t p1 = first + quarter + 1u, p2 = p1 + quarter, p3 = p2 + quarter;
      uint32_t n1 = 0, n23 = 0;                     // keys at or above them
#pragma unroll
      for (int k = 0; k < kTopSteps; ++k) {
        n1 += held[k] >= p1;
        n23 += (held[k] >= p2 ? 1u : 0u) + (held[k] >= p3 ? 0x10000u : 0u);
      }
      n1 = __reduce_add_sync(0xffffffffu, n1);
      n23 = __reduce_add_sync(0xffffffffu, n23);
      if (lane == 0) {
        sm.count[turn][0][warp] = n1;
        sm.count[turn][1][warp] = n23;
      }
      __syncthreads();                              // the counts of the step before are free
      const uint32_t x = lane < 2 * (kTopThreads / 32)
                             ? sm.count[turn][lane >> 3][lane & 7] : 0u;
      n1 = __reduce_add_sync(0xffffffffu, lane < 8 ? x : 0u);
      n23 = __reduce_add_sync(0xffffffffu, lane < 8 ? 0u : x);
      turn ^= 1;
      if ((n23 >> 16) >= rank) {
        first = p3;
      } else if ((n23 & 0xffffu) >= rank) {
        first = p2;
        last = p3 - 1u;
      } else if (n1 >= rank) {
        first = p1;
        last = p2 - 1u;
      } else {
        last = p1 - 1u;
      }
    }
  } else {
    first = last = radix_rank(cd.n, key, [](int) { return true; }, rank, sm);
  }
  // keys above `top` are kept, below `bottom` are not
  const uint32_t top = ordered(unordered(last) + e2);
  const uint32_t bottom = max(1u, ordered(unordered(first) - e2));
  uint32_t in = 0, between = 0;
  if (few) {
#pragma unroll
    for (int k = 0; k < kTopSteps; ++k) {
      in += held[k] > top;
      between += held[k] <= top && held[k] >= bottom;
    }
  } else {
    for (int i = tid; i < cd.n; i += kTopThreads) {
      const uint32_t u = key(i);
      in += u > top;
      between += u <= top && u >= bottom;
    }
  }
  unsigned long long both = (static_cast<unsigned long long>(in) << 32) | between;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
  if (lane == 0) sm.sums[warp] = both;
  __syncthreads();
  both = sm.sums[lane & (kTopThreads / 32 - 1)];
#pragma unroll
  for (int o = 1; o < kTopThreads / 32; o <<= 1) both += __shfl_xor_sync(0xffffffffu, both, o);
  in = static_cast<uint32_t>(both >> 32);
  between = static_cast<uint32_t>(both);
  const uint32_t need = a.top - in;                 // of those between; at least one
  // the smallest key kept, and how many of the pages that have it
  uint32_t least = bottom, equal = 0xffffffffu;
  bool exact = between > need;
  if (exact && cd.n <= cap && between <= kTopBand) {
    // the pages between, ranked exactly in shared memory: the kept ones get the
    // largest key, the others the smallest
    for (int i = tid; i < cd.n; i += kTopThreads) {
      const uint32_t u = sm.keys[i];
      if (u <= top && u >= bottom) {
        const uint32_t at = atomicAdd(&sm.band_n, 1u);
        sm.band[at] = i;
        sm.phys[at] = phys_page(a.q, s, a.sink + i);
      }
    }
    __syncthreads();
    for (uint32_t k = warp; k < between; k += kTopThreads / 32) {
      const float x = exact_score(a, t, g, sm.phys[k]);
      if (lane == 0) sm.exact[k] = ordered(x);
    }
    __syncthreads();
    if (static_cast<uint32_t>(tid) < between) {
      const uint32_t me = sm.exact[tid], at = sm.band[tid];
      uint32_t better = 0;
      for (uint32_t k = 0; k < between; ++k)
        better += sm.exact[k] > me || (sm.exact[k] == me && sm.band[k] < at);
      sm.keys[at] = better < need ? 0xffffffffu : 0u;
    }
    __syncthreads();
    exact = false;
  } else if (exact) {
    // many of them (equal pages), or more candidates than fit: in the score
    // array, marked by a negative magnitude
    __syncthreads();
    for (int base = warp * 32; base < cd.n; base += kTopThreads) {
      const uint32_t u = base + lane < cd.n ? key(base + lane) : 0u;
      uint32_t todo = __ballot_sync(0xffffffffu, base + lane < cd.n && u <= top && u >= bottom);
      while (todo) {
        const int i = base + __ffs(todo) - 1;
        todo &= todo - 1;
        const float x = exact_score(a, t, g, phys_page(a.q, s, a.sink + i));
        if (lane == 0) score[i] = make_float2(x, -1.0f);
      }
    }
    __syncthreads();
    rank = need;
    auto exact_key = [&](int i) { return ordered(score[i].x); };
    auto marked = [&](int i) { return score[i].y < 0.f; };
    least = radix_rank(cd.n, exact_key, marked, rank, sm);
    equal = rank;
  }
  const uint32_t before = (1u << lane) - 1u;
  if (few && !exact) {
    // every key from `bottom` on is kept
    const int i0 = warp * (kTopSteps * 32);
    uint32_t keep[kTopSteps], at = 0;
#pragma unroll
    for (int k = 0; k < kTopSteps; ++k) {
      const int i = i0 + 32 * k + lane;
      keep[k] = __ballot_sync(0xffffffffu, i < cd.n && sm.keys[i] >= bottom);
      at += __popc(keep[k]);
    }
    if (lane == 0) sm.red[0][warp] = at;
    __syncthreads();
    at = __reduce_add_sync(0xffffffffu, lane < warp ? sm.red[0][lane] : 0u);
#pragma unroll
    for (int k = 0; k < kTopSteps; ++k) {
      const uint32_t pos = at + __popc(keep[k] & before);
      if (((keep[k] >> lane) & 1u) && pos < static_cast<uint32_t>(a.top))
        out[head + pos] = a.sink + i0 + 32 * k + lane;
      at += __popc(keep[k]);
    }
    return;
  }
  // pages above the border, and of those between the ones above `least` with
  // the first `equal` that have it
  const int per = (cd.n + kTopThreads - 1) / kTopThreads * 32;   // candidates per warp
  const int i0 = min(cd.n, warp * per), i1 = min(cd.n, i0 + per);
  // 0 dropped, 1 kept, 2 equal to the least
  auto verdict = [&](int i) -> int {
    uint32_t u;
    bool inside;
    if (i < cap) {
      u = sm.keys[i];
      inside = u <= top && u >= bottom;
    } else {
      // a page summed exactly no longer has its fp32 sum, but its mark
      const float2 x = score[i];
      u = ordered(x.x);
      inside = exact ? x.y < 0.f : u <= top && u >= bottom;
    }
    if (!inside) return u > top ? 1 : 0;
    if (!exact) return 1;
    if (i < cap) u = ordered(score[i].x);
    return u > least ? 1 : u == least ? 2 : 0;
  };
  uint32_t gt = 0, eq = 0;                          // kept, equal to the least
  for (int base = i0; base < i1; base += 32) {
    const int vd = base + lane < i1 ? verdict(base + lane) : 0;
    gt += __popc(__ballot_sync(0xffffffffu, vd == 1));
    eq += __popc(__ballot_sync(0xffffffffu, vd == 2));
  }
  if (lane == 0) {
    sm.red[0][warp] = gt;
    sm.red[1][warp] = eq;
  }
  __syncthreads();
  gt = __reduce_add_sync(0xffffffffu, lane < warp ? sm.red[0][lane] : 0u);
  eq = __reduce_add_sync(0xffffffffu, lane < warp ? sm.red[1][lane] : 0u);
  for (int base = i0; base < i1; base += 32) {
    const int vd = base + lane < i1 ? verdict(base + lane) : 0;
    const uint32_t keep = __ballot_sync(0xffffffffu, vd == 1);
    const uint32_t ties = __ballot_sync(0xffffffffu, vd == 2);
    const uint32_t tie = eq + __popc(ties & before);
    const uint32_t at = gt + __popc(keep & before) + min(tie, equal);
    if ((vd == 1 || (vd == 2 && tie < equal)) && at < static_cast<uint32_t>(a.top))
      out[head + at] = a.sink + base + lane;
    gt += __popc(keep);
    eq += __popc(ties);
  }
}

// The largest v with at least `rank` of the warp's keys at or above it, among
// the bits below and at `bit` (v: the bits above); count(v) counts over the warp.
template <class Count>
__device__ __forceinline__ uint32_t bit_rank(uint32_t v, int bit, uint32_t rank, Count count) {
  for (; bit >= 0; --bit) {
    const uint32_t c = v | (1u << bit);
    if (count(c) >= rank) v = c;
  }
  return v;
}

constexpr int kTopWarpThreads = 128;
constexpr int kTopWarpKeys = 512;
// Fewer selections (tokens x kv heads) than about seven per SM go to blocks.  Scores
// and ranking in us, by warps / by blocks, among 128, 256 and 512 candidates:
//     8 selections     12.1 /  9.4    14.9 /  9.9    19.6 / 10.6
//   128 (16 tokens)    14.6 / 10.7    17.4 / 11.7    25.1 / 16.0
//   640 (80 tokens)    21.4 / 20.9    33.0 / 29.5    65.5 / 58.1
//  1024 (two chunks)   17.1 / 20.0    23.2 / 24.8    32.8 / 31.0
//  1536 (two chunks)   18.6 / 25.8    25.5 / 32.0    39.6 / 41.9
//  2000 (two chunks)   22.2 / 33.6    30.8 / 39.9    45.9 / 52.2
constexpr int kTopWarpSelections = 1024;

struct TopWarpSmem {
  uint32_t keys[kTopWarpKeys];
  uint32_t in[kTopWarpKeys / 32], band[kTopWarpKeys / 32];   // kept at once; between
};

__global__ void __launch_bounds__(kTopWarpThreads) page_top_warp_kernel(const SelectArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the attention waits by itself
  extern __shared__ __align__(16) uint8_t top_smem[];
  TopWarpSmem* smem = reinterpret_cast<TopWarpSmem*>(top_smem);
  const long long tg =
      static_cast<long long>(blockIdx.x) * (kTopWarpThreads / 32) + (threadIdx.x >> 5);
  if (tg >= static_cast<long long>(a.q.T) * a.Hkv) return;
  const int t = static_cast<int>(tg / a.Hkv);
  const int g = static_cast<int>(tg - static_cast<long long>(t) * a.Hkv);
  const int lane = threadIdx.x & 31;
  TopWarpSmem& sm = smem[threadIdx.x >> 5];
  int s;
  const Seq q = seq_of_token(a.q, t, s);
  if (q.n == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // not done before the kernel before
    return;
  }
  const Candidates cd = candidates(a, q.kv - q.n + (t - q.q0));
  int32_t* out = a.lists + tg * a.width;
  const int kept = min(cd.n, a.top);
  const int head = min(a.sink, cd.seen);            // sink pages
  const int tail = cd.seen - head - cd.n;           // recent pages
  const int count = head + kept + tail;
  if (lane == 0) a.counts[tg] = count;
  for (int i = lane; i < a.width; i += 32) {
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
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the scores
  if (cd.n <= a.top || a.top == 0) return;
  const float2* score = a.score + tg * a.q.per_seq;
  const int steps = (cd.n + 31) >> 5;               // candidate 32 k + lane; key 0: none
  constexpr int kHeld = kTopWarpKeys / 32;
  uint32_t held[kHeld];
  float big = 0.f;
  uint32_t lo = 0xffffffffu, hi = 0u;
  {
    float2 x[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (32 * k + lane < cd.n) x[k] = score[32 * k + lane];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      held[k] = 0u;
      if (32 * k + lane < cd.n) {
        held[k] = ordered(x[k].x);
        big = fmaxf(big, x[k].y);
        lo = min(lo, held[k]);
        hi = max(hi, held[k]);
      }
      sm.keys[32 * k + lane] = held[k];
    }
  }
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  // The key of rank `top` lies in [first, last], halved until it is no wider than
  // the error of two sums.
  const float e2 = big * (1.0f / 8192.0f);
  uint32_t first = lo, last = hi;
  while (first < last && !(unordered(last) - unordered(first) <= e2)) {
    const uint32_t p = first + ((last - first) >> 1) + 1u;
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) n += held[k] >= p;
    if (__reduce_add_sync(0xffffffffu, n) >= static_cast<uint32_t>(a.top))
      first = p;
    else
      last = p - 1u;
  }
  // keys above `top` are kept, below `bottom` are not
  const uint32_t top = ordered(unordered(last) + e2);
  const uint32_t bottom = max(1u, ordered(unordered(first) - e2));
  uint32_t in = 0, between = 0;
#pragma unroll 4
  for (int k = 0; k < steps; ++k) {
    const uint32_t u = sm.keys[32 * k + lane];
    const uint32_t x = __ballot_sync(0xffffffffu, u > top);
    const uint32_t y = __ballot_sync(0xffffffffu, u <= top && u >= bottom);
    in += __popc(x);
    between += __popc(y);
    if (lane == 0) {
      sm.in[k] = x;
      sm.band[k] = y;
    }
  }
  __syncwarp();
  const uint32_t need = a.top - in;                 // of those between; at least one
  const bool ranked = between > need;
  uint32_t least = 0u, equal = 0xffffffffu;         // of the pages between, when ranked
  if (ranked) {
    uint32_t elo = 0xffffffffu, ehi = 0u;
#pragma unroll 1
    for (int k = 0; k < steps; ++k) {
      uint32_t todo = sm.band[k];
#pragma unroll 1
      while (todo) {
        const int i = 32 * k + __ffs(todo) - 1;
        todo &= todo - 1;
        const uint32_t x = ordered(exact_score(a, t, g, phys_page(a.q, s, a.sink + i)));
        if (lane == 0) sm.keys[i] = x;
        elo = min(elo, x);
        ehi = max(ehi, x);
      }
    }
    __syncwarp();
    const int eb = 31 - __clz(elo ^ ehi);
    auto over = [&](uint32_t c) {
      uint32_t n = 0;
#pragma unroll 4
      for (int k = 0; k < steps; ++k)
        n += ((sm.band[k] >> lane) & 1u) && sm.keys[32 * k + lane] >= c;
      return __reduce_add_sync(0xffffffffu, n);
    };
    least = bit_rank(eb >= 31 ? 0u : ehi & ~((1u << (eb + 1)) - 1u), eb, need, over);
    equal = need - (least == 0xffffffffu ? 0u : over(least + 1u));
  }
  uint32_t at = 0, eq = 0;
  const uint32_t before = (1u << lane) - 1u;
#pragma unroll 2
  for (int k = 0; k < steps; ++k) {
    const uint32_t u = sm.keys[32 * k + lane], band = sm.band[k];
    const bool mine = (band >> lane) & 1u;
    const uint32_t ties = __ballot_sync(0xffffffffu, ranked && mine && u == least);
    bool keep = (sm.in[k] >> lane) & 1u;
    if (mine) keep = !ranked || u > least || (u == least && eq + __popc(ties & before) < equal);
    const uint32_t all = __ballot_sync(0xffffffffu, keep);
    const uint32_t pos = at + __popc(all & before);
    if (keep && pos < static_cast<uint32_t>(a.top)) out[head + pos] = a.sink + 32 * k + lane;
    at += __popc(all);
    eq += __popc(ties);
  }
}

}  // namespace spa

// paged_attn.cuh -- causal attention of new tokens (one per sequence, or a
// chunk) over the pages of a key/value cache, on the 5th-generation tensor
// cores; all pages of a sequence, or a list of pages per token and kv head.
//
// Mathematics: FlashAttention's online softmax, O and the running (max, sum)
// in fp32, P rounded to bf16 for the second product (relative error 2^-8 of
// each probability; the sum is taken of the unrounded values).
//
// Rows.  The q heads of a kv head read the same keys, so a 128-row tile of Q
// is packed token by token with the group's heads inside: row = token * group
// + head.  Keys come in tiles of 128, a tile being 128 / page_size whole pages
// found through the block table, one TMA box per page and 64 columns (small
// pages and few rows: per page).
//
// Three ways through a segment, by the rows of its unit:
//   two row tiles   (more than 128 / group tokens)  A: the first 128 / group
//           tokens, B: the next; both read every key tile, softmax warpgroup
//           A / B works on its own rows;
//   one row tile    the warpgroups take the key tiles in turn (even ones A, odd
//           ones B), each with an accumulator of its own, and warpgroup A
//           joins the two at the end: two independent chains of tiles hide the
//           latency of one another's softmax;
//   few rows        (at most 16: one token, or a few of a small group)  a
//           128-row product would be empty for the most part, and its softmax
//           keeps one warp of four busy; instead each of the eight warps takes
//           16 keys of every tile with mma.sync m16n8k16, from the same shared
//           memory, (max, sum, O) in its registers, and the eight are joined
//           at the end.  Bound by the bytes of K and V: 64 KB a tile against
//           256 such products.
// In the first two step j of a segment (a run of key tiles) uses score slot,
// accumulator and warpgroup j & 1, in the order
//   S_0, S_1, PV_0, S_2, PV_1, S_3, PV_2, ...
// so the tensor core has one product to do while the other slot's softmax runs.
// A step batch that mixes prompt chunks and single tokens has both.
//
// Work split.  All (sequence, kv head, row tiles) units lie end to end on one
// line, as long as they take, and each CTA (one per SM, persistent) takes an
// equal piece of that line, found by a scan over the sequences' lengths: every
// SM has the same work however ragged the batch is, one long sequence included.
// A unit that one CTA covers is finished there; the pieces of the others (at
// most two per CTA) go to the workspace in fp32 and paged_combine_kernel joins
// them in the order of their CTAs, so that the result does not depend on
// timing.  Lists of many tokens are cut into whole units instead (see turn).
//
// Rows of V past the last visible key of a tile (the unfilled end of a page,
// pages not loaded) are cleared before they are read: their probability is 0,
// but 0 * NaN is not.
//
// Roles (384 threads): warps 0-3 / 4-7 softmax of slot 0 / 1, warp 8 loads,
// warp 9 MMA, TMEM and the ends of V tiles, warp 10 walks the CTA's piece and
// hands its segments to the others through a ring of four, so that the lengths,
// lists and page numbers of the next units are read ahead.  Launched with 168
// registers a thread (the compiler spills 176 bytes, 168 with lists), split into
// 56 and 224.  tests/paged_protocol.py plays the roles on the CPU: who waits for
// what, and who may still read what another writes.
//
// Measured (one B200; bound): 2048 tokens at 32K, 32/8 heads, 1.04-1.12 ms, 950
// to 1026 TFLOP/s (the way of a tile's scores through its warpgroup: tensor
// pipe busy for 2048 of some 3600 cycles per pair of tiles); one token at 128K,
// 64/8 heads, 93 us, 5.8 TB/s, and 32 tokens of 300 to 16K keys 128 us, 5.5
// TB/s (memory); one token at 1000 keys 12 us (latency of two kernels).
//
// TMEM columns: S_0 [0,128) (P_0 in [0,64)), S_1 [128,256), O_0 [256,384),
// O_1 [384,512).
#pragma once

#include "common.cuh"
#include "paged_seqs.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace spa {

constexpr int kPagedThreads = 384;
constexpr int kPagedKStages = 3;
constexpr int kPagedVStages = 2;
constexpr uint32_t kPagedBarBytes = 2048u;   // barriers, row statistics, search
constexpr uint32_t kPagedSmemBytes =
    1024u + 2u * kTileBytes + (kPagedKStages + kPagedVStages) * kTileBytes + kPagedBarBytes;
static_assert(kPagedSmemBytes <= 232448u, "more shared memory than a CTA may use");

// What the combine needs of a unit that several CTAs share; written by the
// CTA that starts it, at its own index (c1 < 0: none).
struct PagedRecord {
  int c1;        // last CTA of the unit
  int g;         // kv head
  int tok0;      // first token row
  int ntok;      // tokens
};

// A CTA's share of one unit, handed by the walking warp to the others.
struct PagedSeg {
  int tb, te;    // key tiles [tb, te) of the unit; te < 0: the piece is done
  int flags;     // kSeg*
  int keys;      // keys the unit reads (0: none of its rows sees any)
  int tok0;      // first token row
  int ntok;      // tokens
  int pos0;      // position of the first
  int g;         // kv head
  int seq;       // block table row
  int pad[3];
  int page[32];  // physical numbers of the first 32 pages from tile tb on (-1: none)
};
static_assert(sizeof(PagedSeg) == 176, "ring entries");
constexpr int kPagedSegs = 4;
struct FewSeg {   // what its eight warps need of a segment of few rows
  int tb, te, flags, keys, tok0, ntok, pos0, g;
};
constexpr int kSegDuo = 1;      // two row tiles
constexpr int kSegStart = 2;    // holds the unit's first tile
constexpr int kSegWhole = 4;    // holds all of them
constexpr int kSegFew = 8;      // at most kFewRows rows
// Q buffers (each 32 KB): both for two row tiles, one of them in turn for one,
// both as the exchange area of few rows
constexpr int kSegBuf = 16;     // the one in turn
constexpr int kSegPar = 32;     // << i: parity of buffer i's use
constexpr int kSegOld = 128;    // << i: it was used before
constexpr int kFewRows = 16;
// Pages up to these sizes come as one box of whole rows when rows are few, a key's
// two 128-byte lines beside one another: a box costs some 50 cycles beside its
// rows, more than the two-way bank conflicts of reading this layout.  32 tokens
// of 300 to 16K keys in pages of 16: 185 us instead of 209, but in pages of 32
// 182.5 instead of 180.5; lists of 1024 keys, which many tokens read from L2, in
// pages of 32: 159 us instead of 163, of 64: 161 instead of 151.
constexpr int kWholeRowPages = 16, kWholeRowListPages = 32;
// Arrivals that free a K, V or Q buffer: of the eight softmax warps and the MMA
// warp when rows are few, else of the MMA's commit, which counts for all.
constexpr uint32_t kReaders = 9;
// Lengths on the line of work, in units of about 0.55 us: a key tile (64 KB of K
// and V from memory: 1.6 us; with two row tiles 2.2 us of products), and what a
// unit costs beside its tiles (Q, the first tile's way through, joining and
// storing: measured 2 us for few rows, 6 us for row tiles).
constexpr int kTileOne = 3, kTileDuo = 4, kEdgeFew = 4, kEdgeRows = 11;
static_assert(kTileDuo > kTileOne, "tells two row tiles");

struct PagedAttnArgs {
  Seqs q;
  Rows xq, o;
  float* lse;                // [T][Hq] or null
  const int32_t* lists;      // [T][Hkv][width] or null
  const int32_t* counts;     // [T][Hkv]
  int width;                 // list entries per (token, kv head)
  int unit_length;           // length on the line of a full list
  int whole_units;           // lists: CTAs take whole units in turn
  int q_by_rows;             // q's heads lie further apart than its tokens
  int whole_rows;            // few rows: pages as one box of 256-byte rows
  int Hq, Hkv, group;
  int tpt1;                  // tokens per 128-row tile
  int pitch;                 // 128-element rows between pages
  float sl2;                 // softmax scale * log2(e)
  PagedRecord* rec;          // [G]
  float* part;               // [2 G] slots of kPagedSlotFloats
  uint64_t wait_ns;
  uint32_t debug;
};

// One partial slot: O [32 groups of four columns][256 rows][4], m [256], l [256]:
// threads that own a row each store 512 contiguous bytes together, and four
// rows by eight groups are whole sectors to the combine.
constexpr int kPagedSlotRows = 256;
constexpr long long kPagedSlotFloats = 130LL * kPagedSlotRows;

// The CTA whose piece [total * c / G, total * (c + 1) / G) holds point x.
__device__ __forceinline__ int piece_of(long long x, long long total, int G) {
  return static_cast<int>(quotient((x + 1) * G - 1, total));
}

// ---------------------------------------------------------------------------
// The units of a CTA's piece, in order.
// ---------------------------------------------------------------------------
template <bool LIST>
struct PagedWalk {
  const PagedAttnArgs& a;
  long long x0, x1;          // the CTA's piece of the line
  long long base;            // where the current unit starts on it
  int s = 0, g = 0, r = 0;   // sequence (LIST: token row), kv head, row tile
  int q0, n, pos_first;      // of the sequence
  int nr;                    // its row tiles
  // the current unit
  int seq = 0, tok0 = 0, ntok = 0, pos0 = 0, keys = 0, nt = 0;
  int w, edge, flat;         // lengths on the line: a tile, what precedes them, all

  __device__ __forceinline__ explicit PagedWalk(const PagedAttnArgs& args) : a(args) {}

  __device__ __forceinline__ static int tiles_of(int keys) { return keys > 0 ? (keys + 127) >> 7 : 1; }

  // keys that the last token of row tile r sees
  __device__ __forceinline__ static int tile_keys(int pos_first, int n, int tpt, int r) {
    return max(0, pos_first + min((r + 1) * tpt, n));
  }

  // Lengths on the line: of one key tile of a unit of `tokens` tokens, and of
  // the unit's start and end.
  __device__ __forceinline__ static int tile_length(const PagedAttnArgs& a, int tokens) {
    return tokens > a.tpt1 ? kTileDuo : kTileOne;
  }
  __device__ __forceinline__ static int edge_length(const PagedAttnArgs& a, int tokens) {
    return tokens * a.group <= kFewRows ? kEdgeFew : kEdgeRows;
  }
  __device__ __forceinline__ static int unit_length(const PagedAttnArgs& a, int tokens, int keys) {
    return edge_length(a, tokens) + tiles_of(keys) * tile_length(a, tokens);
  }

  // Length on the line of sequence s, one kv head.
  __device__ __forceinline__ static long long head_length(const PagedAttnArgs& a, int s, bool& duo) {
    const Seq q = seq_at(a.q, s);
    const int tpt = 2 * a.tpt1;
    long long len = 0;
    for (int r = 0; r * tpt < q.n; ++r)
      len += unit_length(a, min(tpt, q.n - r * tpt), tile_keys(q.kv - q.n, q.n, tpt, r));
    duo = q.n > a.tpt1;
    return len;
  }

  __device__ __forceinline__ void load_seq() {
    if (LIST) {
      const Seq q = seq_of_token(a.q, s, seq);
      n = q.n;
      q0 = s;
      pos_first = q.kv - q.n + (s - q.q0);
      nr = 1;
    } else {
      const Seq q = seq_at(a.q, s);
      seq = s;
      q0 = q.q0;
      n = q.n;
      pos_first = q.kv - q.n;
      nr = (n + 2 * a.tpt1 - 1) / (2 * a.tpt1);
    }
  }

  __device__ __forceinline__ void set_unit() {
    if (LIST) {
      tok0 = s;
      ntok = n > 0 ? 1 : 0;
      pos0 = pos_first;
      keys = 0;
      flat = a.unit_length;
      if (n > 0 && pos0 >= 0) {
        const long long at = static_cast<long long>(s) * a.Hkv + g;
        int cnt = a.counts[at];
        if (cnt < 0 || cnt > a.width) {
          atomicOr(a.q.err, kErrBadIndex);
          cnt = 0;
        }
        if (cnt > 0) {
          // full pages but the last one, which may hold the token itself
          const int last = a.lists[at * a.width + cnt - 1];
          if (last < 0 || last > (pos0 >> a.q.shift)) {
            atomicOr(a.q.err, kErrBadIndex);
          } else {
            keys = ((cnt - 1) << a.q.shift) + min(a.q.page, pos0 - (last << a.q.shift) + 1);
          }
        }
      }
      nt = tiles_of(keys);
      w = kTileOne;
      edge = edge_length(a, 1);
    } else {
      const int tpt = 2 * a.tpt1;
      tok0 = q0 + r * tpt;
      ntok = min(tpt, n - r * tpt);
      pos0 = pos_first + r * tpt;
      keys = tile_keys(pos_first, n, tpt, r);
      nt = tiles_of(keys);
      w = tile_length(a, ntok);
      edge = edge_length(a, ntok);
      flat = edge + nt * w;
    }
  }

  // Goes to the unit that holds x0.  s0, base0, length0: the sequence that holds
  // it, where that starts and its length (not LIST).
  __device__ __forceinline__ void start(int s0, long long base0, long long length0) {
    if (LIST) {
      const long long u = quotient(x0, a.unit_length);
      s = static_cast<int>(quotient(u, a.Hkv));
      g = static_cast<int>(u - static_cast<long long>(s) * a.Hkv);
      base = u * a.unit_length;
      r = 0;
      load_seq();
    } else {
      s = s0;
      base = base0;
      load_seq();
      const long long per_head = quotient(length0, a.Hkv);
      g = static_cast<int>(quotient(x0 - base0, per_head));
      base += g * per_head;
      r = 0;
      while (true) {
        const int len = unit_length(a, min(2 * a.tpt1, n - 2 * r * a.tpt1),
                                    tile_keys(pos_first, n, 2 * a.tpt1, r));
        if (x0 < base + len || r + 1 >= nr) break;
        base += len;
        ++r;
      }
    }
    set_unit();
  }

  __device__ __forceinline__ bool more() const { return base < x1; }

  // Lists, whole units in turn: unit u is kv head u / T, token u % T, so that
  // the CTAs are on the same head at the same time and tokens of one sequence
  // find the pages they share in L2.
  __device__ __forceinline__ void turn(long long u) {
    base = u;
    if (base >= x1) return;
    g = static_cast<int>(u / a.q.T);
    s = static_cast<int>(u - static_cast<long long>(g) * a.q.T);
    r = 0;
    load_seq();
    set_unit();
  }

  __device__ __forceinline__ void next() {
    if (LIST && a.whole_units) {
      turn(base + gridDim.x);
      return;
    }
    base += flat;
    if (base >= x1) return;
    if (++r >= nr || LIST) {
      r = 0;
      if (++g >= a.Hkv) {
        g = 0;
        do {                      // base < x1 <= total: a sequence with tokens follows
          if (++s >= (LIST ? a.q.T : a.q.S)) {
            base = x1;
            return;
          }
          load_seq();
        } while (!LIST && n == 0);
      }
    }
    set_unit();
  }

  // The CTA's tiles [b, e) of the current unit: those that begin on its piece;
  // false: none of them exist.
  __device__ __forceinline__ bool range(int& b, int& e) const {
    if (LIST && a.whole_units) {
      b = 0;
      e = nt;
      return ntok > 0;
    }
    const long long t0 = base + edge;
    const long long all = static_cast<long long>(nt) * w;          // below 2^32
    const uint32_t p0 = static_cast<uint32_t>(min(max(x0 - t0, 0LL), all));
    const uint32_t p1 = static_cast<uint32_t>(min(max(x1 - t0, 0LL), all));
    b = static_cast<int>(w == kTileDuo ? (p0 + kTileDuo - 1) / kTileDuo : (p0 + kTileOne - 1) / kTileOne);
    e = static_cast<int>(w == kTileDuo ? (p1 + kTileDuo - 1) / kTileDuo : (p1 + kTileOne - 1) / kTileOne);
    return b < e && ntok > 0;
  }
};

// Physical number of page j of a unit's keys; -1 behind its last.  A bad entry is
// reported, and any page does for it.
template <bool LIST>
__device__ __forceinline__ int unit_page(const PagedAttnArgs& a, int j, int keys, int tok, int g,
                                         int seq, int pos) {
  if (j >= (keys + a.q.page - 1) >> a.q.shift) return -1;
  int lp = j;
  if (LIST) {
    const int32_t* list = a.lists + (static_cast<long long>(tok) * a.Hkv + g) * a.width;
    lp = list[j];
    const int before = j > 0 ? list[j - 1] : -1;
    if (lp <= before || lp < 0 || lp > (pos >> a.q.shift)) {
      atomicOr(a.q.err, kErrBadIndex);
      lp = 0;
    }
  }
  const int p = phys_page(a.q, seq, lp);
  return p < 0 ? 0 : p;
}

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// Float index of (row, column) of a warp's 16 x 128 exchange area: groups of
// eight columns are permuted by the row, so that neither the fragments' 8-byte
// stores nor the rows' 16-byte loads meet in a bank.
__device__ __forceinline__ int few_at(int row, int col) {
  return row * 128 + (col ^ ((row & 7) << 3));
}

// Index of a warp's (m, l) of a row when rows are few.  Warps of warpgroup 0 may
// still read the second accumulator's statistics of the segment before, warp w
// those of rows 32 w .. 32 w + 31, and nothing orders them against one another:
// each overwrites only entries that it alone reads.  Warpgroup 1 waits for them.
__device__ constexpr int few_ml(int warp, int row) {
  return (warp & 3) * 32 + (warp >> 2) * 16 + row;
}

// Barriers, 8 bytes each from b0.
struct PagedBars {
  uint32_t b0;
  __device__ __forceinline__ uint32_t at(int i) const { return b0 + 8u * i; }
  __device__ __forceinline__ uint32_t kfull(int s) const { return at(s); }
  __device__ __forceinline__ uint32_t kempty(int s) const { return at(3 + s); }
  __device__ __forceinline__ uint32_t vfull(int s) const { return at(6 + s); }
  __device__ __forceinline__ uint32_t vempty(int s) const { return at(8 + s); }
  __device__ __forceinline__ uint32_t phalf(int h) const { return at(10 + h); }
  __device__ __forceinline__ uint32_t sfull(int h) const { return at(12 + h); }
  __device__ __forceinline__ uint32_t pfull(int h) const { return at(14 + h); }
  __device__ __forceinline__ uint32_t odone(int h) const { return at(16 + h); }
  __device__ __forceinline__ uint32_t ofree(int h) const { return at(18 + h); }
  __device__ __forceinline__ uint32_t qfull(int i) const { return at(20 + i); }
  __device__ __forceinline__ uint32_t qfree(int i) const { return at(22 + i); }
  __device__ __forceinline__ uint32_t wfull(int i) const { return at(24 + i); }
  __device__ __forceinline__ uint32_t wempty(int i) const { return at(28 + i); }
  __device__ __forceinline__ uint32_t xch() const { return at(32); }
  __device__ __forceinline__ uint32_t drain() const { return at(33); }
  __device__ __forceinline__ uint32_t stall() const { return at(34); }
  __device__ __forceinline__ uint32_t few() const { return at(35); }
};
static_assert(kPagedKStages == 3 && kPagedVStages == 2, "barrier numbers");
// Offsets behind the barriers (36 of them).
// The search of a CTA's piece is over before the ring is used.
constexpr int kPagedTmem = 304, kPagedSegRing = 320, kPagedFind = 320, kPagedMl = 1024;
static_assert(kPagedSegRing + kPagedSegs * sizeof(PagedSeg) <= kPagedMl, "ring");

// A segment of few rows (see above), by one of the eight warps; kt: the CTA's
// tiles before it, parity: of this segment's exchange, uses1: of accumulator 1
// before it.  False when a wait gave up.  A function of its own, so that its
// registers and those of the 128-row softmax are allotted apart.
template <bool LIST, bool WHOLE_ROWS>
__device__ __noinline__ bool few_segment(const PagedAttnArgs& a, const FewSeg sg, uint8_t* smem,
                                         uint32_t s_base, uint32_t b0, const WaitCtx wc, int kt,
                                         uint32_t parity, int uses1) {
  const PagedBars bars{b0};
  volatile float* ml = reinterpret_cast<volatile float*>(
      smem + (2 + kPagedKStages + kPagedVStages) * kTileBytes + kPagedMl);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  const int tb = sg.tb, te = sg.te, keys = sg.keys, g = sg.g, tok0 = sg.tok0, flags = sg.flags;
  const int nrows = sg.ntok * a.group;
  const int r0 = lane >> 2, c2 = 2 * (lane & 3);
  // a key's two 128-byte lines: 16 KB apart, or beside one another
  constexpr uint32_t key_bytes = WHOLE_ROWS ? 256u : 128u;
  constexpr uint32_t half_bytes = WHOLE_ROWS ? 128u : kHalfBytes;
  int seen[2];
  uint32_t qf[8][4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    // rows r0 and r0 + 8; rows behind the last are zero
    const int rr = r0 + 8 * e, ti = rr / a.group;
    const bool on = rr < nrows;
    seen[e] = !on ? 0 : LIST ? keys : max(0, sg.pos0 + ti + 1);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        a.xq.at(0, tok0 + (on ? ti : 0), g * a.group + (on ? rr - ti * a.group : 0)));
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qf[ks][e] = on ? src[(16 * ks + c2) >> 1] : 0u;
      qf[ks][2 + e] = on ? src[(16 * ks + 8 + c2) >> 1] : 0u;
    }
  }
  float acc[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  for (int t = tb; t < te; ++t, ++kt) {
    const int ks_ = kt % kPagedKStages, vs_ = kt % kPagedVStages;
    const int left = keys - 128 * t - 16 * warp;   // keys from this warp's sixteen on
    if (!warp_wait(bars.kfull(ks_), (kt / kPagedKStages) & 1, wc)) return false;
    uint32_t pf[4];
    if (left > 0) {
      float sc2[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc2[n][e] = 0.f;
      // matrix i of a load: key half i / 2 (8 keys each), 16-byte chunk i % 2
      const int key = 16 * warp + ((lane >> 4) << 3) + (lane & 7);
      const uint32_t kat = s_base + (2u + ks_) * kTileBytes + key * key_bytes;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t kf[4];
        const uint32_t line = kat + (ks >> 2) * half_bytes;    // its chunks are permuted by its address
        const uint32_t chunk = (2 * ks + ((lane >> 3) & 1)) & 7;
        ldsm4(kf, line + ((chunk << 4) ^ ((line >> 3) & 0x70u)));
        mma_16816(sc2[0], qf[ks], kf[0], kf[1]);
        mma_16816(sc2[1], qf[ks], kf[2], kf[3]);
      }
      const int k0 = 128 * t + 16 * warp + c2;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (k0 + 8 * n + (e & 1) >= seen[e >> 1]) sc2[n][e] = -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], sc2[n][e]);
        }
      float fac[2];
      bool grow = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2)) * a.sl2;
        fac[e] = 1.f;
        if (mx[e] > m[e] + 8.0f) {              // as above: the maximum may lag
          fac[e] = fast_exp2(m[e] - mx[e]);
          m[e] = mx[e];
          l[e] *= fac[e];
          grow = true;
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] *= fac[e >> 1];
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float nm = m[e] == -INFINITY ? 0.f : -m[e];
          const float p0 = fast_exp2(fmaf(sc2[n][2 * e], a.sl2, nm));
          const float p1 = fast_exp2(fmaf(sc2[n][2 * e + 1], a.sl2, nm));
          l[e] += p0 + p1;
          pf[2 * n + e] = pack_bf16x2(p0, p1);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.kempty(ks_));
    if (!warp_wait(bars.vfull(vs_), (kt / kPagedVStages) & 1, wc)) return false;
    if (left > 0) {
      // matrix i: key half i % 2, 16-byte chunk i / 2 of a pair
      const int key = 16 * warp + (lane & 15);
      const uint32_t vat = s_base + (2u + kPagedKStages + vs_) * kTileBytes + key * key_bytes;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t vf[4];
        const uint32_t line = vat + (j >> 2) * half_bytes;
        const uint32_t chunk = (2 * j + (lane >> 4)) & 7;
        ldsm4_t(vf, line + ((chunk << 4) ^ ((line >> 3) & 0x70u)));
        if (left < 16) {
          // rows behind the last key: their probability is 0, but 0 * NaN is not
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k0 = c2 + 8 * (e & 1);
            vf[e] &= k0 + 1 < left ? 0xffffffffu : k0 < left ? 0xffffu : 0u;
          }
        }
        mma_16816(acc[2 * j], pf, vf[0], vf[1]);
        mma_16816(acc[2 * j + 1], pf, vf[2], vf[3]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.vempty(vs_));
  }
  // join the eight warps: the Q buffers are the exchange area
  for (int b = 0; b < 2; ++b)
    if (!warp_wait(bars.qfull(b), (flags & (kSegPar << b)) ? 1 : 0, wc)) return false;
  // (warpgroup 0 may still read ml for an earlier segment's second accumulator, see few_ml)
  if (warp >= 4 && uses1 > 0 && !warp_wait(bars.ofree(1), (uses1 - 1) & 1, wc)) return false;
  float* area = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    const int rr = r0 + 8 * e;
    if (rr < nrows) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        *reinterpret_cast<float2*>(area + warp * 2048 + few_at(rr, 8 * j + c2)) =
            make_float2(acc[j][2 * e], acc[j][2 * e + 1]);
      if ((lane & 3) == 0) {
        ml[few_ml(warp, rr)] = m[e];
        ml[128 + few_ml(warp, rr)] = l[e];
      }
    }
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(bars.few());
  if (!warp_wait(bars.few(), parity, wc)) return false;
  float* part = a.part + (2LL * c + ((flags & kSegStart) ? 1 : 0)) * kPagedSlotFloats;
  const bool whole = (flags & kSegWhole) != 0;
  for (int rr = warp; rr < nrows; rr += 8) {
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) mm = fmaxf(mm, ml[few_ml(w, rr)]);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float mw = ml[few_ml(w, rr)];
      const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - mm);
      ll = fmaf(ml[128 + few_ml(w, rr)], f, ll);
      const float4 x = *reinterpret_cast<const float4*>(area + w * 2048 + few_at(rr, 4 * lane));
      y.x = fmaf(x.x, f, y.x);
      y.y = fmaf(x.y, f, y.y);
      y.z = fmaf(x.z, f, y.z);
      y.w = fmaf(x.w, f, y.w);
    }
    const int ti = rr / a.group;
    const long long tok = static_cast<long long>(tok0) + ti;
    const int head = g * a.group + (rr - ti * a.group);
    if (whole) {
      const float inv = ll > 0.f ? 1.0f / ll : 0.f;
      uint2 z;
      z.x = pack_bf16x2(y.x * inv, y.y * inv);
      z.y = pack_bf16x2(y.z * inv, y.w * inv);
      *reinterpret_cast<uint2*>(a.o.at(0, tok, head) + 4 * lane) = z;
      if (a.lse && lane == 0)
        a.lse[tok * a.Hq + head] =
            ll > 0.f ? mm * 0.69314718055994531f + logf(ll) : -INFINITY;
    } else {
      *reinterpret_cast<float4*>(part + (lane * kPagedSlotRows + rr) * 4) = y;
      if (lane == 0) {
        part[128 * kPagedSlotRows + rr] = mm;
        part[129 * kPagedSlotRows + rr] = ll;
      }
    }
  }
  // the next contents of the area may come by a copy (async proxy)
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(bars.qfree(0));
    mbar_arrive(bars.qfree(1));
  }
  return true;
}

template <bool LIST>
__global__ void __launch_bounds__(kPagedThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_k2,   // whole rows
                  const __grid_constant__ CUtensorMap tm_v2,
                  const __grid_constant__ PagedAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_u32(smem);
  auto s_q = [&](int i) { return s_base + i * kTileBytes; };
  auto s_k = [&](int st) { return s_base + (2u + st) * kTileBytes; };
  auto s_v = [&](int st) { return s_base + (2u + kPagedKStages + st) * kTileBytes; };
  uint8_t* ctl = smem + (2 + kPagedKStages + kPagedVStages) * kTileBytes;
  const uint32_t b0 = smem_u32(ctl);
  const PagedBars bars{b0};
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ctl + kPagedTmem);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  PagedSeg* segs = reinterpret_cast<PagedSeg*>(ctl + kPagedSegRing);
  FindSmem& find = *reinterpret_cast<FindSmem*>(ctl + kPagedFind);
  static_assert(sizeof(FindSmem) <= kPagedMl - kPagedFind, "search area");
  volatile float* ml = reinterpret_cast<volatile float*>(ctl + kPagedMl);   // slot 1's m, l [128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the combine waits by itself
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPagedKStages; ++i) {
      mbar_init(bars.kfull(i), 1);
      mbar_init(bars.kempty(i), kReaders);
    }
    for (int i = 0; i < kPagedVStages; ++i) {
      mbar_init(bars.vfull(i), 1);
      mbar_init(bars.vempty(i), kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.sfull(i), 1);
      mbar_init(bars.phalf(i), 4);        // warps, by one lane each
      mbar_init(bars.pfull(i), 4);
      mbar_init(bars.odone(i), 1);
      mbar_init(bars.ofree(i), i == 0 ? 8 : 4);
      mbar_init(bars.qfull(i), 1);
      mbar_init(bars.qfree(i), kReaders);
    }
    for (int i = 0; i < kPagedSegs; ++i) {
      mbar_init(bars.wfull(i), 1);
      mbar_init(bars.wempty(i), 10);     // loads, MMA, eight softmax warps
    }
    mbar_init(bars.few(), 8);
    mbar_init(bars.xch(), 4);
    mbar_init(bars.drain(), 1);
    mbar_init(bars.stall(), 1);
    *abort_flag = 0u;
    fence_barrier_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    if (a.whole_rows) {
      prefetch_tensormap(&tm_k2);
      prefetch_tensormap(&tm_v2);
    }
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what the stream did before is visible
  // this CTA's piece of the line: only the walking warp needs it, and finds it
  // by itself when the sequences are few
  const int c = blockIdx.x;
  // pieces: none without a tile of a unit that spans it, so that every CTA
  // between the first and the last of a shared unit has a part of it
  bool any_duo = false;
  auto pieces = [&](long long total) {
    return static_cast<int>(
        min(static_cast<long long>(gridDim.x), max(total / (any_duo ? kTileDuo : kTileOne), 1LL)));
  };
  Found f{0, 0, 0, 0, 0};
  if (LIST) {
    f.total = static_cast<long long>(a.q.T) * a.Hkv * a.unit_length;
  } else {
    bool duo = false;
    auto length = [&](int s) {
      bool d;
      const long long len = PagedWalk<LIST>::head_length(a, s, d) * a.Hkv;
      duo |= d;
      return len;
    };
    if (a.q.S <= 32 * kWarpFind) {
      if (warp == 10) {
        f = warp_find(a.q.S, length, [&](long long total) {
          any_duo = __any_sync(0xffffffffu, duo);
          return quotient(total * c, pieces(total));
        });
      }
    } else {
      f = block_find(
          a.q.S, length,
          [&](long long total) {
            any_duo = __syncthreads_or(duo);
            return quotient(total * c, pieces(total));
          },
          find);
    }
  }
  const int G = pieces(f.total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
  const WaitCtx wc{abort_flag, a.q.err, a.wait_ns};
  // Segment i of the piece, copied out of the ring; false at its end.
  auto take = [&](int i, PagedSeg& sg, int* page = nullptr) -> bool {
    const int r = i % kPagedSegs;
    if (!warp_wait(bars.wfull(r), (i / kPagedSegs) & 1, wc)) return false;
    const PagedSeg& x = segs[r];
    sg.tb = x.tb;
    sg.te = x.te;
    sg.flags = x.flags;
    sg.keys = x.keys;
    sg.tok0 = x.tok0;
    sg.ntok = x.ntok;
    sg.pos0 = x.pos0;
    sg.g = x.g;
    sg.seq = x.seq;
    if (page) *page = x.page[lane];
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.wempty(r));
    return sg.te >= 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;" ::: "memory");
    if (warp == 8) {
      // ----------------------------------------------------------- loads
      const int ppt = 128 >> a.q.shift;             // pages per tile
      const uint32_t page_half = 128u * a.q.page;   // bytes of a page's 64 columns
      int kt = 0, qlast[2] = {-1, -1};              // key tiles; parity of the Q loads in flight
      bool ok = true;
      PagedSeg sg;
      int mine = -1;                                // the lane's page of the first batch
      for (int i = 0; ok && take(i, sg, &mine); ++i) {
        if (sg.keys == 0) continue;
        const bool duo = (sg.flags & kSegDuo) != 0, few = (sg.flags & kSegFew) != 0;
        const bool rows256 = few && a.whole_rows;
        for (int buf = 0; buf < 2; ++buf) {
          if (!duo && !few && buf != ((sg.flags & kSegBuf) ? 1 : 0)) continue;
          const int par = (sg.flags & (kSegPar << buf)) ? 1 : 0;
          if ((sg.flags & (kSegOld << buf)) && !(ok = warp_wait(bars.qfree(buf), par ^ 1, wc))) break;
          if (few) {                                // nothing to load: the area is free
            if (lane == 0) mbar_arrive(bars.qfull(buf));
            qlast[buf] = -1;
            continue;
          }
          const int tok = sg.tok0 + (duo ? buf * a.tpt1 : 0);
          if (a.q_by_rows) {
            const int rows = min(a.tpt1, sg.ntok - (duo ? buf * a.tpt1 : 0)) * a.group;
            if (lane == 0) mbar_arrive_expect_tx(bars.qfull(buf), rows * 256u);
            __syncwarp();
            for (int k = lane; k < rows; k += 32) {
              const int ti = k / a.group, head = sg.g * a.group + (k - ti * a.group);
              tma_load_3d(s_q(buf) + k * 128u, &tm_q, bars.qfull(buf), 0, tok + ti, head);
              tma_load_3d(s_q(buf) + kHalfBytes + k * 128u, &tm_q, bars.qfull(buf), 64, tok + ti,
                          head);
            }
          } else if (lane == 0) {
            // one box of whole tokens per 64 columns; the rows behind the unit's
            // last token are other tokens' or zero, and their results are not stored
            mbar_arrive_expect_tx(bars.qfull(buf), a.tpt1 * a.group * 256u);
            tma_load_3d(s_q(buf), &tm_q, bars.qfull(buf), 0, sg.g * a.group, tok);
            tma_load_3d(s_q(buf) + kHalfBytes, &tm_q, bars.qfull(buf), 64, sg.g * a.group, tok);
          }
          qlast[buf] = par;
        }
        if (!ok) break;
        __syncwarp();
        // Pages come in batches of 32, one per lane: the first with the segment,
        // each further one read while the tiles before it are loaded.
        const int per = 32 / ppt;                   // tiles per batch
        auto batch = [&](int k) {
          return unit_page<LIST>(a, (sg.tb + k * per) * ppt + lane, sg.keys, sg.tok0, sg.g, sg.seq,
                                 sg.pos0);
        };
        int cur = mine, ahead = batch(1);
        for (int t = sg.tb; t < sg.te; ++t, ++kt) {
          const int in = (t - sg.tb) % per;         // tile of the batch
          if (in == 0 && t > sg.tb) {
            cur = ahead;
            ahead = batch((t - sg.tb) / per + 1);
          }
          const int from = __shfl_sync(0xffffffffu, cur, (in * ppt + lane) & 31);
          const int phys = lane < ppt ? from : -1;
          const uint32_t live = __popc(__ballot_sync(0xffffffffu, phys >= 0));
          const int row = phys * a.pitch + (sg.g << a.q.shift);
          const int ks = kt % kPagedKStages, vs = kt % kPagedVStages;
          const int ku = kt / kPagedKStages, vu = kt / kPagedVStages;
          if (ku > 0 && !(ok = warp_wait(bars.kempty(ks), (ku - 1) & 1, wc))) break;
          if (lane == 0) mbar_arrive_expect_tx(bars.kfull(ks), live * 2u * page_half);
          __syncwarp();
          if (phys >= 0) {
            if (rows256) {
              tma_load_3d(s_k(ks) + 2u * lane * page_half, &tm_k2, bars.kfull(ks), 0, 0, row);
            } else {
              const uint32_t at = s_k(ks) + lane * page_half;
              tma_load_2d(at, &tm_k, bars.kfull(ks), 0, row);
              tma_load_2d(at + kHalfBytes, &tm_k, bars.kfull(ks), 64, row);
            }
          }
          __syncwarp();
          if (vu > 0 && !(ok = warp_wait(bars.vempty(vs), (vu - 1) & 1, wc))) {
            // K of this tile is in flight and counted: drain it below
            ++kt;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bars.vfull(vs), live * 2u * page_half);
          __syncwarp();
          if (phys >= 0) {
            if (rows256) {
              tma_load_3d(s_v(vs) + 2u * lane * page_half, &tm_v2, bars.vfull(vs), 0, 0, row);
            } else {
              const uint32_t at = s_v(vs) + lane * page_half;
              tma_load_2d(at, &tm_v, bars.vfull(vs), 0, row);
              tma_load_2d(at + kHalfBytes, &tm_v, bars.vfull(vs), 64, row);
            }
          }
          __syncwarp();
        }
      }
      // no copy may be in flight when the CTA gives its shared memory back
      // (immediate in normal operation, bounded after an abort)
      if (lane == 0) {
        for (int i = max(0, kt - kPagedKStages); i < kt; ++i)
          mbar_drain(bars.kfull(i % kPagedKStages), (i / kPagedKStages) & 1, a.wait_ns);
        for (int i = max(0, kt - kPagedVStages); i < kt; ++i)
          mbar_drain(bars.vfull(i % kPagedVStages), (i / kPagedVStages) & 1, a.wait_ns);
        for (int i = 0; i < 2; ++i)
          if (qlast[i] >= 0) mbar_drain(bars.qfull(i), qlast[i], a.wait_ns);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------- MMA issuer
      bool ok = true;
      if (a.debug & 1u) ok = warp_wait(bars.stall(), 0, wc);   // never signalled: test hook
      int kt = 0, pc0 = 0, pc1 = 0, oc0 = 0, oc1 = 0;
      auto commit_all = [](uint32_t bar) {
        mbar_arrive_n(bar, kReaders - 1);
        mma_commit(bar);
      };
      PagedSeg sg;
      for (int i = 0; ok && take(i, sg); ++i) {
        if (sg.keys == 0) continue;
        if (sg.flags & kSegFew) {
          // No product of this warp, but it sees every phase of the barriers it
          // will wait on again, and holds up the next one until it has: a wait
          // tells phase n only from n - 1.
          for (int b = 0; ok && b < 2; ++b) {
            ok = warp_wait(bars.qfull(b), (sg.flags & (kSegPar << b)) ? 1 : 0, wc);
            if (ok && lane == 0) mbar_arrive(bars.qfree(b));
          }
          for (int t = sg.tb; ok && t < sg.te; ++t, ++kt) {
            const int ks = kt % kPagedKStages, vs = kt % kPagedVStages;
            if (!(ok = warp_wait(bars.kfull(ks), (kt / kPagedKStages) & 1, wc))) break;
            if (lane == 0) mbar_arrive(bars.kempty(ks));
            if (!(ok = warp_wait(bars.vfull(vs), (kt / kPagedVStages) & 1, wc))) break;
            if (lane == 0) mbar_arrive(bars.vempty(vs));
          }
          continue;
        }
        // Everything an MMA is told is the same in all lanes, and the compiler
        // has to see that (broadcasts from lane 0): descriptors then stay in
        // uniform registers.  Computed by the issuing lane alone they cost some
        // 150 cycles per MMA, more than the MMA itself.
        const int flags = __shfl_sync(0xffffffffu, sg.flags, 0);
        const int tiles = __shfl_sync(0xffffffffu, sg.te - sg.tb, 0);
        const int kt0 = __shfl_sync(0xffffffffu, kt, 0);
        const int duo = (flags & kSegDuo) ? 1 : 0;
        const int steps = tiles << duo;
        const int buf = (flags & kSegBuf) ? 1 : 0;
        auto qk = [&](int j) -> bool {
          const int h = j & 1, k = kt0 + (j >> duo), st = k % kPagedKStages;
          const int qb = duo ? h : buf;
          if (j < 2 && (duo || j == 0)) {
            if (!warp_wait(bars.qfull(qb), (flags & (kSegPar << qb)) ? 1 : 0, wc)) return false;
          }
          if (!warp_wait(bars.kfull(st), (k / kPagedKStages) & 1, wc)) return false;
          tc_fence_after();
          const uint64_t qd = smem_desc_sw128(s_q(qb), 16), kd = smem_desc_sw128(s_k(st), 16);
          const uint32_t d = tmem + 128u * h;
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint64_t off = ((ks >> 2) * kHalfBytes + (ks & 3) * 32u) >> 4;
              mma_bf16_ss(d, qd + off, kd + off, kIdescQK, ks > 0 ? 1u : 0u);
            }
            mma_commit(bars.sfull(h));
            if (!duo || h == 1) commit_all(bars.kempty(st));
            if (j + 1 + duo >= steps) commit_all(bars.qfree(qb));
          }
          __syncwarp();
          return true;
        };
        auto pv = [&](int j) -> bool {
          const int h = j & 1, k = kt0 + (j >> duo), st = k % kPagedVStages;
          const bool first = j < 2;
          const int uses_p = (h ? pc1 : pc0)++;
          if (!warp_wait(bars.vfull(st), (k / kPagedVStages) & 1, wc)) return false;
          const int valid = sg.keys - 128 * (sg.tb + (j >> duo));
          if (valid < 128 && (!duo || h == 0)) {
            // zeros behind the last V row: whole 128-byte rows, so the swizzle
            // within a row does not matter
            uint8_t* tile = smem + (2 + kPagedKStages + st) * kTileBytes;
            for (int x = valid * 8 + lane; x < 128 * 8; x += 32) {
              reinterpret_cast<uint4*>(tile)[x] = make_uint4(0, 0, 0, 0);
              reinterpret_cast<uint4*>(tile + kHalfBytes)[x] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (first) {
            // this accumulator of the segment before has been read
            int& uses = h ? oc1 : oc0;
            if (uses > 0 && !warp_wait(bars.ofree(h), (uses - 1) & 1, wc)) return false;
            ++uses;
          }
          const uint64_t vd = smem_desc_sw128(s_v(st), kHalfBytes);
          const uint32_t d = tmem + 256u + 128u * h, p = tmem + 128u * h;
          if (!warp_wait(bars.phalf(h), uses_p & 1, wc)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_ts(d, p + 8u * ks, vd + ks * (2048u >> 4), kIdescPV,
                          (!first || ks > 0) ? 1u : 0u);
          }
          __syncwarp();
          if (!warp_wait(bars.pfull(h), uses_p & 1, wc)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 4; ks < 8; ++ks)
              mma_bf16_ts(d, p + 8u * ks, vd + ks * (2048u >> 4), kIdescPV, 1u);
            if (!duo || h == 1) commit_all(bars.vempty(st));
            if (j + 2 >= steps) mma_commit(bars.odone(h));
          }
          __syncwarp();
          return true;
        };
        for (int j = 0; ok && j < 2 && j < steps; ++j) ok = qk(j);
        for (int j = 0; ok && j < steps; ++j) {
          ok = pv(j);
          if (ok && j + 2 < steps) ok = qk(j + 2);
        }
        kt += tiles;
      }
      // every MMA issued by this warp's elected lane has completed once this
      // arrives (elect.sync picks the same lane each time)
      if (elect_one()) {
        mma_commit(bars.drain());
        mbar_drain(bars.drain(), 0, a.wait_ns);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ----------------------------------------------- the CTA's segments
      PagedWalk<LIST> walk(a);
      walk.x0 = LIST ? quotient(f.total * c, G) : f.x;
      walk.x1 = quotient(f.total * (c + 1), G);
      if (LIST && a.whole_units) {
        walk.x0 = c;
        walk.x1 = static_cast<long long>(a.q.T) * a.Hkv;
      }
      PagedRecord mine{-1, 0, 0, 0};
      int qn = 0, qu[2] = {0, 0};                   // next Q buffer, uses of each
      int i = 0;
      bool ok = true;
      auto hand = [&](int tb, int te, int flags) {
        const int r = i % kPagedSegs;
        const int page = te >= 0 ? unit_page<LIST>(a, tb * (128 >> a.q.shift) + lane, walk.keys,
                                                   walk.tok0, walk.g, walk.seq, walk.pos0)
                                 : -1;
        if (i >= kPagedSegs) {
          // a long wait as a rule: the warp sleeps in between, out of the others' way
          const uint32_t parity = (i / kPagedSegs - 1) & 1;
          bool there = false;
          for (int k = 0; k < 64 && !there; ++k) {
            there = __all_sync(0xffffffffu, mbar_try_wait(bars.wempty(r), parity));
            if (!there) __nanosleep(500);
          }
          if (!there && !(ok = warp_wait(bars.wempty(r), parity, wc))) return;
        }
        PagedSeg& x = segs[r];
        x.page[lane] = page;
        if (lane == 0) {
          x.tb = tb;
          x.te = te;
          x.flags = flags;
          x.keys = walk.keys;
          x.tok0 = walk.tok0;
          x.ntok = walk.ntok;
          x.pos0 = walk.pos0;
          x.g = walk.g;
          x.seq = walk.seq;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.wfull(r));
        ++i;
      };
      if (c < G && walk.x0 < walk.x1 && f.s >= 0) {
        if (LIST && a.whole_units)
          walk.turn(walk.x0);
        else
          walk.start(f.s, f.base, f.cost);
        for (; ok && walk.more(); walk.next()) {
          int tb, te;
          if (!walk.range(tb, te)) continue;
          if (tb == 0 && te < walk.nt) {            // other CTAs go on with it
            mine.c1 = piece_of(walk.base + walk.edge + static_cast<long long>(walk.w) * (walk.nt - 1),
                               f.total, G);
            mine.g = walk.g;
            mine.tok0 = walk.tok0;
            mine.ntok = walk.ntok;
          }
          int flags = (tb == 0 ? kSegStart : 0) | (tb == 0 && te == walk.nt ? kSegWhole : 0);
          if (walk.w == kTileDuo) flags |= kSegDuo;
          if (walk.ntok * a.group <= kFewRows) flags |= kSegFew;
          if (walk.keys > 0) {
            const bool both = (flags & (kSegDuo | kSegFew)) != 0;
            if (!both) flags |= qn ? kSegBuf : 0;
            for (int b = 0; b < 2; ++b) {
              if (!both && b != qn) continue;
              flags |= ((qu[b] & 1) ? kSegPar << b : 0) | (qu[b] > 0 ? kSegOld << b : 0);
              ++qu[b];
            }
            if (!both) qn ^= 1;
          }
          hand(tb, te, flags);
        }
      }
      if (lane == 0) a.rec[c] = mine;
      if (ok) hand(0, -1, 0);
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;" ::: "memory");
    const int hd = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = 128u * hd, o_col = 256u + 128u * hd;
    // a warp's TMEM and shared-memory accesses so far, then one arrival
    auto warp_arrive = [&](uint32_t bar) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int sc = 0, oc[2] = {0, 0}, xc = 0;           // steps, accumulator uses, hand-overs
    int kt = 0, fc = 0;                           // key tiles, few-row segments
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!warp_wait(bars.wfull(i % kPagedSegs), (i / kPagedSegs) & 1, wc)) break;
      // The segment stays in the ring until its end and is read again there:
      // its fields would not fit beside a row of scores in the registers.
      const volatile PagedSeg& sg = segs[i % kPagedSegs];
      const int te = sg.te, flags = sg.flags;
      if (te < 0) break;
      if ((flags & kSegFew) && sg.keys > 0) {
        const FewSeg own{sg.tb, te, flags, sg.keys, sg.tok0, sg.ntok, sg.pos0, sg.g};
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.wempty(i % kPagedSegs));
        ok = a.whole_rows
                 ? few_segment<LIST, true>(a, own, smem, s_base, b0, wc, kt, fc & 1, oc[1])
                 : few_segment<LIST, false>(a, own, smem, s_base, b0, wc, kt, fc & 1, oc[1]);
        if (!ok) break;
        ++fc;
        kt += te - own.tb;
        continue;
      }
      const bool duo = (flags & kSegDuo) != 0;
      int t = sg.tb + (duo ? 0 : hd);
      const bool two = !duo && te - t > (hd ^ 1);  // both accumulators belong to these rows
      // keys of this thread's row, counted along the unit's key tiles
      int seen;
      bool busy;
      {
        const int rt = row / a.group;             // the row's token within a 128-row tile
        const int ti = rt + (duo ? hd * a.tpt1 : 0);
        const bool valid = rt < a.tpt1 && ti < sg.ntok;
        seen = !valid ? 0 : LIST ? sg.keys : max(0, sg.pos0 + ti + 1);
        busy = __any_sync(0xffffffffu, valid);
      }
      const bool none = sg.keys == 0;              // no row of the unit sees a key
      float m_used = -INFINITY, lsum = 0.f;
      bool started = false;
      for (; !none && t < te; t += duo ? 1 : 2) {
        if (!(ok = warp_wait(bars.sfull(hd), sc & 1, wc))) break;
        ++sc;
        tc_fence_after();
        if (busy) {
          const int limit = min(128, seen - 128 * t);
          uint32_t sr[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tmem + lane_off + s_col + 32u * q, sr[q]);
          tmem_ld_wait();
          if (limit < 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * q + e >= limit) sr[q][e] = 0xff800000u;
          }
          float mxv[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            mxv[u] = fmaxf(__uint_as_float(sr[0][2 * u]), __uint_as_float(sr[0][2 * u + 1]));
#pragma unroll
          for (int e = 16; e < 128; e += 2)
            mxv[(e >> 1) & 7] = max3(mxv[(e >> 1) & 7], __uint_as_float(sr[e >> 5][e & 31]),
                                     __uint_as_float(sr[e >> 5][(e & 31) + 1]));
          const float mx2 = max3(max3(mxv[0], mxv[1], mxv[2]), max3(mxv[3], mxv[4], mxv[5]),
                                 fmaxf(mxv[6], mxv[7])) * a.sl2;
          // the maximum in use may lag by up to 2^8 before O is rescaled
          const bool grow = mx2 > m_used + 8.0f;
          if (!started) {
            m_used = mx2;
          } else if (__any_sync(0xffffffffu, grow)) {
            // every PV of this slot issued before S_t has completed
            const float fac = grow ? fast_exp2(m_used - mx2) : 1.0f;
            if (grow) {
              lsum *= fac;
              m_used = mx2;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t ov[32];
              tmem_ld32(tmem + lane_off + o_col + 32u * q, ov);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * fac);
              tmem_st32(tmem + lane_off + o_col + 32u * q, ov);
            }
            tmem_st_wait();
          }
          started = true;
          const float neg_m = (m_used == -INFINITY) ? 0.f : -m_used;
          const uint64_t scale2 = pack_f32x2(a.sl2, a.sl2), neg2 = pack_f32x2(neg_m, neg_m);
          uint64_t ps[2] = {0ull, 0ull};
          auto exps = [&](uint32_t(&x)[32]) {        // packed into the first 16
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float p0, p1;
              unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                     scale2, neg2), p0, p1);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              ps[(e >> 1) & 1] = add_f32x2(ps[(e >> 1) & 1], pack_f32x2(p0, p1));
              x[e >> 1] = pack_bf16x2(p0, p1);
            }
          };
          exps(sr[0]);
          exps(sr[1]);
          tmem_st32_halves(tmem + lane_off + s_col, sr[0], sr[1]);
          tmem_st_wait();
          warp_arrive(bars.phalf(hd));               // PV over the first 64 keys may begin
          exps(sr[2]);
          exps(sr[3]);
          tmem_st32_halves(tmem + lane_off + s_col + 32u, sr[2], sr[3]);
          float l0, l1;
          unpack_f32x2(add_f32x2(ps[0], ps[1]), l0, l1);
          lsum += l0 + l1;
          tmem_st_wait();
        } else {
          warp_arrive(bars.phalf(hd));
        }
        warp_arrive(bars.pfull(hd));
      }
      if (!ok) break;
      // ----------------------------------------------------- segment's end
      const int use0 = oc[0], use1 = oc[1];
      if (!none) {
        kt += te - sg.tb;
        ++oc[0];
        if (duo || two) ++oc[1];
      }
      const bool whole = (flags & kSegWhole) != 0;
      const int rt = row / a.group, ti = rt + (duo ? hd * a.tpt1 : 0);
      const int tok0 = sg.tok0, ntok = sg.ntok, g0 = sg.g * a.group;
      const bool valid_row = rt < a.tpt1 && ti < ntok;
      const long long tok = static_cast<long long>(tok0) + ti;
      const int head = g0 + (row - rt * a.group);
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.wempty(i % kPagedSegs));
      if (none) {
        if (valid_row && (duo || hd == 0)) {
          uint4* dst = reinterpret_cast<uint4*>(a.o.at(0, tok, head));
          for (int k = 0; k < 16; ++k) dst[k] = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[tok * a.Hq + head] = -INFINITY;
        }
        continue;
      }
      // Warpgroup 1 waits for accumulator 0 too, and its arrival frees it with
      // warpgroup 0's: all loads of the segment have landed then, and it has not
      // skipped a phase of the barriers it waits on when rows are few.
      if (!duo && hd == 1) {
        if (two) {
          // hand (m, l) to warpgroup 0, which joins the two accumulators; it has
          // read the last pair once it has freed the second accumulator
          if (use1 > 0 && !(ok = warp_wait(bars.ofree(1), (use1 - 1) & 1, wc))) break;
          ml[row] = m_used;
          ml[128 + row] = lsum;
          warp_arrive(bars.xch());
          if (!(ok = warp_wait(bars.odone(1), use1 & 1, wc))) break;
        }
        if (!(ok = warp_wait(bars.odone(0), use0 & 1, wc))) break;
        warp_arrive(bars.ofree(0));
        continue;
      }
      if (two && !(ok = warp_wait(bars.xch(), xc++ & 1, wc))) break;
      if (!(ok = warp_wait(bars.odone(0), use0 & 1, wc))) break;
      if (hd == 1) {
        warp_arrive(bars.ofree(0));
        if (!(ok = warp_wait(bars.odone(1), use1 & 1, wc))) break;
      }
      if (two && !(ok = warp_wait(bars.odone(1), use1 & 1, wc))) break;
      tc_fence_after();
      float* part = a.part + (2LL * c + ((flags & kSegStart) ? 1 : 0)) * kPagedSlotFloats;
      const int prow = (duo ? hd * 128 : 0) + row;
      float fac0 = 1.f, fac1 = 0.f, m = m_used, l = lsum;
      if (two) {
        const float m1 = ml[row];
        m = fmaxf(m_used, m1);
        const float base = m == -INFINITY ? 0.f : m;
        fac0 = fast_exp2(m_used - base);
        fac1 = fast_exp2(m1 - base);
        l = lsum * fac0 + ml[128 + row] * fac1;
      }
      const float inv = whole ? (l > 0.f ? 1.0f / l : 0.f) : 1.f;
      fac0 *= inv;
      fac1 *= inv;
      if (busy) {
        // rows of this lane's four, when stored: null behind the last
        __nv_bfloat16* dst[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int rk = quad * 32 + (lane & ~3) + k, rkt = rk / a.group;
          const int tk = rkt + (duo ? hd * a.tpt1 : 0);
          dst[k] = rkt < a.tpt1 && tk < ntok
                       ? a.o.at(0, static_cast<long long>(tok0) + tk, g0 + (rk - rkt * a.group))
                       : nullptr;
        }
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t ov[32];
          tmem_ld32(tmem + lane_off + o_col + 32u * q, ov);
          tmem_ld_wait();
          // a row that sees no key has accumulated nothing but 0 * V
#pragma unroll
          for (int e = 0; e < 32; ++e)
            ov[e] = __float_as_uint(l > 0.f ? __uint_as_float(ov[e]) * fac0 : 0.f);
          if (two) {
            uint32_t ow[32];
            tmem_ld32(tmem + lane_off + 384u + 32u * q, ow);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              ov[e] = __float_as_uint(
                  l > 0.f ? fmaf(__uint_as_float(ow[e]), fac1, __uint_as_float(ov[e])) : 0.f);
          }
          if (!whole) {
            if (valid_row) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(part + ((8 * q + i) * kPagedSlotRows + prow) * 4) =
                    make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
            }
            continue;
          }
          // Four lanes exchange the 16-byte quarters of their rows' 64 bytes, so
          // that a store covers eight rows of 64 bytes instead of 32 of 16.
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t* y = ov + 8 * i;
            x[i] = make_uint4(pack_bf16x2(__uint_as_float(y[0]), __uint_as_float(y[1])),
                              pack_bf16x2(__uint_as_float(y[2]), __uint_as_float(y[3])),
                              pack_bf16x2(__uint_as_float(y[4]), __uint_as_float(y[5])),
                              pack_bf16x2(__uint_as_float(y[6]), __uint_as_float(y[7])));
          }
#pragma unroll
          for (int st = 1; st <= 2; ++st) {
            const bool up = (lane & st) != 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int lo = st == 1 ? 2 * k : k, hi = lo + st;
              uint4 z = up ? x[lo] : x[hi];
              z.x = __shfl_xor_sync(0xffffffffu, z.x, st);
              z.y = __shfl_xor_sync(0xffffffffu, z.y, st);
              z.z = __shfl_xor_sync(0xffffffffu, z.z, st);
              z.w = __shfl_xor_sync(0xffffffffu, z.w, st);
              if (up)
                x[lo] = z;
              else
                x[hi] = z;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (dst[k] != nullptr)
              *reinterpret_cast<uint4*>(dst[k] + 32 * q + 8 * (lane & 3)) = x[k];
        }
        if (valid_row) {
          if (whole) {
            if (a.lse)
              a.lse[tok * a.Hq + head] =
                  l > 0.f ? m * 0.69314718055994531f + logf(l) : -INFINITY;
          } else {
            part[128 * kPagedSlotRows + prow] = m;
            part[129 * kPagedSlotRows + prow] = l;
          }
        }
      }
      warp_arrive(bars.ofree(hd));
      if (two) warp_arrive(bars.ofree(1));
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the pieces of every unit that several CTAs share: blocks x look at the
// record of CTA x.  O = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.  A warp
// has four rows by 32 columns, a lane four columns of a row; the (m, l, O) of
// eight pieces are read side by side (a serial merge took 17 us for 8 pieces of
// one token).  Bound by the partials of 133 KB per slot, from L2: 24 us of the
// 1.04 ms of 2048 tokens at 32K, 5 to 7 us for single tokens.
constexpr int kCombineThreads = 256;
constexpr int kCombinePieces = 8;

__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedRecord rec = a.rec[blockIdx.x];
  if (rec.c1 < 0) return;
  const int c0 = blockIdx.x, np = rec.c1 - c0 + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = rec.ntok * a.group;
  const int items = (rows + 3) / 4 * 4;            // row quads x four column blocks
  for (int it = blockIdx.y * (kCombineThreads / 32) + warp; it < items;
       it += gridDim.y * (kCombineThreads / 32)) {
    const int i = (it >> 2) * 4 + (lane & 3);
    if (i >= rows) continue;
    const int c4 = 8 * (it & 3) + (lane >> 2);
    const int ti = i / a.group, hh = i - ti * a.group;
    const int tile = ti >= a.tpt1 ? 1 : 0;
    const int prow = tile * 128 + (ti - tile * a.tpt1) * a.group + hh;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < np; p0 += kCombinePieces) {
      float mp[kCombinePieces], lp[kCombinePieces];
      float4 x[kCombinePieces];
      float mn = m;
#pragma unroll
      for (int p = 0; p < kCombinePieces; ++p) {
        // slot of a piece: the first CTA's is its second
        const float* slot =
            a.part + (2LL * (c0 + p0 + p) + (p0 + p == 0 ? 1 : 0)) * kPagedSlotFloats;
        const bool on = p0 + p < np;
        mp[p] = on ? slot[128 * kPagedSlotRows + prow] : -INFINITY;
        lp[p] = on ? slot[129 * kPagedSlotRows + prow] : 0.f;
        x[p] = on ? *reinterpret_cast<const float4*>(slot + (c4 * kPagedSlotRows + prow) * 4)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int p = 0; p < kCombinePieces; ++p) mn = fmaxf(mn, mp[p]);
      if (mn == -INFINITY) continue;
      const float fo = exp2f(m - mn);
      l *= fo;
      acc.x *= fo;
      acc.y *= fo;
      acc.z *= fo;
      acc.w *= fo;
#pragma unroll
      for (int p = 0; p < kCombinePieces; ++p) {
        const float w = exp2f(mp[p] - mn);
        l = fmaf(lp[p], w, l);
        acc.x = fmaf(x[p].x, w, acc.x);
        acc.y = fmaf(x[p].y, w, acc.y);
        acc.z = fmaf(x[p].z, w, acc.z);
        acc.w = fmaf(x[p].w, w, acc.w);
      }
      m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const long long tok = static_cast<long long>(rec.tok0) + ti;
    const int head = rec.g * a.group + hh;
    uint2 y;
    y.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    y.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.o.at(0, tok, head) + 4 * c4) = y;
    if (a.lse && c4 == 0)
      a.lse[tok * a.Hq + head] = l > 0.f ? m * 0.69314718055994531f + logf(l) : -INFINITY;
  }
}

}  // namespace spa

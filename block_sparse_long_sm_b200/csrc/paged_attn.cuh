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
// found through the block table, one TMA box per page and 64 columns.
//
// Two ways through a segment, by the rows of its unit:
//   two row tiles   (more than 128 / group tokens)  A: the first 128 / group
//           tokens, B: the next; both read every key tile, softmax warpgroup
//           A / B works on its own rows;
//   one row tile    the warpgroups take the key tiles in turn (even ones A, odd
//           ones B), each with an accumulator of its own, and warpgroup A
//           joins the two at the end.  A single token is bound by the bytes of
//           K and V, and two independent chains of tiles hide the latency of
//           one another's softmax.
// Either way step j of a segment (a run of key tiles) uses score slot,
// accumulator and warpgroup j & 1, in the order
//   S_0, S_1, PV_0, S_2, PV_1, S_3, PV_2, ...
// so the tensor core has one product to do while the other slot's softmax runs.
// A step batch that mixes prompt chunks and single tokens has both.
//
// Work split.  All (sequence, kv head, row tiles) units lie end to end on one
// line, a key tile being one step long (two with two row tiles: twice the
// products), and each CTA (one per SM, persistent) takes an equal piece of
// that line, found by a scan over the sequences' lengths: every SM has the same
// work however ragged the batch is, one long sequence included.  A unit that one CTA covers is finished there; the pieces
// of the others (at most two per CTA) go to the workspace in fp32 and
// paged_combine_kernel joins them in the order of their CTAs, so that the
// result does not depend on timing.
//
// Rows of V past the last visible key of a tile (the unfilled end of a page,
// pages not loaded) are cleared in shared memory by a warp of their own: their
// probability is 0, but 0 * NaN is not.
//
// Roles (384 threads): warps 0-3 / 4-7 softmax of slot 0 / 1, warp 8 loads,
// warp 9 MMA and TMEM, warp 10 clears the ends of V tiles, warp 11 walks the
// CTA's piece and hands its segments to the others through a ring of four, so
// that the lengths and lists of the next units are read ahead.
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
};
static_assert(sizeof(PagedSeg) == 48, "ring entries");
constexpr int kPagedSegs = 4;
constexpr int kSegDuo = 1;      // two row tiles
constexpr int kSegStart = 2;    // holds the unit's first tile
constexpr int kSegWhole = 4;    // holds all of them

struct PagedAttnArgs {
  Seqs q;
  Rows o;
  float* lse;                // [T][Hq] or null
  const int32_t* lists;      // [T][Hkv][width] or null
  const int32_t* counts;     // [T][Hkv]
  int width;                 // list entries per (token, kv head)
  int wu;                    // key tiles of a full list
  int Hq, Hkv, group;
  int tpt1;                  // tokens per 128-row tile
  int pitch;                 // 128-element rows between pages
  float sl2;                 // softmax scale * log2(e)
  PagedRecord* rec;          // [G]
  float* part;               // [2 G] slots of kPagedSlotFloats
  uint64_t wait_ns;
  uint32_t debug;
};

// One partial slot: O [256 rows][128], m [256], l [256].
constexpr int kPagedSlotRows = 256;
constexpr long long kPagedSlotFloats = 130LL * kPagedSlotRows;

// The CTA whose piece [total * c / G, total * (c + 1) / G) holds point x.
__device__ __forceinline__ int piece_of(long long x, long long total, int G) {
  return static_cast<int>(((x + 1) * G - 1) / total);
}

// ---------------------------------------------------------------------------
// The units of a CTA's piece, in order.
// ---------------------------------------------------------------------------
template <bool LIST>
struct PagedWalk {
  const PagedAttnArgs& a;
  long long x0, x1;          // the CTA's piece of the line
  long long base;            // where the current unit starts on it
  int s, g, r;               // sequence (LIST: token row), kv head, row tile
  int q0, n, pos_first;      // of the sequence
  int nr;                    // its row tiles
  // the current unit
  int seq, tok0, ntok, pos0, keys, nt;
  int w, flat;               // length of one of its tiles on the line, of all

  __device__ __forceinline__ explicit PagedWalk(const PagedAttnArgs& args) : a(args) {}

  __device__ __forceinline__ static int tiles_of(int keys) { return keys > 0 ? (keys + 127) >> 7 : 1; }

  // keys that the last token of row tile r sees
  __device__ __forceinline__ static int tile_keys(int pos_first, int n, int tpt, int r) {
    return max(0, pos_first + min((r + 1) * tpt, n));
  }

  // Length on the line of one tile of a unit of `tokens` tokens.
  __device__ __forceinline__ static int tile_length(int tokens, int tpt1) {
    return tokens > tpt1 ? 2 : 1;
  }

  // Length on the line of sequence s, one kv head.
  __device__ __forceinline__ static long long head_length(const PagedAttnArgs& a, int s, bool& duo) {
    const Seq q = seq_at(a.q, s);
    const int tpt = 2 * a.tpt1;
    long long len = 0;
    for (int r = 0; r * tpt < q.n; ++r)
      len += tiles_of(tile_keys(q.kv - q.n, q.n, tpt, r)) * tile_length(q.n - r * tpt, a.tpt1);
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
      flat = a.wu;
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
      w = 1;
    } else {
      const int tpt = 2 * a.tpt1;
      tok0 = q0 + r * tpt;
      ntok = min(tpt, n - r * tpt);
      pos0 = pos_first + r * tpt;
      keys = tile_keys(pos_first, n, tpt, r);
      nt = tiles_of(keys);
      w = tile_length(ntok, a.tpt1);
      flat = nt * w;
    }
  }

  // Goes to the unit that holds x0.  s0, base0: the sequence that holds it and
  // where that starts (not LIST).
  __device__ __forceinline__ void start(int s0, long long base0) {
    if (LIST) {
      const long long u = x0 / a.wu;
      s = static_cast<int>(u / a.Hkv);
      g = static_cast<int>(u - static_cast<long long>(s) * a.Hkv);
      base = u * a.wu;
      r = 0;
      load_seq();
    } else {
      s = s0;
      base = base0;
      load_seq();
      bool duo;
      const long long per_head = head_length(a, s, duo);
      g = static_cast<int>((x0 - base0) / per_head);
      base += g * per_head;
      r = 0;
      while (true) {
        const int len = tiles_of(tile_keys(pos_first, n, 2 * a.tpt1, r)) *
                        tile_length(n - 2 * r * a.tpt1, a.tpt1);
        if (x0 < base + len || r + 1 >= nr) break;
        base += len;
        ++r;
      }
    }
    set_unit();
  }

  __device__ __forceinline__ bool more() const { return base < x1; }

  __device__ __forceinline__ void next() {
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
    b = static_cast<int>((max(x0 - base, 0LL) + w - 1) / w);
    e = static_cast<int>(min((x1 - base + w - 1) / w, static_cast<long long>(nt)));
    return b < e && ntok > 0;
  }
};

template <bool LIST>
__global__ void __launch_bounds__(kPagedThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PagedAttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t s_base = smem_u32(smem);
  auto s_q = [&](int i) { return s_base + i * kTileBytes; };
  auto s_k = [&](int st) { return s_base + (2u + st) * kTileBytes; };
  auto s_v = [&](int st) { return s_base + (2u + kPagedKStages + st) * kTileBytes; };
  uint8_t* ctl = smem + (2 + kPagedKStages + kPagedVStages) * kTileBytes;
  const uint32_t b0 = smem_u32(ctl);
  auto bar_kfull = [&](int s) { return b0 + 8u * s; };
  auto bar_kempty = [&](int s) { return b0 + 8u * (3 + s); };
  auto bar_vfull = [&](int s) { return b0 + 8u * (6 + s); };
  auto bar_vempty = [&](int s) { return b0 + 8u * (8 + s); };
  auto bar_vclean = [&](int s) { return b0 + 8u * (10 + s); };
  auto bar_sfull = [&](int h) { return b0 + 8u * (12 + h); };
  auto bar_pfull = [&](int h) { return b0 + 8u * (14 + h); };
  auto bar_odone = [&](int h) { return b0 + 8u * (16 + h); };
  auto bar_ofree = [&](int h) { return b0 + 8u * (18 + h); };
  auto bar_qfull = [&](int i) { return b0 + 8u * (20 + i); };
  auto bar_qfree = [&](int i) { return b0 + 8u * (22 + i); };
  auto bar_wfull = [&](int i) { return b0 + 8u * (24 + i); };
  auto bar_wempty = [&](int i) { return b0 + 8u * (28 + i); };
  const uint32_t bar_xch = b0 + 8u * 32, bar_drain = b0 + 8u * 33, bar_stall = b0 + 8u * 34;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ctl + 288);
  PagedSeg* segs = reinterpret_cast<PagedSeg*>(ctl + 320);
  volatile uint32_t* abort_flag = tmem_holder + 1;
  FindSmem& find = *reinterpret_cast<FindSmem*>(ctl + 512);
  static_assert(sizeof(FindSmem) <= 512, "search area");
  volatile float* ml = reinterpret_cast<volatile float*>(ctl + 1024);   // slot 1's m, l [128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the combine waits by itself
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPagedKStages; ++i) {
      mbar_init(bar_kfull(i), 1);
      mbar_init(bar_kempty(i), 1);
    }
    for (int i = 0; i < kPagedVStages; ++i) {
      mbar_init(bar_vfull(i), 1);
      mbar_init(bar_vempty(i), 1);
      mbar_init(bar_vclean(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_sfull(i), 1);
      mbar_init(bar_pfull(i), 128);
      mbar_init(bar_odone(i), 1);
      mbar_init(bar_ofree(i), 128);
      mbar_init(bar_qfull(i), 1);
      mbar_init(bar_qfree(i), 1);
    }
    for (int i = 0; i < kPagedSegs; ++i) {
      mbar_init(bar_wfull(i), 1);
      mbar_init(bar_wempty(i), 11);     // loads, MMA, clearing, eight softmax warps
    }
    mbar_init(bar_xch, 128);
    mbar_init(bar_drain, 1);
    mbar_init(bar_stall, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  // this CTA's piece of the line
  const int c = blockIdx.x;
  // pieces: none without a tile of a unit that spans it, so that every CTA
  // between the first and the last of a shared unit has a part of it
  bool any_duo = false;
  auto pieces = [&](long long total) {
    return static_cast<int>(
        min(static_cast<long long>(gridDim.x), max(total / (any_duo ? 2 : 1), 1LL)));
  };
  Found f{0, 0, 0, 0};
  if (LIST) {
    f.total = static_cast<long long>(a.q.T) * a.Hkv * a.wu;
  } else {
    bool duo = false;
    f = block_find(
        a.q.S,
        [&](int s) {
          bool d;
          const long long len = PagedWalk<LIST>::head_length(a, s, d) * a.Hkv;
          duo |= d;
          return len;
        },
        [&](long long total) {
          any_duo = __syncthreads_or(duo);
          return total * c / pieces(total);
        },
        find);
  }
  const int G = pieces(f.total);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const WaitCtx wc{abort_flag, a.q.err, a.wait_ns};
  // Segment i of the piece, copied out of the ring; false at its end.
  auto take = [&](int i, PagedSeg& sg) -> bool {
    const int r = i % kPagedSegs;
    if (!warp_wait(bar_wfull(r), (i / kPagedSegs) & 1, wc)) return false;
    sg = segs[r];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_wempty(r));
    return sg.te >= 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
    if (warp == 8) {
      // ----------------------------------------------------------- loads
      const int ppt = 128 >> a.q.shift;             // pages per tile
      const uint32_t page_half = 128u * a.q.page;   // bytes of a page's 64 columns
      int kt = 0, qu[2] = {0, 0}, qn = 0;           // key tiles, Q buffer uses, next buffer
      bool ok = true;
      PagedSeg sg;
      for (int i = 0; ok && take(i, sg); ++i) {
        if (sg.keys == 0) continue;
        // Q: both buffers for two row tiles, else the buffers in turn
        const bool duo = (sg.flags & kSegDuo) != 0;
        const int first = duo ? 0 : qn, tiles = duo ? 2 : 1;
        if (!duo) qn ^= 1;
        for (int q = 0; ok && q < tiles; ++q) {
          const int buf = first + q;
          if (qu[buf] > 0 && !(ok = warp_wait(bar_qfree(buf), (qu[buf] - 1) & 1, wc))) break;
          const int tok = sg.tok0 + q * a.tpt1;
          const int n = min(a.tpt1, sg.ntok - q * a.tpt1);
          if (lane == 0) mbar_arrive_expect_tx(bar_qfull(buf), n * a.group * 256u);
          __syncwarp();
          for (int k = lane; k < n; k += 32) {
            const uint32_t at = s_q(buf) + k * a.group * 128u;
            tma_load_3d(at, &tm_q, bar_qfull(buf), 0, sg.g * a.group, tok + k);
            tma_load_3d(at + kHalfBytes, &tm_q, bar_qfull(buf), 64, sg.g * a.group, tok + k);
          }
          ++qu[buf];
        }
        if (!ok) break;
        __syncwarp();
        // lane l < ppt: page l of the tile; its physical number is fetched one
        // tile ahead so that the table's latency overlaps the wait for a stage
        const int32_t* list = nullptr;
        int npages = (sg.keys + a.q.page - 1) >> a.q.shift;
        if (LIST) list = a.lists + (static_cast<long long>(sg.tok0) * a.Hkv + sg.g) * a.width;
        auto fetch = [&](int t) -> int {
          const int j = t * ppt + lane;
          if (lane >= ppt || j >= npages) return -1;
          int lp = j;
          if (LIST) {
            lp = list[j];
            const int before = j > 0 ? list[j - 1] : -1;
            if (lp <= before || lp < 0 || lp > (sg.pos0 >> a.q.shift)) {
              atomicOr(a.q.err, kErrBadIndex);
              lp = 0;
            }
          }
          const int p = phys_page(a.q, sg.seq, lp);
          return p < 0 ? 0 : p;                     // reported; any page will do
        };
        int ahead = fetch(sg.tb);
        for (int t = sg.tb; t < sg.te; ++t, ++kt) {
          const int phys = ahead;
          if (t + 1 < sg.te) ahead = fetch(t + 1);
          const uint32_t live = __popc(__ballot_sync(0xffffffffu, phys >= 0));
          const int row = phys * a.pitch + (sg.g << a.q.shift);
          const int ks = kt % kPagedKStages, vs = kt % kPagedVStages;
          const int ku = kt / kPagedKStages, vu = kt / kPagedVStages;
          if (ku > 0 && !(ok = warp_wait(bar_kempty(ks), (ku - 1) & 1, wc))) break;
          if (lane == 0) mbar_arrive_expect_tx(bar_kfull(ks), live * 2u * page_half);
          __syncwarp();
          if (phys >= 0) {
            const uint32_t at = s_k(ks) + lane * page_half;
            tma_load_2d(at, &tm_k, bar_kfull(ks), 0, row);
            tma_load_2d(at + kHalfBytes, &tm_k, bar_kfull(ks), 64, row);
          }
          __syncwarp();
          if (vu > 0 && !(ok = warp_wait(bar_vempty(vs), (vu - 1) & 1, wc))) {
            // K of this tile is in flight and counted: drain it below
            ++kt;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar_vfull(vs), live * 2u * page_half);
          __syncwarp();
          if (phys >= 0) {
            const uint32_t at = s_v(vs) + lane * page_half;
            tma_load_2d(at, &tm_v, bar_vfull(vs), 0, row);
            tma_load_2d(at + kHalfBytes, &tm_v, bar_vfull(vs), 64, row);
          }
          __syncwarp();
        }
      }
      // no copy may be in flight when the CTA gives its shared memory back
      // (immediate in normal operation, bounded after an abort)
      if (lane == 0) {
        for (int i = max(0, kt - kPagedKStages); i < kt; ++i)
          mbar_drain(bar_kfull(i % kPagedKStages), (i / kPagedKStages) & 1, a.wait_ns);
        for (int i = max(0, kt - kPagedVStages); i < kt; ++i)
          mbar_drain(bar_vfull(i % kPagedVStages), (i / kPagedVStages) & 1, a.wait_ns);
        for (int i = 0; i < 2; ++i)
          if (qu[i] > 0) mbar_drain(bar_qfull(i), (qu[i] - 1) & 1, a.wait_ns);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------- MMA issuer
      bool ok = true;
      if (a.debug & 1u) ok = warp_wait(bar_stall, 0, wc);   // never signalled: test hook
      int kt = 0, qn = 0, qu[2] = {0, 0}, pc[2] = {0, 0}, oc[2] = {0, 0};
      PagedSeg sg;
      for (int i = 0; ok && take(i, sg); ++i) {
        if (sg.keys == 0) continue;
        if (lane == 0) {
          const int duo = (sg.flags & kSegDuo) ? 1 : 0;
          const int tiles = sg.te - sg.tb, steps = tiles << duo;
          const int buf = qn;
          if (!duo) qn ^= 1;
          auto qk = [&](int j) -> bool {
            const int h = j & 1, k = kt + (j >> duo), st = k % kPagedKStages;
            const int qb = duo ? h : buf;
            if (j < 2 && (duo || j == 0)) {
              if (!mbar_wait(bar_qfull(qb), qu[qb] & 1, wc)) return false;
              ++qu[qb];
            }
            if (!mbar_wait(bar_kfull(st), (k / kPagedKStages) & 1, wc)) return false;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint32_t off = (ks >> 2) * kHalfBytes + (ks & 3) * 32u;
              mma_bf16_ss(tmem + 128u * h, smem_desc_sw128(s_q(qb) + off, 16),
                          smem_desc_sw128(s_k(st) + off, 16), kIdescQK, ks > 0 ? 1u : 0u);
            }
            mma_commit(bar_sfull(h));
            if (!duo || h == 1) mma_commit(bar_kempty(st));
            if (j + 1 + duo >= steps) mma_commit(bar_qfree(qb));
            return true;
          };
          auto pv = [&](int j) -> bool {
            const int h = j & 1, k = kt + (j >> duo), st = k % kPagedVStages;
            const bool first = j < 2;
            if (!mbar_wait(bar_pfull(h), pc[h] & 1, wc)) return false;
            ++pc[h];
            if (!mbar_wait(bar_vfull(st), (k / kPagedVStages) & 1, wc)) return false;
            if (!mbar_wait(bar_vclean(st), (k / kPagedVStages) & 1, wc)) return false;
            if (first) {
              // this accumulator of the segment before has been read
              if (oc[h] > 0 && !mbar_wait(bar_ofree(h), (oc[h] - 1) & 1, wc)) return false;
              ++oc[h];
            }
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              mma_bf16_ts(tmem + 256u + 128u * h, tmem + 128u * h + 8u * ks,
                          smem_desc_sw128(s_v(st) + ks * 2048u, kHalfBytes), kIdescPV,
                          (!first || ks > 0) ? 1u : 0u);
            }
            if (!duo || h == 1) mma_commit(bar_vempty(st));
            if (j + 2 >= steps) mma_commit(bar_odone(h));
            return true;
          };
          for (int j = 0; ok && j < 2 && j < steps; ++j) ok = qk(j);
          for (int j = 0; ok && j < steps; ++j) {
            ok = pv(j);
            if (ok && j + 2 < steps) ok = qk(j + 2);
          }
          kt += tiles;
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      }
      // every MMA issued by this thread has completed once this arrives
      if (lane == 0) {
        mma_commit(bar_drain);
        mbar_drain(bar_drain, 0, a.wait_ns);
      }
      __syncwarp();
    } else if (warp == 10) {
      // ------------------------------------- zeros behind the last V rows
      int kt = 0;
      bool ok = true;
      PagedSeg sg;
      for (int i = 0; ok && take(i, sg); ++i) {
        if (sg.keys == 0) continue;
        for (int t = sg.tb; t < sg.te; ++t, ++kt) {
          const int st = kt % kPagedVStages;
          if (!(ok = warp_wait(bar_vfull(st), (kt / kPagedVStages) & 1, wc))) break;
          const int valid = sg.keys - 128 * t;
          if (valid < 128) {
            // whole 128-byte rows, so the swizzle within a row does not matter
            uint8_t* tile = smem + (2 + kPagedKStages + st) * kTileBytes;
            for (int i = valid * 8 + lane; i < 128 * 8; i += 32) {
              reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
              reinterpret_cast<uint4*>(tile + kHalfBytes)[i] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_vclean(st));
        }
      }
    } else if (lane == 0) {
      // ----------------------------------------------- the CTA's segments
      PagedWalk<LIST> walk(a);
      walk.x0 = f.total * c / G;
      walk.x1 = f.total * (c + 1) / G;
      PagedRecord mine{-1, 0, 0, 0};
      int i = 0;
      bool ok = true;
      auto hand = [&](const PagedSeg& sg) {
        const int r = i % kPagedSegs;
        if (i >= kPagedSegs && !(ok = mbar_wait(bar_wempty(r), (i / kPagedSegs - 1) & 1, wc)))
          return;
        segs[r] = sg;
        mbar_arrive(bar_wfull(r));
        ++i;
      };
      if (c < G && walk.x0 < walk.x1 && f.s >= 0) {
        for (walk.start(f.s, f.base); ok && walk.more(); walk.next()) {
          int tb, te;
          if (!walk.range(tb, te)) continue;
          if (tb == 0 && te < walk.nt) {            // other CTAs go on with it
            mine.c1 = piece_of(walk.base + static_cast<long long>(walk.w) * (walk.nt - 1), f.total, G);
            mine.g = walk.g;
            mine.tok0 = walk.tok0;
            mine.ntok = walk.ntok;
          }
          const int flags = (walk.w == 2 ? kSegDuo : 0) | (tb == 0 ? kSegStart : 0) |
                            (tb == 0 && te == walk.nt ? kSegWhole : 0);
          hand(PagedSeg{tb, te, flags, walk.keys, walk.tok0, walk.ntok, walk.pos0, walk.g,
                        walk.seq, {0, 0, 0}});
        }
      }
      a.rec[c] = mine;
      if (ok) hand(PagedSeg{0, -1, 0, 0, 0, 0, 0, 0, 0, {0, 0, 0}});
    }
  } else {
    // ------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    const int hd = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = 128u * hd, o_col = 256u + 128u * hd;
    int sc = 0, oc[2] = {0, 0}, xc = 0;           // steps, accumulator uses, hand-overs
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!warp_wait(bar_wfull(i % kPagedSegs), (i / kPagedSegs) & 1, wc)) break;
      // The segment stays in the ring until its end and is read again there:
      // its fields would not fit beside a row of scores in the registers.
      const volatile PagedSeg& sg = segs[i % kPagedSegs];
      const int te = sg.te, flags = sg.flags;
      if (te < 0) break;
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
        if (!(ok = warp_wait(bar_sfull(hd), sc & 1, wc))) break;
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
          for (int u = 0; u < 8; ++u) mxv[u] = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e) mxv[e & 7] = fmaxf(mxv[e & 7], __uint_as_float(sr[q][e]));
          const float mx2 = fmaxf(fmaxf(fmaxf(mxv[0], mxv[1]), fmaxf(mxv[2], mxv[3])),
                                  fmaxf(fmaxf(mxv[4], mxv[5]), fmaxf(mxv[6], mxv[7]))) * a.sl2;
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
          float ps[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) ps[u] = 0.f;
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const int q = 2 * h2 + cc;
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float p0 = fast_exp2(fmaf(__uint_as_float(sr[q][e]), a.sl2, neg_m));
                const float p1 = fast_exp2(fmaf(__uint_as_float(sr[q][e + 1]), a.sl2, neg_m));
                ps[(e >> 1) & 7] += p0 + p1;
                sr[q][e >> 1] = pack_bf16x2(p0, p1);
              }
            }
            tmem_st32_halves(tmem + lane_off + s_col + 32u * h2, sr[2 * h2], sr[2 * h2 + 1]);
          }
          lsum += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(bar_pfull(hd));
      }
      if (!ok) break;
      // ----------------------------------------------------- segment's end
      const int use0 = oc[0], use1 = oc[1];
      if (!none) {
        ++oc[0];
        if (duo || two) ++oc[1];
      }
      const bool whole = (flags & kSegWhole) != 0;
      const int rt = row / a.group, ti = rt + (duo ? hd * a.tpt1 : 0);
      const bool valid_row = rt < a.tpt1 && ti < sg.ntok;
      const long long tok = static_cast<long long>(sg.tok0) + ti;
      const int head = sg.g * a.group + (row - rt * a.group);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_wempty(i % kPagedSegs));
      if (none) {
        if (valid_row && (duo || hd == 0)) {
          uint4* dst = reinterpret_cast<uint4*>(a.o.at(0, tok, head));
          for (int k = 0; k < 16; ++k) dst[k] = make_uint4(0, 0, 0, 0);
          if (a.lse) a.lse[tok * a.Hq + head] = -INFINITY;
        }
        continue;
      }
      if (!duo && hd == 1) {
        if (!two) continue;
        // hand (m, l) to warpgroup 0, which joins the two accumulators; it has
        // read the last pair once it has freed the second accumulator
        if (use1 > 0 && !(ok = warp_wait(bar_ofree(1), (use1 - 1) & 1, wc))) break;
        ml[row] = m_used;
        ml[128 + row] = lsum;
        mbar_arrive(bar_xch);
        if (!(ok = warp_wait(bar_odone(1), use1 & 1, wc))) break;
        continue;
      }
      if (two && !(ok = warp_wait(bar_xch, xc++ & 1, wc))) break;
      if (!(ok = warp_wait(bar_odone(hd), (hd ? use1 : use0) & 1, wc))) break;
      if (two && !(ok = warp_wait(bar_odone(1), use1 & 1, wc))) break;
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
          if (valid_row) {
            if (whole) {
              uint4* dst = reinterpret_cast<uint4*>(a.o.at(0, tok, head) + 32 * q);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t* x = ov + 8 * i;
                dst[i] = make_uint4(
                    pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                    pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                    pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                    pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7])));
              }
            } else {
              uint4* dst = reinterpret_cast<uint4*>(part + prow * 128 + 32 * q);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[i] = make_uint4(ov[4 * i], ov[4 * i + 1], ov[4 * i + 2], ov[4 * i + 3]);
            }
          }
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
      tc_fence_before();
      mbar_arrive(bar_ofree(hd));
      if (two) mbar_arrive(bar_ofree(1));
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// Joins the pieces of every unit that several CTAs share: blocks x look at the
// record of CTA x.  O = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c.  A warp
// per row: the lanes read the pieces' (m, l) side by side and turn them into
// weights, then each lane sums four columns over the pieces, all loads
// independent (a serial merge took 17 us for 8 pieces of one token).
constexpr int kCombineThreads = 256;

__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const PagedAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PagedRecord rec = a.rec[blockIdx.x];
  if (rec.c1 < 0) return;
  const int c0 = blockIdx.x, np = rec.c1 - c0 + 1;
  const int lane = threadIdx.x & 31;
  const int rows = rec.ntok * a.group;
  const int stride = gridDim.y * (kCombineThreads / 32);
  // slot of piece i: the first CTA's is its second
  auto slot = [&](int i) {
    return a.part + (2LL * (c0 + i) + (i == 0 ? 1 : 0)) * kPagedSlotFloats;
  };
  for (int i = blockIdx.y * (kCombineThreads / 32) + (threadIdx.x >> 5); i < rows; i += stride) {
    const int ti = i / a.group, hh = i - ti * a.group;
    const int tile = ti >= a.tpt1 ? 1 : 0;
    const int prow = tile * 128 + (ti - tile * a.tpt1) * a.group + hh;
    constexpr int kGroups = 5;                     // of 32 pieces: up to 160 CTAs
    float mw[kGroups], lw[kGroups], m = -INFINITY;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int p = 32 * k + lane;
      mw[k] = p < np ? slot(p)[128 * kPagedSlotRows + prow] : -INFINITY;
      lw[k] = p < np ? slot(p)[129 * kPagedSlotRows + prow] : 0.f;
      m = fmaxf(m, mw[k]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      mw[k] = mw[k] == -INFINITY ? 0.f : exp2f(mw[k] - m);
      l = fmaf(lw[k], mw[k], l);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      const int n = min(32, np - 32 * k);
#pragma unroll 8
      for (int p = 0; p < n; ++p) {
        const float wgt = __shfl_sync(0xffffffffu, mw[k], p);
        const float4 x =
            *reinterpret_cast<const float4*>(slot(32 * k + p) + prow * 128 + 4 * lane);
        acc.x = fmaf(x.x, wgt, acc.x);
        acc.y = fmaf(x.y, wgt, acc.y);
        acc.z = fmaf(x.z, wgt, acc.z);
        acc.w = fmaf(x.w, wgt, acc.w);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const long long tok = static_cast<long long>(rec.tok0) + ti;
    const int head = rec.g * a.group + hh;
    uint2 y;
    y.x = pack_bf16x2(acc.x * inv, acc.y * inv);
    y.y = pack_bf16x2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(a.o.at(0, tok, head) + 4 * lane) = y;
    if (a.lse && lane == 0)
      a.lse[tok * a.Hq + head] = l > 0.f ? m * 0.69314718055994531f + logf(l) : -INFINITY;
  }
}

}  // namespace spa

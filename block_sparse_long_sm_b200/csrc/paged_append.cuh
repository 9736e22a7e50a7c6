// paged_append.cuh -- new tokens' keys and values into the pages of a cache,
// normed and rotated on the way, with the per-page key minima and maxima that
// the page selection reads, and the same tokens' queries beside them.
//
// Work unit: the rows that one sequence adds to one of its pages, for one kv
// head -- contiguous in the cache, and all that the page's summary can depend
// on, so the summary needs no atomics and no second pass: the unit takes the
// minimum and maximum over the rows it writes and, when the page held rows
// before, over those as well.  (Updating the old summary instead would keep
// values of rows that were since overwritten, as after rejected draft tokens.)
// One block of 16 row slots (eight lanes each) per unit; the blocks behind the
// units take the queries, a warp per token and group of heads.
#pragma once

#include "paged_seqs.cuh"
#include "rope.cuh"

namespace spa {

struct AppendArgs {
  Seqs q;
  Rows xq, xk, xv, qo;
  const __nv_bfloat16 *qw, *kw;
  RopeSpec r;
  __nv_bfloat16 *kc, *vc, *summary;
  long long page_stride;
  int Hq, Hkv;
  long long kv_blocks;       // blocks of the k/v part
  int heads_per_warp, groups;
  long long q_warps;
};

constexpr int kAppendThreads = 128;
constexpr int kAppendSlots = kAppendThreads / kRowLanes;

// Pages that sequence s touches: 0 when it has no new tokens, or (reported)
// more new tokens than its length.
__device__ __forceinline__ int append_segments(const Seqs& v, int s) {
  const Seq q = seq_at(v, s);
  if (q.n == 0) return 0;
  if (q.n > q.kv) {
    atomicOr(v.err, kErrBadIndex);
    return 0;
  }
  return ((q.kv - 1) >> v.shift) - ((q.kv - q.n) >> v.shift) + 1;
}

// Five blocks per SM (96 registers, 8 bytes spilled): the 760 blocks of
// five ragged chunks, 7300 tokens of 8 kv heads, run in about one round, 14.0 us
// (3.4 TB/s; four blocks 19.7 us, six 17.7 us); one token each of 64 sequences
// takes 5.6 us.  Held off the memory's rate by the latency of a block's way, each
// step after the one before: lengths, table, its rows 16 at a time, the rows that
// the page held, summary.
__global__ void __launch_bounds__(kAppendThreads, 5) paged_append_kernel(const AppendArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the attention waits by itself
  const int lane = threadIdx.x & 31, li = lane & 7, warp = threadIdx.x >> 5;
  const Seqs& v = a.q;
  if (blockIdx.x >= a.kv_blocks) {
    // ------------------------------------------------------------- queries
    const long long w = (blockIdx.x - a.kv_blocks) * (kAppendThreads / 32) + warp;
    if (w >= a.q_warps) return;
    const int t = static_cast<int>(w / a.groups);
    int s;
    const Seq q = seq_of_token(v, t, s);
    const int pos = q.kv - q.n + (t - q.q0);
    if (q.n == 0 || q.n > q.kv) return;               // reported by the k/v part
    if (a.r.rot != 0 && pos >= a.r.rows) {
      if (lane == 0) atomicOr(v.err, kErrBadIndex);
      return;
    }
    const Angles ang = load_angles(a.r, pos, li);
    const NormWeights nw = load_weights(a.qw, li);
    const int h0 = static_cast<int>(w % a.groups) * a.heads_per_warp;
    const int h1 = min(h0 + a.heads_per_warp, a.Hq);
#pragma unroll 4
    for (int hb = h0; hb < h1; hb += 4) {
      const int h = hb + (lane >> 3);
      const bool on = h < h1;
      const __nv_bfloat16* src = a.xq.at(0, t, on ? h : h0);
      Row16 x;
      unpack8(*reinterpret_cast<const uint4*>(src + 8 * li), x.x);
      unpack8(*reinterpret_cast<const uint4*>(src + 64 + 8 * li), x.x + 8);
      norm_rotate(x, a.qw != nullptr, true, nw, a.r, ang, li);
      if (on) {
        __nv_bfloat16* dst = a.qo.at(0, t, h);
        *reinterpret_cast<uint4*>(dst + 8 * li) = pack8(x.x);
        *reinterpret_cast<uint4*>(dst + 64 + 8 * li) = pack8(x.x + 8);
      }
    }
    return;
  }

  // ------------------------------------------------------- keys and values
  __shared__ FindSmem find;
  __shared__ float red[kAppendThreads / 32][2][128];
  const long long unit = blockIdx.x / a.Hkv;
  const int g = static_cast<int>(blockIdx.x - unit * a.Hkv);
  // every warp finds the unit's sequence by itself when the sequences are few
  auto pages = [&](int s) { return static_cast<long long>(append_segments(v, s)); };
  auto place = [&](long long) { return unit; };
  const Found f = v.S <= 32 * kWarpFind ? warp_find(v.S, pages, place)
                                        : block_find(v.S, pages, place, find);
  if (f.s < 0) return;
  const Seq q = seq_at(v, f.s);
  const int pos0 = q.kv - q.n;                        // >= 0: it has segments
  const int j = (pos0 >> v.shift) + static_cast<int>(unit - f.base);
  const int lo = max(pos0, j << v.shift);             // positions of the new rows
  const int hi = min(q.kv, (j + 1) << v.shift);
  const int phys = phys_page(v, f.s, j);
  if (phys < 0) return;
  const int slot = threadIdx.x >> 3;
  const long long page0 = phys * a.page_stride + static_cast<long long>(g) * v.page * 128;
  __nv_bfloat16* kp = a.kc + page0;
  __nv_bfloat16* vp = a.vc + page0;
  float mn[16], mx[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    mn[i] = INFINITY;
    mx[i] = -INFINITY;
  }
  auto note = [&](const Row16& x) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      mn[i] = fminf(mn[i], x.x[i]);
      mx[i] = fmaxf(mx[i], x.x[i]);
    }
  };
  const NormWeights nw = load_weights(a.kw, li);
#pragma unroll 2
  for (int base = lo; base < hi; base += kAppendSlots) {
    const int pos = base + slot;
    const bool in = pos < hi;
    const bool on = in && (a.r.rot == 0 || pos < a.r.rows);
    if (in && !on && li == 0) atomicOr(v.err, kErrBadIndex);
    const long long t = static_cast<long long>(q.q0) + (on ? pos : lo) - pos0;
    const __nv_bfloat16* ks = a.xk.at(0, t, g);
    const __nv_bfloat16* vs = a.xv.at(0, t, g);
    Row16 x;
    unpack8(*reinterpret_cast<const uint4*>(ks + 8 * li), x.x);
    unpack8(*reinterpret_cast<const uint4*>(ks + 64 + 8 * li), x.x + 8);
    const uint4 v0 = *reinterpret_cast<const uint4*>(vs + 8 * li);
    const uint4 v1 = *reinterpret_cast<const uint4*>(vs + 64 + 8 * li);
    const Angles ang = load_angles(a.r, on ? pos : 0, li);
    norm_rotate(x, a.kw != nullptr, true, nw, a.r, ang, li);
    if (on) {
      const int r = pos & (v.page - 1);
      *reinterpret_cast<uint4*>(kp + r * 128 + 8 * li) = pack8(x.x);
      *reinterpret_cast<uint4*>(kp + r * 128 + 64 + 8 * li) = pack8(x.x + 8);
      *reinterpret_cast<uint4*>(vp + r * 128 + 8 * li) = v0;
      *reinterpret_cast<uint4*>(vp + r * 128 + 64 + 8 * li) = v1;
      note(x);                       // rounding is monotone: round the result once
    }
  }
  if (a.summary == nullptr) return;
  // rows the page held before
  const int old = lo - (j << v.shift);
#pragma unroll 4
  for (int r = slot; r < old; r += kAppendSlots) {
    Row16 x;
    unpack8(*reinterpret_cast<const uint4*>(kp + r * 128 + 8 * li), x.x);
    unpack8(*reinterpret_cast<const uint4*>(kp + r * 128 + 64 + 8 * li), x.x + 8);
    note(x);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      mn[i] = fminf(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], o));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
    }
  }
  if (lane < kRowLanes) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = (i < 8 ? 0 : 56) + 8 * li + i;
      red[warp][0][d] = mn[i];
      red[warp][1][d] = mx[i];
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    // lane: minima (0-15) or maxima (16-31) of dims 8 (lane % 16) ..
    const int which = lane >> 4, d0 = 8 * (lane & 15);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = red[0][which][d0 + i];
      for (int w = 1; w < kAppendThreads / 32; ++w) {
        const float z = red[w][which][d0 + i];
        y[i] = which ? fmaxf(y[i], z) : fminf(y[i], z);
      }
    }
    __nv_bfloat16* dst =
        a.summary + ((static_cast<long long>(phys) * a.Hkv + g) * 2 + which) * 128 + d0;
    *reinterpret_cast<uint4*>(dst) = pack8(y);
  }
}

}  // namespace spa

// rope.cuh -- RMS norm of every q and k head with the position rotation in the
// same pass (sparse_qk_norm_rope), and the same on the way into a paged cache
// (sparse_paged_append).
//
// A row is one head of one token: 128 bf16.  Eight lanes hold it, lane i the
// elements [8i, 8i+8) and [64+8i, 64+8i+8) -- two 16-byte loads, 128 contiguous
// bytes per load and row -- so that the two halves of a rotation over all 128
// dims (i, i + 64) meet in one lane.  A narrower rotation over r dims pairs
// lane i with lane i ^ (r / 16); interleaved pairs lie in one lane anyway.
// Everything is fp32 between the load and the one rounding at the store.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace spa {

constexpr int kRowLanes = 8;

struct Rows {
  __nv_bfloat16* p;
  long long sb, st, sh;
  __device__ __forceinline__ __nv_bfloat16* at(long long b, long long t, int h) const {
    return p + b * sb + t * st + static_cast<long long>(h) * sh;
  }
};

struct RopeSpec {
  const float* table;   // [rows][rot]: cosines, then sines
  int rot;              // rotated dims (0: none)
  int interleaved;
  int rows;
  float eps;
};

struct Row16 {
  float x[16];
};

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// The angles a lane needs: c[0..7], s[0..7] belong to its first eight elements
// (and, over 128 dims in halves, to the second eight as the other member of
// the same pairs).  Interleaved: c[0..3] for the first eight, c[4..7] for the
// second eight.
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load4(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}

__device__ __forceinline__ Angles load_angles(const RopeSpec& r, int pos, int li) {
  Angles a;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a.c[i] = 1.f;
    a.s[i] = 0.f;
  }
  if (r.rot == 0) return a;
  const int half = r.rot >> 1;
  const float* row = r.table + static_cast<long long>(pos) * r.rot;
  if (r.interleaved) {
    if (8 * li < r.rot) {                       // pairs 4 li .. 4 li + 3
      load4(row + 4 * li, a.c);
      load4(row + half + 4 * li, a.s);
    }
    if (r.rot == 128) {                         // pairs 32 + 4 li ..
      load4(row + 32 + 4 * li, a.c + 4);
      load4(row + half + 32 + 4 * li, a.s + 4);
    }
  } else if (8 * li < r.rot) {
    const int m = (8 * li) & (half - 1);        // half is a power of two
    load8(row + m, a.c);
    load8(row + half + m, a.s);
  }
  return a;
}

// The lane's sixteen weights of a row's norm, as they come (1 without).
struct NormWeights {
  uint4 lo, hi;
};
__device__ __forceinline__ NormWeights load_weights(const __nv_bfloat16* weight, int li) {
  NormWeights n;
  n.lo = n.hi = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  if (weight != nullptr) {
    n.lo = *reinterpret_cast<const uint4*>(weight + 8 * li);
    n.hi = *reinterpret_cast<const uint4*>(weight + 64 + 8 * li);
  }
  return n;
}

__device__ __forceinline__ void rotate_halves(Row16& v, const Angles& a) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float e = v.x[i], o = v.x[8 + i];
    v.x[i] = e * a.c[i] - o * a.s[i];
    v.x[8 + i] = o * a.c[i] + e * a.s[i];
  }
}

// Norm (of this row when `mine`; `any`, the same for the whole warp: of some
// row) and rotation of the row held by the eight lanes; every lane of the warp
// takes part (shuffles).  rsqrtf is off by at most 2 units in the last place of fp32.
template <bool HALVES = false>   // rotation of all 128 dims in halves, known beforehand
__device__ __forceinline__ void norm_rotate(Row16& v, bool any, bool mine, const NormWeights& n,
                                            const RopeSpec& r, const Angles& a, int li) {
  if (any) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(v.x[i], v.x[i], ss);
#pragma unroll
    for (int o = 1; o < kRowLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float f = mine ? rsqrtf(ss * (1.0f / 128.0f) + r.eps) : 1.0f;
    float w[8];
    unpack8(n.lo, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x[i] = v.x[i] * f * w[i];
    unpack8(n.hi, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v.x[8 + i] = v.x[8 + i] * f * w[i];
  }
  if (HALVES) {
    rotate_halves(v, a);
    return;
  }
  if (r.rot == 0) return;
  if (r.interleaved) {
    // lanes past rotary_dim hold c = 1, s = 0
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = v.x[2 * i], o = v.x[2 * i + 1];
      v.x[2 * i] = e * a.c[i] - o * a.s[i];
      v.x[2 * i + 1] = o * a.c[i] + e * a.s[i];
    }
  } else if (r.rot == 128) {
    rotate_halves(v, a);
  } else {
    const int hl = r.rot >> 4;                  // lanes per half
    const float sign = (li & hl) ? 1.f : -1.f;  // second half: + s * first
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, v.x[i], hl);
      if (8 * li < r.rot) v.x[i] = v.x[i] * a.c[i] + sign * o * a.s[i];
    }
  }
}

// ---------------------------------------------------------------------------
// sparse_qk_norm_rope
// ---------------------------------------------------------------------------
struct NormRopeArgs {
  Rows q, k, qo, ko;
  const __nv_bfloat16 *qw, *kw;
  const int32_t* positions;
  RopeSpec r;
  int L, hq, hk;            // hq / hk: 0 when that side is left out
  int heads_per_warp;       // multiple of 4
  int groups;               // warps per token
  long long warps;
  uint32_t* err;
};

constexpr int kRopeThreads = 256;

// One warp: one token, heads_per_warp of its heads, four at a time.  The angles
// are loaded once per warp (40 heads per warp instead of 20: 259 us instead of
// 274 on 65536 tokens of 40 heads), the weights with every row (from L1; kept in
// registers, in a loop per side, they cost more in loads under way than they
// save: 299 us).  The rows of a step are independent, so the loop is unrolled
// to keep several 16-byte loads per lane in flight, and four blocks per SM bound
// the registers (three: 271 us, five: 266 us).  The usual rotation, all 128 dims
// in halves, has a kernel of its own: 243 us, 5.65 TB/s, against 259.
template <bool HALVES>
__global__ void __launch_bounds__(kRopeThreads, 4) norm_rope_kernel(const NormRopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long w = (static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5;
  if (w >= a.warps) return;
  const int lane = threadIdx.x & 31, li = lane & 7, slot = lane >> 3;
  const long long tok = w / a.groups;
  const int h0 = static_cast<int>(w - tok * a.groups) * a.heads_per_warp;
  const long long b = tok / a.L, t = tok - b * a.L;
  const int pos = a.positions ? a.positions[tok] : static_cast<int>(t);
  if (a.r.rot != 0 && (pos < 0 || pos >= a.r.rows)) {
    if (lane == 0) atomicOr(a.err, kErrBadIndex);
    return;
  }
  const Angles ang = load_angles(a.r, pos, li);
  const int heads = a.hq + a.hk;
  const int h1 = min(h0 + a.heads_per_warp, heads);
#pragma unroll 4
  for (int hb = h0; hb < h1; hb += 4) {
    const int h = hb + slot;
    const bool on = h < h1;
    const int hh = on ? h : h0;
    const bool isq = hh < a.hq;
    const int hr = isq ? hh : hh - a.hq;
    const __nv_bfloat16* src = isq ? a.q.at(b, t, hr) : a.k.at(b, t, hr);
    Row16 v;
    unpack8(*reinterpret_cast<const uint4*>(src + 8 * li), v.x);
    unpack8(*reinterpret_cast<const uint4*>(src + 64 + 8 * li), v.x + 8);
    const __nv_bfloat16* weight = isq ? a.qw : a.kw;
    norm_rotate<HALVES>(v, a.qw != nullptr || a.kw != nullptr, weight != nullptr,
                load_weights(weight, li), a.r, ang, li);
    if (on) {
      __nv_bfloat16* dst = isq ? a.qo.at(b, t, hr) : a.ko.at(b, t, hr);
      *reinterpret_cast<uint4*>(dst + 8 * li) = pack8(v.x);
      *reinterpret_cast<uint4*>(dst + 64 + 8 * li) = pack8(v.x + 8);
    }
  }
}

}  // namespace spa

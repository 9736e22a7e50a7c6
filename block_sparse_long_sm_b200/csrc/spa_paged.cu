// spa_paged.cu -- the serving step around a paged key/value cache
// (include/spa.h): sparse_qk_norm_rope, sparse_paged_append,
// sparse_paged_select, sparse_paged_attn and their helpers.  Nothing here
// allocates device memory.
#include <climits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/spa.h"
#include "host.cuh"
#include "paged_append.cuh"
#include "paged_attn.cuh"
#include "paged_select.cuh"
#include "rope.cuh"

namespace {

using namespace spa;

// CTAs of the attention: one per SM of the chip's 148.
constexpr int kPagedGrid = 148;

bool rows_ok(const spa_rows* r) {
  return r && r->data && aligned16(r->data) && r->stride_batch % 8 == 0 &&
         r->stride_token % 8 == 0 && r->stride_head % 8 == 0;
}

Rows rows_of(const spa_rows* r) {
  Rows x{nullptr, 0, 0, 0};
  if (!r) return x;
  x.p = static_cast<__nv_bfloat16*>(const_cast<void*>(r->data));
  x.sb = r->stride_batch;
  x.st = r->stride_token;
  x.sh = r->stride_head;
  return x;
}

bool word_ok(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

spa_status validate_rope(const spa_rope_params* r) {
  if (!r) return SPA_ERR_INVALID;
  if (r->batch < 0 || r->tokens < 0 || r->heads_q < 1 || r->heads_kv < 1) return SPA_ERR_INVALID;
  if (r->head_dim != 128) return SPA_ERR_UNSUPPORTED;
  if (r->rotary_dim < 0 || r->rotary_dim > 128) return SPA_ERR_INVALID;
  if (r->rotary_dim != 0 && r->rotary_dim != 16 && r->rotary_dim != 32 && r->rotary_dim != 64 &&
      r->rotary_dim != 128)
    return SPA_ERR_UNSUPPORTED;
  if (r->interleaved != 0 && r->interleaved != 1) return SPA_ERR_INVALID;
  if (r->rotary_dim != 0 && r->table_rows < 1) return SPA_ERR_INVALID;
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps)) return SPA_ERR_INVALID;
  if (r->heads_q > 65535 || r->heads_kv > 65535) return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

spa_status validate_paged(const spa_paged_params* p) {
  if (!p) return SPA_ERR_INVALID;
  if (p->heads_q < 1 || p->heads_kv < 1 || p->heads_q % p->heads_kv != 0) return SPA_ERR_INVALID;
  if (p->head_dim != 128) return SPA_ERR_UNSUPPORTED;
  if (p->page_size < 1) return SPA_ERR_INVALID;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return SPA_ERR_UNSUPPORTED;
  if (p->num_pages < 1 || p->pages_per_seq < 1 || p->seqs < 0 || p->tokens < 0)
    return SPA_ERR_INVALID;
  const long long own = (long long)p->heads_kv * p->page_size * 128;
  if (p->page_stride < 0 || p->page_stride % 128 != 0 ||
      (p->page_stride != 0 && p->page_stride < own))
    return SPA_ERR_INVALID;
  if (!(p->softmax_scale >= 0.f) || !std::isfinite(p->softmax_scale)) return SPA_ERR_INVALID;
  if (p->sink_pages < 0 || p->local_pages < 1 || p->top_pages < 0) return SPA_ERR_INVALID;
  if (p->heads_q / p->heads_kv > 128 || p->heads_q > 65535) return SPA_ERR_UNSUPPORTED;
  const long long pitch = (p->page_stride ? p->page_stride : own) / 128;
  if (pitch * p->num_pages >= (1LL << 31)) return SPA_ERR_UNSUPPORTED;      // TMA row index
  if ((long long)p->pages_per_seq * p->page_size >= (1LL << 30)) return SPA_ERR_UNSUPPORTED;
  if ((long long)p->sink_pages + p->local_pages + p->top_pages >= (1LL << 30) / p->page_size)
    return SPA_ERR_UNSUPPORTED;
  if ((long long)p->tokens * p->heads_q >= (1LL << 31)) return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

int log2i(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

Seqs seqs_of(const spa_paged_params* p, const int32_t* cu_q, const int32_t* kv_lens,
             const int32_t* table, uint32_t* err) {
  Seqs v;
  v.cu_q = cu_q;
  v.kv_lens = kv_lens;
  v.table = table;
  v.S = p->seqs;
  v.T = p->tokens;
  v.per_seq = p->pages_per_seq;
  v.num_pages = p->num_pages;
  v.page = p->page_size;
  v.shift = log2i(p->page_size);
  v.err = err;
  return v;
}

RopeSpec rope_of(const spa_rope_params* r, const float* table) {
  RopeSpec s{nullptr, 0, 0, 0, 0.f};
  if (!r) return s;
  s.table = table;
  s.rot = r->rotary_dim;
  s.interleaved = r->interleaved;
  s.rows = r->table_rows;
  s.eps = r->eps;
  return s;
}

// Heads a warp takes of one token: a large batch's angles are loaded once per
// 40 heads, a small one is spread over more warps instead.
int heads_per_warp(long long tokens, int heads) {
  const long long quads = tokens * ((heads + 3) / 4);
  int per = 4;
  while (per < 40 && quads * 4 / per > 148LL * 32) per += 4;
  return per;
}

int pitch_rows(const spa_paged_params* p) {
  return p->page_stride ? (int)(p->page_stride / 128) : p->heads_kv * p->page_size;
}

struct PagedLayout {
  size_t rec = 0, part = 0, score = 0, total = 0;
};

// Workspace (byte offsets, each region 256-aligned): unit records, partial
// results of the attention (two slots of 256 rows per CTA), page scores.  The
// attention uses what lies before the scores.
PagedLayout paged_layout(const spa_paged_params* p) {
  PagedLayout lo;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes);
    return at;
  };
  lo.rec = take(kPagedGrid * sizeof(PagedRecord));
  lo.part = take((size_t)2 * kPagedGrid * kPagedSlotFloats * 4);
  lo.score = take((size_t)p->tokens * p->heads_kv * p->pages_per_seq * 8);
  lo.total = off;
  return lo;
}

spa_status paged_checks(const spa_paged_params* p, const spa_rows* q, const int32_t* cu_q,
                        const int32_t* kv_lens, const int32_t* table, const void* workspace,
                        size_t bytes, const uint32_t* err, bool scores) {
  spa_status st = validate_paged(p);
  if (st != SPA_OK) return st;
  if (!workspace || !aligned16(workspace) || !word_ok(err)) return SPA_ERR_INVALID;
  const PagedLayout lo = paged_layout(p);
  if (bytes < (scores ? lo.total : lo.score)) return SPA_ERR_WORKSPACE;
  if (p->tokens == 0 || p->seqs == 0) return SPA_OK;
  if (!rows_ok(q) || !word_ok(cu_q) || !word_ok(kv_lens) || !word_ok(table))
    return SPA_ERR_INVALID;
  return SPA_OK;
}

// Whether a token can have more candidate pages than the selection keeps.
bool ranks(const spa_paged_params* p) {
  return p->top_pages > 0 &&
         (long long)p->pages_per_seq - p->sink_pages - p->local_pages > p->top_pages;
}

// Launch that, with `early`, may begin before the stream's previous kernel has
// ended (2 us less between two kernels); the kernel itself waits for that one
// before it reads or writes memory.
template <typename... P, typename... A>
bool launch_after(bool early, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                  cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Shared memory that spreads `blocks` evenly over the SMs: more than a block's
// share when one more were to fit.  Blocks that begin as the kernel before
// leaves the SMs would crowd on the first ones that it leaves (ranking for 16
// tokens of 8 kv heads, 128 blocks: the whole selecting step 82 us, spread 74).
size_t spread_smem(long long blocks, size_t own) {
  const long long per_sm = (blocks + kPagedGrid - 1) / kPagedGrid;
  const size_t share = (size_t)(233472 / (per_sm + 1)) + 1024;
  return share > own ? share : own;
}
constexpr int kSpreadMax = 233472 / 2 + 1024;

template <bool LIST>
bool launch_paged(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                  const CUtensorMap& tk2, const CUtensorMap& tv2, const PagedAttnArgs& a,
                  int combine_y, cudaStream_t stream) {
  if (set_smem(paged_attn_kernel<LIST>, kPagedSmemBytes) != cudaSuccess) return false;
  if (!launch_after(true, paged_attn_kernel<LIST>, dim3(kPagedGrid), kPagedThreads, kPagedSmemBytes,
                    stream, tq, tk, tv, tk2, tv2, a))
    return false;
  if (a.whole_units) return true;
  return launch_after(true, paged_combine_kernel, dim3(kPagedGrid, combine_y), kCombineThreads, 0,
                      stream, a);
}

}  // namespace

extern "C" {

SPA_API spa_status sparse_qk_norm_rope(const spa_rope_params* r, const spa_rows* q,
                                       const spa_rows* k, const void* q_weight,
                                       const void* k_weight, const int32_t* positions,
                                       const float* table, const spa_rows* q_out,
                                       const spa_rows* k_out, uint32_t* error_word,
                                       cudaStream_t stream) {
  spa_status st = validate_rope(r);
  if (st != SPA_OK) return st;
  if (!word_ok(error_word)) return SPA_ERR_INVALID;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
    return SPA_ERR_INVALID;
  if ((long long)r->batch * r->tokens >= (1LL << 31)) return SPA_ERR_UNSUPPORTED;
  if (r->batch == 0 || r->tokens == 0 || (!q && !k)) return SPA_OK;
  if ((q && (!rows_ok(q) || !rows_ok(q_out))) || (k && (!rows_ok(k) || !rows_ok(k_out))))
    return SPA_ERR_INVALID;
  if (r->rotary_dim != 0 && (!table || !aligned16(table))) return SPA_ERR_INVALID;
  if (positions && !word_ok(positions)) return SPA_ERR_INVALID;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return SPA_ERR_INVALID;
  NormRopeArgs a;
  a.q = rows_of(q);
  a.k = rows_of(k);
  a.qo = rows_of(q_out);
  a.ko = rows_of(k_out);
  a.qw = static_cast<const __nv_bfloat16*>(q ? q_weight : nullptr);
  a.kw = static_cast<const __nv_bfloat16*>(k ? k_weight : nullptr);
  a.positions = positions;
  a.r = rope_of(r, table);
  a.L = r->tokens;
  a.hq = q ? r->heads_q : 0;
  a.hk = k ? r->heads_kv : 0;
  const long long tokens = (long long)r->batch * r->tokens;
  const int heads = a.hq + a.hk;
  a.heads_per_warp = heads_per_warp(tokens, heads);
  a.groups = (heads + a.heads_per_warp - 1) / a.heads_per_warp;
  a.warps = tokens * a.groups;
  a.err = error_word;
  const long long blocks = (a.warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > INT_MAX) return SPA_ERR_UNSUPPORTED;
  const bool ok = r->rotary_dim == 128 && !r->interleaved
                      ? launch_after(true, norm_rope_kernel<true>, dim3((unsigned)blocks),
                                     kRopeThreads, 0, stream, a)
                      : launch_after(true, norm_rope_kernel<false>, dim3((unsigned)blocks),
                                     kRopeThreads, 0, stream, a);
  return ok ? SPA_OK : SPA_ERR_CUDA;
}

SPA_API spa_status sparse_paged_append(const spa_paged_params* p, const spa_rope_params* r,
                                       const spa_rows* q, const spa_rows* k, const spa_rows* v,
                                       const void* q_weight, const void* k_weight,
                                       const float* table, const int32_t* cu_q,
                                       const int32_t* kv_lens, const int32_t* block_table,
                                       const spa_rows* q_out, void* k_cache, void* v_cache,
                                       void* summary, uint32_t* error_word, cudaStream_t stream) {
  spa_status st = validate_paged(p);
  if (st != SPA_OK) return st;
  if (r) {
    if ((st = validate_rope(r)) != SPA_OK) return st;
    if (r->batch != 1 || r->tokens != p->tokens || r->heads_q != p->heads_q ||
        r->heads_kv != p->heads_kv)
      return SPA_ERR_INVALID;
  }
  if (!word_ok(error_word)) return SPA_ERR_INVALID;
  if ((q == nullptr) != (q_out == nullptr)) return SPA_ERR_INVALID;
  if (p->tokens == 0 || p->seqs == 0) return SPA_OK;
  if (!rows_ok(k) || !rows_ok(v) || (q && (!rows_ok(q) || !rows_ok(q_out))))
    return SPA_ERR_INVALID;
  if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(summary) ||
      !word_ok(cu_q) || !word_ok(kv_lens) || !word_ok(block_table))
    return SPA_ERR_INVALID;
  if (r && r->rotary_dim != 0 && (!table || !aligned16(table))) return SPA_ERR_INVALID;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return SPA_ERR_INVALID;
  AppendArgs a;
  a.q = seqs_of(p, cu_q, kv_lens, block_table, error_word);
  a.xq = rows_of(q);
  a.xk = rows_of(k);
  a.xv = rows_of(v);
  a.qo = rows_of(q_out);
  a.qw = static_cast<const __nv_bfloat16*>(r ? q_weight : nullptr);
  a.kw = static_cast<const __nv_bfloat16*>(r ? k_weight : nullptr);
  a.r = rope_of(r, table);
  a.kc = static_cast<__nv_bfloat16*>(k_cache);
  a.vc = static_cast<__nv_bfloat16*>(v_cache);
  a.summary = static_cast<__nv_bfloat16*>(summary);
  a.page_stride = (long long)pitch_rows(p) * 128;
  a.Hq = p->heads_q;
  a.Hkv = p->heads_kv;
  // a sequence of n new tokens touches at most n pages, and at most n / page_size + 2
  long long units = (long long)p->tokens / p->page_size + 2LL * p->seqs;
  if (units > p->tokens) units = p->tokens;
  a.kv_blocks = units * p->heads_kv;
  a.heads_per_warp = heads_per_warp(p->tokens, p->heads_q);
  a.groups = (p->heads_q + a.heads_per_warp - 1) / a.heads_per_warp;
  a.q_warps = q ? (long long)p->tokens * a.groups : 0;
  const long long blocks =
      a.kv_blocks + (a.q_warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks > INT_MAX) return SPA_ERR_UNSUPPORTED;
  paged_append_kernel<<<(unsigned)blocks, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SPA_OK : SPA_ERR_CUDA;
}

SPA_API size_t sparse_paged_workspace_bytes(const spa_paged_params* p) {
  if (validate_paged(p) != SPA_OK) return 0;
  return paged_layout(p).total;
}

SPA_API size_t sparse_paged_attn_workspace_bytes(const spa_paged_params* p) {
  if (validate_paged(p) != SPA_OK) return 0;
  return paged_layout(p).score;
}

SPA_API spa_status sparse_paged_select(const spa_paged_params* p, const spa_rows* q,
                                       const void* summary, const int32_t* cu_q,
                                       const int32_t* kv_lens, const int32_t* block_table,
                                       int32_t* lists, int32_t* counts, void* workspace,
                                       size_t workspace_bytes, uint32_t* error_word,
                                       cudaStream_t stream) {
  spa_status st = paged_checks(p, q, cu_q, kv_lens, block_table, workspace, workspace_bytes,
                               error_word, p && ranks(p));
  if (st != SPA_OK) return st;
  if (p->tokens == 0 || p->seqs == 0) return SPA_OK;
  if (!summary || !aligned16(summary) || !word_ok(lists) || !word_ok(counts))
    return SPA_ERR_INVALID;
  SelectArgs a;
  a.q = seqs_of(p, cu_q, kv_lens, block_table, error_word);
  a.xq = rows_of(q);
  a.summary = static_cast<const __nv_bfloat16*>(summary);
  a.score = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + paged_layout(p).score);
  a.lists = lists;
  a.counts = counts;
  a.Hkv = p->heads_kv;
  a.group = p->heads_q / p->heads_kv;
  a.sink = p->sink_pages;
  a.local = p->local_pages;
  a.top = p->top_pages;
  a.width = a.sink + a.local + a.top;
  // tokens beside one another share a block's loads when they can be of one sequence
  a.tm = a.group <= 16 && p->tokens > p->seqs ? 16 / a.group : 1;
  const long long most = (long long)p->pages_per_seq - a.sink - a.local;   // candidates
  const long long tg = (long long)p->tokens * p->heads_kv;
  if (tg > INT_MAX) return SPA_ERR_UNSUPPORTED;
  const bool scored = ranks(p);
  if (scored) {
    const long long groups = ((long long)p->tokens + a.tm - 1) / a.tm * p->heads_kv;
    a.chunks = (int)((most + kScorePages - 1) / kScorePages);
    const long long blocks = groups * a.chunks;
    if (blocks > INT_MAX) return SPA_ERR_UNSUPPORTED;
    page_score_kernel<<<(unsigned)blocks, kScoreThreads, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return SPA_ERR_CUDA;
  }
  // (begins while the scores are computed: it reads the lengths meanwhile)
  bool ok;
  if (most > kTopWarpKeys || tg < kTopWarpSelections) {
    static_assert(top_smem_bytes(INT_MAX) <= kSpreadMax, "one limit for both");
    if (set_smem(page_top_kernel, kSpreadMax) != cudaSuccess) return SPA_ERR_CUDA;
    ok = launch_after(scored, page_top_kernel, dim3((unsigned)tg), kTopThreads,
                      spread_smem(tg, top_smem_bytes(p->pages_per_seq)), stream, a);
  } else {
    constexpr int warps = kTopWarpThreads / 32;
    const long long blocks = (tg + warps - 1) / warps;
    if (set_smem(page_top_warp_kernel, kSpreadMax) != cudaSuccess) return SPA_ERR_CUDA;
    ok = launch_after(scored, page_top_warp_kernel, dim3((unsigned)blocks), kTopWarpThreads,
                      spread_smem(blocks, warps * sizeof(TopWarpSmem)), stream, a);
  }
  return ok ? SPA_OK : SPA_ERR_CUDA;
}

SPA_API spa_status sparse_paged_attn(const spa_paged_params* p, const spa_rows* q,
                                     const void* k_cache, const void* v_cache,
                                     const int32_t* cu_q, const int32_t* kv_lens,
                                     const int32_t* block_table, const int32_t* lists,
                                     const int32_t* counts, const spa_rows* o, float* lse,
                                     void* workspace, size_t workspace_bytes,
                                     uint32_t* error_word, cudaStream_t stream) {
  spa_status st = paged_checks(p, q, cu_q, kv_lens, block_table, workspace, workspace_bytes,
                               error_word, false);
  if (st != SPA_OK) return st;
  if ((lists == nullptr) != (counts == nullptr)) return SPA_ERR_INVALID;
  if (p->tokens == 0 || p->seqs == 0) return SPA_OK;
  if (!rows_ok(o) || !k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache))
    return SPA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(lists) & 3u) || (reinterpret_cast<uintptr_t>(counts) & 3u) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return SPA_ERR_INVALID;
  // The q tensor map wants positive strides, the larger a multiple of the
  // smaller.  Tokens further apart than heads: boxes of whole tokens; the other
  // way round (head-major rows): row by row.
  long long sh = q->stride_head, st_q = q->stride_token;
  if (p->heads_q == 1) sh = p->tokens == 1 ? 128 : st_q;
  if (p->tokens == 1) st_q = sh;
  if (sh <= 0 || st_q <= 0 || sh >= (1LL << 38) || st_q >= (1LL << 38)) return SPA_ERR_UNSUPPORTED;
  const bool by_rows = st_q < sh;
  if ((by_rows ? sh % st_q : st_q % sh) != 0) return SPA_ERR_UNSUPPORTED;
  const int group = p->heads_q / p->heads_kv;
  PagedAttnArgs a;
  a.q = seqs_of(p, cu_q, kv_lens, block_table, error_word);
  a.xq = rows_of(q);
  a.o = rows_of(o);
  a.lse = lse;
  a.lists = lists;
  a.counts = counts;
  a.width = p->sink_pages + p->local_pages + p->top_pages;
  a.unit_length = (group <= kFewRows ? kEdgeFew : kEdgeRows) +
                  kTileOne * (int)(((long long)a.width * p->page_size + 127) / 128);
  // Eight or more units per CTA: whole ones in turn (the last round costs at
  // most an eighth, and nothing is left to join).
  a.whole_units = lists && (long long)p->tokens * p->heads_kv >= 8LL * kPagedGrid;
  a.q_by_rows = by_rows;
  a.Hq = p->heads_q;
  a.Hkv = p->heads_kv;
  a.group = group;
  a.tpt1 = 128 / group;
  a.pitch = pitch_rows(p);
  a.sl2 = (p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt(128.0f)) *
          1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const PagedLayout lo = paged_layout(p);
  a.rec = reinterpret_cast<PagedRecord*>(ws + lo.rec);
  a.part = reinterpret_cast<float*>(ws + lo.part);
  a.wait_ns = (uint64_t)(p->wait_limit_us ? p->wait_limit_us : 250000u) * 1000ull;
  a.debug = p->debug_flags;
  const uint64_t cache_rows =
      (uint64_t)a.pitch * (p->num_pages - 1) + (uint64_t)p->heads_kv * p->page_size;
  CUtensorMap tq, tk, tv, tk2 = {}, tv2 = {};
  const bool q_map =
      by_rows ? map_rows(&tq, q->data, p->tokens, p->heads_q, st_q, sh, 1, 1)
              : map_rows(&tq, q->data, p->heads_q, p->tokens, sh, st_q, group, a.tpt1);
  if (!q_map ||
      !map_2d(&tk, kBF16, 2, k_cache, 128, cache_rows, 64, p->page_size, kSW128) ||
      !map_2d(&tv, kBF16, 2, v_cache, 128, cache_rows, 64, p->page_size, kSW128))
    return SPA_ERR_CUDA;
  a.whole_rows = p->page_size <= (lists ? kWholeRowListPages : kWholeRowPages);
  if (a.whole_rows &&
      (!map_rows(&tk2, k_cache, 2, cache_rows, 64, 128, 2, p->page_size, 64) ||
       !map_rows(&tv2, v_cache, 2, cache_rows, 64, 128, 2, p->page_size, 64)))
    return SPA_ERR_CUDA;
  // combine blocks beside one another: a warp per row of a usual unit (four
  // rows by a quarter of the columns)
  long long rows = lists ? group : (long long)p->tokens * group / p->seqs;
  if (rows > kPagedSlotRows) rows = kPagedSlotRows;
  const int cy = rows > 16 ? (int)(rows + 15) / 16 : 1;
  const bool ok = lists ? launch_paged<true>(tq, tk, tv, tk2, tv2, a, cy, stream)
                        : launch_paged<false>(tq, tk, tv, tk2, tv2, a, cy, stream);
  return ok ? SPA_OK : SPA_ERR_CUDA;
}

SPA_API spa_status sparse_paged_status(uint32_t* error_word, cudaStream_t stream) {
  if (!word_ok(error_word)) return SPA_ERR_INVALID;
  uint32_t bits = 0;
  if (cudaMemcpyAsync(&bits, error_word, 4, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaMemsetAsync(error_word, 0, 4, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return SPA_ERR_CUDA;
  if (bits & kErrTimeout) return SPA_ERR_TIMEOUT;
  if (bits & kErrBadIndex) return SPA_ERR_INVALID;
  return SPA_OK;
}

}  // extern "C"

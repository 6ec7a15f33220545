// C ABI of the paged cache (declared and documented in cache.h): argument
// validation, the choice of a variant and the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "launch.h"

namespace attn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status_t check_step(const attn_cache_problem_t* p) {
  if (!p) return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs <= 0 || p->tokens < 0 || p->heads_q <= 0 || p->heads_kv <= 0 ||
      p->head_dim <= 0 || p->num_pages <= 0 || p->max_pages <= 0 || p->max_new < 0)
    return ATTN_ERR_INVALID_ARG;
  if (p->tokens > 0 && p->max_new == 0) return ATTN_ERR_INVALID_ARG;
  if (p->heads_q % p->heads_kv) return ATTN_ERR_INVALID_ARG;
  if (p->cache_type != ATTN_CACHE_BF16 && p->cache_type != ATTN_CACHE_E4M3)
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(p->scale)) return ATTN_ERR_INVALID_ARG;
  if (!p->cu_seqlens || !p->seqlens_kv || !p->page_table) return ATTN_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
    return ATTN_ERR_UNSUPPORTED;
  const int64_t lim = int64_t(1) << 31;
  if (p->heads_q > 65535 || static_cast<int64_t>(p->tokens) * p->heads_q >= lim ||
      static_cast<int64_t>(p->num_pages) * p->heads_kv >= lim / p->page_size)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(p->cu_seqlens, 4) || !aligned(p->seqlens_kv, 4) || !aligned(p->page_table, 4) ||
      !aligned(p->error_word, 4))
    return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

// A token stride: 0 stands for dense rows.
bool good_stride(int64_t stride, int heads, int dim, int64_t* out) {
  const int64_t dense = static_cast<int64_t>(heads) * dim;
  *out = stride == 0 ? dense : stride;
  return *out >= dense && *out % 8 == 0;
}

CacheStep to_step(const attn_cache_problem_t* p) {
  CacheStep s;
  s.num_seqs = p->num_seqs;
  s.tokens = p->tokens;
  s.heads_q = p->heads_q;
  s.heads_kv = p->heads_kv;
  s.group = p->heads_q / p->heads_kv;
  s.ps_shift = p->page_size == 16 ? 4 : p->page_size == 32 ? 5 : p->page_size == 64 ? 6 : 7;
  s.num_pages = p->num_pages;
  s.max_pages = p->max_pages;
  s.max_new = p->max_new;
  s.cu = p->cu_seqlens;
  s.kv_len = p->seqlens_kv;
  s.table = p->page_table;
  s.err = p->error_word;
  return s;
}

// Query rows that one KV head has in the longest sequence of the step.
int step_rows(const attn_cache_problem_t* p) {
  const int64_t r = static_cast<int64_t>(p->max_new) * (p->heads_q / p->heads_kv);
  return static_cast<int>(r < 1 << 30 ? r : 1 << 30);
}

// Which kernels serve a step.  The one for few rows goes over the keys once for
// every 16 rows of a KV head (8 where no sequence has more), the tcgen05 kernel
// once for 256, but pays more for an item, above all with e4m3 keys.  Measured, few
// rows / tcgen05, in us, with 8 KV heads of 128 where nothing else is said:
//  - 32 sequences of 4096 keys, all with the same rows: bf16 101 / 115 at 16 rows, 179 / 116
//    at 20 (heads of 64: 58 / 75 and 103 / 75); e4m3 81 / 148 at 16, 143 / 150 at 32,
//    203 / 150 at 40;
//  - bf16, drafts of 1 to 5 tokens, group 4 (20 rows at most), by the rows on average: 64
//    sequences of up to 8192 keys 80 / 89 at 10, 81 / 90 at 11, 93 / 90 at 12, 91 / 90 at
//    14; 16 of up to 16000 56 / 57 at 8, 63 / 57 at 10; heads of 64, the first batch 48 / 72
//    at 10, 57 / 72 at 16, 68 / 73 at 18, 74 / 73 at 20, the second 37 / 43, 44 / 43, 45 / 43
//    and 49 / 43.  One sequence of 64 rows among them: 85 / 91 and 68 / 57 at 8;
//  - e4m3, 64 of up to 8192 keys with 64 rows at most: 109 / 156 at 24, 135 / 153 at 32,
//    137 / 161 at 36; with 128 at most 93 / 149 at 10 and 143 / 156 at 32; with 160 at most
//    101 / 148 and 152 / 155, but for 16 of up to 16000 115 / 82 at 32 with 128 at most.
// A batch of decoding sequences with a prompt's chunk among them: both kernels, each
// for its own sequences, cost two launches more.  Both / tcgen05 alone, e4m3, sequences
// of up to 2000 and of up to 8192 keys with a chunk of 128 | 512 tokens: 8 sequences 38 / 27
// and 45 / 42 | 48 / 37 and 59 / 58; 16: 39 / 35 and 50 / 58 | 48 / 48 and 62 / 78; 20: 42 / 42
// and 61 / 73 | 60 / 56 and 93 / 94; 24, the first where both won everywhere: 40 / 48 and
// 59 / 71 | 51 / 62 and 76 / 96; 64: 50 / 83 and 81 / 154 | 61 / 107 and 92 / 159.  bf16, 64:
// 51 / 55 and 88 / 93 | 61 / 61 and 98 / 101: the tcgen05 kernel alone.
// The averages are over `tokens`, padding included: the lists of lengths are the device's.
struct Kernels {
  bool few, tc;
  int split;       // rows above which a sequence is the tcgen05 kernel's
  int few_rows;    // rows of an item of the other
};
Kernels pick_kernels(const attn_cache_problem_t* p) {
  const int group = p->heads_q / p->heads_kv, rows = step_rows(p);
  const bool e4m3 = p->cache_type == ATTN_CACHE_E4M3;
  const int64_t average = static_cast<int64_t>(p->tokens) * group / p->num_seqs;
  const Kernels few = {true, false, 0x7fffffff, cache_fwd_rows(rows)};
  if (rows <= (e4m3 ? 32 : 16) || group > kCacheTcTile) return few;
  if (rows <= (e4m3 ? 128 : 32) && average <= (e4m3 ? 32 : p->head_dim == 64 ? 16 : 10)) return few;
  if (e4m3 && p->num_seqs >= 24 && group <= 16 &&
      p->tokens < static_cast<int64_t>(p->num_seqs) * p->max_new)
    return {true, true, 16, cache_fwd_rows(group)};
  return {false, true, 0, 0};
}

struct Workspace {
  size_t o, stash, ml, meta, bytes;
};
// The workspace of one kernel, from `at` on.
Workspace kernel_workspace(size_t at, int item_rows, int head_dim, bool tc, bool e4m3) {
  const size_t rows = 2 * static_cast<size_t>(kCacheCtas) * item_rows;
  Workspace w;
  w.o = at;
  w.stash = w.o + rows * head_dim * sizeof(float);
  w.ml = w.stash + (tc ? 0 : static_cast<size_t>(kCacheCtas) * cache_warps(e4m3, item_rows) * item_rows * head_dim * sizeof(float));
  w.meta = w.ml + rows * sizeof(float2);
  w.bytes = w.meta + 2 * kCacheCtas * sizeof(int4);
  return w;
}
size_t fwd_workspace(const attn_cache_problem_t* p, const Kernels& k) {
  const bool e4m3 = p->cache_type == ATTN_CACHE_E4M3;
  size_t n = 0;
  if (k.few) n = kernel_workspace(n, k.few_rows, p->head_dim, false, e4m3).bytes;
  if (k.tc) n = kernel_workspace(n, kCacheTcRows, p->head_dim, true, e4m3).bytes;
  return n;
}

attn_status_t status_of(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

attn_status_t attn_cache_append(const attn_cache_problem_t* p, const void* q, const void* k,
                                const void* v, const float* cos_sin, void* q_out, void* k_cache,
                                void* v_cache, float* k_scale, float* v_scale,
                                attn_stream_t stream) {
  const attn_status_t st = check_step(p);
  if (st != ATTN_OK) return st;
  const bool e4m3 = p->cache_type == ATTN_CACHE_E4M3;
  if (!k_cache || !v_cache || (e4m3 && (!k_scale || !v_scale))) return ATTN_ERR_INVALID_ARG;
  if (p->tokens > 0 && (!k || !v || (q == nullptr) != (q_out == nullptr))) return ATTN_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > p->head_dim || p->rot_dim % 16 ||
      (p->rot_dim > 0 && (!cos_sin || p->max_position <= 0)))
    return ATTN_ERR_INVALID_ARG;
  AppendArgs a;
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &a.q_stride) ||
      !good_stride(p->k_stride, p->heads_kv, p->head_dim, &a.k_stride) ||
      !good_stride(p->v_stride, p->heads_kv, p->head_dim, &a.v_stride))
    return ATTN_ERR_INVALID_ARG;
  if (q && q == q_out && a.q_stride != static_cast<int64_t>(p->heads_q) * p->head_dim)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(cos_sin, 16) ||
      !aligned(q_out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return ATTN_ERR_ALIGNMENT;
  if (p->tokens == 0) return ATTN_OK;

  a.s = to_step(p);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.cos_sin = cos_sin;
  a.rot_dim = p->rot_dim;
  a.interleaved = p->rot_interleaved ? 1 : 0;
  a.max_position = p->max_position;
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  // e4m3: pages that a sequence's new tokens can touch, and over all sequences
  const int64_t slots = (static_cast<int64_t>(p->max_new) - 1 + p->page_size - 1) / p->page_size + 1;
  const bool small = p->max_new <= kAppendSmall;
  int64_t items = slots * p->num_seqs;
  if (!small) {
    const int64_t packed = p->tokens / p->page_size + 2 * static_cast<int64_t>(p->num_seqs);
    if (packed < items) items = packed;
  }
  const int64_t units = items * 2 * p->heads_kv;
  // slots == 0: as many units (up to 8) go to one thread as leaves a block for every SM.
  // One, this rule, always eight: 89, 75, 75 us for four prompts, 46, 29, 29 us for 256
  // sequences with 12 new tokens, 11, 8.2, 11 us for 64, and 3.3, 3.3, 9.3 us for one.
  const int wide = append_units(p->head_dim, p->page_size);
  a.loop = 8;
  while (a.loop > 1 && units / (wide * a.loop) < 152) a.loop /= 2;
  a.head_blocks = (2 * p->heads_kv + wide * a.loop - 1) / (wide * a.loop);
  const int64_t unit_blocks = !e4m3 ? 0 : small ? (units + 7) / 8 : items * a.head_blocks;
  // Rows: blocks of tokens for groups of heads, as large (up to 8) as leaves two
  // blocks for every SM.  One head, this rule, always eight: 94, 75, 75 us for four
  // prompts, 2.7, 2.7, 4.3 us for one token, 6.5, 4.7, 6.2 us for 512 sequences' tokens.
  const int per = append_row_tokens(p->head_dim);
  a.row_blocks = (p->tokens + per - 1) / per;
  const int64_t heads = (q ? p->heads_q : 0) + (e4m3 ? 0 : 2 * p->heads_kv);
  a.hb = 8;
  while (a.hb > 1 && a.row_blocks * heads / a.hb < 304) a.hb /= 2;
  a.q_groups = q ? (p->heads_q + a.hb - 1) / a.hb : 0;
  a.kv_groups = e4m3 ? 0 : (p->heads_kv + a.hb - 1) / a.hb;
  const int64_t row_blocks = static_cast<int64_t>(a.row_blocks) * (a.q_groups + 2 * a.kv_groups);
  if (units >= (int64_t(1) << 30) || unit_blocks + row_blocks >= (int64_t(1) << 31))
    return ATTN_ERR_UNSUPPORTED;
  a.units = static_cast<int>(units);
  a.unit_blocks = static_cast<int>(unit_blocks);
  a.slots = small ? static_cast<int>(slots) : 0;
  a.fd_slots = make_fastdiv(static_cast<uint32_t>(a.slots > 0 ? a.slots : 1));
  return status_of(launch_cache_append(a, p->head_dim, e4m3, p->page_size,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

size_t attn_cache_fwd_workspace_size(const attn_cache_problem_t* p) {
  if (check_step(p) != ATTN_OK) return 0;
  return fwd_workspace(p, pick_kernels(p));
}

attn_status_t attn_cache_fwd(const attn_cache_problem_t* p, const void* q, const void* k_cache,
                             const void* v_cache, const float* k_scale, const float* v_scale,
                             void* o, float* lse, void* workspace, size_t workspace_bytes,
                             attn_stream_t stream) {
  const attn_status_t st = check_step(p);
  if (st != ATTN_OK) return st;
  const bool e4m3 = p->cache_type == ATTN_CACHE_E4M3;
  if (!k_cache || !v_cache || (e4m3 && (!k_scale || !v_scale))) return ATTN_ERR_INVALID_ARG;
  if (p->tokens > 0 && (!q || !o || !lse)) return ATTN_ERR_INVALID_ARG;
  CacheFwdArgs both[2];   // of the kernel for few rows, of the tcgen05 kernel
  CacheFwdArgs& base = both[0];
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &base.q_stride)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) ||
      !aligned(lse, 16) || !aligned(workspace, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return ATTN_ERR_ALIGNMENT;
  if (p->tokens == 0) return ATTN_OK;
  const Kernels kern = pick_kernels(p);
  if (!workspace || workspace_bytes < fwd_workspace(p, kern)) return ATTN_ERR_WORKSPACE;

  base.s = to_step(p);
  base.causal = p->causal ? 1 : 0;
  base.scale_log2 = p->scale * kLog2e;
  base.q = static_cast<const __nv_bfloat16*>(q);
  base.k_cache = k_cache;
  base.v_cache = v_cache;
  base.k_scale = k_scale;
  base.v_scale = v_scale;
  base.o = static_cast<__nv_bfloat16*>(o);
  base.lse = lse;
  const int64_t pool_rows = static_cast<int64_t>(p->num_pages) * p->heads_kv * p->page_size;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  size_t used = 0;
  int grids[2];
  both[1] = base;
  for (int tc = 0; tc < 2; ++tc) {
    if (!(tc ? kern.tc : kern.few)) continue;
    CacheFwdArgs& a = both[tc];
    a.rows_lo = tc && kern.few ? kern.split : 0;
    a.rows_hi = tc ? 0x7fffffff : kern.split;
    a.pad = tc ? !kern.few : 1;
    const int chunk = tc ? cache_tc_chunk(p->head_dim, e4m3) : kChunk;
    const int box = p->page_size < chunk ? p->page_size : chunk;
    if (!(tc && e4m3) &&
        (!make_cache_rows_map(&a.tm_k, k_cache, pool_rows, p->head_dim, e4m3, box) ||
         !make_cache_rows_map(&a.tm_v, v_cache, pool_rows, p->head_dim, e4m3, box)))
      return ATTN_ERR_CUDA;
    a.tiles = tc ? kCacheTcRows / kCacheTcTile : 1;
    a.tile_tokens = tc ? kCacheTcTile / a.s.group : 0;
    a.tile_rows = tc ? a.tile_tokens * a.s.group : kern.few_rows;
    if (tc && !e4m3 &&
        !make_bf16_heads_map(&a.tm_q, q, p->tokens, p->heads_q, p->head_dim, a.q_stride, a.s.group,
                             a.tile_tokens))
      return ATTN_ERR_CUDA;
    const Workspace w = kernel_workspace(used, a.tiles * (tc ? kCacheTcTile : kern.few_rows), p->head_dim, tc, e4m3);
    a.part_o = reinterpret_cast<float*>(ws + w.o);
    a.stash = reinterpret_cast<float*>(ws + w.stash);
    a.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    a.part_meta = reinterpret_cast<int4*>(ws + w.meta);
    used = w.bytes;
    // The most chunks that the step can have.  A CTA takes at least one per warp, of
    // the tcgen05 kernel one.
    const double items =
        (static_cast<double>(p->tokens) * a.s.group / (a.tiles * a.tile_rows) + p->num_seqs) * p->heads_kv;
    const double chunks = items * ((static_cast<double>(p->max_pages) * p->page_size) / chunk + 3);
    const double ctas = chunks / (tc ? 1 : cache_warps(e4m3, kern.few_rows)) + 1;
    grids[tc] = ctas < kCacheCtas ? static_cast<int>(ctas) : kCacheCtas;
  }
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (kern.few) e = launch_cache_fwd(both[0], p->head_dim, e4m3, kern.few_rows, grids[0], cs);
  if (e == cudaSuccess && kern.tc) e = launch_cache_fwd_tc(both[1], p->head_dim, e4m3, grids[1], cs);
  return status_of(e);
}

}  // extern "C"

// Kernel-side view of a paged-cache step and the launch wrappers shared by the
// cache kernels and their C ABI layer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "cache.h"
#include "common.cuh"

namespace attn {

struct CacheStep {
  int num_seqs, tokens;
  int heads_q, heads_kv, group;
  int ps_shift;              // log2 of page_size
  int num_pages, max_pages;
  int max_new;
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int32_t* err;
};

// Sequence n of a step: its new tokens are rows t0 .. t0 + m - 1 at positions
// pos0 .. (negative where there are more of them than the length), its keys
// are 0 .. len - 1.  Rows outside [0, tokens) and keys past the page table are
// cut off, so that arrays breaking their contract move no access out of its
// buffer; so are the last 255 keys below 2^31, so that a length rounded up to
// whole chunks stays an int.
struct StepSeq {
  int t0, m, pos0, len;
};

__device__ __forceinline__ StepSeq step_seq(const CacheStep& s, int n, int* bad = nullptr) {
  const int a = __ldg(s.cu + n), b = __ldg(s.cu + n + 1), l = __ldg(s.kv_len + n);
  StepSeq q;
  q.t0 = min(max(a, 0), s.tokens);
  q.m = min(max(b, q.t0), s.tokens) - q.t0;
  const int cap = static_cast<int>(
      min(static_cast<long long>(s.max_pages) << s.ps_shift, static_cast<long long>(0x7fffff00)));
  q.len = min(max(l, 0), cap);
  q.pos0 = max(l, 0) - q.m;
  if (bad && (l > cap || l < 0 || q.m > s.max_new || q.m > l)) *bad |= ATTN_DEVERR_SEQLEN;
  return q;
}

// Allows `kern` its dynamic shared memory, once per device (`ready`: a bit each):
// the call takes 1 to 2 us of the host's time, of some 30 for a step.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (ready.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

struct AppendArgs {
  CacheStep s;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float* cos_sin;
  int rot_dim, interleaved, max_position;
  __nv_bfloat16* q_out;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;
  // e4m3: leading blocks of the grid, and how they find their pages
  int unit_blocks;
  int slots;         // page slots per sequence, 0: found by a scan over the sequences
  int units;         // slots > 0: (page item, KV head, K or V) units
  int head_blocks, loop;   // slots == 0: blocks of a page item, units that a thread goes over
  FastDiv fd_slots;
  // the other blocks: row_blocks blocks of tokens for each group of hb heads of q and,
  // bf16, of k and v
  int row_blocks, hb, q_groups, kv_groups;
};

cudaError_t launch_cache_append(const AppendArgs& a, int head_dim, bool e4m3, int page_size,
                                cudaStream_t st);
// e4m3 units of pages of page_size rows that a block works on at a time.
int append_units(int head_dim, int page_size);
// Tokens of a block of the row path.
int append_row_tokens(int head_dim);

// e4m3 calls with at most this many new tokens per sequence give each (page, KV
// head, K or V) unit to one warp, the others to as many threads as a page needs,
// found by a scan over the sequences.  256 sequences with 1, 8, 12 new tokens: 6.3,
// 16.3, 39 us by warps (of 16 rows for the 12), 13, 23, 29 us by the scan.
constexpr int kAppendSmall = 8;

// Chunks of 32 keys are the unit in which attn_cache_fwd deals work.
constexpr int kChunk = 32;
// Warps of a CTA of the kernel for few rows, by the rows of its items.  e4m3 keys take
// as many instructions as bf16 ones in half the time: one sequence of 262144 of them,
// 8 and 12 warps, 103 and 98 us; but 16 rows at 12 warps have too few registers (32
// sequences of 4096 keys with 20 rows each: 136 and 161 us).  bf16: 65 and 75 us for 64
// sequences of up to 8192 keys.
constexpr int cache_warps(bool e4m3, int rows) { return e4m3 && rows == 8 ? 12 : 8; }
// CTAs of attn_cache_fwd (fewer for small steps): a fixed count, not the
// device's SM count, so that the result does not depend on the device.
constexpr int kCacheCtas = 152;

struct CacheFwdArgs {
  CacheStep s;
  int causal;
  int rows_lo, rows_hi;   // sequences with more than rows_lo, at most rows_hi query rows per KV head
  int pad;                // whether this launch writes the padding rows
  float scale_log2;
  const __nv_bfloat16* q;
  int64_t q_stride;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;     // [grid][2][head_dim / 4][rows][4] partial outputs
  float* stash;      // [grid][warps][rows][head_dim] parts that a warp finished early
  float2* part_ml;   // [grid][2][rows] running maximum (log2) and sum
  int4* part_meta;   // [grid][2] {kind bits, sequence, KV head, row block}
  int tiles, tile_rows;     // an item's row tiles, and the query rows in each
  int tile_tokens;          // cache_fwd_tc: tile_rows / group
  CUtensorMap tm_k, tm_v;   // the pools' rows in boxes of min(page_size, chunk)
  CUtensorMap tm_q;         // cache_fwd_tc: q in boxes of tile_tokens x group heads x 64 dims
};

// e4m3 caches: P enters its product with the codes as fp16, as
//   p_j scale_j 2^(kPHead - R),   R (log2) at most kPSlack below the largest p_j scale_j
// of the keys that the row has seen (p over the running maximum, scale of the values'
// page).  R goes by the product, so that neither a page of a large scale that weighs
// nothing nor a key of no value but a large weight takes the others' bits; it rises by
// more than kPSlack at a time, which spares O most rescalings.  P is off by 2^-11 of
// itself and, where fp16 ends, by 2^-25 2^-kPHead = 2^-33 of the largest product.  It
// stays below 2^11: the five powers of two to fp16's end are for logits so large that
// their rounding is whole powers (R is held relative to the maximum for the same reason).
// Head and slack of 8 and 3, 7 and 4: 585 and 583 us for the chunk of 2 x 2048 tokens over
// 8192, 76.9 and 76.7 us for 12 sequences of up to 700 new tokens.
constexpr float kPHead = 8.f, kPSlack = 3.f;
constexpr float kPUp = 256.f, kPDown = 1.f / 256.f;   // 2^kPHead and back

// e4m3 caches: a row of q is held in fp16 times a power of two that takes its largest
// element to [2^kQUp, 2^(kQUp + 1)): a bf16 element is exact down to 2^-31 of that, and
// then off by 2^-39 of it at most.
constexpr int kQUp = 14;

// Rows of an item of the tcgen05 kernel, and of each of its two tiles.
constexpr int kCacheTcRows = 256, kCacheTcTile = 128;
// The number of keys of its chunks.
int cache_tc_chunk(int head_dim, bool e4m3);
cudaError_t launch_cache_fwd_tc(const CacheFwdArgs& a, int head_dim, bool e4m3, int grid,
                                cudaStream_t st);
// Joins the items that several CTAs hold parts of (parts of item_rows rows).
cudaError_t launch_cache_join(const CacheFwdArgs& a, int head_dim, int item_rows, int grid,
                              cudaStream_t st);

// Rows per work item of the variant that serves `rows` query rows per KV head.
int cache_fwd_rows(int rows);
cudaError_t launch_cache_fwd(const CacheFwdArgs& a, int head_dim, bool e4m3, int item_rows,
                             int grid, cudaStream_t st);

// Whether a launch serves sequence q, its new tokens' rows being m * group.
__device__ __forceinline__ bool serves(const CacheFwdArgs& a, const StepSeq& q) {
  const int rows = q.m * a.s.group;
  return rows > a.rows_lo && rows <= a.rows_hi;
}

}  // namespace attn

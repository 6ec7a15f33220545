// Shared definitions of the linear-attention kernels (linear.h).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"
#include "linear.h"
#include "places.h"

namespace attn {

constexpr int kLinearJobs = 3;      // outputs of one launch at most

// The output and the three gradients are one recurrence over rows x, y, z:
//   forwards   S = l S + y_t z_t^T,  out_t = scale S^T x_t
//   backwards  S = S + scale y_t z_t^T,  out_t = S^T x_t,  then S = l S
//              (over t from the last token down; y, z of every query head of x's KV head)
// with (x, y, z) = (q, k, v) -> o;  (dout, v, k) -> dq;  backwards (k, q, dout) -> dv and
// (v, dout, q) -> dk.  The state of the second and the last is the transposed
// one of the first and the third.
struct LinearJob {
  CUtensorMap mx, my, mz, mo;   // maps over [tokens, heads, head_dim], boxes of a chunk and 64 dims
  const __nv_bfloat16 *x, *y, *z;           // the same rows, for the kernel without maps
  int64_t x_stride, y_stride, z_stride;     // elements from token to token
  __nv_bfloat16* out;       // dense, heads_x heads; null: states only
  int heads_x;              // heads that the job's items go over (states only: KV heads)
  int backwards;
  int terms;                // bf16 terms of a decayed key: 3 where `last` is returned; 2 of a pass over the
                            // states whose walks hold them in one (see state_terms); else 1
  int inner;                // heads of y and z that meet one head of x
  FastDiv fd_heads;         // heads_x
  FastDiv fd_kv;            // heads of x per KV head
  const float* first;       // state before the first token of the walk, or null
  float* last;              // state after its last token, or null
  int transposed;           // `first` is held transposed
  int seg_chunks;           // chunks of a segment at most
  int slots;                // (sequence, segment) pairs at most, without `out` those that hand a state on
  // States that the segments add, but for the last of each sequence in the walk's direction, fp32
  // [places, heads_kv, D/4, D, 4] (columns in fours, rows within): read by a job with `out`, written
  // by one without, which also writes them transposed where that is not null.
  float* parts;
  float* parts_t;
};

// The bf16 terms in which a state meets its rows, in a walk of a launch whose keys come in up to `terms`:
// two, or, where there is no room (heads of 128 or two CTAs on an SM, with terms of the keys
// beside them), one, the keys then in two or three, in the pass over the states as well.  So two roundings to
// bf16 are on a product's way besides the output's at most, one of them for most: 1.41 times
// the error of the output's alone, 1.6 to 1.7 with one term of each (then 104 us for 124 of 4 x 4096 tokens).
constexpr int state_terms(int head_dim, int terms, bool pairs) {
  return terms == 1 || (head_dim == 64 && !pairs) ? 2 : 1;
}

struct LinearArgs {
  LinearJob job[kLinearJobs];
  int jobs;
  int merged;               // 1: one job's items after the other's; `jobs` (all have as many): in turn
  int num_seqs, seqlen, tokens, heads_kv;
  float scale;
  const int32_t* cu;
  const float* log_decay;
  int32_t* err;
};

// The logarithm of a head's decay, at most 0.  -inf becomes a number whose products with 0
// and with token counts stay finite.
__device__ __forceinline__ float log_decay_of(const LinearArgs& a, int h) {
  float g = __ldg(a.log_decay + h);
  if (!(g <= 0.f)) {
    if (a.err) atomicOr(a.err, ATTN_DEVERR_DECAY);
    g = 0.f;
  }
  return fmaxf(g, -1e6f);
}

// The rows of sequence n alone, kept within the tensors whatever cu holds; two of them may overlap
// where it decreases.
__device__ __forceinline__ void sequence_rows(const LinearArgs& a, int n, int& row0, int& len) {
  if (!a.cu) {
    row0 = n * a.seqlen;
    len = a.seqlen;
    return;
  }
  const int b = __ldg(a.cu + n), e = __ldg(a.cu + n + 1);
  row0 = min(max(b, 0), a.tokens);
  const int end = min(max(e, row0), a.tokens);
  len = end - row0;
  if ((b != row0 || e != end || (n == 0 && b != 0)) && a.err) atomicOr(a.err, ATTN_DEVERR_SEQLEN);
}

// The rows of sequences n0 .. n0 + 31, one a lane (any past the last one), disjoint whatever cu holds;
// `top` is the end of the sequence before (0 at n0 = 0), then that of the last one.
__device__ __forceinline__ void packed_rows(const LinearArgs& a, int n0, int& top, int& row0, int& len) {
  const int lane = lane_id();
  const bool live = n0 + lane < a.num_seqs;
  const int first = n0 == 0 ? __ldg(a.cu) : top;
  const int e = live ? __ldg(a.cu + n0 + lane + 1) : a.tokens;
  top = packed_end(first, top, a.tokens);
  int end = packed_end(e, top, a.tokens);
  row0 = __shfl_up_sync(0xffffffffu, end, 1);
  if (lane == 0) row0 = top;
  if (__any_sync(0xffffffffu, end < row0)) {
#pragma unroll 1
    for (int d = 1; d < 32; d *= 2) end = max(end, __shfl_up_sync(0xffffffffu, end, d));
    row0 = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) row0 = top;
  }
  len = end - row0;
  if (((live && e != end) || (n0 == 0 && first != 0)) && a.err) atomicOr(a.err, ATTN_DEVERR_SEQLEN);
  top = __shfl_sync(0xffffffffu, end, 31);
}

// `pairs` (head_dim 64): two CTAs on an SM.  `follows`: the launch before on the stream is the pass
// over its states.
cudaError_t launch_linear(const LinearArgs& a, int head_dim, bool states_only, bool pairs, bool follows,
                          cudaStream_t st);

// Sequences of at most this many tokens (packed: all of them together) go token by token
// (linear_short.cu).  us with and without, 32 heads, a graph's launch of 5 us included:
//                                   8 tokens       64 x 8
//   128 dims, forward              12.4 / 13.5     83 / 111
//     forward, states              12.4 / 19.6     93 / 202
//     backward, 8 KV heads         18.6 / 23.6    172 / 217
//   64 dims, forward               11.4 / 13.4     34 / 55
//     backward, 8 KV heads         16.5 / 18.6     65 / 119
// 16 tokens of 8 KV heads, backward, would take 27 for 23.
constexpr int kLinearShort = 8;
cudaError_t launch_linear_short(const LinearArgs& a, int head_dim, cudaStream_t st);

}  // namespace attn

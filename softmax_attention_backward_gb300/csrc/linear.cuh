// Shared definitions of the linear-attention kernels (linear.h).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"
#include "linear.h"

namespace attn {

// The three gradients and the output are one recurrence over rows x, y, z:
//   forwards   S = l S + y_t z_t^T,  out_t = scale S^T x_t
//   backwards  S = S + scale y_t z_t^T,  out_t = S^T x_t,  then S = l S
//              (over t from the last token down; y, z of every query head of x's KV head)
// with (x, y, z) = (q, k, v) -> o;  (dout, v, k) -> dq;  backwards (k, q, dout) -> dv and
// (v, dout, q) -> dk.  The state of the second and the last is the transposed
// one of the first and the third.
struct LinearJob {
  const __nv_bfloat16* x;
  const __nv_bfloat16* y;
  const __nv_bfloat16* z;
  int64_t x_stride, y_stride, z_stride;   // elements from token to token
  __nv_bfloat16* out;                     // dense, heads_x heads
  int heads_x;
  int backwards;
  int inner;              // heads of y and z that meet one head of x
  FastDiv fd_kv;          // heads of x per KV head
  const float* first;     // state before the first token of the walk, or null
  float* last;            // state after its last token, or null
  int transposed;         // `first` is held transposed
};

struct LinearArgs {
  int num_seqs, seqlen, tokens, heads_kv;
  float scale;
  const int32_t* cu;
  const float* log_decay;
  int32_t* err;
};

// log2 of a head's decay, at most 0.  -inf becomes a number whose products with 0
// and with token counts stay finite.
__device__ __forceinline__ double log2_decay(const LinearArgs& a, int h) {
  float g = __ldg(a.log_decay + h);
  if (!(g <= 0.f)) {
    if (a.err) atomicOr(a.err, ATTN_DEVERR_DECAY);
    g = 0.f;
  }
  return fmax(g * 1.4426950408889634, -1e6);
}

// The rows of sequence n, kept within the tensors whatever cu holds.
__device__ __forceinline__ void linear_sequence(const LinearArgs& a, int n, int& row0, int& len) {
  if (!a.cu) {
    row0 = n * a.seqlen;
    len = a.seqlen;
    return;
  }
  const int b = __ldg(a.cu + n), e = __ldg(a.cu + n + 1);
  row0 = min(max(b, 0), a.tokens);
  const int end = min(max(e, row0), a.tokens);
  len = end - row0;
  if ((b != row0 || e != end) && a.err) atomicOr(a.err, ATTN_DEVERR_SEQLEN);
}

cudaError_t launch_linear_walk(int head_dim, const LinearArgs& a, const LinearJob& j,
                               cudaStream_t st);

}  // namespace attn

// Shared definitions of the linear-attention kernels (linear.h).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"
#include "launch.h"
#include "linear.h"

namespace attn {

constexpr int kLinearChunk = 128;   // tokens of a chunk
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
  __nv_bfloat16* out;       // dense, heads_x heads; null: states only
  int heads_x;              // heads that the job's items go over (states only: KV heads)
  int backwards;
  int terms;                // bf16 terms of a decayed key: 1, or 3 where `last` is returned
  int inner;                // heads of y and z that meet one head of x
  FastDiv fd_heads;         // heads_x
  FastDiv fd_kv;            // heads of x per KV head
  const float* first;       // state before the first token of the walk, or null
  float* last;              // state after its last token, or null
  int transposed;           // `first` is held transposed
  int seg_chunks;           // chunks of a segment at most
  int slots;                // (sequence, segment) places of the job
  // States that the segments add, fp32 [slots, heads_kv, D/4, D, 4] (columns in fours,
  // rows within): read by a job with `out`, written by one without, which also
  // writes them transposed where that is not null.
  float* parts;
  float* parts_t;
};

struct LinearArgs {
  LinearJob job[kLinearJobs];
  int jobs;
  int num_seqs, seqlen, tokens, heads_kv;
  float scale;
  const int32_t* cu;
  const float* log_decay;
  int32_t* err;
};

cudaError_t launch_linear(const LinearArgs& a, int head_dim, bool states_only, cudaStream_t st);

}  // namespace attn

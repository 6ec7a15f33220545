// The recurrent step of linear attention (linear_attn_step, linear.h): one token
// for each sequence.  Bound by memory: a state of head_dim^2 fp32 is read and
// written for 6 operations an element and query head.
//
// A CTA takes a block of columns of one (sequence, KV head): a thread owns four
// columns (16 bytes) of every eighth to 32nd row, loads them all before it uses
// the first, stores l S + k v^T and keeps its part of q^T S for each query head;
// the parts are joined over the rows through shared memory, in a fixed order.  64
// sequences of 32 heads of 128 (268 MB): 45 us and 5 for the launch, 40 for the bytes alone.
#include <cmath>

#include "linear.cuh"

namespace attn {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepHeads = 4;    // query heads of one pass over the registers

struct StepArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* o;
  float* state;
  int64_t q_stride, k_stride, v_stride;
  int num_slots, heads_kv, group;
  float scale;
  const int32_t* slots;
  const float* log_decay;
  int32_t* err;
};

// D: head_dim; C: columns of a CTA
template <int D, int C>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(const StepArgs a) {
  constexpr int CT = C / 4;                    // threads over the columns
  constexpr int RT = kStepThreads / CT;        // threads over the rows
  constexpr int R = D / RT;                    // rows of a thread
  static_assert(R >= 1, "rows");
  __shared__ float sk[D], sq[kStepHeads][D], s_decay[2];
  __shared__ __align__(16) float sv[C];   // (read and written in 16-byte pieces)
  __shared__ __align__(16) float part[kStepHeads][RT][C];
  const int n = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * C;
  const int ct = threadIdx.x % CT, rt = threadIdx.x / CT;
  const int slot = a.slots ? __ldg(a.slots + n) : n;
  bool live = slot >= 0 && slot < a.num_slots;
  bool bad = slot < -1 || slot >= a.num_slots;
  // a slot that an earlier sequence has is that sequence's
  int twice = 0;
  if (live && a.slots)
    for (int i = threadIdx.x; i < n; i += kStepThreads) twice |= __ldg(a.slots + i) == slot;
  float* base = a.state + ((static_cast<int64_t>(live ? slot : 0) * a.heads_kv + h) * D + rt) * D + c0 + ct * 4;
  float4 s[R];
  if (live)
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = *reinterpret_cast<const float4*>(base + i * RT * D);
  if (threadIdx.x < D) sk[threadIdx.x] = __bfloat162float(a.k[n * a.k_stride + h * D + threadIdx.x]);
  if (threadIdx.x < C) sv[threadIdx.x] = __bfloat162float(a.v[n * a.v_stride + h * D + c0 + threadIdx.x]);
  // The decay in two parts: the rounding of one would be the same in every step (log_decay near -2^-11: a
  // steady state off by up to 2^-14).  By one thread, while the others' loads are under way.
  if (threadIdx.x == kStepThreads - 1) {
    float g = __ldg(a.log_decay + h);
    if (!(g <= 0.f)) {
      if (live && a.err) atomicOr(a.err, ATTN_DEVERR_DECAY);
      g = 0.f;
    }
    const double l = exp(static_cast<double>(g));
    s_decay[0] = static_cast<float>(l);
    s_decay[1] = static_cast<float>(l - s_decay[0]);
  }
  if (__syncthreads_or(twice)) {
    live = false;
    bad = true;
  }
  if (bad && threadIdx.x == 0 && a.err) atomicOr(a.err, ATTN_DEVERR_INDEX_RANGE);
  if (!live) {
    for (int i = threadIdx.x; i < a.group * C; i += kStepThreads)
      a.o[(static_cast<int64_t>(n) * a.heads_kv * a.group + h * a.group + i / C) * D + c0 + i % C] =
          __float2bfloat16_rn(0.f);
    return;
  }
  const float l = s_decay[0], l2 = s_decay[1];
  const float4 v = *reinterpret_cast<const float4*>(sv + ct * 4);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float k = sk[rt + i * RT];
    s[i].x = fmaf(l, s[i].x, fmaf(l2, s[i].x, k * v.x));
    s[i].y = fmaf(l, s[i].y, fmaf(l2, s[i].y, k * v.y));
    s[i].z = fmaf(l, s[i].z, fmaf(l2, s[i].z, k * v.z));
    s[i].w = fmaf(l, s[i].w, fmaf(l2, s[i].w, k * v.w));
    *reinterpret_cast<float4*>(base + i * RT * D) = s[i];
  }
  for (int g0 = 0; g0 < a.group; g0 += kStepHeads) {
    const int gn = min(kStepHeads, a.group - g0);
    const __nv_bfloat16* q = a.q + n * a.q_stride + (static_cast<int64_t>(h) * a.group + g0) * D;
    for (int i = threadIdx.x; i < gn * D; i += kStepThreads) sq[i / D][i % D] = __bfloat162float(q[i]);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kStepHeads; ++j) {
      if (j >= gn) break;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float x = sq[j][rt + i * RT];
        o.x = fmaf(x, s[i].x, o.x);
        o.y = fmaf(x, s[i].y, o.y);
        o.z = fmaf(x, s[i].z, o.z);
        o.w = fmaf(x, s[i].w, o.w);
      }
      *reinterpret_cast<float4*>(&part[j][rt][ct * 4]) = o;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < gn * C; i += kStepThreads) {
      const int j = i / C, c = i % C;
      float o = 0.f;
#pragma unroll
      for (int r = 0; r < RT; ++r) o += part[j][r][c];
      a.o[(static_cast<int64_t>(n) * a.heads_kv * a.group + h * a.group + g0 + j) * D + c0 + c] =
          __float2bfloat16_rn(o * a.scale);
    }
    __syncthreads();
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool good_stride(int64_t stride, int heads, int dim, int64_t* out) {
  const int64_t dense = static_cast<int64_t>(heads) * dim;
  *out = stride == 0 ? dense : stride;
  return *out >= dense && *out % 8 == 0;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" attn_status_t linear_attn_step(const linear_attn_step_t* p, const void* q, const void* k,
                                          const void* v, float* state, void* o,
                                          attn_stream_t stream) {
  if (!p) return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs < 0 || p->num_slots <= 0 || p->heads_q <= 0 || p->heads_kv <= 0 ||
      p->head_dim <= 0 || p->heads_q % p->heads_kv || !std::isfinite(p->scale))
    return ATTN_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->heads_q > 65535) return ATTN_ERR_UNSUPPORTED;
  if (!p->slots && p->num_seqs > p->num_slots) return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs == 0) return ATTN_OK;
  if (!q || !k || !v || !state || !o || !p->log_decay) return ATTN_ERR_INVALID_ARG;
  StepArgs a{};
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &a.q_stride) ||
      !good_stride(p->k_stride, p->heads_kv, p->head_dim, &a.k_stride) ||
      !good_stride(p->v_stride, p->heads_kv, p->head_dim, &a.v_stride))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(state, 16) ||
      !aligned(o, 16) || !aligned(p->slots, 4) || !aligned(p->log_decay, 4) ||
      !aligned(p->error_word, 4))
    return ATTN_ERR_ALIGNMENT;
  const int64_t n = p->num_seqs, wq = static_cast<int64_t>(p->heads_q) * p->head_dim;
  const int64_t wk = static_cast<int64_t>(p->heads_kv) * p->head_dim;
  if (overlap({span_of(o, n, wq, wq, 2), span_of(state, p->num_slots, wk * p->head_dim, wk * p->head_dim, 4),
               span_of(q, n, a.q_stride, wq, 2), span_of(k, n, a.k_stride, wk, 2), span_of(v, n, a.v_stride, wk, 2),
               span_of(p->slots, 1, 0, n, 4), span_of(p->log_decay, 1, 0, p->heads_kv, 4),
               span_of(p->error_word, 1, 0, 1, 4)},
              2))
    return ATTN_ERR_INVALID_ARG;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.state = state;
  a.num_slots = p->num_slots;
  a.heads_kv = p->heads_kv;
  a.group = p->heads_q / p->heads_kv;
  a.scale = p->scale;
  a.slots = p->slots;
  a.log_decay = p->log_decay;
  a.err = p->error_word;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->head_dim == 64) linear_step_kernel<64, 64><<<dim3(p->num_seqs, p->heads_kv, 1), kStepThreads, 0, st>>>(a);
  else linear_step_kernel<128, 64><<<dim3(p->num_seqs, p->heads_kv, 2), kStepThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

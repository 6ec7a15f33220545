// C ABI of the chunked linear attention (declared and documented in linear.h):
// argument validation and the launches.
#include <cuda_runtime.h>

#include <cmath>

#include "linear.cuh"

namespace attn {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool good_stride(int64_t stride, int heads, int dim, int64_t* out) {
  const int64_t dense = static_cast<int64_t>(heads) * dim;
  *out = stride == 0 ? dense : stride;
  return *out >= dense && *out % 8 == 0;
}

attn_status_t check(const linear_attn_problem_t* p) {
  if (!p) return ATTN_ERR_INVALID_ARG;
  if (p->num_seqs <= 0 || p->tokens < 0 || p->heads_q <= 0 || p->heads_kv <= 0 || p->head_dim <= 0 ||
      p->heads_q % p->heads_kv || !std::isfinite(p->scale))
    return ATTN_ERR_INVALID_ARG;
  if (!p->cu_seqlens &&
      (p->seqlen < 0 || static_cast<int64_t>(p->num_seqs) * p->seqlen != p->tokens))
    return ATTN_ERR_INVALID_ARG;
  if (!p->log_decay) return ATTN_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->heads_q > 65535 || static_cast<int64_t>(p->tokens) * p->heads_q >= (int64_t(1) << 31))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(p->cu_seqlens, 4) || !aligned(p->log_decay, 4) || !aligned(p->error_word, 4))
    return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

LinearArgs make_args(const linear_attn_problem_t* p) {
  LinearArgs a{};
  a.num_seqs = p->num_seqs;
  a.seqlen = p->seqlen;
  a.tokens = p->tokens;
  a.heads_kv = p->heads_kv;
  a.scale = p->scale;
  a.cu = p->cu_seqlens;
  a.log_decay = p->log_decay;
  a.err = p->error_word;
  return a;
}

struct Rows {
  const __nv_bfloat16* p;
  int64_t stride;
};

// The job of x's heads over y and z; `shared`: heads of x per KV head.
LinearJob make_job(Rows x, Rows y, Rows z, void* out, int heads_x, int shared, int inner,
                   bool backwards, const float* first, float* last, bool transposed) {
  LinearJob j{};
  j.x = x.p, j.y = y.p, j.z = z.p;
  j.x_stride = x.stride, j.y_stride = y.stride, j.z_stride = z.stride;
  j.out = static_cast<__nv_bfloat16*>(out);
  j.heads_x = heads_x;
  j.backwards = backwards;
  j.inner = inner;
  j.fd_kv = make_fastdiv(shared);
  j.first = first;
  j.last = last;
  j.transposed = transposed;
  return j;
}

// A problem without a token: the last state is the first one.
attn_status_t pass_state(const linear_attn_problem_t* p, const float* first, float* last,
                         cudaStream_t st) {
  if (!last) return ATTN_OK;
  const size_t n = sizeof(float) * p->num_seqs * p->heads_kv * p->head_dim * p->head_dim;
  const cudaError_t e = first ? cudaMemcpyAsync(last, first, n, cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(last, 0, n, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" size_t linear_attn_fwd_workspace_size(const linear_attn_problem_t* p) {
  if (check(p) != ATTN_OK) return 0;
  return 0;
}

extern "C" size_t linear_attn_bwd_workspace_size(const linear_attn_problem_t* p) {
  if (check(p) != ATTN_OK) return 0;
  return 0;
}

extern "C" attn_status_t linear_attn_fwd(const linear_attn_problem_t* p, const void* q,
                                         const void* k, const void* v, const float* initial_state,
                                         void* o, float* final_state, void* workspace,
                                         size_t workspace_bytes, attn_stream_t stream) {
  const attn_status_t s = check(p);
  if (s != ATTN_OK) return s;
  if (initial_state && initial_state == final_state) return ATTN_ERR_INVALID_ARG;
  if (!aligned(initial_state, 16) || !aligned(final_state, 16)) return ATTN_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->tokens == 0) return pass_state(p, initial_state, final_state, st);
  if (!q || !k || !v || !o) return ATTN_ERR_INVALID_ARG;
  Rows rq{static_cast<const __nv_bfloat16*>(q)}, rk{static_cast<const __nv_bfloat16*>(k)},
      rv{static_cast<const __nv_bfloat16*>(v)};
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &rq.stride) ||
      !good_stride(p->k_stride, p->heads_kv, p->head_dim, &rk.stride) ||
      !good_stride(p->v_stride, p->heads_kv, p->head_dim, &rv.stride))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return ATTN_ERR_ALIGNMENT;
  const size_t need = linear_attn_fwd_workspace_size(p);
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  const int group = p->heads_q / p->heads_kv;
  const LinearJob j = make_job(rq, rk, rv, o, p->heads_q, group, 1, false, initial_state,
                               final_state, false);
  return launch_linear_walk(p->head_dim, make_args(p), j, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t linear_attn_bwd(const linear_attn_problem_t* p, const void* q,
                                         const void* k, const void* v, const void* dout,
                                         const float* initial_state, const float* dfinal_state,
                                         void* dq, void* dk, void* dv, float* dinitial_state,
                                         void* workspace, size_t workspace_bytes,
                                         attn_stream_t stream) {
  const attn_status_t s = check(p);
  if (s != ATTN_OK) return s;
  if (dfinal_state && dfinal_state == dinitial_state) return ATTN_ERR_INVALID_ARG;
  if (!aligned(initial_state, 16) || !aligned(dfinal_state, 16) || !aligned(dinitial_state, 16))
    return ATTN_ERR_ALIGNMENT;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (p->tokens == 0) return pass_state(p, dfinal_state, dinitial_state, st);
  if (!q || !k || !v || !dout || !dq || !dk || !dv) return ATTN_ERR_INVALID_ARG;
  Rows rq{static_cast<const __nv_bfloat16*>(q)}, rk{static_cast<const __nv_bfloat16*>(k)},
      rv{static_cast<const __nv_bfloat16*>(v)}, rd{static_cast<const __nv_bfloat16*>(dout)};
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &rq.stride) ||
      !good_stride(p->k_stride, p->heads_kv, p->head_dim, &rk.stride) ||
      !good_stride(p->v_stride, p->heads_kv, p->head_dim, &rv.stride) ||
      !good_stride(p->dout_stride, p->heads_q, p->head_dim, &rd.stride))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return ATTN_ERR_ALIGNMENT;
  const size_t need = linear_attn_bwd_workspace_size(p);
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  const int group = p->heads_q / p->heads_kv;
  const LinearArgs a = make_args(p);
  const LinearJob jobs[3] = {
      make_job(rd, rv, rk, dq, p->heads_q, group, 1, false, initial_state, nullptr, true),
      make_job(rk, rq, rd, dv, p->heads_kv, 1, group, true, dfinal_state, dinitial_state, false),
      make_job(rv, rd, rq, dk, p->heads_kv, 1, group, true, dfinal_state, nullptr, true)};
  for (const LinearJob& j : jobs)
    if (launch_linear_walk(p->head_dim, a, j, st) != cudaSuccess) return ATTN_ERR_CUDA;
  return ATTN_OK;
}

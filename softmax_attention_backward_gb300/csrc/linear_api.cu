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

// How sequences are cut into segments: chunks of a segment for the jobs that walk
// forwards (o, dq) and backwards (dk, dv), and the places that this makes.
struct Cut {
  int chunks[2], slots[2];
  bool parts[2];   // a sequence may have several segments
};

// Costs are counted in tiles of 128 x 128 bf16, the units that a walk loads and
// stores: a chunk of o or dq takes 4, of dk or dv 2 + 2 group, of the states between
// segments 2 (2 group).  A walk that is cut costs the pass over the states and its
// own start (about 3 us, 4 tiles' time at an SM's share of the bandwidth).
struct Kind {
  int heads, chunk, state_heads, state_chunk, count;
};
Cut cut_sequences(const linear_attn_problem_t* p, bool backward) {
  const int sms = sm_count() > 0 ? sm_count() : 152;
  const int group = p->heads_q / p->heads_kv;
  const double unit = p->head_dim / 128.0, start = 4.0;
  const Kind kinds[2] = {{p->heads_q, 4, p->heads_kv, 2, 1}, {p->heads_kv, 2 + 2 * group, p->heads_kv, 2 * group, 2}};
  const bool packed = p->cu_seqlens != nullptr;
  // packed sequences: any may hold nearly all tokens
  const int64_t total = packed ? (static_cast<int64_t>(p->tokens) + kLinearChunk - 1) / kLinearChunk + p->num_seqs / 2
                               : 0;
  const int longest = ((packed ? p->tokens : p->seqlen) + kLinearChunk - 1) / kLinearChunk;
  const int n_kinds = backward ? 2 : 1;
  struct Option {
    int chunks;
    double items, cost, state;   // walks, tiles of one, tiles of all state walks
  };
  Option opt[2][64];
  int n_opt[2] = {0, 0};
  for (int i = 0; i < n_kinds; ++i) {
    const Kind& k = kinds[i];
    for (int nseg = 1; nseg <= 64 && nseg <= (longest > 1 ? longest : 1); ++nseg) {
      const int per = longest > 0 ? (longest + nseg - 1) / nseg : 1;
      if (n_opt[i] && opt[i][n_opt[i] - 1].chunks == per) continue;
      Option o;
      o.chunks = per;
      const double walks = packed ? static_cast<double>(total) / per + 0.5 * p->num_seqs
                                  : static_cast<double>(p->num_seqs) * ((longest + per - 1) / per);
      o.items = walks * k.heads * k.count;
      o.cost = start + unit * per * k.chunk;
      const double cut = packed ? static_cast<double>(total) * (nseg - 1) / nseg
                                : static_cast<double>(p->num_seqs) * (longest - per);
      o.state = nseg == 1 ? 0.0 : unit * cut * k.state_heads * k.state_chunk;
      opt[i][n_opt[i]++] = o;
    }
  }
  auto time = [&](const Option& x, const Option* y) {
    const double items = x.items + (y ? y->items : 0), most = y && y->cost > x.cost ? y->cost : x.cost;
    const double all = packed ? x.items * (start + 0.7 * (x.cost - start)) + (y ? y->items * (start + 0.7 * (y->cost - start)) : 0)
                              : x.items * x.cost + (y ? y->items * y->cost : 0);
    double t;
    if (items <= sms) t = most;
    else if (!packed && !y) t = static_cast<double>((static_cast<int64_t>(items) + sms - 1) / sms) * most;
    else t = all / sms + 0.6 * most;
    const double state = x.state + (y ? y->state : 0);
    if (state > 0) t += 2 * start + 1.3 * state / sms;
    return t;
  };
  int best[2] = {0, 0};
  double least = 0;
  for (int i = 0; i < n_opt[0]; ++i)
    for (int j = 0; j < (backward ? n_opt[1] : 1); ++j) {
      const double t = time(opt[0][i], backward ? &opt[1][j] : nullptr);
      if ((i == 0 && j == 0) || t < least) least = t, best[0] = i, best[1] = j;
    }
  Cut c{};
  for (int i = 0; i < n_kinds; ++i) {
    c.chunks[i] = opt[i][best[i]].chunks;
    c.slots[i] = packed ? p->tokens / (c.chunks[i] * kLinearChunk) + p->num_seqs
                        : p->num_seqs * (longest > 0 ? (longest + c.chunks[i] - 1) / c.chunks[i] : 1);
    c.parts[i] = c.chunks[i] < longest;
  }
  return c;
}

size_t state_bytes(const linear_attn_problem_t* p, int slots) {
  return sizeof(float) * static_cast<size_t>(slots) * p->heads_kv * p->head_dim * p->head_dim;
}
// The states of one launch: forwards those of o or dq, backwards those of dv and, transposed, dk.
size_t workspace_bytes_of(const linear_attn_problem_t* p, const Cut& c) {
  return (c.parts[0] ? state_bytes(p, c.slots[0]) : 0) + (c.parts[1] ? 2 * state_bytes(p, c.slots[1]) : 0);
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
  const void* p;
  int64_t stride;
  int heads;
};

bool map_rows(CUtensorMap* m, const linear_attn_problem_t* p, const Rows& r) {
  return make_bf16_heads_map(m, r.p, p->tokens, r.heads, p->head_dim, r.stride, 1, kLinearChunk);
}

bool map_out(LinearJob* j, const linear_attn_problem_t* p, void* out, int heads) {
  j->out = static_cast<__nv_bfloat16*>(out);
  return map_rows(&j->mo, p, {out, static_cast<int64_t>(heads) * p->head_dim, heads});
}

// What a job takes from the problem; `shared`: heads of x per KV head, `way`: 0 forwards, 1 backwards.
void set_job(LinearJob& j, const linear_attn_problem_t* p, int heads_x, int shared, int inner, const Cut& c, int way) {
  j.heads_x = heads_x;
  j.backwards = way;
  j.inner = inner;
  j.fd_heads = make_fastdiv(heads_x);
  j.fd_kv = make_fastdiv(shared);
  j.seg_chunks = c.chunks[way];
  j.slots = c.slots[way];
}
// The job that fills `j`'s states, and their transposes where those are wanted.
LinearJob state_job(const LinearJob& j, const linear_attn_problem_t* p, int inner, float* transposes) {
  LinearJob s = j;
  s.out = nullptr;
  s.heads_x = p->heads_kv;
  s.inner = inner;
  s.fd_heads = make_fastdiv(p->heads_kv);
  s.fd_kv = make_fastdiv(1);
  s.parts_t = transposes;
  return s;
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
  if (check(p) != ATTN_OK || p->tokens == 0) return 0;
  return workspace_bytes_of(p, cut_sequences(p, false));
}

extern "C" size_t linear_attn_bwd_workspace_size(const linear_attn_problem_t* p) {
  if (check(p) != ATTN_OK || p->tokens == 0) return 0;
  return workspace_bytes_of(p, cut_sequences(p, true));
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
  Rows rq{q, 0, p->heads_q}, rk{k, 0, p->heads_kv}, rv{v, 0, p->heads_kv};
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &rq.stride) ||
      !good_stride(p->k_stride, p->heads_kv, p->head_dim, &rk.stride) ||
      !good_stride(p->v_stride, p->heads_kv, p->head_dim, &rv.stride))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16))
    return ATTN_ERR_ALIGNMENT;
  const Cut cut = cut_sequences(p, false);
  const size_t need = workspace_bytes_of(p, cut);
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  LinearArgs a = make_args(p);
  a.jobs = 1;
  LinearJob& j = a.job[0];
  if (!map_rows(&j.mx, p, rq) || !map_rows(&j.my, p, rk) || !map_rows(&j.mz, p, rv) ||
      !map_out(&j, p, o, p->heads_q))
    return ATTN_ERR_CUDA;
  set_job(j, p, p->heads_q, p->heads_q / p->heads_kv, 1, cut, 0);
  j.first = initial_state;
  j.last = final_state;
  j.parts = static_cast<float*>(workspace);
  if (cut.parts[0]) {
    LinearArgs s = make_args(p);
    s.job[s.jobs++] = state_job(j, p, 1, nullptr);
    if (launch_linear(s, p->head_dim, final_state ? 3 : 1, true, st) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  return launch_linear(a, p->head_dim, final_state ? 3 : 1, false, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
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
  Rows rq{q, 0, p->heads_q}, rk{k, 0, p->heads_kv}, rv{v, 0, p->heads_kv}, rd{dout, 0, p->heads_q};
  if (!good_stride(p->q_stride, p->heads_q, p->head_dim, &rq.stride) ||
      !good_stride(p->k_stride, p->heads_kv, p->head_dim, &rk.stride) ||
      !good_stride(p->v_stride, p->heads_kv, p->head_dim, &rv.stride) ||
      !good_stride(p->dout_stride, p->heads_q, p->head_dim, &rd.stride))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dout, 16) ||
      !aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16))
    return ATTN_ERR_ALIGNMENT;
  const Cut cut = cut_sequences(p, true);
  const size_t need = workspace_bytes_of(p, cut);
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  const int group = p->heads_q / p->heads_kv;
  LinearArgs a = make_args(p);
  a.jobs = 3;
  // dv and dk first: their walks are the longer ones
  LinearJob &jv = a.job[0], &jk = a.job[1], &jq = a.job[2];
  if (!map_rows(&jv.mx, p, rk) || !map_rows(&jv.my, p, rq) || !map_rows(&jv.mz, p, rd) || !map_rows(&jk.mx, p, rv) ||
      !map_out(&jv, p, dv, p->heads_kv) || !map_out(&jk, p, dk, p->heads_kv) || !map_out(&jq, p, dq, p->heads_q))
    return ATTN_ERR_CUDA;
  jk.my = jv.mz, jk.mz = jv.my;
  jq.mx = jv.mz, jq.my = jk.mx, jq.mz = jv.mx;
  set_job(jv, p, p->heads_kv, 1, group, cut, 1);
  set_job(jk, p, p->heads_kv, 1, group, cut, 1);
  set_job(jq, p, p->heads_q, group, 1, cut, 0);
  jv.first = jk.first = dfinal_state;
  jv.last = dinitial_state;
  jq.first = initial_state;
  jk.transposed = jq.transposed = 1;
  float* ws = static_cast<float*>(workspace);
  if (cut.parts[1]) {
    jv.parts = ws;
    jk.parts = ws + state_bytes(p, cut.slots[1]) / sizeof(float);
    ws = jk.parts + state_bytes(p, cut.slots[1]) / sizeof(float);
  }
  jq.parts = ws;
  const int terms = dinitial_state ? 3 : 1;
  if (cut.parts[0] || cut.parts[1]) {
    LinearArgs s = make_args(p);
    if (cut.parts[1]) s.job[s.jobs++] = state_job(jv, p, group, jk.parts);
    if (cut.parts[0]) s.job[s.jobs++] = state_job(jq, p, 1, nullptr);
    if (launch_linear(s, p->head_dim, terms, true, st) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  return launch_linear(a, p->head_dim, terms, false, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

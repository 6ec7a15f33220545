// C ABI of the chunked linear attention (declared and documented in linear.h):
// argument validation and the launches.
#include <cuda_runtime.h>

#include <algorithm>
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
  if (p->num_seqs < 0 || p->tokens < 0 || (p->num_seqs == 0 && p->tokens > 0) ||
      p->heads_q <= 0 || p->heads_kv <= 0 || p->head_dim <= 0 || p->heads_q % p->heads_kv ||
      !std::isfinite(p->scale))
    return ATTN_ERR_INVALID_ARG;
  if (!p->cu_seqlens &&
      (p->seqlen < 0 || static_cast<int64_t>(p->num_seqs) * p->seqlen != p->tokens))
    return ATTN_ERR_INVALID_ARG;
  if (!p->log_decay) return ATTN_ERR_INVALID_ARG;
  if (p->head_dim != 64 && p->head_dim != 128) return ATTN_ERR_UNSUPPORTED;
  if (p->heads_q > 65535 || static_cast<int64_t>(p->tokens) * p->heads_q >= (int64_t(1) << 31) ||
      static_cast<int64_t>(p->num_seqs) * p->heads_q >= (int64_t(1) << 29))
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(p->cu_seqlens, 4) || !aligned(p->log_decay, 4) || !aligned(p->error_word, 4))
    return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

// How sequences are cut into segments: chunks of a segment for the jobs that walk
// forwards (o, dq) and backwards (dk, dv), the segments that this makes at most, and the states that
// they hand on.
struct Cut {
  int chunks[2], slots[2], places[2];
  bool parts[2];   // a sequence may have several segments
  bool dq_first;   // backward: the walks of dq are the longer ones
  bool pairs;      // head_dim 64: two CTAs on an SM
  double us;       // what it is taken to cost
};

// What a walk takes, in us on one SM: `base` for a chunk, `step` for each of its inner
// heads (S, P Z and the state's product), `state` for each inner head of a chunk in the pass over
// the states alone.  Measured, 64 chunks against 32 of 8192 and 4096 tokens: head_dim 128,
// 1, 2, 4 and 8 inner heads, 195, 315, 530 and 970 us; head_dim 64, 140, 229, 412 and 775.  Where many
// SMs read, a chunk takes longer (head_dim 128, 1 inner head, 128 walks 3.07 us, 152 walks 3.26, for 2.88 here),
// and a walk's start and end 12 us: cuts are compared with each other, not with the clock.
struct Rates {
  double base, step, state, part;   // part: a segment's state on the way to another's first
  double start;                     // a walk's start and end
};
constexpr Rates kRates[2] = {{0.58, 1.41, 0.80, 0.2, 4.0}, {1.15, 1.73, 0.94, 0.65, 4.0}};
// Two CTAs of head_dim 64 on an SM hide each other's starts, ends and waits, but leave a walk fewer
// tiles and registers.  us with one and with two, 32 heads: 16 sequences of 100 tokens 34 and 24, 64
// of 100 97 and 61, 8 of 4096 with 38 heads 153 and 150, 4 of 4096 with 38 81 and 104; packed, 64
// of 16 to 400, 16 heads 92 and 69, their backward 231 and 174, 12 of up to 8192 83 and 75.
constexpr Rates kPairs = {1.39, 2.96, 1.4, 0.3, 3.0};
constexpr double kLaunch = 1.5;    // of the pass over the states, whose end the walks overlap
constexpr double kBytes = 5.9e6;   // bytes per us that all walks together get

// The time of na walks of ca and then nb of cb on `sms` SMs, each taking the next as it is free.
double makespan(int sms, double na, double ca, double nb, double cb) {
  const double k = std::floor(na / sms), r = na - k * sms;
  const double low = k * ca, high = r > 0 ? low + ca : low;   // of sms - r SMs, and of r
  if (nb <= 0) return high;
  auto fits = [&](double t) {
    double n = t > low ? (sms - r) * std::floor((t - low) / cb + 1e-9) : 0;
    if (t > high) n += r * std::floor((t - high) / cb + 1e-9);
    return n >= nb;
  };
  double lo = 0, hi = high + (std::floor(nb / sms) + 1) * cb;
  for (int i = 0; i < 12; ++i) {
    const double mid = 0.5 * (lo + hi);
    if (fits(mid)) hi = mid;
    else lo = mid;
  }
  return hi > high ? hi : high;
}

// Measured against cuts of every size (us): backward of 2 x 8192 tokens, 32 heads on 8 of 128, dq
// uncut and the others in 8 segments of a sequence 278, in 6 307, in 4 306 with dq in 2; one
// sequence of 65536 tokens, 8 heads on 2 of 128, segments of 27 chunks 133, of 32 149, of 16 165; packed, forward of
// 12 sequences of up to 8192 tokens, 16 heads on 4 of 64, segments of 7 chunks (taken) 75, of 12 73, of
// 4 81; 40 of 16 to 4096, 16 heads of 128, of 13 179, of 16 167, uncut 191.
Cut find_cut(const linear_attn_problem_t* p, bool backward, int sms, bool pairs) {
  const int group = p->heads_q / p->heads_kv;
  const Rates& rate = pairs ? kPairs : kRates[p->head_dim == 128];
  if (pairs) sms *= 2;
  const double tile = 2.0 * kLinearChunk * p->head_dim;
  const bool packed = p->cu_seqlens != nullptr;
  const int most = ((packed ? p->tokens : p->seqlen) + kLinearChunk - 1) / kLinearChunk;   // of a sequence
  // packed sequences have lengths that the host does not know: half a chunk is taken to be empty in
  // each, and the longest to be six times the average.  Forward and backward of 16 heads on 4 of 64, 32 on 8 and 16
  // of 128, of 6, 12, 40 and 200 sequences of one length (8192 to 200 tokens), 12 and 40 of 1 to 4096,
  // one of 16384 beside 30 of 100, two of 6000 beside 60 of 700: with 1, 2, 4, 6 and 10 times, 10,
  // 6, 4, 2.6 and 3.2 % over the best of them in the mean, 51, 29, 30, 23 and 23 % at most
  const double chunks = packed ? most + 0.5 * p->num_seqs : static_cast<double>(most) * p->num_seqs;
  const int longest = packed ? std::min(most, std::max(4, static_cast<int>(6 * chunks / p->num_seqs))) : most;
  struct Option {
    int chunks;
    double walks, cost, longest, states, state_cost, bytes;   // of one job
  };
  Option opt[2][16];
  int n_opt[2] = {0, 0};
  for (int i = 0; i < (backward ? 2 : 1); ++i) {
    const int inner = i ? group : 1, heads = i ? p->heads_kv : p->heads_q;
    // (the first: as many as fill the SMs once)
    const int fill = packed ? 1 : sms / std::max(1, std::min(sms, p->num_seqs * heads));
    for (const int nseg : {fill, 1, 2, 3, 4, 5, 6, 8, 11, 16, 22, 32, 45, 64, 90}) {
      if (nseg > 1 && nseg > longest) continue;
      const int per = longest > 0 ? (longest + nseg - 1) / nseg : 1;
      const int segs = longest > 0 ? (longest + per - 1) / per : 1;
      Option o;
      o.chunks = per;
      const double chunk = rate.base + rate.step * inner;
      const double walks = packed ? std::max<double>(p->num_seqs, chunks / per + 0.5 * p->num_seqs)
                                  : static_cast<double>(p->num_seqs) * segs;
      const double before = rate.part * (packed ? 0.3 : 0.75) * (segs - 1);
      o.walks = walks * heads;
      o.longest = rate.start + before + chunk * per;
      o.cost = packed ? rate.start + before + chunk * std::min<double>(per, chunks / walks) : o.longest;
      o.states = (walks - p->num_seqs) * p->heads_kv;
      o.state_cost = rate.start + rate.state * inner * per;
      o.bytes = tile * (chunks * heads * (i ? 2 + 2 * inner : 2 + 2.0 / group) +
                        chunks * (walks - p->num_seqs) / walks * p->heads_kv * 2 * inner);
      opt[i][n_opt[i]++] = o;
    }
  }
  const Option none{};
  int best[2] = {0, 0};
  double least = 0;
  for (int i = 0; i < n_opt[0]; ++i)
    for (int j = 0; j < (backward ? n_opt[1] : 1); ++j) {
      const Option &x = opt[0][i], &y = backward ? opt[1][j] : none;
      double t;
      if (packed) {
        // walks of many lengths, the longest first (of each job, or merged of all): the SMs fill up,
        // but for a part of the longest, of two on an SM less, as the last ones run alone
        const double tail = pairs ? 0.25 : 0.5;
        t = (x.walks * x.cost + 2 * y.walks * y.cost) / sms + tail * std::max(x.longest, y.longest);
        if (backward && !(group == 1 && x.chunks == y.chunks))
          t += 0.5 * std::max(x.longest - x.cost, y.longest - y.cost);
        t = std::max(t, std::max(x.longest, y.longest));
        if (x.states + y.states > 0)
          t += kLaunch + (x.states * x.state_cost + y.states * y.state_cost) / sms +
               tail * std::max(x.state_cost, y.state_cost);
      } else {
        t = x.longest > y.longest ? makespan(sms, x.walks, x.cost, 2 * y.walks, y.cost)
                                  : makespan(sms, 2 * y.walks, y.cost, x.walks, x.cost);
        if (x.states + y.states > 0)
          t += kLaunch + makespan(sms, y.states, y.state_cost, x.states, x.state_cost);
      }
      t = std::max(t, (x.bytes + 2 * y.bytes) / kBytes);
      if ((i == 0 && j == 0) || t < least) least = t, best[0] = i, best[1] = j;
    }
  Cut c{};
  for (int i = 0; i < (backward ? 2 : 1); ++i) {
    c.chunks[i] = opt[i][best[i]].chunks;
    const int segs = most > 0 ? (most + c.chunks[i] - 1) / c.chunks[i] : 1;   // of a sequence, dense
    c.slots[i] = packed ? packed_walks(p->tokens, p->num_seqs, c.chunks[i]) : p->num_seqs * segs;
    c.places[i] = packed ? packed_places(p->tokens, c.chunks[i]) : p->num_seqs * (segs - 1);
    c.parts[i] = c.chunks[i] < most;
  }
  c.pairs = pairs;
  c.us = least;
  c.dq_first = backward && opt[0][best[0]].longest > opt[1][best[1]].longest;
  return c;
}

// The cut depends on the sizes alone; a thread keeps the last ones it asked for (finding one takes
// some 10 us of the host's time).
Cut cut_sequences(const linear_attn_problem_t* p, bool backward) {
  const int sms = sm_count() > 0 ? sm_count() : 152;
  struct Kept {
    int key[8];
    Cut cut;
  };
  constexpr int kKept = 8;
  static thread_local Kept kept[kKept] = {};
  static thread_local int next = 0;
  const int key[8] = {sms, backward ? 2 : 1, p->cu_seqlens != nullptr, p->num_seqs,
                      p->tokens, p->heads_q, p->heads_kv, p->head_dim};
  for (const Kept& k : kept)
    if (std::equal(key, key + 8, k.key)) return k.cut;
  Kept& k = kept[next];
  next = (next + 1) % kKept;
  std::copy(key, key + 8, k.key);
  k.cut = find_cut(p, backward, sms, false);
  if (p->head_dim == 64) {
    const Cut two = find_cut(p, backward, sms, true);
    if (two.us < k.cut.us) k.cut = two;
  }
  return k.cut;
}

size_t state_bytes(const linear_attn_problem_t* p, int states) {
  return sizeof(float) * static_cast<size_t>(states) * p->heads_kv * p->head_dim * p->head_dim;
}
// The states of one launch: forwards those of o or dq, backwards those of dv and, transposed, dk.
size_t workspace_bytes_of(const linear_attn_problem_t* p, const Cut& c) {
  return (c.parts[0] ? state_bytes(p, c.places[0]) : 0) + (c.parts[1] ? 2 * state_bytes(p, c.places[1]) : 0);
}

LinearArgs make_args(const linear_attn_problem_t* p) {
  LinearArgs a{};
  a.merged = 1;
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

// Whether no sequence can have more than a few tokens.
bool all_short(const linear_attn_problem_t* p) {
  return (p->cu_seqlens ? p->tokens : p->seqlen) <= kLinearShort && p->num_seqs < (1 << 24);
}

void set_rows(LinearJob* j, const Rows& x, const Rows& y, const Rows& z) {
  j->x = static_cast<const __nv_bfloat16*>(x.p), j->x_stride = x.stride;
  j->y = static_cast<const __nv_bfloat16*>(y.p), j->y_stride = y.stride;
  j->z = static_cast<const __nv_bfloat16*>(z.p), j->z_stride = z.stride;
}

bool map_rows(CUtensorMap* m, const linear_attn_problem_t* p, const Rows& r) {
  return make_bf16_heads_map(m, r.p, p->tokens, r.heads, p->head_dim, r.stride, 1, kLinearChunk);
}

bool map_out(LinearJob* j, const linear_attn_problem_t* p) {
  return map_rows(&j->mo, p, {j->out, static_cast<int64_t>(j->heads_x) * p->head_dim, j->heads_x});
}

// What a job takes from the problem; `shared`: heads of x per KV head, `way`: 0 forwards, 1 backwards.
void set_job(LinearJob& j, const linear_attn_problem_t* p, int heads_x, int shared, int inner,
             const Cut& c, int way) {
  j.heads_x = heads_x;
  j.backwards = way;
  j.terms = 1;
  j.inner = inner;
  j.fd_heads = make_fastdiv(heads_x);
  j.fd_kv = make_fastdiv(shared);
  j.seg_chunks = c.chunks[way];
  j.slots = c.slots[way];
}
// The job that fills `j`'s states, and their transposes where those are wanted.
LinearJob state_job(const LinearJob& j, const linear_attn_problem_t* p, int inner, const Cut& c, float* transposes) {
  LinearJob s = j;
  s.out = nullptr;
  s.slots = c.places[j.backwards];
  s.heads_x = p->heads_kv;
  s.inner = inner;
  s.fd_heads = make_fastdiv(p->heads_kv);
  s.fd_kv = make_fastdiv(1);
  s.parts_t = transposes;
  return s;
}

Span span(const linear_attn_problem_t* p, const Rows& r) {
  return span_of(r.p, p->tokens, r.stride, static_cast<int64_t>(r.heads) * p->head_dim, sizeof(__nv_bfloat16));
}

Span span(const linear_attn_problem_t* p, const float* state) {
  return span_of(state, 1, 0, state_bytes(p, p->num_seqs), 1);
}

// What else a call reads, or (its error word) adds to.
struct Small {
  Span decay, cu, word;
};
Small small(const linear_attn_problem_t* p) {
  return {span_of(p->log_decay, 1, 0, p->heads_kv, sizeof(float)),
          span_of(p->cu_seqlens, 1, 0, static_cast<int64_t>(p->num_seqs) + 1, sizeof(int32_t)),
          span_of(p->error_word, 1, 0, 1, sizeof(int32_t))};
}

// A problem without a token: the last state is the first one.
attn_status_t pass_state(const linear_attn_problem_t* p, const float* first, float* last,
                         cudaStream_t st) {
  if (!last || p->num_seqs == 0) return ATTN_OK;
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
  const Small in = small(p);
  if (overlap({span(p, final_state), span(p, initial_state), in.decay, in.cu, in.word}, 1)) return ATTN_ERR_INVALID_ARG;
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
  const int64_t dense = static_cast<int64_t>(p->heads_q) * p->head_dim;
  const Cut cut = cut_sequences(p, false);
  const size_t need = workspace_bytes_of(p, cut);
  if (overlap({span(p, Rows{o, dense, p->heads_q}), span(p, final_state), span_of(workspace, 1, 0, need, 1), span(p, rq),
               span(p, rk), span(p, rv), span(p, initial_state), in.decay, in.cu, in.word}, 3))
    return ATTN_ERR_INVALID_ARG;
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  LinearArgs a = make_args(p);
  a.jobs = 1;
  LinearJob& j = a.job[0];
  set_job(j, p, p->heads_q, p->heads_q / p->heads_kv, 1, cut, 0);
  set_rows(&j, rq, rk, rv);
  j.out = static_cast<__nv_bfloat16*>(o);
  j.first = initial_state;
  j.last = final_state;
  j.terms = final_state ? 3 : 1;
  if (all_short(p)) return launch_linear_short(a, p->head_dim, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  if (!map_rows(&j.mx, p, rq) || !map_rows(&j.my, p, rk) || !map_rows(&j.mz, p, rv) || !map_out(&j, p))
    return ATTN_ERR_CUDA;
  j.parts = static_cast<float*>(workspace);
  if (cut.parts[0]) {
    LinearArgs s = make_args(p);
    s.job[s.jobs++] = state_job(j, p, 1, cut, nullptr);
    if (launch_linear(s, p->head_dim, true, false, false, st) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  return launch_linear(a, p->head_dim, false, cut.pairs, cut.parts[0], st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t linear_attn_bwd(const linear_attn_problem_t* p, const void* q,
                                         const void* k, const void* v, const void* dout,
                                         const float* initial_state, const float* dfinal_state,
                                         void* dq, void* dk, void* dv, float* dinitial_state,
                                         void* workspace, size_t workspace_bytes,
                                         attn_stream_t stream) {
  const attn_status_t s = check(p);
  if (s != ATTN_OK) return s;
  const Small in = small(p);
  if (overlap({span(p, dinitial_state), span(p, initial_state), span(p, dfinal_state), in.decay, in.cu, in.word}, 1))
    return ATTN_ERR_INVALID_ARG;
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
  const int64_t dense_q = static_cast<int64_t>(p->heads_q) * p->head_dim;
  const int64_t dense_kv = static_cast<int64_t>(p->heads_kv) * p->head_dim;
  const Cut cut = cut_sequences(p, true);
  const size_t need = workspace_bytes_of(p, cut);
  if (overlap({span(p, Rows{dq, dense_q, p->heads_q}), span(p, Rows{dk, dense_kv, p->heads_kv}),
               span(p, Rows{dv, dense_kv, p->heads_kv}), span(p, dinitial_state), span_of(workspace, 1, 0, need, 1),
               span(p, rq), span(p, rk), span(p, rv), span(p, rd), span(p, initial_state), span(p, dfinal_state),
               in.decay, in.cu, in.word}, 5))
    return ATTN_ERR_INVALID_ARG;
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return ATTN_ERR_ALIGNMENT;
  const int group = p->heads_q / p->heads_kv;
  LinearArgs a = make_args(p);
  a.jobs = 3;
  // the longest walks first
  LinearJob &jv = a.job[cut.dq_first], &jk = a.job[cut.dq_first + 1], &jq = a.job[cut.dq_first ? 0 : 2];
  set_job(jv, p, p->heads_kv, 1, group, cut, 1);
  set_job(jk, p, p->heads_kv, 1, group, cut, 1);
  set_job(jq, p, p->heads_q, group, 1, cut, 0);
  set_rows(&jv, rk, rq, rd);
  set_rows(&jk, rv, rd, rq);
  set_rows(&jq, rd, rv, rk);
  jv.out = static_cast<__nv_bfloat16*>(dv);
  jk.out = static_cast<__nv_bfloat16*>(dk);
  jq.out = static_cast<__nv_bfloat16*>(dq);
  jv.first = jk.first = dfinal_state;
  jv.last = dinitial_state;
  jq.first = initial_state;
  jk.transposed = jq.transposed = 1;
  if (all_short(p)) return launch_linear_short(a, p->head_dim, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  if (!map_rows(&jv.mx, p, rk) || !map_rows(&jv.my, p, rq) || !map_rows(&jv.mz, p, rd) || !map_rows(&jk.mx, p, rv))
    return ATTN_ERR_CUDA;
  jk.my = jv.mz, jk.mz = jv.my;
  jq.mx = jv.mz, jq.my = jk.mx, jq.mz = jv.mx;
  if (!map_out(&jv, p) || !map_out(&jk, p) || !map_out(&jq, p)) return ATTN_ERR_CUDA;
  float* ws = static_cast<float*>(workspace);
  if (cut.parts[1]) {
    jv.parts = ws;
    jk.parts = ws + state_bytes(p, cut.places[1]) / sizeof(float);
    ws = jk.parts + state_bytes(p, cut.places[1]) / sizeof(float);
  }
  jq.parts = ws;
  jv.terms = dinitial_state ? 3 : 1;
  // walks of one length: the jobs' in turn, so that none's longest come late and the rows that
  // they share are read together (12 packed sequences of up to 2500 tokens, 16 heads of 64, 130 ->
  // 110 us; 4 x 4096 tokens of 32 heads of 128 339 -> 331 at the time)
  if (group == 1 && cut.chunks[0] == cut.chunks[1]) a.merged = a.jobs;
  if (cut.parts[0] || cut.parts[1]) {
    LinearArgs s = make_args(p);
    if (cut.parts[1]) s.job[s.jobs++] = state_job(jv, p, group, cut, jk.parts);
    if (cut.parts[0]) {
      LinearJob& sq = s.job[s.jobs++];
      sq = state_job(jq, p, 1, cut, nullptr);
      if (state_terms(p->head_dim, jv.terms, cut.pairs) == 1) sq.terms = 2;
    }
    if (launch_linear(s, p->head_dim, true, false, false, st) != cudaSuccess) return ATTN_ERR_CUDA;
  }
  const bool follows = cut.parts[0] || cut.parts[1];
  return launch_linear(a, p->head_dim, false, cut.pairs, follows, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

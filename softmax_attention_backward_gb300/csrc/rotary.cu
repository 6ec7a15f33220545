// Rotation by position (declared and documented in rotary.h): the table of
// cosines and sines, and the rotation of queries and keys with its transpose.
//
// Table.  A frequency f is held as Phi = f / 2 pi modulo 1 in 64-bit fixed point,
// so that position p has the phase p Phi modulo 2^64, one turn: integer sums give
// the angle reduced, where a product in fp64 (two per clock and SM on this chip)
// took most of the time.  The two leading bits of the phase plus an eighth of a turn are the
// quadrant, the rest is t quarter turns with |t| <= 1/2, and with q = pi / 2
//   sin(q t) = q t - (q t)^3 / 3! + ... - (q t)^11 / 11!...,  cos(q t) = 1 - (q t)^2 / 2! + ...
// (Taylor's series, cut behind t^9 and t^10: 2^-29 and 2^-33 of the sum).  Bound by
// memory: 4 cosines and sines a thread, 16 bytes each.  131072 positions of 128 (67 MB):
// 17.5 us, 5 of them a graph's launch; 52 with the angle in fp64 and sincospi.
//
// Rotation.  Bound by memory: every row is read and written once.  A thread holds
// the angles of one unit of dims (two 16-byte pieces half the rotated part
// apart, or one piece of adjacent pairs) and rotates it in up to four heads of a
// token, all loads first; the angles come from L1 or L2, once for four heads.  4 x 4096
// tokens of 32 + 8 heads of 128: 56.5 us with the launch, 50 for the bytes alone.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.h"
#include "rotary.h"

namespace attn {
namespace {

constexpr int kMaxRot = 256;
constexpr int kHeads = 4;        // heads of a thread
constexpr int kTableThreads = 256;

struct Frequencies {
  uint64_t phi[kMaxRot / 2];   // turns per position, modulo 1, times 2^64
};

// The sine and cosine of a phase.
__device__ __forceinline__ void phase_sincos(uint64_t phase, float& sn, float& cs) {
  const uint32_t hi = static_cast<uint32_t>(phase >> 32), lo = static_cast<uint32_t>(phase);
  const uint32_t quad = (hi + 0x20000000u) >> 30;
  // t in units of 2^-32: its leading 32 bits, and the 30 below (a small angle's only ones)
  const int32_t lead = static_cast<int32_t>(((hi - (quad << 30)) << 2) | (lo >> 30));
  const float t = fmaf(static_cast<float>(lo << 2), 0x1p-64f, static_cast<float>(lead) * 0x1p-32f);
  const float u = t * t;
  float s = 1.60441184787e-4f;                 // (pi/2)^9 / 9!
  s = fmaf(s, u, -4.68175413531e-3f);          // (pi/2)^7 / 7!
  s = fmaf(s, u, 7.96926262461e-2f);           // (pi/2)^5 / 5!
  s = fmaf(s, u, -6.45964097506e-1f);          // (pi/2)^3 / 3!
  s = fmaf(s, u, -4.37113900e-8f);             // pi / 2 less its fp32 value
  s = fmaf(t, 1.57079637050f, t * s);
  float c = -2.52020423731e-5f;                // (pi/2)^10 / 10!
  c = fmaf(c, u, 9.19260274839e-4f);           // (pi/2)^8 / 8!
  c = fmaf(c, u, -2.08634807633e-2f);          // (pi/2)^6 / 6!
  c = fmaf(c, u, 2.53669507901e-1f);           // (pi/2)^4 / 4!
  c = fmaf(c, u, -1.23370055014f);             // (pi/2)^2 / 2!
  c = fmaf(c, u, 1.f);
  const bool odd = quad & 1;
  const float a = odd ? c : s, b = odd ? s : c;
  sn = __uint_as_float(__float_as_uint(a) ^ ((quad & 2) << 30));
  cs = __uint_as_float(__float_as_uint(b) ^ (((quad + 1) & 2) << 30));
}

__global__ void __launch_bounds__(kTableThreads)
    rotary_table_kernel(const __grid_constant__ Frequencies fr, float* out, int rows, int rot,
                        float m, float m2) {   // m + m2: the magnitude
  // a thread writes 4 cosines and their 4 sines of every `step`th row
  const int quads = rot / 8, per = kTableThreads / quads;   // rows of a block at a time
  const int lane = static_cast<int>(threadIdx.x) / quads, a = (static_cast<int>(threadIdx.x) - lane * quads) * 4;
  if (lane >= per) return;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int64_t p = static_cast<int64_t>(blockIdx.x) * per + lane;
  uint64_t phase[4], add[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t phi = fr.phi[a + j];
    phase[j] = static_cast<uint64_t>(p) * phi;
    add[j] = static_cast<uint64_t>(step) * phi;
  }
  for (; p < rows; p += step) {
    float c[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      phase_sincos(phase[j], s[j], c[j]);
      phase[j] += add[j];
    }
    float* row = out + p * rot + a;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = fmaf(m, c[j], m2 * c[j]);
      s[j] = fmaf(m, s[j], m2 * s[j]);
    }
    *reinterpret_cast<float4*>(row) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(row + rot / 2) = make_float4(s[0], s[1], s[2], s[3]);
  }
}

struct RotArgs {
  const __nv_bfloat16* in[2];
  __nv_bfloat16* out[2];
  int64_t in_stride[2];
  int heads[2], groups[2];   // groups of kHeads heads
  int tokens, dim, rot, offset, max_position, num_seqs;
  const float* cos_sin;
  const int32_t* cu;
  const int32_t* positions;
  int32_t* err;
  FastDiv fd_units, fd_groups, fd_seqlen;
  int64_t items;
};

// The position of token t: -1 for rows that are to be zeros.
__device__ __forceinline__ int position_of(const RotArgs& a, int t) {
  int pos, flag;
  if (a.positions) {
    pos = __ldg(a.positions + t);
    if (pos == -1) return -1;
    flag = ATTN_DEVERR_INDEX_RANGE;
  } else if (a.cu) {
    if (t >= __ldg(a.cu + a.num_seqs)) return -1;
    int lo = 0, hi = a.num_seqs;   // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid;
      else hi = mid;
    }
    pos = t - __ldg(a.cu + lo);
    flag = ATTN_DEVERR_SEQLEN;
  } else {
    pos = static_cast<int>(fmod_u(static_cast<uint32_t>(t), a.fd_seqlen));
    flag = ATTN_DEVERR_SEQLEN;
  }
  if (pos >= 0 && pos < a.max_position) return pos;
  if (a.err) atomicOr(a.err, flag);
  return -1;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
// x c - y s and y c + x s, each product and sum rounded once
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}

// Units of a head: the rotated ones (rot / 16 pairs of pieces, or rot / 8 pieces of
// adjacent pairs), then the pieces of 8 dims that are copied.
template <bool kInterleaved, bool kInverse>
__global__ void __launch_bounds__(256) rotary_kernel(const RotArgs a) {
  const int64_t item = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x;
  if (item >= a.items) return;
  // groups vary slower than units, tokens slowest; a token has fewer than 2^31 items
  const uint32_t per_token = a.fd_units.d * a.fd_groups.d;
  int t;
  uint32_t rem;
  if (a.items < (int64_t(1) << 32)) {
    const uint32_t q = fdiv(static_cast<uint32_t>(item), a.fd_units);
    t = static_cast<int>(fdiv(q, a.fd_groups));
    rem = static_cast<uint32_t>(item) - t * per_token;
  } else {
    t = static_cast<int>(item / per_token);
    rem = static_cast<uint32_t>(item - static_cast<int64_t>(t) * per_token);
  }
  uint32_t g = fdiv(rem, a.fd_units);
  const int u = static_cast<int>(rem - g * a.fd_units.d);
  const int which = g >= static_cast<uint32_t>(a.groups[0]);
  if (which) g -= a.groups[0];
  const int h0 = g * kHeads;
  const int n = min(kHeads, a.heads[which] - h0);
  const int rotated = kInterleaved ? a.rot / 8 : a.rot / 16;
  int at, second = 0;   // the first dim of the unit's piece, and the distance of the other piece
  bool turned = u < rotated;
  if (turned) {
    at = a.offset + u * 8;
    second = kInterleaved ? 0 : a.rot / 2;
  } else {
    at = (u - rotated) * 8;
    if (at >= a.offset) at += a.rot;
  }
  const __nv_bfloat16* src = a.in[which] + t * a.in_stride[which] + static_cast<int64_t>(h0) * a.dim + at;
  uint4 x[kHeads], y[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i)
    if (i < n) {
      x[i] = *reinterpret_cast<const uint4*>(src + i * a.dim);
      if (!kInterleaved && turned) y[i] = *reinterpret_cast<const uint4*>(src + i * a.dim + second);
    }
  const int pos = position_of(a, t);
  float c[8], s[8];
  if (pos >= 0 && turned) {
    const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
    if (kInterleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(row + u * 4));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + u * 4));
      c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
      s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(row + u * 8) + j);
        const float4 sv = __ldg(reinterpret_cast<const float4*>(row + a.rot / 2 + u * 8) + j);
        c[4 * j] = cv.x, c[4 * j + 1] = cv.y, c[4 * j + 2] = cv.z, c[4 * j + 3] = cv.w;
        s[4 * j] = sv.x, s[4 * j + 1] = sv.y, s[4 * j + 2] = sv.z, s[4 * j + 3] = sv.w;
      }
    }
    if (kInverse)
#pragma unroll
      for (int j = 0; j < (kInterleaved ? 4 : 8); ++j) s[j] = -s[j];
  }
  __nv_bfloat16* dst = a.out[which] +
                       (static_cast<int64_t>(t) * a.heads[which] + h0) * a.dim + at;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i >= n) break;
    uint4 xo = x[i], yo = y[i];
    if (pos < 0) {
      xo = yo = make_uint4(0, 0, 0, 0);
    } else if (turned) {
      float xf[8], yf[8];
      unpack8(x[i], xf);
      if (kInterleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn(xf[2 * j], xf[2 * j + 1], c[j], s[j]);
      } else {
        unpack8(y[i], yf);
#pragma unroll
        for (int j = 0; j < 8; ++j) turn(xf[j], yf[j], c[j], s[j]);
        yo = pack8(yf);
      }
      xo = pack8(xf);
    }
    *reinterpret_cast<uint4*>(dst + i * a.dim) = xo;
    if (!kInterleaved && turned) *reinterpret_cast<uint4*>(dst + i * a.dim + second) = yo;
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status_t rotate(const attn_rotary_problem_t* p, const void* q, const void* k,
                     const float* cos_sin, void* q_out, void* k_out, bool inverse,
                     attn_stream_t stream) {
  if (!p) return ATTN_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->heads_q <= 0 || p->heads_k < 0 || p->head_dim <= 0 || p->rot_dim <= 0 ||
      p->rot_offset < 0 || p->max_position <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (!p->positions && (p->cu_seqlens ? p->num_seqs <= 0 : p->seqlen <= 0 && p->tokens > 0))
    return ATTN_ERR_INVALID_ARG;
  if (p->head_dim % 8 || p->head_dim > 1024 || p->rot_dim % 16 || p->rot_dim > kMaxRot ||
      p->rot_offset % 8)
    return ATTN_ERR_UNSUPPORTED;
  if (p->rot_offset > p->head_dim - p->rot_dim) return ATTN_ERR_INVALID_ARG;
  const int64_t heads = static_cast<int64_t>(p->heads_q) + p->heads_k;
  // (a token's work items then stay below 2^31 as well)
  if (heads * p->head_dim >= (int64_t(1) << 31) ||
      p->tokens >= (int64_t(1) << 40) / (heads * p->head_dim))
    return ATTN_ERR_UNSUPPORTED;
  if (p->tokens == 0) return ATTN_OK;
  if (!q || !q_out || !cos_sin || (k == nullptr) != (k_out == nullptr) ||
      (k != nullptr) != (p->heads_k > 0))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(cos_sin, 16) || !aligned(p->cu_seqlens, 4) || !aligned(p->positions, 4) ||
      !aligned(p->error_word, 4))
    return ATTN_ERR_ALIGNMENT;
  RotArgs a{};
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int64_t stride[2] = {p->q_stride, p->k_stride};
  for (int i = 0; i < 2; ++i) {
    a.in[i] = static_cast<const __nv_bfloat16*>(in[i]);
    a.out[i] = static_cast<__nv_bfloat16*>(out[i]);
    a.heads[i] = i ? p->heads_k : p->heads_q;
    a.groups[i] = (a.heads[i] + kHeads - 1) / kHeads;
    const int64_t dense = static_cast<int64_t>(a.heads[i]) * p->head_dim;
    a.in_stride[i] = stride[i] == 0 ? dense : stride[i];
    if (a.in_stride[i] < dense) return ATTN_ERR_INVALID_ARG;
    if (a.in_stride[i] % 8) return ATTN_ERR_ALIGNMENT;
    if (in[i] && in[i] == out[i] && a.in_stride[i] != dense) return ATTN_ERR_INVALID_ARG;
  }
  Span from[2], to[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t dense = static_cast<int64_t>(a.heads[i]) * p->head_dim;
    from[i] = span_of(in[i], p->tokens, a.in_stride[i], dense, 2);
    to[i] = span_of(out[i], p->tokens, dense, dense, 2);
    if (in[i] != out[i] && overlap({to[i], from[i]}, 1)) return ATTN_ERR_INVALID_ARG;
  }
  if (overlap({to[0], to[1], from[1]}, 1) || overlap({to[1], from[0]}, 1)) return ATTN_ERR_INVALID_ARG;
  if (overlap({to[0], to[1], span_of(cos_sin, p->max_position, p->rot_dim, p->rot_dim, 4),
               span_of(p->cu_seqlens, 1, 0, static_cast<int64_t>(p->num_seqs) + 1, 4),
               span_of(p->positions, 1, 0, p->tokens, 4), span_of(p->error_word, 1, 0, 1, 4)},
              2))
    return ATTN_ERR_INVALID_ARG;
  a.tokens = p->tokens;
  a.dim = p->head_dim;
  a.rot = p->rot_dim;
  a.offset = p->rot_offset;
  a.max_position = p->max_position;
  a.num_seqs = p->num_seqs;
  a.cos_sin = cos_sin;
  a.cu = p->cu_seqlens;
  a.positions = p->positions;
  a.err = p->error_word;
  const int units = (p->interleaved ? p->rot_dim / 8 : p->rot_dim / 16) + (p->head_dim - p->rot_dim) / 8;
  const int groups = a.groups[0] + a.groups[1];
  a.fd_units = make_fastdiv(units);
  a.fd_groups = make_fastdiv(groups);
  a.fd_seqlen = make_fastdiv(p->seqlen > 0 ? p->seqlen : 1);
  a.items = static_cast<int64_t>(p->tokens) * units * groups;
  const int64_t blocks = (a.items + 255) / 256;
  if (blocks >= (int64_t(1) << 31)) return ATTN_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (p->interleaved) {
    if (inverse) rotary_kernel<true, true><<<grid, 256, 0, st>>>(a);
    else rotary_kernel<true, false><<<grid, 256, 0, st>>>(a);
  } else {
    if (inverse) rotary_kernel<false, true><<<grid, 256, 0, st>>>(a);
    else rotary_kernel<false, false><<<grid, 256, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" attn_status_t attn_rotary_table(const attn_rotary_table_t* t, float* cos_sin,
                                           attn_stream_t stream) {
  if (!t || t->max_position < 0 || t->rot_dim <= 0) return ATTN_ERR_INVALID_ARG;
  if (t->rot_dim % 16 || t->rot_dim > kMaxRot) return ATTN_ERR_UNSUPPORTED;
  if (!(t->base > 0.0) || !std::isfinite(t->base) || !std::isfinite(static_cast<float>(t->magnitude)))
    return ATTN_ERR_INVALID_ARG;
  if (t->scaling < ATTN_ROTARY_NONE || t->scaling > ATTN_ROTARY_PARTS) return ATTN_ERR_INVALID_ARG;
  if (t->scaling != ATTN_ROTARY_NONE && (!(t->factor > 0.0) || !std::isfinite(t->factor)))
    return ATTN_ERR_INVALID_ARG;
  if (t->scaling == ATTN_ROTARY_PARTS &&
      (t->original <= 0 || !std::isfinite(t->fast) || !std::isfinite(t->slow) || !(t->fast > t->slow)))
    return ATTN_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  Frequencies fr{};
  const double r = t->rot_dim;
  const double base = t->scaling == ATTN_ROTARY_BASE ? t->base * std::pow(t->factor, r / (r - 2.0)) : t->base;
  for (int a = 0; a < t->rot_dim / 2; ++a) {
    double f = std::pow(base, -2.0 * a / r);
    if (t->scaling == ATTN_ROTARY_LINEAR) f /= t->factor;
    if (t->scaling == ATTN_ROTARY_PARTS) {
      double w = (t->original * f / two_pi - t->slow) / (t->fast - t->slow);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      f *= w + (1.0 - w) / t->factor;
    }
    if (!std::isfinite(f)) return ATTN_ERR_INVALID_ARG;
    double turns = f / two_pi;
    turns -= std::floor(turns);
    const double scaled = std::ldexp(turns, 64);   // below 2^64, an integer from 2^53 on
    fr.phi[a] = scaled >= 18446744073709551616.0 ? 0 : static_cast<uint64_t>(scaled + (scaled < 0x1p52 ? 0.5 : 0.0));
  }
  if (t->max_position == 0) return ATTN_OK;
  if (!cos_sin) return ATTN_ERR_INVALID_ARG;
  if (!aligned(cos_sin, 16)) return ATTN_ERR_ALIGNMENT;
  const int per = kTableThreads / (t->rot_dim / 8);
  const size_t blocks = (static_cast<size_t>(t->max_position) + per - 1) / per;
  const int grid = resident_grid(rotary_table_kernel, blocks * kTableThreads, kTableThreads, 1);
  const float m = static_cast<float>(t->magnitude);
  rotary_table_kernel<<<grid, kTableThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      fr, cos_sin, t->max_position, t->rot_dim, m, static_cast<float>(t->magnitude - m));
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

extern "C" attn_status_t attn_rotary_fwd(const attn_rotary_problem_t* p, const void* q,
                                         const void* k, const float* cos_sin, void* q_out,
                                         void* k_out, attn_stream_t stream) {
  return rotate(p, q, k, cos_sin, q_out, k_out, false, stream);
}

extern "C" attn_status_t attn_rotary_bwd(const attn_rotary_problem_t* p, const void* dq,
                                         const void* dk, const float* cos_sin, void* dq_out,
                                         void* dk_out, attn_stream_t stream) {
  return rotate(p, dq, dk, cos_sin, dq_out, dk_out, true, stream);
}

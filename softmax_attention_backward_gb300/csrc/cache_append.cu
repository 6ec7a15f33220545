// Appending keys and values to the paged cache, the position rotation of
// queries and keys applied on the way.
//
// Pair a = (x, y) of a row at position p becomes (x c - y s, y c + x s) with
// c = cos_sin[p, a], s = cos_sin[p, rot/2 + a].  An e4m3 page and head share one
// scale 2^e, e the least integer with amax <= 448 * 2^e, so a unit of work is
// the part of a call that falls into one page for one KV head and K or V: its
// threads read the rows once, keep the rotated values in registers, reduce
// their largest magnitude and write the codes.  Everything is one pass over
// the inputs, bound by HBM for prompts and by latency for single tokens.
//
// A group of G threads takes a unit.  Sixteen elements of a row, two 16-byte
// chunks, belong to one thread: with half-split pairs the chunks rot/2 apart,
// so that both members of a pair meet in it.
#include "cache.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;

// (x c - y s, y c + x s), every product and sum rounded once (no contraction,
// so the result does not depend on the compiler's choices)
__device__ __forceinline__ void rotate(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  const float b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = a;
  y = b;
}

// Two chunks (ca, cb) of 8 elements of one row in v[0..7], v[8..15].
struct Chunks {
  int ca, cb, rot;   // rot: pair index of the first pair, -1 = not rotated
};

// Chunk pair p of a row of which the first `rot` elements are rotated.
__device__ __forceinline__ Chunks chunk_pair(int p, int rot, int interleaved) {
  const int rp = rot >> 4;
  Chunks c;
  if (p < rp) {
    c.ca = interleaved ? 2 * p : p;
    c.cb = interleaved ? 2 * p + 1 : p + rp;
    c.rot = 8 * p;
  } else {
    c.ca = 2 * p;
    c.cb = 2 * p + 1;
    c.rot = -1;
  }
  return c;
}

__device__ __forceinline__ void load_rotated(const __nv_bfloat16* row, const Chunks& c,
                                             const float* cs, int half, int interleaved,
                                             float (&v)[16]) {
  const uint4 a = *reinterpret_cast<const uint4*>(row + c.ca * 8);
  const uint4 b = *reinterpret_cast<const uint4*>(row + c.cb * 8);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  if (c.rot >= 0) {
    float cv[8], sv[8];
    const float4* c4 = reinterpret_cast<const float4*>(cs + c.rot);
    const float4* s4 = reinterpret_cast<const float4*>(cs + half + c.rot);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(c4 + i), y = __ldg(s4 + i);
      cv[4 * i] = x.x, cv[4 * i + 1] = x.y, cv[4 * i + 2] = x.z, cv[4 * i + 3] = x.w;
      sv[4 * i] = y.x, sv[4 * i + 1] = y.y, sv[4 * i + 2] = y.z, sv[4 * i + 3] = y.w;
    }
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rotate(v[2 * i], v[2 * i + 1], cv[i], sv[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) rotate(v[i], v[8 + i], cv[i], sv[i]);
    }
  }
}

__device__ __forceinline__ void store_bf16(__nv_bfloat16* row, const Chunks& c,
                                           const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(row + c.ca * 8) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(row + c.cb * 8) = make_uint4(w[4], w[5], w[6], w[7]);
}

// Four e4m3 codes, round to nearest even, magnitudes above 448 to 448.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void unpack_e4m3(uint32_t w, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint16_t two = static_cast<uint16_t>(w >> (16 * i));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 x = __half22float2(*reinterpret_cast<__half2*>(&h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// The exponent e of a page's scale: the least integer e >= -100 with
// amax <= 448 * 2^e; 448 = 1.75 * 2^8, so it follows from the exponent and
// mantissa fields of amax (finite, non-negative).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = static_cast<int>(u >> 23) - 127;
  return max((u & 0x7fffffu) <= 0x600000u ? k - 8 : k - 7, -100);
}
__device__ __forceinline__ float exp2_int(int e) {   // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The sequence of token t: the number of entries of cu[1 .. num_seqs] that are
// <= t.  A 32-way search by one warp (t is the same in all its lanes).
__device__ __forceinline__ int warp_seq_of(const CacheStep& s, int t) {
  int lo = 0, hi = s.num_seqs;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + (lane_id() + 1) * step - 1;
    const bool below = i < hi && __ldg(s.cu + i + 1) <= t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, below));
    const int base = lo + cnt * step;
    hi = min(hi, base + step - 1);
    lo = base;
  }
  return min(lo, s.num_seqs);
}

// Positions of sequence q that this call appends: [lo, hi).
__device__ __forceinline__ void append_range(const AppendArgs& a, const StepSeq& q, int& lo,
                                             int& hi) {
  lo = max(q.pos0, 0);
  hi = min(q.len, q.pos0 + min(q.m, a.s.max_new));
  if (a.rot_dim > 0) hi = min(hi, a.max_position);
}

// D: head dim.  G: threads of a unit.  PASSES * (G / (D / 16)) rows at most
// fall into one unit.
template <int D, bool E4M3, int G, int PASSES>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendArgs a) {
  constexpr int CPR = D / 16;              // threads of a row
  constexpr int RP = G / CPR;              // rows of a pass
  const CacheStep& s = a.s;
  const int half = a.rot_dim >> 1;

  if (static_cast<int>(blockIdx.x) >= a.unit_blocks) {
    // ---------------- queries: one row (token, head) per CPR threads ----------------
    const int64_t rows = static_cast<int64_t>(s.tokens) * s.heads_q;
    const int p = threadIdx.x % CPR;
    const Chunks c = chunk_pair(p, a.rot_dim, a.interleaved);
    const int64_t row0 = static_cast<int64_t>(blockIdx.x - a.unit_blocks) * (kThreads / CPR);
    const int64_t wrow = row0 + (threadIdx.x / 32) * (32 / CPR);   // first row of the warp
    if (wrow >= rows) return;
    int n = warp_seq_of(s, static_cast<int>(fdiv(static_cast<uint32_t>(wrow), a.fd_hq)));
    const int64_t row = row0 + threadIdx.x / CPR;
    if (row >= rows) return;
    const int t = static_cast<int>(fdiv(static_cast<uint32_t>(row), a.fd_hq));
    const int h = static_cast<int>(row) - t * s.heads_q;
    while (n < s.num_seqs && __ldg(s.cu + n + 1) <= t) ++n;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    if (n < s.num_seqs && t >= __ldg(s.cu)) {
      const StepSeq q = step_seq(s, n);
      const int pos = q.pos0 + (t - q.t0);
      if (t >= q.t0 && pos >= 0 && (a.rot_dim == 0 || pos < a.max_position))
        load_rotated(a.q + t * a.q_stride + h * D, c, a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim,
                     half, a.interleaved, v);
    }
    store_bf16(a.q_out + row * D, c, v);
    return;
  }

  // ---------------- keys and values: one unit per G threads ----------------
  __shared__ int sh_scan[kThreads / 32 + 1];
  __shared__ int sh_unit[2];
  __shared__ float sh_amax[kThreads / 32];
  const int unit = blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const int tid = threadIdx.x % G;
  const int item = unit / (2 * s.heads_kv);   // page item
  const int hw = unit - item * 2 * s.heads_kv;
  const int h = hw >> 1;
  const bool is_v = hw & 1;
  int n = -1, j = 0;   // sequence and its page among those that the call touches
  if (a.slots > 0) {
    const int nn = static_cast<int>(fdiv(static_cast<uint32_t>(item), a.fd_slots));
    if (unit < a.units && nn < s.num_seqs) {
      n = nn;
      j = item - n * a.slots;
    }
  } else {
    // block-wide scan over the sequences' touched pages (one unit per block)
    if (threadIdx.x == 0) sh_unit[0] = -1;
    int base = 0;
    for (int n0 = 0; n0 < s.num_seqs; n0 += kThreads) {
      const int nn = n0 + threadIdx.x;
      int cnt = 0;
      if (nn < s.num_seqs) {
        int lo, hi;
        append_range(a, step_seq(s, nn), lo, hi);
        if (hi > lo) cnt = ((hi - 1) >> s.ps_shift) - (lo >> s.ps_shift) + 1;
      }
      int inc = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (static_cast<int>(lane_id()) >= o) inc += x;
      }
      __syncthreads();
      if (lane_id() == 31) sh_scan[warp_id()] = inc;
      __syncthreads();
      int before = base, all = base;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < static_cast<int>(warp_id())) before += sh_scan[w];
        all += sh_scan[w];
      }
      const int end = before + inc;
      if (item >= end - cnt && item < end) {
        sh_unit[0] = nn;
        sh_unit[1] = item - (end - cnt);
      }
      base = all;
      if (base > item) break;
    }
    __syncthreads();
    n = sh_unit[0];
    j = sh_unit[1];
  }

  bool live = n >= 0;
  int lo = 0, hi = 0, pos0 = 0, t0 = 0, bad = 0;
  if (live) {
    const StepSeq q = step_seq(s, n, &bad);
    t0 = q.t0;
    pos0 = q.pos0;
    append_range(a, q, lo, hi);
    if (q.m > 0 && a.rot_dim > 0 && pos0 > a.max_position - q.m) bad |= ATTN_DEVERR_SEQLEN;
    live = hi > lo;
  }
  int page = 0, first = 0, cnt = 0;   // first: row in the page of the first new key
  if (live) {
    const int col = (lo >> s.ps_shift) + j;
    const int p0 = max(lo, col << s.ps_shift);
    const int p1 = min(hi, (col + 1) << s.ps_shift);
    cnt = p1 - p0;
    live = cnt > 0;
    if (live) {
      page = __ldg(s.table + static_cast<int64_t>(n) * s.max_pages + col);
      if (page < 0 || page >= s.num_pages) {
        bad |= ATTN_DEVERR_INDEX_RANGE;
        live = false;
      }
      first = p0 - (col << s.ps_shift);
      t0 += p0 - pos0;
      pos0 = p0;
    }
  }
  if (bad && s.err && tid == 0) atomicOr(s.err, bad);
  if (!live) return;   // uniform over the unit's threads

  const int p = tid % CPR;
  const int rot = is_v ? 0 : a.rot_dim;
  const Chunks c = chunk_pair(p, rot, a.interleaved);
  const __nv_bfloat16* src = (is_v ? a.v + t0 * a.v_stride : a.k + t0 * a.k_stride) + h * D;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int64_t ph = static_cast<int64_t>(page) * s.heads_kv + h;
  const int64_t slab = (ph << s.ps_shift) * D;
  float v[PASSES][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * RP + tid / CPR;
    if (r < cnt) {
      load_rotated(src + r * stride, c, a.cos_sin + static_cast<int64_t>(pos0 + r) * a.rot_dim, half,
                   a.interleaved, v[i]);
      if constexpr (E4M3) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float m = fabsf(v[i][e]);
          if (m < INFINITY) amax = fmaxf(amax, m);   // neither infinities nor NaN
        }
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + slab;
        store_bf16(dst + (first + r) * D, c, v[i]);
      }
    }
  }
  if constexpr (E4M3) {
    // (a unit that left above took all G threads of it along, so the masks and
    // barriers below see whole groups)
    const uint32_t mask = 0xffffffffu;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, o));
    if constexpr (G == kThreads) {
      if (lane_id() == 0) sh_amax[warp_id()] = amax;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, sh_amax[w]);
    }
    uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + slab;
    float* scale = (is_v ? a.v_scale : a.k_scale) + ph;
    const int e = scale_exponent(amax);
    float sc = exp2_int(e);
    float inv = exp2_int(-e);
    if (first > 0) {
      const float old = *scale;
      if (old >= sc) {
        sc = old;
        inv = 1.f / old;   // exact: a power of two
      } else {
        // the page's earlier codes again, under the larger scale
        const float f = old * inv;
        uint32_t* w = reinterpret_cast<uint32_t*>(dst);
        for (int i = tid; i < first * D / 4; i += G) {
          float x[4];
          unpack_e4m3(w[i], x);
          w[i] = pack_e4m3(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
        }
      }
      // every thread has read the old scale before one replaces it
      if constexpr (G == kThreads) __syncthreads();
      else __syncwarp();
    }
    if (tid == 0) *scale = sc;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RP + tid / CPR;
      if (r < cnt) {
        uint32_t w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          w[x] = pack_e4m3(v[i][4 * x] * inv, v[i][4 * x + 1] * inv, v[i][4 * x + 2] * inv,
                           v[i][4 * x + 3] * inv);
        uint8_t* row = dst + (first + r) * D;
        *reinterpret_cast<uint2*>(row + c.ca * 8) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + c.cb * 8) = make_uint2(w[2], w[3]);
      }
    }
  }
}

template <int D>
cudaError_t launch(const AppendArgs& a, bool e4m3, bool small, int q_blocks, cudaStream_t st) {
  const int grid = a.unit_blocks + q_blocks;
  if (grid == 0) return cudaSuccess;
  // rows of a unit: up to 8 for the small form (a warp), a whole page (128) else
  constexpr int PS = 8 * (D / 16) / 32, PB = 128 * (D / 16) / kThreads;
  if (small) {
    if (e4m3) cache_append_kernel<D, true, 32, PS><<<grid, kThreads, 0, st>>>(a);
    else cache_append_kernel<D, false, 32, PS><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (e4m3) cache_append_kernel<D, true, kThreads, PB><<<grid, kThreads, 0, st>>>(a);
    else cache_append_kernel<D, false, kThreads, PB><<<grid, kThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, int head_dim, bool e4m3, bool small,
                                int q_blocks, cudaStream_t st) {
  return head_dim == 64 ? launch<64>(a, e4m3, small, q_blocks, st)
                        : launch<128>(a, e4m3, small, q_blocks, st);
}

}  // namespace attn

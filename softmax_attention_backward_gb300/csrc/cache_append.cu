// Appending keys and values to the paged cache, the position rotation of
// queries and keys applied on the way.
//
// Pair a = (x, y) of a row at position p becomes (x c - y s, y c + x s) with
// c = cos_sin[p, a], s = cos_sin[p, rot/2 + a].  Sixteen elements of a row, two
// 16-byte chunks, belong to one thread: with half-split pairs the chunks rot/2
// apart, so that both members of a pair meet in it.
//
// Queries, and bf16 keys and values: a thread keeps the angles of its token's
// chunks and goes over a group of heads (an fp32 table row is as large as two
// bf16 rows, so reading it once per head would double the traffic).
//
// An e4m3 page and head share one scale 2^e, e the least integer with
// amax <= 448 * 2^e, so a unit of work is the part of a call that falls into one
// page for one KV head and K or V: its threads read the rows once, keep the
// rotated values in registers, reduce their largest magnitude and write the
// codes.
//
// Everything is one pass over the inputs.  Four prompts of 8192 to 758 tokens, 16 heads
// of 128, into e4m3 pages: 75 us, 3.9 TB/s over what is read and written, bound by the
// latency of a unit (rows, angles, the maximum, codes) with the 16 warps that the
// registers leave an SM.  8 chunks of up to 1000 tokens into bf16 pages, 32 heads of 64:
// 14 us, 3.9 TB/s.  A token for each of 64 sequences, e4m3: 3.5 us, for one: 2.8 us,
// both the latency of a chain of dependent loads (lengths, page, rows).
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

// The cosines and sines of eight pairs.
struct Angles {
  float c[8], s[8];
  __device__ __forceinline__ void load(const float* at, int half) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(at) + i);
      const float4 y = __ldg(reinterpret_cast<const float4*>(at + half) + i);
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
  }
  // v: the two chunks; pairs are neighbours, or the chunks' elements of one index
  __device__ __forceinline__ void apply(float (&v)[16], int interleaved) const {
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rotate(v[2 * i], v[2 * i + 1], c[i], s[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) rotate(v[i], v[8 + i], c[i], s[i]);
    }
  }
};

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float (&v)[16]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
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

// The rows of a group of heads for a block of tokens.
template <int D>
__device__ __forceinline__ void append_rows(const AppendArgs& a, int block) {
  constexpr int CPR = D / 16;              // threads of a row
  const CacheStep& s = a.s;
  const int grp = block / a.row_blocks;
  const int tok0 = (block - grp * a.row_blocks) * (kThreads / CPR);
  // what the group is of: 0 q, 1 k, 2 v
  const int kind = grp < a.q_groups ? 0 : grp < a.q_groups + a.kv_groups ? 1 : 2;
  const int h0 = (kind == 0 ? grp : grp - a.q_groups - (kind - 1) * a.kv_groups) * a.hb;
  const int h1 = min(h0 + a.hb, kind == 0 ? s.heads_q : s.heads_kv);
  const int wtok = tok0 + threadIdx.x / 32 * (32 / CPR);   // first token of the warp
  if (wtok >= s.tokens) return;
  int n = warp_seq_of(s, wtok);
  const int t = tok0 + threadIdx.x / CPR;
  if (t >= s.tokens) return;
  while (n < s.num_seqs && __ldg(s.cu + n + 1) <= t) ++n;
  const Chunks c = chunk_pair(threadIdx.x % CPR, kind == 2 ? 0 : a.rot_dim, a.interleaved);
  int pos = -1, bad = 0;
  __nv_bfloat16* dst = nullptr;   // the token's row of head 0, and the elements to the next head's
  int64_t step = D;
  if (n < s.num_seqs && t >= __ldg(s.cu)) {
    const StepSeq q = step_seq(s, n, &bad);
    pos = q.pos0 + (t - q.t0);
    if (a.rot_dim > 0 && pos >= a.max_position) {
      bad |= ATTN_DEVERR_SEQLEN;
      pos = -1;
    }
    if (kind != 0 && pos >= 0 && pos < q.len && t - q.t0 < s.max_new) {
      const int page = __ldg(s.table + static_cast<int64_t>(n) * s.max_pages + (pos >> s.ps_shift));
      if (page < 0 || page >= s.num_pages) {
        bad |= ATTN_DEVERR_INDEX_RANGE;
      } else {
        step = static_cast<int64_t>(D) << s.ps_shift;
        dst = static_cast<__nv_bfloat16*>(kind == 1 ? a.k_cache : a.v_cache) +
              static_cast<int64_t>(page) * s.heads_kv * step + (pos & ((1 << s.ps_shift) - 1)) * D;
      }
    }
    if (bad && s.err && threadIdx.x % CPR == 0) atomicOr(s.err, bad);
  }
  if (kind == 0) dst = a.q_out + static_cast<int64_t>(t) * s.heads_q * D;
  if (!dst) return;
  const __nv_bfloat16* src = kind == 0   ? a.q + t * a.q_stride
                             : kind == 1 ? a.k + t * a.k_stride
                                         : a.v + t * a.v_stride;
  const bool live = pos >= 0;   // a query without a position: zeros
  Angles ang;
  if (c.rot >= 0 && live)
    ang.load(a.cos_sin + static_cast<int64_t>(pos) * a.rot_dim + c.rot, a.rot_dim >> 1);
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (live) {
      x = *reinterpret_cast<const uint4*>(src + h * D + c.ca * 8);
      y = *reinterpret_cast<const uint4*>(src + h * D + c.cb * 8);
    }
    float v[16];
    unpack16(x, y, v);
    if (c.rot >= 0 && live) ang.apply(v, a.interleaved);
    store_bf16(dst + h * step, c, v);
  }
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D: head dim.  G: threads of an e4m3 unit, into which PASSES * (G / (D / 16)) rows
// fall at most; SCAN: blocks of a page item each, found by a scan over the sequences,
// of which a group of G threads takes a.loop units, the next one's rows on their way
// into shared memory while it works on one (else slots of a sequence, a warp each).
template <int D, bool E4M3, int G, int PASSES, bool SCAN>
__global__ void __launch_bounds__(kThreads, SCAN ? 2 : 3) cache_append_kernel(const AppendArgs a) {
  if (!E4M3 || static_cast<int>(blockIdx.x) >= a.unit_blocks) {
    append_rows<D>(a, blockIdx.x - a.unit_blocks);
    return;
  }
  if constexpr (E4M3) {
    constexpr int CPR = D / 16;              // threads of a row
    constexpr int RP = G / CPR;              // rows of a pass
    constexpr int UNITS = kThreads / G;      // units of a block at a time
    const CacheStep& s = a.s;
    const int group = threadIdx.x / G, tid = threadIdx.x % G;
    __shared__ float sh_amax[4][kThreads / 32];
    int n = -1, j = 0;   // sequence and its page among those that the call touches
    int hw, hw_end;      // 2 KV head + (0: K, 1: V), of the first unit; their end, UNITS apart
    if constexpr (!SCAN) {
      const int unit = blockIdx.x * UNITS + group;
      const int item = unit / (2 * s.heads_kv);
      hw = unit - item * 2 * s.heads_kv;
      hw_end = hw + 1;
      const int nn = static_cast<int>(fdiv(static_cast<uint32_t>(item), a.fd_slots));
      if (unit < a.units && nn < s.num_seqs) {
        n = nn;
        j = item - n * a.slots;
      }
    } else {
      __shared__ int sh_scan[kThreads / 32];
      __shared__ int sh_unit[2];
      const int item = blockIdx.x / a.head_blocks;
      hw = (blockIdx.x - item * a.head_blocks) * UNITS * a.loop + group;
      hw_end = min(hw + UNITS * a.loop, 2 * s.heads_kv);
      // block-wide scan over the sequences' touched pages; the first block, which looks at all
      // sequences, flags those that bring nothing because their positions are out of range
      if (threadIdx.x == 0) sh_unit[0] = -1;
      int base = 0;
      for (int n0 = 0; n0 < s.num_seqs; n0 += kThreads) {
        const int nn = n0 + threadIdx.x;
        int cnt = 0;
        if (nn < s.num_seqs) {
          int lo, hi, wrong = 0;
          const StepSeq q = step_seq(s, nn, &wrong);
          append_range(a, q, lo, hi);
          if (hi > lo) cnt = ((hi - 1) >> s.ps_shift) - (lo >> s.ps_shift) + 1;
          else if (q.m > 0) wrong = ATTN_DEVERR_SEQLEN;
          if (wrong && s.err && blockIdx.x == 0) atomicOr(s.err, wrong);
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
        if (base > item && blockIdx.x > 0) break;
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
    auto sync = [&] {
      if constexpr (G > 32) named_bar_sync(1 + group, G);
      else __syncwarp();
    };
    // the largest of a unit's threads; `at`: 0 to 3, another in each of two calls in a row
    auto largest = [&](float x, int at) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
      if constexpr (G > 32) {
        if (lane_id() == 0) sh_amax[at][warp_id()] = x;
        sync();
#pragma unroll
        for (int w = 0; w < G / 32; ++w) x = fmaxf(x, sh_amax[at][group * (G / 32) + w]);
      }
      return x;
    };
    const int row0 = tid / CPR;   // the thread's first row
    // The rows of unit hw: into registers, or (SCAN) to the thread's own place in buffer b
    extern __shared__ uint4 sh_rows[];   // [buffer][PASSES][2][kThreads]
    auto load = [&](int hw, int b, uint4 (&x)[PASSES], uint4 (&y)[PASSES]) {
      const Chunks c = chunk_pair(tid % CPR, hw & 1 ? 0 : a.rot_dim, a.interleaved);
      const int64_t stride = hw & 1 ? a.v_stride : a.k_stride;
      const __nv_bfloat16* src = (hw & 1 ? a.v : a.k) + t0 * stride + (hw >> 1) * D;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = i * RP + row0;
        if constexpr (SCAN) {
          uint4* at = sh_rows + (b * PASSES + i) * 2 * kThreads + threadIdx.x;
          if (r < cnt) {
            cp_async16(at, src + r * stride + c.ca * 8);
            cp_async16(at + kThreads, src + r * stride + c.cb * 8);
          }
        } else {
          x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < cnt) {
            x[i] = *reinterpret_cast<const uint4*>(src + r * stride + c.ca * 8);
            y[i] = *reinterpret_cast<const uint4*>(src + r * stride + c.cb * 8);
          }
        }
      }
      if constexpr (SCAN) cp_async_commit();
    };

    uint4 x[PASSES], y[PASSES];
    if (hw < hw_end) load(hw, 0, x, y);
    for (int k = 0; hw < hw_end; ++k, hw += UNITS) {
      const bool is_v = hw & 1;
      const Chunks c = chunk_pair(tid % CPR, is_v ? 0 : a.rot_dim, a.interleaved);
      const int64_t ph = static_cast<int64_t>(page) * s.heads_kv + (hw >> 1);
      uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + (ph << s.ps_shift) * D;
      float* scale = (is_v ? a.v_scale : a.k_scale) + ph;
      float old = 0.f;
      if (first > 0) old = *scale;
      if constexpr (SCAN) {
        if (hw + UNITS < hw_end) {
          load(hw + UNITS, (k + 1) & 1, x, y);
          cp_async_wait<1>();
        } else {
          cp_async_wait<0>();
        }
#pragma unroll
        for (int i = 0; i < PASSES; ++i) {
          const uint4* at = sh_rows + ((k & 1) * PASSES + i) * 2 * kThreads + threadIdx.x;
          x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
          if (i * RP + row0 < cnt) x[i] = at[0], y[i] = at[kThreads];
        }
      }
      float v[PASSES][16];
#pragma unroll
      for (int i = 0; i < PASSES; ++i) unpack16(x[i], y[i], v[i]);
      float amax = 0.f;   // (fmaxf leaves NaN out)
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = i * RP + row0;
        if (r < cnt && c.rot >= 0) {
          Angles ang;
          ang.load(a.cos_sin + static_cast<int64_t>(pos0 + r) * a.rot_dim + c.rot, a.rot_dim >> 1);
          ang.apply(v[i], a.interleaved);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(v[i][e]));
      }
      amax = largest(amax, k & 1);
      if (amax == INFINITY) {   // once more, without the infinities
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < PASSES; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (fabsf(v[i][e]) < INFINITY) amax = fmaxf(amax, fabsf(v[i][e]));
        amax = largest(amax, 2 + (k & 1));
      }
      const int e = scale_exponent(amax);
      float sc = exp2_int(e);
      float inv = exp2_int(-e);
      if (first > 0) {
        if (old >= sc) {
          sc = old;
          inv = 1.f / old;   // exact: a power of two
        } else {
          // the page's earlier codes again, under the larger scale
          const float f = old * inv;
          uint32_t* w = reinterpret_cast<uint32_t*>(dst);
          for (int i = tid; i < first * D / 4; i += G) {
            float z[4];
            unpack_e4m3(w[i], z);
            w[i] = pack_e4m3(z[0] * f, z[1] * f, z[2] * f, z[3] * f);
          }
        }
        sync();   // every thread has read the old scale
      }
      if (tid == 0) *scale = sc;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int r = i * RP + row0;
        if (r < cnt) {
          uint32_t w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            w[z] = pack_e4m3(v[i][4 * z] * inv, v[i][4 * z + 1] * inv, v[i][4 * z + 2] * inv,
                             v[i][4 * z + 3] * inv);
          uint8_t* row = dst + (first + r) * D;
          *reinterpret_cast<uint2*>(row + c.ca * 8) = make_uint2(w[0], w[1]);
          *reinterpret_cast<uint2*>(row + c.cb * 8) = make_uint2(w[2], w[3]);
        }
      }
    }
  }
}

// Threads of a unit that holds a page of `page_size` rows: four rows a thread, two
// where that would leave less than a warp.
constexpr int page_threads(int head_dim, int page_size) {
  return page_size * (head_dim / 16) / 4 < 32 ? 32 : page_size * (head_dim / 16) / 4;
}

template <int D, int PS>
cudaError_t launch_pages(const AppendArgs& a, int grid, cudaStream_t st) {
  constexpr int G = page_threads(D, PS), PASSES = PS * (D / 16) / G, SMEM = 2 * PASSES * 2 * kThreads * 16;
  auto kern = cache_append_kernel<D, true, G, PASSES, true>;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = allow_smem(kern, SMEM, ready);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, SMEM, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const AppendArgs& a, bool e4m3, int page_size, cudaStream_t st) {
  const int grid = a.unit_blocks + a.row_blocks * (a.q_groups + 2 * a.kv_groups);
  if (grid == 0) return cudaSuccess;
  if (!e4m3) {
    cache_append_kernel<D, false, 32, 1, false><<<grid, kThreads, 0, st>>>(a);
  } else if (a.slots > 0) {   // units of up to kAppendSmall rows, a warp each
    cache_append_kernel<D, true, 32, kAppendSmall * (D / 16) / 32, false><<<grid, kThreads, 0, st>>>(a);
  } else {
    switch (page_size) {
      case 16: return launch_pages<D, 16>(a, grid, st);
      case 32: return launch_pages<D, 32>(a, grid, st);
      case 64: return launch_pages<D, 64>(a, grid, st);
      default: return launch_pages<D, 128>(a, grid, st);
    }
  }
  return cudaGetLastError();
}

}  // namespace

int append_units(int head_dim, int page_size) { return kThreads / page_threads(head_dim, page_size); }
int append_row_tokens(int head_dim) { return kThreads / (head_dim / 16); }

cudaError_t launch_cache_append(const AppendArgs& a, int head_dim, bool e4m3, int page_size,
                                cudaStream_t st) {
  return head_dim == 64 ? launch<64>(a, e4m3, page_size, st) : launch<128>(a, e4m3, page_size, st);
}

}  // namespace attn

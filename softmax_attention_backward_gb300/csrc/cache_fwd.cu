// Attention of new queries over the paged cache: few query rows against long
// key ranges, where every key and value has to cross HBM once and little is
// computed for each.
//
// Work.  An item is (sequence, KV head, block of up to ROWS query rows); the
// rows of a KV head are its (new token, query head of the group) pairs, token
// major, so the heads that share a key read it once.  An item's keys are cut
// into chunks of 16.  All items' chunks, in one line, are dealt to the CTAs in
// equal contiguous ranges, and a CTA's range to its warps, so every SM streams
// the same number of bytes whatever the sequences' lengths are.  An item that
// ends up in several warps is joined in shared memory, one that ends up in
// several CTAs by a second kernel, in a fixed order.
//
// A warp runs on its own, without barriers: each thread copies with cp.async
// exactly the 16-byte vectors that it will feed to the tensor cores
// (mma.sync.m16n8k16) itself, into a ring of its own, in which neither bank
// conflicts nor other threads' copies matter.  That works because the order of
// the contracted index is free as long as both operands agree on it, and the
// order of the output columns as long as the epilogue undoes it:
//   S = Q K^T: the thread of column g (key g of 8) and quad index t takes the
//     vector of dims [V t, V t + V) of its key (V = 8 bf16 or 16 codes) in each
//     4 V dims, and Q is loaded in the same order;
//   O = P V: it takes vector g of keys 2t, 2t+1, 2t+8, 2t+9; output column g of
//     the j-th MMA is then dim V g + j, and a byte permutation pairs the keys.
// Tensor-core work is a small part of what mma.sync can do (one 16-row tile
// meets each key), so tcgen05, whose operands have to lie in shared memory
// in a swizzled order, would add data movement and gain nothing here.
//
// Softmax statistics, sums and O are fp32.  bf16 caches: S is exact products in
// fp32, and with ROWS = 8 the unused half of the 16-row tile carries the
// rounding residue of P (P = hi + lo in bf16), at no cost; with more rows P is
// rounded to bf16 once, as in attn_fwd.  e4m3 caches: codes convert to fp16
// exactly; q, scaled by a power of two per row, is exact in fp16 too, and P is
// rounded to fp16 (2^-11).  The page scales multiply the logits of a chunk and
// its P; O is kept relative to the largest value scale seen so far, so that P
// times scale stays within fp16.
#include "cache.cuh"

namespace attn {
namespace {

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// two e4m3 codes (low and high byte of the 16 bits) as two fp16, exactly
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// MT: 16-row tiles of an item.  HALF: only rows 0..7 of the one tile are used
// (bf16), the others carry the residue of P.
template <int D, bool E4M3, int MT, bool HALF>
struct Cfg {
  static constexpr int ROWS = HALF ? 8 : 16 * MT;
  static constexpr int WARPS = (D == 128 && !(E4M3 && MT == 1)) ? (HALF ? 7 : 6) : 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int EL = E4M3 ? 1 : 2;
  // 16-byte vectors a thread copies for the keys of a chunk; the values' are
  // as many, of 8 bytes for e4m3 at D = 64
  static constexpr int NK = kChunk * D * EL / 512;
  static constexpr int NV = (E4M3 && D == 64) ? 4 : NK;
  static constexpr int VB = (E4M3 && D == 64) ? 8 : 16;
  static constexpr int STAGE = NK * 512 + NV * VB * 32;
  static constexpr int SLOT_LD = D + 4;   // fp32 row stride of a partial result
  static constexpr int SLOT = ROWS * SLOT_LD * 4;
  static constexpr int BUDGET = 216 * 1024;
  static constexpr int RING_MAX = (BUDGET / WARPS - SLOT) / STAGE;
  static constexpr int STAGES = RING_MAX < 8 ? RING_MAX : 8;
  // (a warp's last partial goes into its drained ring)
  static constexpr int RING = STAGES * STAGE > SLOT ? STAGES * STAGE : SLOT;
  static_assert(STAGES >= 2 && WARPS * (RING + SLOT) <= BUDGET, "shared memory");
  static constexpr int SMEM = WARPS * (RING + SLOT);
};

// Chunks of an item of sequence q (all items of a sequence count the same, the
// causal ones with fewer visible keys too), and its items per KV head.
__device__ __forceinline__ int seq_chunks(const StepSeq& q) {
  return q.len > 0 ? (q.len + kChunk - 1) / kChunk : 1;   // 1: an item always writes its rows
}
template <int ROWS>
__device__ __forceinline__ int seq_blocks(const CacheFwdArgs& a, const StepSeq& q) {
  return static_cast<int>((static_cast<int64_t>(q.m) * a.s.group + ROWS - 1) / ROWS);
}

// A partial result: which item, and whether it holds the item's first / last
// chunk.
struct PartMeta {
  int kind;   // bit 0 valid, bit 1 begins, bit 2 ends
  int n, h, rb;
};

template <int D>
__device__ __forceinline__ void store_row8(__nv_bfloat16* dst, const float4& x, const float4& y,
                                           float f) {
  uint4 w;
  w.x = pack_bf16(x.x * f, x.y * f);
  w.y = pack_bf16(x.z * f, x.w * f);
  w.z = pack_bf16(y.x * f, y.y * f);
  w.w = pack_bf16(y.z * f, y.w * f);
  *reinterpret_cast<uint4*>(dst) = w;
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.f || l != l ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

template <int D, bool E4M3, int MT, bool HALF>
__global__ void __launch_bounds__(Cfg<D, E4M3, MT, HALF>::THREADS, 1)
    cache_fwd_kernel(const CacheFwdArgs a) {
  using C = Cfg<D, E4M3, MT, HALF>;
  constexpr int ROWS = C::ROWS;
  constexpr int NT = D / 8;                 // 8-column output tiles
  constexpr int VN = E4M3 ? (D == 64 ? 8 : 16) : 8;   // dims of a value vector
  constexpr int NH = D / (8 * VN);          // value vectors per key and thread
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t sh_pre[C::THREADS + 1];
  __shared__ int64_t sh_warp[C::WARPS];
  __shared__ float4 sh_scale[C::WARPS][C::STAGES];    // {k scale, v scale, valid keys, -}
  __shared__ PartMeta sh_meta[C::WARPS][2];
  __shared__ float2 sh_ml[C::WARPS][2][ROWS];

  const CacheStep& s = a.s;
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- every thread sums a slice of the sequences, a block scan joins them ----
  const int per = (s.num_seqs + C::THREADS - 1) / C::THREADS;
  int64_t mine = 0;
  {
    int bad = 0;
    const int n1 = min(s.num_seqs, static_cast<int>(threadIdx.x + 1) * per);
    for (int n = threadIdx.x * per; n < n1; ++n) {
      const StepSeq q = step_seq(s, n, &bad);
      mine += static_cast<int64_t>(s.heads_kv) * seq_blocks<ROWS>(a, q) * seq_chunks(q);
    }
    if (bad && s.err && blockIdx.x == 0) atomicOr(s.err, bad);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sh_warp[warp] = inc;
    if (lane < 2) sh_meta[warp][lane].kind = 0;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += sh_warp[w];
    sh_pre[threadIdx.x + 1] = before + inc;
    if (threadIdx.x == 0) sh_pre[0] = 0;
    __syncthreads();
  }
  const int64_t total = sh_pre[C::THREADS];
  int64_t quota = (total + gridDim.x - 1) / gridDim.x;
  if (quota < C::WARPS) quota = C::WARPS;
  const int64_t cta0 = min(total, quota * static_cast<int64_t>(blockIdx.x));
  const int64_t cta1 = min(total, cta0 + quota);
  const int64_t f0 = cta0 + (cta1 - cta0) * warp / C::WARPS;
  const int64_t f1 = cta0 + (cta1 - cta0) * (warp + 1) / C::WARPS;

  uint8_t* ring = smem + warp * (C::RING + C::SLOT);
  float* slot_a = reinterpret_cast<float*>(ring + C::RING);   // a part that began before f0
  float* slot_b = reinterpret_cast<float*>(ring);             // one that goes on past f1
  const uint32_t ring_u = smem_u32(ring);

  if (f0 < f1) {
    // ---- the item of chunk f0 ----
    int sl = 0;
    {
      int lo = 0, hi = C::THREADS - 1;   // last slice that starts at or before f0 and is not empty
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sh_pre[mid] <= f0) lo = mid; else hi = mid - 1;
      }
      sl = lo;
    }
    int n = sl * per;
    int64_t base = sh_pre[sl];
    StepSeq q = step_seq(s, n);
    int nc = seq_chunks(q), nb = seq_blocks<ROWS>(a, q);
    while (true) {
      const int64_t w = static_cast<int64_t>(s.heads_kv) * nb * nc;
      if (base + w > f0) break;
      base += w;
      ++n;
      q = step_seq(s, n);
      nc = seq_chunks(q);
      nb = seq_blocks<ROWS>(a, q);
    }
    int64_t off = f0 - base;
    int h = static_cast<int>(off / (static_cast<int64_t>(nb) * nc));
    off -= static_cast<int64_t>(h) * nb * nc;
    int rb = static_cast<int>(off / nc);
    int c0 = static_cast<int>(off - static_cast<int64_t>(rb) * nc);
    int64_t left = f1 - f0;

    while (true) {
      const int c1 = static_cast<int>(min(static_cast<int64_t>(nc), c0 + left));   // chunks [c0, c1)
      // last chunk that any of the block's rows sees
      const int rows_all = q.m * s.group;
      const int r_hi = min(rows_all, (rb + 1) * ROWS) - 1;
      const int vis_hi = min(q.len, a.causal ? q.pos0 + r_hi / s.group + 1 : q.len);
      const int ce = min(c1, vis_hi > 0 ? (vis_hi + kChunk - 1) / kChunk : 0);   // exclusive

      // ---- page look-ahead: lane l holds the page of column pg0 + l ----
      int pg0 = -1, pid = -1;
      float pks = 1.f, pvs = 1.f;
      const int32_t* trow = s.table + static_cast<int64_t>(n) * s.max_pages;
      auto fetch_pages = [&](int col) {
        pg0 = col;
        const int cc = col + lane;
        const int last = (q.len - 1) >> s.ps_shift;
        pid = cc <= last ? __ldg(trow + cc) : 0;
        if (pid < 0 || pid >= s.num_pages) {
          pid = -1;
          if (s.err) atomicOr(s.err, ATTN_DEVERR_INDEX_RANGE);
        }
        if constexpr (E4M3) {
          if (cc <= last && pid >= 0) {
            pks = __ldg(a.k_scale + static_cast<int64_t>(pid) * s.heads_kv + h);
            pvs = __ldg(a.v_scale + static_cast<int64_t>(pid) * s.heads_kv + h);
          }
        }
      };
      auto issue = [&](int c, int st) {
        const int col = (c * kChunk) >> s.ps_shift;
        if (pg0 < 0 || col >= pg0 + 32) fetch_pages(col);
        const int page = __shfl_sync(0xffffffffu, pid, col - pg0);
        int valid = min(q.len - c * kChunk, kChunk);
        if (page < 0) valid = 0;
        const float kf = E4M3 ? __shfl_sync(0xffffffffu, pks, col - pg0) : 1.f;
        const float vf = E4M3 ? __shfl_sync(0xffffffffu, pvs, col - pg0) : 1.f;
        if (lane == 0) sh_scale[warp][st] = make_float4(kf, vf, __int_as_float(valid), 0.f);
        const int64_t row = ((static_cast<int64_t>(max(page, 0)) * s.heads_kv + h) << s.ps_shift) +
                            ((c * kChunk) & ((1 << s.ps_shift) - 1));
        const uint8_t* kp = static_cast<const uint8_t*>(a.k_cache) + row * (D * C::EL);
        const uint8_t* vp = static_cast<const uint8_t*>(a.v_cache) + row * (D * C::EL);
        const uint32_t dst = ring_u + st * C::STAGE;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < C::NK / 2; ++j) {
            const int key = x * 8 + g;
            cp_async16(dst + ((x * (C::NK / 2) + j) * 32 + lane) * 16,
                       kp + key * (D * C::EL) + j * 64 + t * 16, key < valid ? 16u : 0u);
          }
        const uint32_t dv = dst + C::NK * 512;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int j = 0; j < C::NV / 4; ++j) {
            const int key = 2 * t + (x & 1) + (x >> 1) * 8;
            const uint8_t* src = vp + key * (D * C::EL) + j * 128 + g * C::VB;
            if constexpr (C::VB == 16)
              cp_async16(dv + ((x * (C::NV / 4) + j) * 32 + lane) * 16, src, key < valid ? 16u : 0u);
            else
              cp_async8(dv + (x * 32 + lane) * 8, src, key < valid ? 8u : 0u);
          }
      };
#pragma unroll
      for (int i = 0; i < C::STAGES - 1; ++i) {
        if (c0 + i < ce) issue(c0 + i, i);
        cp_async_commit();
      }

      // ---- the block's query rows ----
      uint32_t qf[MT][D / 16][4];
      float qs[MT][2];          // logit factor of the thread's rows
      int vis[MT][2];           // keys its rows see
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int r = rb * ROWS + mt * 16 + hh * 8 + g;
          const bool ok = r < rows_all && !(HALF && hh == 1);
          const int i = r / s.group;
          const __nv_bfloat16* src =
              a.q + (q.t0 + (ok ? i : 0)) * a.q_stride + (h * s.group + (ok ? r - i * s.group : 0)) * D;
          vis[mt][hh] = !ok ? 0 : min(q.len, a.causal ? q.pos0 + i + 1 : q.len);
          qs[mt][hh] = a.scale_log2;
          if constexpr (!E4M3) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (ok) w = *reinterpret_cast<const uint4*>(src + j * 32 + t * 8);
              qf[mt][2 * j][hh] = w.x;
              qf[mt][2 * j][2 + hh] = w.y;
              qf[mt][2 * j + 1][hh] = w.z;
              qf[mt][2 * j + 1][2 + hh] = w.w;
            }
          } else {
            uint32_t w[D / 8];
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {   // 16 dims: two vectors per 64 dims
              uint4 x = make_uint4(0u, 0u, 0u, 0u);
              if (ok) x = *reinterpret_cast<const uint4*>(src + (j >> 1) * 64 + t * 16 + (j & 1) * 8);
              w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                       fabsf(__uint_as_float(w[j] & 0xffff0000u))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // q 2^(8 - k), k the exponent of the row's largest element: below
            // 512, exact in fp16 down to 2^-32 of it and then within 2^-33 of it
            const int k = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
            const float f = __uint_as_float(static_cast<uint32_t>(8 - k + 127) << 23);
            qs[mt][hh] *= __uint_as_float(static_cast<uint32_t>(k - 8 + 127) << 23);
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              w[j] = pack_f16(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xffff0000u) * f);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              qf[mt][j][hh] = w[2 * j];
              qf[mt][j][2 + hh] = w[2 * j + 1];
            }
          }
        }

      float acc[MT][NT][4];
      float mrun[MT][2], lrun[MT][2], vref = 0.f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[mt][i][e] = 0.f;
        mrun[mt][0] = mrun[mt][1] = -INFINITY;
        lrun[mt][0] = lrun[mt][1] = 0.f;
      }

      // ---- the chunks ----
      int st = 0;
      for (int c = c0; c < ce; ++c) {
        {
          const int nx = c + C::STAGES - 1;
          int sx = st + C::STAGES - 1;
          if (sx >= C::STAGES) sx -= C::STAGES;
          if (nx < ce) issue(nx, sx);
          cp_async_commit();
        }
        cp_async_wait<C::STAGES - 1>();
        __syncwarp();
        const float4 sc = sh_scale[warp][st];
        const int kend = c * kChunk + __float_as_int(sc.z);   // keys of the chunk end here
        const uint32_t src = ring_u + st * C::STAGE;

        float x[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][nt][e] = 0.f;
#pragma unroll
        for (int j = 0; j < C::NK / 2; ++j)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const uint4 w = lds128(src + ((nt * (C::NK / 2) + j) * 32 + lane) * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            if constexpr (E4M3) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t b0 = e4m3x2_f16x2(ww[i]), b1 = e4m3x2_f16x2(ww[i] >> 16);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  const uint32_t(&q4)[4] = qf[mt][4 * j + i];
                  mma16816<true>(x[mt][nt], q4[0], q4[1], q4[2], q4[3], b0, b1);
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  const uint32_t(&q4)[4] = qf[mt][2 * j + i];
                  mma16816<false>(x[mt][nt], q4[0], q4[1], q4[2], q4[3], ww[2 * i], ww[2 * i + 1]);
                }
            }
          }

        // values' factor relative to the largest value scale so far
        float vratio = 1.f, vfac = 1.f;
        if constexpr (E4M3) {
          const bool any = __float_as_int(sc.z) > 0;
          const float vs = any ? sc.y : 0.f;
          if (vs > vref) {
            vratio = vref / vs;
            vref = vs;
          } else {
            vfac = vref > 0.f ? vs / vref : 0.f;
          }
        }
        uint32_t pa[MT][4];
        bool grow = vratio != 1.f;
        float alpha[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            alpha[mt][hh] = 1.f;
            if (HALF && hh == 1) continue;
            const float f = E4M3 ? qs[mt][hh] * sc.x : qs[mt][hh];
            const int lim = min(vis[mt][hh], kend) - c * kChunk - 2 * t;
            float y[4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float v = x[mt][nt][2 * hh + e] * f;
                y[2 * nt + e] = nt * 8 + e < lim ? v : -INFINITY;
              }
            float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(mrun[mt][hh], mx);
            const float ms = mn == -INFINITY ? 0.f : mn;
            alpha[mt][hh] = ex2(mrun[mt][hh] - ms);   // 0 while nothing has been seen
            grow |= mn > mrun[mt][hh];
            mrun[mt][hh] = mn;
            float p[4], sum;
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = ex2(y[e] - ms);
            sum = (p[0] + p[1]) + (p[2] + p[3]);
            lrun[mt][hh] = lrun[mt][hh] * alpha[mt][hh] + sum;
            if constexpr (E4M3) {
              pa[mt][hh] = pack_f16(p[0] * vfac, p[1] * vfac);
              pa[mt][2 + hh] = pack_f16(p[2] * vfac, p[3] * vfac);
            } else {
              pa[mt][hh] = pack_bf16(p[0], p[1]);
              pa[mt][2 + hh] = pack_bf16(p[2], p[3]);
              if constexpr (HALF) {   // the residues, as rows 8..15
                pa[mt][1] = pack_bf16(p[0] - __uint_as_float(pa[mt][0] << 16),
                                      p[1] - __uint_as_float(pa[mt][0] & 0xffff0000u));
                pa[mt][3] = pack_bf16(p[2] - __uint_as_float(pa[mt][2] << 16),
                                      p[3] - __uint_as_float(pa[mt][2] & 0xffff0000u));
              }
            }
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float a0 = alpha[mt][0] * vratio, a1 = (HALF ? alpha[mt][0] : alpha[mt][1]) * vratio;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              acc[mt][i][0] *= a0;
              acc[mt][i][1] *= a0;
              acc[mt][i][2] *= a1;
              acc[mt][i][3] *= a1;
            }
          }
        }

        // O += P V: keys (2t, 2t+1) are the low and high half of b0, (2t+8, 2t+9) of b1
        const uint32_t sv = src + C::NK * 512;
#pragma unroll
        for (int j = 0; j < NH; ++j) {
          uint32_t vw[4][VN * C::EL / 4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (C::VB == 16) {
              const uint4 w = lds128(sv + ((k * NH + j) * 32 + lane) * 16);
              vw[k][0] = w.x, vw[k][1] = w.y, vw[k][2] = w.z, vw[k][3] = w.w;
            } else {
              const uint2 w = lds64(sv + (k * 32 + lane) * 8);
              vw[k][0] = w.x, vw[k][1] = w.y;
            }
          }
          if constexpr (E4M3) {
#pragma unroll
            for (int i = 0; i < VN / 2; ++i) {   // dims 2i, 2i+1
              const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
              const uint32_t b0 = __byte_perm(vw[0][i / 2], vw[1][i / 2], sel);
              const uint32_t b1 = __byte_perm(vw[2][i / 2], vw[3][i / 2], sel);
              const uint32_t e0 = e4m3x2_f16x2(b0), o0 = e4m3x2_f16x2(b0 >> 16);
              const uint32_t e1 = e4m3x2_f16x2(b1), o1 = e4m3x2_f16x2(b1 >> 16);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<true>(acc[mt][j * VN + 2 * i], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], e0, e1);
                mma16816<true>(acc[mt][j * VN + 2 * i + 1], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], o0, o1);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < VN / 2; ++i) {
              const uint32_t e0 = __byte_perm(vw[0][i], vw[1][i], 0x5410u);
              const uint32_t o0 = __byte_perm(vw[0][i], vw[1][i], 0x7632u);
              const uint32_t e1 = __byte_perm(vw[2][i], vw[3][i], 0x5410u);
              const uint32_t o1 = __byte_perm(vw[2][i], vw[3][i], 0x7632u);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma16816<false>(acc[mt][j * VN + 2 * i], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], e0, e1);
                mma16816<false>(acc[mt][j * VN + 2 * i + 1], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3], o0, o1);
              }
            }
          }
        }
        if (++st == C::STAGES) st = 0;
      }
      cp_async_wait<0>();
      __syncwarp();

      // ---- the end of the item's part ----
      const bool begins = c0 == 0, ends = c1 == nc;
      const bool part_b = begins && !ends;     // goes on past f1: the warp's last part
      float* slot = part_b ? slot_b : slot_a;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < (HALF ? 1 : 2); ++hh) {
          float l = lrun[mt][hh];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          const int rl = mt * 16 + hh * 8 + g, r = rb * ROWS + rl;
          const float vf = E4M3 ? vref : 1.f;
          // columns 2t and 2t+1 of the VN MMAs of vector j: dims (8 j + 2t + col) VN + i
#pragma unroll
          for (int j = 0; j < NH; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int i = 0; i < VN; i += 8) {
                float o[8];
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                  const float(&ac)[4] = acc[mt][j * VN + i + z];
                  o[z] = (HALF ? ac[e] + ac[2 + e] : ac[2 * hh + e]) * vf;
                }
                const int d = (8 * j + 2 * t + e) * VN + i;
                const float4 lo = make_float4(o[0], o[1], o[2], o[3]);
                const float4 hi = make_float4(o[4], o[5], o[6], o[7]);
                if (begins && ends) {
                  if (r < rows_all) {
                    const int tok = r / s.group;
                    store_row8<D>(a.o + (static_cast<int64_t>(q.t0 + tok) * s.heads_q + h * s.group +
                                         (r - tok * s.group)) * D + d,
                                  lo, hi, l > 0.f || l != l ? 1.f / l : 0.f);
                  }
                } else {
                  float4* dst = reinterpret_cast<float4*>(slot + rl * C::SLOT_LD + d);
                  dst[0] = lo;
                  dst[1] = hi;
                }
              }
          if (t == 0) {
            if (begins && ends) {
              if (r < rows_all) {
                const int tok = r / s.group;
                a.lse[static_cast<int64_t>(h * s.group + (r - tok * s.group)) * s.tokens + q.t0 + tok] =
                    lse_of(mrun[mt][hh], l);
              }
            } else {
              sh_ml[warp][part_b][rl] = make_float2(mrun[mt][hh], l);
            }
          }
        }
      if (!(begins && ends) && lane == 0)
        sh_meta[warp][part_b] = PartMeta{1 | (begins ? 2 : 0) | (ends ? 4 : 0), n, h, rb};

      // ---- the next item ----
      left -= c1 - c0;
      if (left <= 0) break;
      c0 = 0;
      if (++rb == nb) {
        rb = 0;
        if (++h == s.heads_kv) {
          h = 0;
          do {
            ++n;
            q = step_seq(s, n);
            nb = seq_blocks<ROWS>(a, q);
          } while (nb == 0);
          nc = seq_chunks(q);
        }
      }
    }
  }
  __syncthreads();

  // ---- join the warps' parts (in order: part a, then part b of each warp) ----
  if (threadIdx.x < 2) a.part_meta[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  int i = 0;
  while (i < 2 * C::WARPS) {
    const PartMeta first = sh_meta[i >> 1][i & 1];
    if (!(first.kind & 1)) {
      ++i;
      continue;
    }
    // the chain of one item: parts until one ends it, or the last of the CTA
    int last = i, kind = first.kind;
    for (int k = i + 1; !(kind & 4) && k < 2 * C::WARPS; ++k) {
      const int kk = sh_meta[k >> 1][k & 1].kind;
      if (kk & 1) {
        last = k;
        kind |= kk & 4;
      }
    }
    const StepSeq q = step_seq(s, first.n);
    const bool whole = (kind & 6) == 6;
    const int which = (kind & 2) ? 1 : 0;   // the CTA's part that goes on, or came from before
    const int rows_all = q.m * s.group;
    for (int e = threadIdx.x; e < ROWS * (D / 8); e += C::THREADS) {
      const int rl = e / (D / 8), d = (e - rl * (D / 8)) * 8, r = first.rb * ROWS + rl;
      float m = -INFINITY;
      for (int k = i; k <= last; ++k)
        if (sh_meta[k >> 1][k & 1].kind & 1) m = fmaxf(m, sh_ml[k >> 1][k & 1][rl].x);
      const float ms = m == -INFINITY ? 0.f : m;
      float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
      float l = 0.f;
      for (int k = i; k <= last; ++k) {
        if (!(sh_meta[k >> 1][k & 1].kind & 1)) continue;
        const float2 ml = sh_ml[k >> 1][k & 1][rl];
        const float w = ex2(ml.x - ms);
        const float* sp = reinterpret_cast<const float*>(smem + (k >> 1) * (C::RING + C::SLOT) +
                                                         ((k & 1) ? 0 : C::RING)) +
                          rl * C::SLOT_LD + d;
        const float4 x = *reinterpret_cast<const float4*>(sp);
        const float4 y = *reinterpret_cast<const float4*>(sp + 4);
        l += w * ml.y;
        lo.x += w * x.x, lo.y += w * x.y, lo.z += w * x.z, lo.w += w * x.w;
        hi.x += w * y.x, hi.y += w * y.y, hi.z += w * y.z, hi.w += w * y.w;
      }
      if (whole) {
        if (r < rows_all) {
          const int tok = r / s.group, hd = first.h * s.group + (r - tok * s.group);
          store_row8<D>(a.o + (static_cast<int64_t>(q.t0 + tok) * s.heads_q + hd) * D + d, lo, hi,
                        l > 0.f || l != l ? 1.f / l : 0.f);
          if (d == 0) a.lse[static_cast<int64_t>(hd) * s.tokens + q.t0 + tok] = lse_of(m, l);
        }
      } else {
        const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + which) * ROWS + rl;
        float4* dst = reinterpret_cast<float4*>(a.part_o + at * D + d);
        dst[0] = lo;
        dst[1] = hi;
        if (d == 0) a.part_ml[at] = make_float2(m, l);
      }
    }
    if (!whole && threadIdx.x == 0)
      a.part_meta[2 * blockIdx.x + which] = make_int4(kind, first.n, first.h, first.rb);
    i = last + 1;
  }

  // ---- padding rows: at or past cu_seqlens[num_seqs] ----
  const int end = min(max(__ldg(s.cu + s.num_seqs), 0), s.tokens);
  const int64_t words = static_cast<int64_t>(s.tokens - end) * s.heads_q * (D / 8);
  uint4* o4 = reinterpret_cast<uint4*>(a.o + static_cast<int64_t>(end) * s.heads_q * D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * C::THREADS;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(C::THREADS) + threadIdx.x; w < words; w += step)
    o4[w] = make_uint4(0u, 0u, 0u, 0u);
  const int64_t pad = s.tokens - end, lses = pad * s.heads_q;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(C::THREADS) + threadIdx.x; w < lses; w += step)
    a.lse[w / pad * s.tokens + end + w % pad] = -INFINITY;
}

// Joins the items that several CTAs hold parts of.  Block b looks after the
// item that begins in CTA b and goes on in CTA b + 1 (there is at most one):
// its parts are CTA b's second, then the first of each following CTA until one
// ends the item.
constexpr int kJoinThreads = 512;

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const CacheFwdArgs a, int grid) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int POS = ROWS * (D / 4);                    // float4 positions of a partial
  constexpr int SPLIT = POS >= kJoinThreads ? 1 : kJoinThreads / POS;
  __shared__ float sh_w[kCacheCtas][ROWS];
  __shared__ float sh_l[ROWS], sh_m[ROWS];
  __shared__ float4 sh_o[SPLIT > 1 ? kJoinThreads : 1];
  const int b = blockIdx.x;
  const int4 meta = a.part_meta[2 * b + 1];
  if (!(meta.x & 1)) return;   // (kind bit 1, "begins", is set in every second part)
  int parts = 1;
  {
    // the following CTAs' first parts, until one ends the item
    __shared__ int sh_end;
    if (threadIdx.x == 0) sh_end = grid;
    __syncthreads();
    for (int c = b + 1 + threadIdx.x; c < grid; c += kJoinThreads)
      if (a.part_meta[2 * c].x & 4) atomicMin(&sh_end, c);
    __syncthreads();
    parts = min(sh_end, grid - 1) - b + 1;
  }
  const int warp = warp_id(), lane = lane_id();
  auto part_at = [&](int p) { return static_cast<int64_t>(p == 0 ? 2 * b + 1 : 2 * (b + p)) * ROWS; };
  for (int r = warp; r < ROWS; r += kJoinThreads / 32) {
    float m = -INFINITY;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_ml[part_at(p) + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float2 ml = a.part_ml[part_at(p) + r];
      const float w = ex2(ml.x - ms);
      sh_w[p][r] = w;
      l += w * ml.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) {
      sh_l[r] = l;
      sh_m[r] = m;
    }
  }
  __syncthreads();
  const CacheStep& s = a.s;
  const StepSeq q = step_seq(s, meta.y);
  const int rows_all = q.m * s.group;
  for (int e0 = 0; e0 < POS; e0 += kJoinThreads) {
    const int e = SPLIT > 1 ? threadIdx.x % POS : e0 + threadIdx.x;
    const int sp = SPLIT > 1 ? threadIdx.x / POS : 0;
    const int rl = e / (D / 4), d = (e - rl * (D / 4)) * 4, r = meta.w * ROWS + rl;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows_all) {
#pragma unroll 4
      for (int p = sp; p < parts; p += SPLIT) {
        const float w = sh_w[p][rl];
        const float4 x = *reinterpret_cast<const float4*>(a.part_o + (part_at(p) + rl) * D + d);
        o.x += w * x.x, o.y += w * x.y, o.z += w * x.z, o.w += w * x.w;
      }
    }
    if constexpr (SPLIT > 1) {
      sh_o[threadIdx.x] = o;
      __syncthreads();
      if (sp > 0) return;
#pragma unroll
      for (int k = 1; k < SPLIT; ++k) {
        const float4 x = sh_o[k * POS + e];
        o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
      }
    }
    if (r < rows_all) {
      const int tok = r / s.group, hd = meta.z * s.group + (r - tok * s.group);
      const float l = sh_l[rl], f = l > 0.f || l != l ? 1.f / l : 0.f;
      uint2 w;
      w.x = pack_bf16(o.x * f, o.y * f);
      w.y = pack_bf16(o.z * f, o.w * f);
      *reinterpret_cast<uint2*>(a.o + (static_cast<int64_t>(q.t0 + tok) * s.heads_q + hd) * D + d) = w;
      if (d == 0) a.lse[static_cast<int64_t>(hd) * s.tokens + q.t0 + tok] = lse_of(sh_m[rl], l);
    }
  }
}

template <int D, bool E4M3, int MT, bool HALF>
cudaError_t launch(const CacheFwdArgs& a, int grid, cudaStream_t st) {
  using C = Cfg<D, E4M3, MT, HALF>;
  auto kern = cache_fwd_kernel<D, E4M3, MT, HALF>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::THREADS, C::SMEM, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid - 1);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, C::ROWS>, a, grid);
}

template <int D, bool E4M3>
cudaError_t launch_rows(const CacheFwdArgs& a, int rows, int grid, cudaStream_t st) {
  switch (cache_fwd_rows(rows, E4M3)) {
    case 8:
      if constexpr (!E4M3) return launch<D, false, 1, true>(a, grid, st);
    case 16: return launch<D, E4M3, 1, false>(a, grid, st);
    default: return launch<D, E4M3, 2, false>(a, grid, st);
  }
}

}  // namespace

int cache_fwd_rows(int rows, bool e4m3) {
  if (rows <= 8 && !e4m3) return 8;
  return rows <= 16 ? 16 : 32;
}

cudaError_t launch_cache_fwd(const CacheFwdArgs& a, int head_dim, bool e4m3, int rows, int grid,
                             cudaStream_t st) {
  if (head_dim == 64)
    return e4m3 ? launch_rows<64, true>(a, rows, grid, st) : launch_rows<64, false>(a, rows, grid, st);
  return e4m3 ? launch_rows<128, true>(a, rows, grid, st) : launch_rows<128, false>(a, rows, grid, st);
}

}  // namespace attn

// Attention of new queries over the paged cache: few query rows against long
// key ranges, where every key and value has to cross HBM once and little is
// computed for each.
//
// Work.  An item is (sequence, KV head, block of up to ROWS query rows); the
// rows of a KV head are its (new token, query head of the group) pairs, token
// major, so the heads that share a key read it once.  An item's keys are cut
// into chunks of 32.  All items' chunks, in one line, are dealt to the CTAs in
// equal contiguous ranges, and a CTA's range to its warps, so every SM streams
// the same number of bytes whatever the sequences' lengths are.  An item that
// ends up in several warps is joined in shared memory, one that ends up in
// several CTAs by a second kernel, in a fixed order.
//
// A warp runs on its own, without block barriers: its lane 0 has TMA copy the
// keys and the values of a chunk, in turn, into the warp's ring, running ahead
// across items, and its lanes feed them to the tensor cores straight from
// 16-byte vectors.  The few query rows are the N side of mma.sync.m16n8k16, the
// keys and then the output dims its M side, so that 8 rows fill an MMA:
//   S^T = K Q^T: a thread of row g (of 8) and quad index t takes vector 4 j + t of
//     its keys (V = 8 bf16 or 16 codes); Q is loaded in the same order, in
//     which the contracted index is free;
//   O^T = V^T P^T: movmatrix turns P over, and the thread takes vector g of the
//     four keys that it holds probabilities of; rows g and g + 8 of the i-th MMA
//     are dims V g + 2 i and V g + 2 i + 1, and a byte permutation pairs keys.
// Row 2t of an 8-key tile is its key 2t, row 2t + 1 its key (2t) ^ 5: with the
// 128-byte swizzle, in which the copies arrive, both reads are then free of
// bank conflicts.  mma.sync has several times the rate that the HBM bound asks
// for here, and tcgen05, whose smallest tile has 64 rows and whose operands
// would have to be converted in shared memory, has nothing to gain.
//
// Bound by HBM once it runs (6.1 to 6.3 TB/s for bf16, of 6.8 measured for a copy), and
// around that by latency: about 5 us from the launch to the first keys (the dealing, the
// page lists, the first copies), 3 us for the join in a CTA and 3 for that of CTAs.
// 64 sequences of 15 to 8192 keys, 32 query heads on 8 KV heads of 128: 66 us for bf16
// (5.4 TB/s over all), 48 us for e4m3 (3.7 TB/s: half the bytes for 1.16 times the
// instructions, whose own latency the warps wait for); one sequence of 262144 e4m3 keys:
// 97 us (5.5 TB/s); one token over 1000 keys: 12 us, latency alone.
//
// Softmax statistics, sums and O are fp32.  bf16 caches: S is exact products in
// fp32; P goes in as hi + lo, two bf16 (2^-16): one would double the output's own
// rounding of 2^-8, and the MMAs are far from what bounds this kernel.  e4m3
// caches: codes convert to fp16 exactly, q nearly always (kQUp in cache.cuh), and
// P is rounded to fp16 once (2^-11, an eighth of the output's rounding).  The
// page scales multiply the logits of a page and its P, relative to the largest
// product of P and scale that the row has seen (kPHead in cache.cuh); O is kept
// in that unit.
#include "cache.cuh"

namespace attn {
namespace {

__device__ __forceinline__ void tma_load_2d(const CUtensorMap* m, uint64_t* bar, uint32_t dst,
                                            int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
// One fp32 into shared memory.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// An arrival on `bar` once this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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
// 8 x 8 matrix of 16-bit elements over a warp (row = lane / 4, columns 2 (lane % 4)
// and the next), transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// NQ: tiles of 8 query rows of an item.
template <int D, bool E4M3, int NQ>
struct Cfg {
  static constexpr int ROWS = 8 * NQ;
  static constexpr int WARPS = cache_warps(E4M3, ROWS);
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int EL = E4M3 ? 1 : 2;
  static constexpr int RB = D * EL < 128 ? D * EL : 128;   // bytes of a row in a panel
  static constexpr int PANELS = D * EL / RB;
  static constexpr int SLOT = kChunk * D * EL;             // keys or values of a chunk
  // 16 KB a warp, 128 KB an SM with 8 warps: 24 KB measured 3-7% slower, the copies queueing
  // longer at HBM in front of what an item's start waits for
  static constexpr int RING_MAX = 16384;
  static constexpr int SLOTS = RING_MAX / SLOT < 8 ? RING_MAX / SLOT : 8;
  static constexpr int PART_LD = D + 4;   // fp32 row stride of a partial result
  static constexpr int PART = ROWS * PART_LD * 4;
  // the ring; a warp's last partial goes into it once it is drained
  static constexpr int RING = SLOTS * SLOT;
  static_assert(RING >= PART && RING % 1024 == 0 && SLOTS >= 2, "ring");
  static constexpr int SMEM = WARPS * RING + 1024;
};

// Chunks that an item of sequence q counts for in the dealing (all items of a
// sequence the same, the causal ones with fewer visible keys too), and its
// items per KV head.  The two chunks more than it has stand for an item's own
// cost, its query rows and outputs, and give items without keys a place: 64
// decoding sequences of 15 to 8192 e4m3 keys took 58 us with one, 49 with two,
// 51 with three (the slowest warps hold ten items of one chunk each).
__device__ __forceinline__ int seq_chunks(const StepSeq& q) { return (q.len + kChunk - 1) / kChunk + 2; }
template <int ROWS>
__device__ __forceinline__ int seq_blocks(const CacheFwdArgs& a, const StepSeq& q) {
  return serves(a, q) ? (q.m * a.s.group + ROWS - 1) / ROWS : 0;
}

// An item and the walk over the items in the order in which they are dealt:
// sequence, KV head, row block.
struct Item {
  int n, h, rb;
  int nb, nc;   // row blocks per KV head, chunks per item
  StepSeq q;
};
template <int ROWS>
__device__ __forceinline__ void item_load(const CacheFwdArgs& a, Item& it) {
  it.q = step_seq(a.s, it.n);
  it.nc = seq_chunks(it.q);
  it.nb = seq_blocks<ROWS>(a, it.q);
}
// The next item; the caller knows that there is one.
template <int ROWS>
__device__ __forceinline__ void item_next(const CacheFwdArgs& a, Item& it) {
  if (++it.rb < it.nb) return;
  it.rb = 0;
  if (++it.h < a.s.heads_kv) return;
  it.h = 0;
  do {
    ++it.n;
    item_load<ROWS>(a, it);
  } while (it.nb == 0);
}
// Chunks of the item that some row of it sees.
template <int ROWS>
__device__ __forceinline__ int item_seen(const CacheFwdArgs& a, const Item& it) {
  const int r_hi = min(it.q.m * a.s.group, (it.rb + 1) * ROWS) - 1;
  const int vis = min(it.q.len, a.causal ? it.q.pos0 + r_hi / a.s.group + 1 : it.q.len);
  return vis > 0 ? (vis + kChunk - 1) / kChunk : 0;
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

template <int D, bool E4M3, int NQ>
__global__ void __launch_bounds__(Cfg<D, E4M3, NQ>::THREADS, 1)
    cache_fwd_kernel(const __grid_constant__ CacheFwdArgs a) {
  using C = Cfg<D, E4M3, NQ>;
  constexpr int ROWS = C::ROWS;
  constexpr int MT = D / 16;                // 16-dim output tiles
  constexpr int VN = E4M3 ? (D == 64 ? 8 : 16) : 8;   // dims of a value vector
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ int64_t sh_pre[C::THREADS + 1];
  __shared__ int64_t sh_warp[C::WARPS];
  __shared__ uint64_t bar_full[C::WARPS][C::SLOTS];
  __shared__ float4 sh_scale[C::WARPS][8];   // {k, v scale} of both halves of a chunk
  __shared__ int sh_bad[C::WARPS][8];        // halves (bits) without a page
  __shared__ PartMeta sh_meta[C::WARPS][2];
  __shared__ float2 sh_ml[C::WARPS][2][ROWS];
  __shared__ const float* sh_part[C::WARPS][2];
  __shared__ int sh_ld[C::WARPS][2];
  __shared__ float sh_w[2 * C::WARPS][ROWS];
  __shared__ float2 sh_sum[2 * C::WARPS][ROWS];
  __shared__ int abort_flag;

  const CacheStep& s = a.s;
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, t = lane & 3;
  AbortCtx ac{&abort_flag, s.err};
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane == 0) {
    // two arrivals: the bytes of TMA, and the scales (or a plain one)
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&bar_full[warp][i], 2);
    fence_mbar_init();
    if (warp == 0) {
      tma_prefetch_desc(&a.tm_k);
      tma_prefetch_desc(&a.tm_v);
    }
  }
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

  uint8_t* ring = smem + warp * C::RING;
  const uint32_t ring_u = smem_u32(ring);
  bool ok = true;

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
    Item it;
    it.n = sl * per;
    it.rb = 0;
    int64_t base = sh_pre[sl];
    item_load<ROWS>(a, it);
    while (true) {
      const int64_t w = static_cast<int64_t>(s.heads_kv) * it.nb * it.nc;
      if (base + w > f0) break;
      base += w;
      ++it.n;
      item_load<ROWS>(a, it);
    }
    const int64_t off = f0 - base;
    int c0;
    if (off >> 32) {
      const int64_t item = off / it.nc;
      c0 = static_cast<int>(off - item * it.nc);
      it.h = static_cast<int>(item / it.nb);
      it.rb = static_cast<int>(item - static_cast<int64_t>(it.h) * it.nb);
    } else {   // short divisions
      const uint32_t item = static_cast<uint32_t>(off) / it.nc;
      c0 = static_cast<int>(static_cast<uint32_t>(off) - item * it.nc);
      it.h = static_cast<int>(item / it.nb);
      it.rb = static_cast<int>(item) - it.h * it.nb;
    }
    int left = static_cast<int>(min(f1 - f0, static_cast<int64_t>(0x7fffffff)));

    // The raw words of row g of the item's tiles: vector 4 j + t of 8 dims; e4m3: half of
    // vector 4 (j / 2) + t of 16 dims.
    uint32_t qw[NQ][D / 8];
    auto load_q = [&](const Item& x) {
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
        const int r = x.rb * ROWS + nq * 8 + g, i = r / s.group;
        const bool in = r < x.q.m * s.group;
        const __nv_bfloat16* src = a.q + (x.q.t0 + (in ? i : 0)) * a.q_stride +
                                   (x.h * s.group + (in ? r - i * s.group : 0)) * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (in)
            v = *reinterpret_cast<const uint4*>(src + (E4M3 ? (j >> 1) * 64 + t * 16 + (j & 1) * 8
                                                            : j * 32 + t * 8));
          qw[nq][4 * j] = v.x, qw[nq][4 * j + 1] = v.y, qw[nq][4 * j + 2] = v.z, qw[nq][4 * j + 3] = v.w;
        }
      }
    };
    load_q(it);

    // ---- the copies, which run ahead of the computation, across items ----
    // lane l holds the page of column pg0 + l of item `cp`, and that of column l of
    // the next sequence
    Item cp = it;
    int cp_c = c0, cp_left = left;                 // next chunk; the warp's chunks from the item on
    int cp_span = min(cp.nc - c0, left);           // those of the item
    int cp_end = min(c0 + cp_span, item_seen<ROWS>(a, cp));   // end of its chunks to copy
    int pg0 = -1, pid = -1, npid = -1, cp_half = 0;       // cp_half: halves issued so far
    auto fetch_pages = [&](int col, bool ahead) {
      const int cc = col + lane;
      pg0 = col;
      if (!ahead) pid = cc < s.max_pages ? __ldg(s.table + static_cast<int64_t>(cp.n) * s.max_pages + cc) : -1;
      else pid = npid;
      if (col == 0)
        npid = cp.n + 1 < s.num_seqs && lane < s.max_pages
                   ? __ldg(s.table + static_cast<int64_t>(cp.n + 1) * s.max_pages + lane)
                   : -1;
      if (cc > (cp.q.len - 1) >> s.ps_shift) {
        pid = -1;
      } else if (pid < 0 || pid >= s.num_pages) {
        pid = -1;
        if (s.err) atomicOr(s.err, ATTN_DEVERR_INDEX_RANGE);
      }
    };
    // A sequence's query rows towards L2 (the first 32 KB), well before their loads
    auto prefetch_q = [&]() {
      const int words = min(min(cp.q.m, 256) * s.heads_q * (D / 64), 256);   // of 128 bytes
      for (int i = lane; i < words; i += 32) {
        const int tok = i / (s.heads_q * (D / 64));
        const __nv_bfloat16* p = a.q + (cp.q.t0 + tok) * a.q_stride + (i - tok * s.heads_q * (D / 64)) * 64;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
      }
    };
    // Half u: the keys (even) or values (odd) of a chunk.  False when all are issued.
    bool ahead = false;   // npid is of the sequence that begins
    int pg_seq = -2;      // the sequence before that of npid
    auto issue = [&]() -> bool {
      if (!(cp_half & 1)) {
        while (cp_c >= cp_end) {   // on to the next item
          const int n_old = cp.n;
          cp_left -= cp_span;
          if (cp_left <= 0) return false;
          item_next<ROWS>(a, cp);
          cp_c = 0;
          cp_span = min(cp.nc, cp_left);
          cp_end = min(cp_span, item_seen<ROWS>(a, cp));
          if (cp.n != n_old) {
            prefetch_q();
            ahead = cp.n == n_old + 1 && pg_seq == n_old;
            pg0 = -1;
          } else if (pg0 != 0) {
            pg0 = -1;
          }
        }
      }
      const int col0 = (cp_c * kChunk) >> s.ps_shift, col1 = (cp_c * kChunk + 16) >> s.ps_shift;
      if (pg0 < 0 || col1 >= pg0 + 32) {
        fetch_pages(col0, ahead && col0 == 0);
        ahead = false;
        if (col0 == 0) pg_seq = cp.n;
      }
      const int p0 = __shfl_sync(0xffffffffu, pid, col0 - pg0);
      const int p1 = __shfl_sync(0xffffffffu, pid, col1 - pg0);
      const bool values = cp_half & 1;
      if (lane == 0) {
        const uint32_t at = static_cast<uint32_t>(cp_half) % C::SLOTS;
        uint64_t* bar = &bar_full[warp][at];
        const int ix = (cp_half >> 1) & 7;
        if (!values) sh_bad[warp][ix] = (p0 < 0 ? 1 : 0) | (p1 < 0 ? 2 : 0);
        if (E4M3 && !values) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int page = b ? p1 : p0;
            float2* sc = reinterpret_cast<float2*>(&sh_scale[warp][ix]) + b;
            if (page >= 0) {
              const int64_t i = static_cast<int64_t>(page) * s.heads_kv + cp.h;
              cp_async4(smem_u32(sc), a.k_scale + i);
              cp_async4(smem_u32(sc) + 4, a.v_scale + i);
            } else {
              *sc = make_float2(0.f, 0.f);
            }
          }
          cp_async_arrive(bar);
        } else {
          mbar_arrive(bar);
        }
        const uint32_t dst = ring_u + at * C::SLOT;
        const CUtensorMap* m = values ? &a.tm_v : &a.tm_k;
        const int in_page = (cp_c * kChunk) & ((1 << s.ps_shift) - 1);
        const int y0 = ((p0 * s.heads_kv + cp.h) << s.ps_shift) + in_page;
        if (s.ps_shift > 4) {   // one box of 32 rows
          mbar_arrive_expect_tx(bar, p0 < 0 ? 0 : C::SLOT);
          if (p0 >= 0)
            for (int pn = 0; pn < C::PANELS; ++pn)
              tma_load_2d(m, bar, dst + pn * kChunk * 128, pn * 64, y0);
        } else {
          const int y1 = (p1 * s.heads_kv + cp.h) << 4;
          mbar_arrive_expect_tx(bar, (p0 < 0 ? 0 : C::SLOT / 2) + (p1 < 0 ? 0 : C::SLOT / 2));
          for (int pn = 0; pn < C::PANELS; ++pn) {
            if (p0 >= 0) tma_load_2d(m, bar, dst + pn * kChunk * 128, pn * 64, y0);
            if (p1 >= 0) tma_load_2d(m, bar, dst + pn * kChunk * 128 + 16 * C::RB, pn * 64, y1);
          }
        }
      }
      if (values) ++cp_c;
      ++cp_half;
      return true;
    };
    for (int u = 0; u < C::SLOTS; ++u)
      if (!issue()) break;
    __syncwarp();

    int half = 0;   // halves computed so far

    while (true) {
      const StepSeq q = it.q;
      const int nc = it.nc, n = it.n, h = it.h, rb = it.rb;
      const int c1 = min(nc, c0 + left);   // chunks [c0, c1), of which those below ce are seen
      const int ce = min(c1, item_seen<ROWS>(a, it));
      const int rows_all = q.m * s.group;

      // ---- the block's query rows: B fragments of row g, statistics of rows 2t and 2t + 1 ----
      uint32_t qf[NQ][D / 8];        // [2 step], [2 step + 1]: k low, k high
      float qs[NQ][2];               // logit factors
      int vis[NQ][2];                // keys that they see
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = rb * ROWS + nq * 8 + 2 * t + e;
          vis[nq][e] = r >= rows_all ? 0 : min(q.len, a.causal ? q.pos0 + r / s.group + 1 : q.len);
          qs[nq][e] = a.scale_log2;
        }
        uint32_t(&w)[D / 8] = qw[nq];
        if constexpr (E4M3) {
          float amax = 0.f;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)),
                                     fabsf(__uint_as_float(w[j] & 0xffff0000u))));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // q 2^(kQUp - k), k the exponent of the row's largest element
          const int k = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
          const float f = __uint_as_float(static_cast<uint32_t>(kQUp - k + 127) << 23);
          const float back = __uint_as_float(static_cast<uint32_t>(k - kQUp + 127) << 23);
          qs[nq][0] *= __shfl_sync(0xffffffffu, back, 8 * t);
          qs[nq][1] *= __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            w[j] = pack_f16(__uint_as_float(w[j] << 16) * f, __uint_as_float(w[j] & 0xffff0000u) * f);
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) qf[nq][j] = w[j];
      }
      left -= c1 - c0;
      const bool last_part = left <= 0;
      Item nx = it;
      if (!last_part) {   // the next item's rows arrive while this one is computed
        item_next<ROWS>(a, nx);
        load_q(nx);
      }

      float acc[NQ][MT][4];
      float mrun[NQ][2], lrun[NQ][2];
      float off[NQ][2];   // e4m3: R of kPHead, less mrun; O is in units of 2^(R - kPHead)
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nq][i][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mrun[nq][e] = -INFINITY;
          lrun[nq][e] = 0.f;
          off[nq][e] = -INFINITY;
        }
      }

      // ---- the chunks ----
      for (int c = c0; c < ce; ++c) {
        uint32_t at = static_cast<uint32_t>(half) % C::SLOTS;
        if (!mbar_wait_w(&bar_full[warp][at], (static_cast<uint32_t>(half) / C::SLOTS) & 1, ac)) {
          ok = false;
          break;
        }
        uint32_t src = ring_u + at * C::SLOT;
        const float4 sc = sh_scale[warp][(half >> 1) & 7];
        const int bad = sh_bad[warp][(half >> 1) & 7];
        const int key0 = c * kChunk;

        // S^T, tiles of 16 keys; row 2t of 8 is key 2t, row 2t + 1 key (2t) ^ 5
        float x[2][NQ][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][nq][e] = 0.f;
        const int krow = (g & 1) ? (g - 1) ^ 5 : g;
#pragma unroll
        for (int j = 0; j < D * C::EL / 64; ++j)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            uint32_t ww[2][4];
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const int row = mt * 16 + hi * 8 + krow;
              uint32_t off;
              if constexpr (C::RB == 128)
                off = (j >> 1) * (kChunk * 128) + row * 128 + ((((j & 1) * 4 + t) ^ krow) << 4);
              else
                off = row * 64 + ((t ^ ((krow >> 1) & 3)) << 4);
              const uint4 w = lds128(src + off);
              ww[hi][0] = w.x, ww[hi][1] = w.y, ww[hi][2] = w.z, ww[hi][3] = w.w;
            }
            if constexpr (E4M3) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = e4m3x2_f16x2(ww[0][i]), a2 = e4m3x2_f16x2(ww[0][i] >> 16);
                const uint32_t a1 = e4m3x2_f16x2(ww[1][i]), a3 = e4m3x2_f16x2(ww[1][i] >> 16);
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq)
                  mma16816<true>(x[mt][nq], a0, a1, a2, a3, qf[nq][8 * j + 2 * i], qf[nq][8 * j + 2 * i + 1]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq)
                  mma16816<false>(x[mt][nq], ww[0][2 * i], ww[1][2 * i], ww[0][2 * i + 1], ww[1][2 * i + 1],
                                  qf[nq][4 * j + 2 * i], qf[nq][4 * j + 2 * i + 1]);
            }
          }
        __syncwarp();
        issue();

        // the values' scales (0 without a page) and their log2
        const float vs0 = sc.y * kPUp, vs1 = sc.w * kPUp;
        const float lv0 = __log2f(sc.y), lv1 = __log2f(sc.w);
        const bool apart = E4M3 && sc.y != sc.w;
        constexpr int LO = E4M3 ? 1 : 2;   // P itself, or its hi and lo parts
        uint32_t pb[2][NQ][LO][2];         // B fragments of P^T: 16 keys each
        bool grow = false;
        float alpha[NQ][2];   // O's factor
        const bool dirty = bad != 0 || key0 + kChunk > q.len;
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          float p[2][2][2];   // [row][16-key tile][lower or upper 8 keys]
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f0 = E4M3 ? qs[nq][e] * sc.x : qs[nq][e], f1 = E4M3 ? qs[nq][e] * sc.z : qs[nq][e];
            float(&y)[2][2] = p[e];
            y[0][0] = x[0][nq][e] * f0;
            y[0][1] = x[0][nq][2 + e] * f0;
            y[1][0] = x[1][nq][e] * f1;
            y[1][1] = x[1][nq][2 + e] * f1;
            if (dirty || key0 + kChunk > vis[nq][e]) {
              const int lim = vis[nq][e] - key0;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (k * 8 + krow >= lim || (bad >> (k >> 1) & 1)) y[k >> 1][k & 1] = -INFINITY;
            }
            auto over_quads = [](float v) {
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            };
            float mx, m0, m1;   // the largest logit; e4m3: those of the two halves
            if (apart) {
              m0 = over_quads(fmaxf(y[0][0], y[0][1])), m1 = over_quads(fmaxf(y[1][0], y[1][1]));
              mx = fmaxf(m0, m1);
            } else {
              mx = over_quads(fmaxf(fmax3(y[0][0], y[0][1], y[1][0]), y[1][1]));
              m0 = m1 = mx;
            }
            const float mn = fmaxf(mrun[nq][e], mx);
            const float ms = mn == -INFINITY ? 0.f : mn;
            const float rise = mrun[nq][e] - ms;
            const float decay = ex2(rise);   // 0 while nothing has been seen
            float vf0, vf1;   // factors of P
            if constexpr (E4M3) {
              // log2 of the largest product, over the maximum (far below which their sum would drown)
              float top = m0 - ms + lv0;
              if (apart) top = fmaxf(top, m1 - ms + lv1);
              float& ref = off[nq][e];
              ref += rise;
              const bool up = top > ref + kPSlack;
              alpha[nq][e] = up ? ex2(ref - top) : 1.f;
              ref = up ? top : ref;
              grow |= up;
              // P of a factor past fp32 (a key of no weight under a scale that far above the
              // others', or no key at all) is 0
              const float f = ex2(-ref);
              vf0 = fminf(vs0 * f, 3.4e38f);
              vf1 = fminf(vs1 * f, 3.4e38f);
            } else {
              alpha[nq][e] = decay;
              grow |= mn > mrun[nq][e];
            }
            mrun[nq][e] = mn;
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k >> 1][k & 1] = ex2(y[k >> 1][k & 1] - ms);
            lrun[nq][e] = lrun[nq][e] * decay + ((y[0][0] + y[0][1]) + (y[1][0] + y[1][1]));
            if constexpr (E4M3) {
              y[0][0] *= vf0, y[0][1] *= vf0;
              y[1][0] *= vf1, y[1][1] *= vf1;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p0 = p[0][k >> 1][k & 1], p1 = p[1][k >> 1][k & 1];
            if constexpr (E4M3) {
              pb[k >> 1][nq][0][k & 1] = transpose8x8(pack_f16(p0, p1));
            } else {
              const uint32_t hi = pack_bf16(p0, p1);
              const uint32_t lo = pack_bf16(p0 - __uint_as_float(hi << 16),
                                            p1 - __uint_as_float(hi & 0xffff0000u));
              pb[k >> 1][nq][0][k & 1] = transpose8x8(hi);
              pb[k >> 1][nq][LO - 1][k & 1] = transpose8x8(lo);
            }
          }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            const float a0 = alpha[nq][0], a1 = alpha[nq][1];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              acc[nq][i][0] *= a0;
              acc[nq][i][1] *= a1;
              acc[nq][i][2] *= a0;
              acc[nq][i][3] *= a1;
            }
          }
        }

        // O^T += V^T P^T: keys (2t, (2t)^5) are the low and high half of a0 and a1, + 8 of a2 and a3
        ++half;
        at = static_cast<uint32_t>(half) % C::SLOTS;
        if (!mbar_wait_w(&bar_full[warp][at], (static_cast<uint32_t>(half) / C::SLOTS) & 1, ac)) {
          ok = false;
          break;
        }
        src = ring_u + at * C::SLOT;
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
          for (int j = 0; j < C::PANELS; ++j) {
            uint32_t vw[4][VN * C::EL / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = 8 * (k >> 1) + ((k & 1) ? (2 * t) ^ 5 : 2 * t);
              if constexpr (C::RB == 128) {
                const uint4 w = lds128(src + j * (kChunk * 128) + (i2 * 16 + row) * 128 + ((g ^ (row & 7)) << 4));
                vw[k][0] = w.x, vw[k][1] = w.y, vw[k][2] = w.z, vw[k][3] = w.w;
              } else {
                const uint2 w = lds64(src + (i2 * 16 + row) * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                vw[k][0] = w.x, vw[k][1] = w.y;
              }
              // values that no key has must not meet P = 0: they may be NaN
              if (dirty && (key0 + i2 * 16 + row >= q.len || (bad >> i2 & 1)))
#pragma unroll
                for (int i = 0; i < VN * C::EL / 4; ++i) vw[k][i] = 0u;
            }
#pragma unroll
            for (int i = 0; i < VN / 2; ++i) {   // dims 2i, 2i+1
              uint32_t a0, a1, a2, a3;
              if constexpr (E4M3) {
                const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
                const uint32_t b0 = __byte_perm(vw[0][i / 2], vw[1][i / 2], sel);
                const uint32_t b1 = __byte_perm(vw[2][i / 2], vw[3][i / 2], sel);
                a0 = e4m3x2_f16x2(b0), a1 = e4m3x2_f16x2(b0 >> 16);
                a2 = e4m3x2_f16x2(b1), a3 = e4m3x2_f16x2(b1 >> 16);
              } else {
                a0 = __byte_perm(vw[0][i], vw[1][i], 0x5410u);
                a1 = __byte_perm(vw[0][i], vw[1][i], 0x7632u);
                a2 = __byte_perm(vw[2][i], vw[3][i], 0x5410u);
                a3 = __byte_perm(vw[2][i], vw[3][i], 0x7632u);
              }
#pragma unroll
              for (int lo = 0; lo < LO; ++lo)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq)
                  mma16816<E4M3>(acc[nq][j * (VN / 2) + i], a0, a1, a2, a3, pb[i2][nq][lo][0],
                                 pb[i2][nq][lo][1]);
            }
          }
        ++half;
        __syncwarp();
        issue();
      }
      if (!ok) {   // a wait ran out: the copies in flight get a moment to land, then the warp leaves
        for (int u = half; u < cp_half; ++u) {
          const uint32_t bar = smem_u32(&bar_full[warp][static_cast<uint32_t>(u) % C::SLOTS]);
          const uint64_t t0 = globaltimer();
          while (!mbar_try_wait(bar, (static_cast<uint32_t>(u) / C::SLOTS) & 1) &&
                 globaltimer() - t0 < 10000000ull) {
          }
        }
        break;
      }

      // ---- the end of the item's part ----
      const bool begins = c0 == 0, ends = c1 == nc, whole = begins && ends;
      const int which = begins ? 1 : 0;   // 1: goes on past f1, 0: began before f0
      // the warp's last part may lie in its drained ring
      float* part = last_part ? reinterpret_cast<float*>(ring)
                              : a.stash + (static_cast<int64_t>(blockIdx.x) * C::WARPS + warp) * ROWS * D;
      const int ld = last_part ? C::PART_LD : D;
#pragma unroll
      for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = lrun[nq][e];
          l += __shfl_xor_sync(0xffffffffu, l, 4);
          l += __shfl_xor_sync(0xffffffffu, l, 8);
          l += __shfl_xor_sync(0xffffffffu, l, 16);
          const int rl = nq * 8 + 2 * t + e, r = rb * ROWS + rl, tok = r / s.group;
          const int hd = h * s.group + (r - tok * s.group);
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
          // e4m3: from O's unit to that of the row's maximum
          const float unit = E4M3 ? ex2(off[nq][e]) : 1.f;
          // dims VN (8 j + g) + 2 i (c0, c1 of MMA i of panel j) and + 2 i + 1 (c2, c3)
#pragma unroll
          for (int j = 0; j < C::PANELS; ++j)
#pragma unroll
            for (int i = 0; i < VN; i += 8) {
              float o[8];
#pragma unroll
              for (int z = 0; z < 8; ++z)
                o[z] = acc[nq][j * (VN / 2) + (i + z) / 2][(z & 1) * 2 + e] * (E4M3 ? kPDown : 1.f) * unit;
              const int d = (8 * j + g) * VN + i;
              const float4 lo = make_float4(o[0], o[1], o[2], o[3]);
              const float4 hi = make_float4(o[4], o[5], o[6], o[7]);
              if (!whole) {
                float4* dst = reinterpret_cast<float4*>(part + rl * ld + d);
                dst[0] = lo;
                dst[1] = hi;
              } else if (r < rows_all) {
                store_row8<D>(a.o + (static_cast<int64_t>(q.t0 + tok) * s.heads_q + hd) * D + d, lo, hi, inv);
              }
            }
          if (g == 0) {
            if (!whole) sh_ml[warp][which][rl] = make_float2(mrun[nq][e], l);
            else if (r < rows_all)
              a.lse[static_cast<int64_t>(hd) * s.tokens + q.t0 + tok] = lse_of(mrun[nq][e], l);
          }
        }
      if (!whole && lane == 0) {
        sh_meta[warp][which] = PartMeta{1 | (begins ? 2 : 0) | (ends ? 4 : 0), n, h, rb};
        sh_part[warp][which] = part;
        sh_ld[warp][which] = ld;
      }

      if (last_part) break;
      it = nx;
      c0 = 0;
    }
  }
  __syncthreads();

  // ---- join the warps' parts (in order: part a, then part b of each warp) ----
  // A chain is the parts of one item: from the first, or the one after an end, to the
  // next end, or the last of the CTA.
  {
    const int kind = lane < 2 * C::WARPS ? sh_meta[lane >> 1][lane & 1].kind : 0;
    const uint32_t valid = __ballot_sync(0xffffffffu, kind & 1), ends = __ballot_sync(0xffffffffu, kind & 4);
    const uint32_t before = valid & ((1u << lane) - 1);
    const bool starts = (kind & 1) && (before == 0 || (ends >> (31 - __clz(before)) & 1));
    const uint32_t first = __ballot_sync(0xffffffffu, starts);
    const int chains = __popc(first);
    // parts [i0, i1) of chain c
    auto chain = [&](int c, int& i0, int& i1) {
      uint32_t f = first;
      for (int k = 0; k < c; ++k) f &= f - 1;
      i0 = __ffs(f) - 1;
      f &= f - 1;
      i1 = f ? __ffs(f) - 1 : 2 * C::WARPS;
    };
    for (int e = threadIdx.x; e < chains * ROWS; e += C::THREADS) {
      const int c = e / ROWS, rl = e - c * ROWS;
      int i0, i1;
      chain(c, i0, i1);
      float m = -INFINITY, l = 0.f;
      for (int k = i0; k < i1; ++k)
        if (valid >> k & 1) m = fmaxf(m, sh_ml[k >> 1][k & 1][rl].x);
      const float ms = m == -INFINITY ? 0.f : m;
      for (int k = i0; k < i1; ++k)
        if (valid >> k & 1) {
          const float2 ml = sh_ml[k >> 1][k & 1][rl];
          const float w = ex2(ml.x - ms);
          l += w * ml.y;
          sh_w[k][rl] = w;
        }
      sh_sum[c][rl] = make_float2(m, l);
    }
    if (threadIdx.x < 2) a.part_meta[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
    __syncthreads();
    for (int e = threadIdx.x; e < chains * ROWS * (D / 8); e += C::THREADS) {
      const int c = e / (ROWS * (D / 8)), er = e - c * (ROWS * (D / 8));
      const int rl = er / (D / 8), d = (er - rl * (D / 8)) * 8;
      int i0, i1;
      chain(c, i0, i1);
      const PartMeta meta = sh_meta[i0 >> 1][i0 & 1];
      float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
#pragma unroll 4
      for (int k = i0; k < i1; ++k) {
        if (!(valid >> k & 1)) continue;
        const float w = sh_w[k][rl];
        const float* sp = sh_part[k >> 1][k & 1] + rl * sh_ld[k >> 1][k & 1] + d;
        const float4 x = *reinterpret_cast<const float4*>(sp);
        const float4 y = *reinterpret_cast<const float4*>(sp + 4);
        lo.x += w * x.x, lo.y += w * x.y, lo.z += w * x.z, lo.w += w * x.w;
        hi.x += w * y.x, hi.y += w * y.y, hi.z += w * y.z, hi.w += w * y.w;
      }
      // of the chain: whether it begins the item, ends it
      const int kinds = (meta.kind & 2) | ((ends & valid) >> i0 << (32 - (i1 - i0)) ? 4 : 0);
      const float2 ml = sh_sum[c][rl];
      if (kinds == 6) {
        const StepSeq q = step_seq(s, meta.n);
        const int r = meta.rb * ROWS + rl;
        if (r < q.m * s.group) {
          const int tok = r / s.group, hd = meta.h * s.group + (r - tok * s.group);
          store_row8<D>(a.o + (static_cast<int64_t>(q.t0 + tok) * s.heads_q + hd) * D + d, lo, hi,
                        ml.y > 0.f || ml.y != ml.y ? 1.f / ml.y : 0.f);
          if (d == 0) a.lse[static_cast<int64_t>(hd) * s.tokens + q.t0 + tok] = lse_of(ml.x, ml.y);
        }
      } else {
        // the CTA's part that goes on in the next (1), or came from the one before (0)
        const int which = kinds >> 1 & 1;
        const int64_t at = static_cast<int64_t>(blockIdx.x) * 2 + which;
        float4* dst = reinterpret_cast<float4*>(a.part_o) + (at * (D / 4) + d / 4) * ROWS + rl;
        dst[0] = lo;
        dst[ROWS] = hi;
        if (d == 0) a.part_ml[at * ROWS + rl] = ml;
        if (er == 0) a.part_meta[at] = make_int4(1 | kinds, meta.n, meta.h, meta.rb);
      }
    }
  }

  // ---- padding rows: at or past cu_seqlens[num_seqs] ----
  if (!a.pad) return;
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

// Joins the items that several CTAs hold parts of.  Block (b, y) looks after rows
// [y ROWS, (y + 1) ROWS) of the item that begins in CTA b and goes on in CTA b + 1
// (there is at most one): its parts are CTA b's second, then the first of each
// following CTA until one ends the item.
//
// A few KB a block: only latency counts, so that all CTAs' notes are read at once,
// and then the sequence, the statistics and the first kAhead parts' outputs.
constexpr int kJoinThreads = 256;   // few enough to wait beside the main kernel's CTA on an SM
constexpr int kAhead = 4;
static_assert(kCacheCtas <= kJoinThreads, "a thread reads each CTA's note");

template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads, 4)
    cache_join_kernel(const __grid_constant__ CacheFwdArgs a, int grid, int item_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int WARPS = kJoinThreads / 32;
  constexpr int POS = ROWS * (D / 4);                    // float4 positions, rows first
  constexpr int SPLIT = POS >= kJoinThreads ? 1 : kJoinThreads / POS;
  constexpr int PER = POS * SPLIT / kJoinThreads;        // positions of a thread
  constexpr int LD = D + 8;                              // bf16 row stride of the result
  __shared__ float sh_w[kCacheCtas][ROWS];
  __shared__ float sh_l[ROWS], sh_m[ROWS];
  __shared__ float4 sh_o[SPLIT > 1 ? kJoinThreads : 1];
  __shared__ __align__(16) __nv_bfloat16 sh_out[ROWS * LD];
  __shared__ int sh_end[WARPS];
  const CacheStep& s = a.s;
  const int b = blockIdx.x, warp = warp_id(), lane = lane_id(), base = blockIdx.y * ROWS;
  const int c = threadIdx.x;
  const int kind = c > b && c < grid ? a.part_meta[2 * c].x : 0;
  const int4 meta = a.part_meta[2 * b + 1];
  if (!(meta.x & 1)) return;   // (kind bit 1, "begins", is set in every second part)
  // the following CTAs' first parts, until one ends the item
  const uint32_t ends = __ballot_sync(0xffffffffu, kind & 4);
  if (lane == 0) sh_end[warp] = ends ? 32 * warp + __ffs(ends) - 1 : grid - 1;
  const StepSeq q = step_seq(s, meta.y);
  __syncthreads();
  int end = grid - 1;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) end = min(end, sh_end[w]);
  const int parts = end - b + 1;
  auto slot_of = [&](int p) { return static_cast<int64_t>(p == 0 ? 2 * b + 1 : 2 * (b + p)); };

  float4 ahead[PER][kAhead];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = SPLIT > 1 ? threadIdx.x % POS : i * kJoinThreads + threadIdx.x;
    const int sp = SPLIT > 1 ? threadIdx.x / POS : 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int p = sp + k * SPLIT;
      ahead[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < parts)
        ahead[i][k] = *(reinterpret_cast<const float4*>(a.part_o) +
                        (slot_of(p) * (D / 4) + e / ROWS) * item_rows + base + e % ROWS);
    }
  }
  // row rl of the item: row tr of its tile, query row r of the sequence and KV head
  const int rows_all = q.m * s.group;
  const int tile_size = item_rows / a.tiles, tile = base / tile_size, tr0 = base - tile * tile_size;
  auto row_of = [&](int rl) {
    return tr0 + rl < a.tile_rows ? (meta.w * a.tiles + tile) * a.tile_rows + tr0 + rl : rows_all;
  };
  float2 ml0[ROWS / WARPS];
#pragma unroll
  for (int i = 0; i < ROWS / WARPS; ++i) {
    ml0[i] = make_float2(-INFINITY, 0.f);
    if (lane < parts) ml0[i] = a.part_ml[slot_of(lane) * item_rows + base + warp + i * WARPS];
  }
  if (row_of(0) >= rows_all) return;   // (a tile's rows that exist come first)
#pragma unroll
  for (int i = 0; i < ROWS / WARPS; ++i) {
    const int r = warp + i * WARPS;
    if (row_of(r) >= rows_all) continue;
    float m = ml0[i].x;
    for (int p = lane + 32; p < parts; p += 32)
      m = fmaxf(m, a.part_ml[slot_of(p) * item_rows + base + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int p = lane; p < parts; p += 32) {
      const float2 ml = p < 32 ? ml0[i] : a.part_ml[slot_of(p) * item_rows + base + r];
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
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = SPLIT > 1 ? threadIdx.x % POS : i * kJoinThreads + threadIdx.x;
    const int sp = SPLIT > 1 ? threadIdx.x / POS : 0;
    const int rl = e % ROWS, d4 = e / ROWS;
    const bool in = row_of(rl) < rows_all;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int p = sp + k * SPLIT;
        if (p >= parts) break;
        const float w = sh_w[p][rl];
        const float4 x = ahead[i][k];
        o.x += w * x.x, o.y += w * x.y, o.z += w * x.z, o.w += w * x.w;
      }
#pragma unroll 4
      for (int p = sp + kAhead * SPLIT; p < parts; p += SPLIT) {
        const float w = sh_w[p][rl];
        const float4 x = *(reinterpret_cast<const float4*>(a.part_o) +
                           (slot_of(p) * (D / 4) + d4) * item_rows + base + rl);
        o.x += w * x.x, o.y += w * x.y, o.z += w * x.z, o.w += w * x.w;
      }
    }
    if constexpr (SPLIT > 1) {
      sh_o[threadIdx.x] = o;
      __syncthreads();
      if (sp == 0) {
#pragma unroll
        for (int k = 1; k < SPLIT; ++k) {
          const float4 x = sh_o[k * POS + e];
          o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
        }
      }
    }
    if (in && sp == 0) {
      const float l = sh_l[rl], f = l > 0.f || l != l ? 1.f / l : 0.f;
      *reinterpret_cast<uint2*>(sh_out + rl * LD + d4 * 4) =
          make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < ROWS * (D / 8); e += kJoinThreads) {
    const int rl = e / (D / 8), d = (e - rl * (D / 8)) * 8, r = row_of(rl);
    if (r >= rows_all) continue;
    const int tok = r / s.group, hd = meta.z * s.group + (r - tok * s.group);
    *reinterpret_cast<uint4*>(a.o + (static_cast<int64_t>(q.t0 + tok) * s.heads_q + hd) * D + d) =
        *reinterpret_cast<const uint4*>(sh_out + rl * LD + d);
    if (d == 0) a.lse[static_cast<int64_t>(hd) * s.tokens + q.t0 + tok] = lse_of(sh_m[rl], sh_l[rl]);
  }
}

template <int D, int ROWS>
cudaError_t launch_join(const CacheFwdArgs& a, int item_rows, int grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid - 1, item_rows / ROWS);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<D, ROWS>, a, grid, item_rows);
}

template <int D, bool E4M3, int NQ>
cudaError_t launch(const CacheFwdArgs& a, int grid, cudaStream_t st) {
  using C = Cfg<D, E4M3, NQ>;
  auto kern = cache_fwd_kernel<D, E4M3, NQ>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::THREADS, C::SMEM, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid < 2) return e;
  return launch_cache_join(a, D, C::ROWS, grid, st);
}

template <int D>
cudaError_t launch_dim(const CacheFwdArgs& a, bool e4m3, int item_rows, int grid, cudaStream_t st) {
  if (item_rows == 8)
    return e4m3 ? launch<D, true, 1>(a, grid, st) : launch<D, false, 1>(a, grid, st);
  return e4m3 ? launch<D, true, 2>(a, grid, st) : launch<D, false, 2>(a, grid, st);
}

}  // namespace

cudaError_t launch_cache_join(const CacheFwdArgs& a, int head_dim, int item_rows, int grid,
                              cudaStream_t st) {
  if (item_rows == 8)
    return head_dim == 64 ? launch_join<64, 8>(a, 8, grid, st) : launch_join<128, 8>(a, 8, grid, st);
  return head_dim == 64 ? launch_join<64, 16>(a, item_rows, grid, st)
                        : launch_join<128, 16>(a, item_rows, grid, st);
}

int cache_fwd_rows(int rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_cache_fwd(const CacheFwdArgs& a, int head_dim, bool e4m3, int item_rows,
                             int grid, cudaStream_t st) {
  return head_dim == 64 ? launch_dim<64>(a, e4m3, item_rows, grid, st)
                        : launch_dim<128>(a, e4m3, item_rows, grid, st);
}

}  // namespace attn

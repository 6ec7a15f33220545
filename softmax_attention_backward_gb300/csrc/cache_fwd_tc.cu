// Attention of many new queries over the paged cache (chunks of prompts, drafts
// of many tokens, and the decoding sequences that share a call with them): the
// tcgen05 counterpart of cache_fwd.cu, with the pipeline of attn_fwd.cu.
//
// An item is (sequence, KV head, two tiles of up to 128 query rows).  A tile's
// rows are TT = 128 / group new tokens times the group's query heads, token major:
// one TMA box of q puts them into shared memory in that order, and the keys are
// read once for all heads that share them.  Keys come in chunks of BN rows, which
// TMA gathers from the pages.  Roles as in attn_fwd: warp 8 copies, warps 9 and 10
// issue the MMAs of tile 0 and 1 (S = Q K^T from shared memory, O += P V with P
// from TMEM), warps 0..3 and 4..7 run the online softmax, a row per thread.
//
// The items' chunks that some row sees, with a few more for an item's own cost,
// form one line that is dealt to the CTAs in equal contiguous ranges, so that a
// step fills the GPU whatever its shape is: one short chunk over a long cached
// prefix as much as many prompts.  An item cut by a range's end leaves fp32 partial
// results (O unnormalized, row maximum, row sum), which the second kernel of
// cache_fwd.cu joins in a fixed order.
//
// Rows of a page past the sequence's length may hold anything: their logits are
// masked, and their values are zeroed in shared memory before the MMA reads them
// (0 * NaN).  The last chunk of an item alone pays for that.
//
// e4m3: all operands are fp16, in which codes are exact.  Warp 8 brings the codes of
// a chunk by bulk copies into a ring of their own, warps 11..14 convert them into
// the slots that the MMAs read; the softmax warps bring and scale their rows of q.
// The scales of 16-key groups enter with the softmax: the key scale as a factor of
// the logits, log2 of the value scale as a summand in the exponent of P, which the
// row sum takes off again (kPHead in cache.cuh says in what unit P and O are held).
//
// Rounding.  Statistics, sums and O are fp32, and the row sum takes P unrounded.  bf16: P
// goes in as one bf16 (2^-8), as in attn_fwd: a second one for the rest would make the
// MMAs half as many again, which at the measured GEMM rate is longer (480 us for the chunk
// below) than all that the kernel takes now.  e4m3: one fp16 (2^-11).
//
// Bound by the softmax (bf16: 1.36 PFLOP/s, 455 us, for 2 x 2048 new tokens over
// 8192 cached ones, 32 query heads of 128, 70% of the measured GEMM rate; the dense
// forward's own rate is 1.27), and for short items by what an item costs beside its
// chunks: about 5 us until the first logits, 2 us for the outputs, 10 us for the join of
// partial results (12 sequences of up to 700 new tokens over up to 4000 keys: 52 us).
// e4m3: 584 us and 77 us for the same two; with the conversion, four scales a chunk
// and 128 registers a thread it issues 1.7 times the instructions, which makes a
// chunk 1.2 us long instead of 0.95.  Converting by shifts and masks (to bf16 for the
// keys, so that q needs none) takes three instructions for one and a check for NaN:
// 827 us without the check, 1414 with it, in the four warps that registers leave for it.
#include "cache.cuh"
#include "launch.h"

namespace attn {
namespace {

template <int D, bool E4M3>
struct TcCfg {
  static constexpr int BM = 128;
  static constexpr int BN = D == 128 || E4M3 ? 64 : 128;   // bf16: as in attn_fwd
  static constexpr int PANELS = D / 64;
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int NSLOT = 6;
  static constexpr int QBUFS = E4M3 ? 1 : 2;   // query tile pairs
  // e4m3: warp 8 brings the codes into a ring of RAW chunks of keys or values, which
  // warps 11..14 convert into the slots
  static constexpr int RAW = 4, RAW_BYTES = E4M3 ? BN * D : 0;
  static constexpr int SMEM = QBUFS * 2 * Q_BYTES + NSLOT * KV_BYTES + RAW * RAW_BYTES + 1024;
  static constexpr int THREADS = E4M3 ? 480 : 352;
  static constexpr int INFOS = 2;   // parts announced at a time
  static_assert(E4M3 || QBUFS == INFOS, "a bf16 part's queries come with its announcement");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_S0 = 0, COL_S1 = BN, COL_O0 = 256, COL_O1 = 256 + D;
  static constexpr uint32_t COL_P0 = D == 128 ? 2 * BN : 256 + 2 * D, COL_P1 = COL_P0 + BN / 2;
  static_assert(D != 128 || 3 * BN <= 256, "S and P of both tiles below O");
  static_assert(D == 128 || 256 + 2 * D + BN <= 512, "TMEM budget");
  static_assert(SMEM <= 227 * 1024 - 700, "shared memory");
};

// Chunks by which an item counts more in the dealing than it has, for its query
// tiles, its first and last chunk and its outputs: 12 sequences of up to 700 new
// tokens over up to 4000 keys took 52.2, 52.5, 54.9 us with 4, 5, 7 (bf16) and 88, 85,
// 78 us with 5, 7, 10 (e4m3, whose queries the softmax warps convert), 2 x 4096 fresh
// tokens 257, 253, 258 us with 4, 5, 7 (77 and 243 us by now, with 10 and 5).
template <bool E4M3>
constexpr int kItemCost = E4M3 ? 10 : 5;

// A contiguous copy, 16-byte aligned on both sides and a multiple of 16 bytes.
__device__ __forceinline__ void bulk_load(uint64_t* bar, void* dst, const void* src, uint32_t bytes) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_2d(const CUtensorMap* m, uint64_t* bar, void* dst, int c0,
                                            int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

struct TcItem {
  int n, h, rb, nb;   // sequence, KV head, block of two tiles, blocks of the sequence
  StepSeq q;
  int seen[2];        // chunks that the tiles' rows see
  int nc;             // chunks of the item in the dealing
};

// Chunks that tile `tile` (of TT tokens) of a sequence sees.
template <int BN>
__device__ __forceinline__ int tile_seen(const CacheFwdArgs& a, const StepSeq& q, int tile) {
  const int tok0 = tile * a.tile_tokens;
  if (tok0 >= q.m) return 0;
  const int hi = min(q.m, tok0 + a.tile_tokens);
  const int vis = a.causal ? min(q.len, q.pos0 + hi) : q.len;
  return vis > 0 ? (vis + BN - 1) / BN : 0;
}
template <int BN, bool E4M3>
__device__ __forceinline__ void item_block(const CacheFwdArgs& a, TcItem& it) {
  it.seen[0] = tile_seen<BN>(a, it.q, 2 * it.rb);
  it.seen[1] = tile_seen<BN>(a, it.q, 2 * it.rb + 1);
  it.nc = max(it.seen[0], it.seen[1]) + kItemCost<E4M3>;
}
__device__ __forceinline__ int seq_blocks(const CacheFwdArgs& a, const StepSeq& q) {
  return serves(a, q) ? (q.m + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens) : 0;
}
// The next item; the caller knows that there is one.
template <int BN, bool E4M3>
__device__ __forceinline__ void item_next(const CacheFwdArgs& a, TcItem& it) {
  if (++it.rb == it.nb) {
    it.rb = 0;
    if (++it.h == a.s.heads_kv) {
      it.h = 0;
      do {
        ++it.n;
        it.q = step_seq(a.s, it.n);
        it.nb = seq_blocks(a, it.q);
      } while (it.nb == 0);
    }
  }
  item_block<BN, E4M3>(a, it);
}
// Chunks in the dealing of block rb of a sequence (its last token sees most).
template <int BN, bool E4M3>
__device__ __forceinline__ int block_chunks(const CacheFwdArgs& a, const StepSeq& q, int rb) {
  const int vis = a.causal ? min(q.len, q.pos0 + min(q.m, (rb + 1) * 2 * a.tile_tokens)) : q.len;
  return (vis > 0 ? (vis + BN - 1) / BN : 0) + kItemCost<E4M3>;
}
// Those of one KV head of a sequence, summed by the lanes of a warp (q the same in all).
template <int BN, bool E4M3>
__device__ __forceinline__ int64_t head_chunks_warp(const CacheFwdArgs& a, const StepSeq& q) {
  const int nb = seq_blocks(a, q);
  int64_t w = 0;
  for (int rb = lane_id(); rb < nb; rb += 32) w += block_chunks<BN, E4M3>(a, q, rb);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}
// The same for a sequence per lane (q.m = 0: none), sequences of many blocks by the warp.
template <int BN, bool E4M3>
__device__ __forceinline__ int64_t head_chunks(const CacheFwdArgs& a, const StepSeq& q) {
  const int nb = seq_blocks(a, q);
  int64_t w = 0;
  for (int rb = 0; rb < (nb <= 16 ? nb : 0); ++rb) w += block_chunks<BN, E4M3>(a, q, rb);
  for (uint32_t many = __ballot_sync(0xffffffffu, nb > 16); many; many &= many - 1) {
    const int src = __ffs(many) - 1;
    StepSeq x;
    x.t0 = 0;
    x.m = __shfl_sync(0xffffffffu, q.m, src);
    x.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
    x.len = __shfl_sync(0xffffffffu, q.len, src);
    const int64_t sum = head_chunks_warp<BN, E4M3>(a, x);
    if (static_cast<int>(lane_id()) == src) w = sum;
  }
  return w;
}

// The part of an item that a CTA computes: chunks [c0, c0 + n_kv), of which tile
// t's rows see the first n_w[t].
struct Part {
  int c0, span;   // span: chunks in the dealing
  int n_w[2], n_kv;
};
__device__ __forceinline__ Part part_of(const TcItem& it, int c0, int64_t left) {
  Part p;
  p.c0 = c0;
  p.span = static_cast<int>(min(static_cast<int64_t>(it.nc - c0), left));
  for (int t = 0; t < 2; ++t) p.n_w[t] = max(0, min(it.seen[t], c0 + p.span) - c0);
  p.n_kv = max(p.n_w[0], p.n_w[1]);
  return p;
}

// What warp 8 tells the other roles about a part, in shared memory beside its query
// tiles: they read it when those have arrived.
struct PartInfo {
  int n_w[2], n_kv, c0;
  StepSeq q;
  int n, h, rb;
  int kind;   // bit 0: a part, bit 1: begins its item, bit 2: ends it; 0: no more parts
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(TcCfg<D, E4M3>::THREADS, 1)
    cache_fwd_tc_kernel(const __grid_constant__ CacheFwdArgs a) {
  using C = TcCfg<D, E4M3>;
  constexpr int BN = C::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sQ = smem;                                // QBUFS x 2 tiles
  uint8_t* sRing = sQ + C::QBUFS * 2 * C::Q_BYTES;   // NSLOT chunks of keys or values

  __shared__ uint64_t bar_q[C::INFOS], bar_qempty[C::INFOS], bar_qready[2];
  __shared__ uint64_t bar_full[C::NSLOT], bar_empty[C::NSLOT], bar_tail;
  __shared__ uint64_t bar_s[2], bar_p[2], bar_o[2], bar_sfree[2], bar_stagger;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ int sh_bad[32];   // by chunk: 16-key groups (bits) without a page
  // e4m3, by chunk: the key scale and log2 of the value scale of its 16-key groups; by raw
  // chunk: its barriers, which rows exist (a bit each), and whether it is one at all
  __shared__ float2 sh_scale[E4M3 ? 32 : 1][4];
  __shared__ uint64_t bar_rfull[C::RAW], bar_rempty[C::RAW], sh_rows[C::RAW];
  __shared__ int sh_more[C::RAW];
  __shared__ int64_t sh_warp[C::THREADS / 32 + 1];
  __shared__ TcItem sh_item;
  __shared__ PartInfo sh_info[C::INFOS];
  __shared__ int sh_c0;
  __shared__ int64_t sh_left;

  const CacheStep& s = a.s;
  const int warp = warp_id(), lane = lane_id();
  AbortCtx ac{&abort_flag, s.err};
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- setup ---------------------------------------------------------------
  if (threadIdx.x == 0) {
    abort_flag = 0;
    sh_left = 0;
    for (int b = 0; b < C::INFOS; ++b) {
      mbar_init(&bar_q[b], 1);
      mbar_init(&bar_qempty[b], 10);     // released by both issuers and 8 softmax warps
    }
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&bar_full[i], E4M3 ? 128 : 1);
      mbar_init(&bar_empty[i], 2);       // released by both issuers
    }
    mbar_init(&bar_tail, 1);
    if constexpr (E4M3)
      for (int i = 0; i < C::RAW; ++i) {
        mbar_init(&bar_rfull[i], 1);
        mbar_init(&bar_rempty[i], 4);    // released by the converting warps
      }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w], 128);
      mbar_init(&bar_o[w], 1);
      mbar_init(&bar_sfree[w], 128);
      mbar_init(&bar_qready[w], 128);
    }
    mbar_init(&bar_stagger, 1);
    fence_mbar_init();
    if constexpr (!E4M3) {
      tma_prefetch_desc(&a.tm_q);
      tma_prefetch_desc(&a.tm_k);
      tma_prefetch_desc(&a.tm_v);
    }
  }
  if (threadIdx.x < 2) a.part_meta[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
  if (warp == 9) tmem_alloc(&tmem_base_sh, C::TMEM_COLS);

  // ---- the dealing: every thread sums a slice of the sequences, the warp whose slices
  // hold the CTA's first chunk finds its item ----
  {
    const int per = (s.num_seqs + C::THREADS - 1) / C::THREADS;
    const int n0 = threadIdx.x * per;
    int64_t mine = 0;
    int bad = 0;
    for (int n = n0; n < n0 + per; ++n) {
      StepSeq q = {0, 0, 0, 0};
      if (n < s.num_seqs) q = step_seq(s, n, &bad);
      mine += s.heads_kv * head_chunks<BN, E4M3>(a, q);
    }
    if (bad && s.err && blockIdx.x == 0) atomicOr(s.err, bad);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sh_warp[warp] = inc;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int64_t total = 0, before = 0;
    for (int w = 0; w < C::THREADS / 32; ++w) {
      if (w == warp) before = total;
      total += sh_warp[w];
    }
    const int64_t quota = (total + gridDim.x - 1) / gridDim.x;
    const int64_t f0 = min(total, quota * static_cast<int64_t>(blockIdx.x));
    const int64_t f1 = min(total, f0 + quota);
    const int64_t end = before + inc;
    const uint32_t who = __ballot_sync(0xffffffffu, f0 < f1 && f0 >= end - mine && f0 < end);
    if (who) {
      const int src = __ffs(who) - 1;
      TcItem it;
      int64_t off = __shfl_sync(0xffffffffu, f0 - (end - mine), src);
      for (it.n = __shfl_sync(0xffffffffu, n0, src);; ++it.n) {
        it.q = step_seq(s, it.n);
        const int64_t w = head_chunks_warp<BN, E4M3>(a, it.q);
        if (off < s.heads_kv * w) {
          it.h = static_cast<int>(off / w);
          off -= it.h * w;
          break;
        }
        off -= s.heads_kv * w;
      }
      it.nb = seq_blocks(a, it.q);
      for (int rb = lane;; rb += 32) {
        const int64_t c = rb < it.nb ? block_chunks<BN, E4M3>(a, it.q, rb) : 0;
        int64_t sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += x;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, off < sum);
        if (in) {
          const int l = __ffs(in) - 1;
          it.rb = __shfl_sync(0xffffffffu, rb, l);
          off -= __shfl_sync(0xffffffffu, sum - c, l);
          break;
        }
        off -= __shfl_sync(0xffffffffu, sum, 31);
      }
      item_block<BN, E4M3>(a, it);
      int64_t left = f1 - f0;
      if (off > 0 && off >= max(it.seen[0], it.seen[1])) {   // the CTA before has all of the item
        left -= it.nc - off;
        off = 0;
        if (left > 0) item_next<BN, E4M3>(a, it);
      }
      if (lane == 0) {
        sh_item = it;
        sh_c0 = static_cast<int>(off);
        sh_left = max(left, static_cast<int64_t>(0));
      }
    }
    __syncthreads();
  }
  const uint32_t tmem = tmem_base_sh;
  const int64_t range = sh_left;   // chunks of the CTA

  if (warp == 8) {
    // ---------------- copies (warp-uniform, lane 0 issues) ----------------
    if (range > 0) {
      const int box = min(BN, 1 << s.ps_shift), boxes = BN / box;
      const int tile_bytes = a.tile_tokens * s.group * 128 * C::PANELS;
      auto issue_q = [&](const TcItem& it, const Part& pt, int icq) {
        if (lane != 0) return;
        const int qb = icq % C::INFOS;
        PartInfo f;
        f.n_w[0] = pt.n_w[0], f.n_w[1] = pt.n_w[1], f.n_kv = pt.n_kv, f.c0 = pt.c0;
        f.q = it.q, f.n = it.n, f.h = it.h, f.rb = it.rb;
        f.kind = 1 | (pt.c0 == 0 ? 2 : 0) | (pt.c0 + pt.span >= max(it.seen[0], it.seen[1]) ? 4 : 0);
        sh_info[qb] = f;
        if constexpr (E4M3) {   // (the softmax warps bring the rows)
          mbar_arrive(&bar_q[qb]);
          return;
        }
        mbar_arrive_expect_tx(&bar_q[qb], 2 * tile_bytes);
        for (int t = 0; t < 2; ++t)
          for (int pn = 0; pn < C::PANELS; ++pn)
            tma_load_3d(&a.tm_q, &bar_q[qb], sQ + (qb * 2 + t) * C::Q_BYTES + pn * C::BM * 128, pn * 64,
                        it.h * s.group, it.q.t0 + (2 * it.rb + t) * a.tile_tokens);
      };
      // the walk: item, part, next
      auto advance = [&](TcItem& it, Part& pt, int64_t& left) -> bool {
        left -= pt.span;
        if (left <= 0) return false;
        item_next<BN, E4M3>(a, it);
        pt = part_of(it, 0, left);
        return true;
      };
      TcItem it = sh_item, nx;
      int64_t left = range;
      Part pt = part_of(it, sh_c0, left), pn_;
      int ic = 0, gring = 0, gchunk = 0, tails = 0;
      // lane l holds the page of column pg0 + l of sequence pg_n, e4m3: and its scales for
      // KV head pg_h
      int pg0 = -1, pg_n = -1, pg_h = -1, pid = -1;
      float pks = 1.f, pvs = -INFINITY;
      bool ok = mbar_wait_w(&bar_qempty[0], 1, ac);
      if (ok) issue_q(it, pt, 0);
      while (ok) {
        nx = it;
        pn_ = pt;
        int64_t left_nx = left;
        const bool have_next = advance(nx, pn_, left_nx);
        bool q_pending = have_next;
        const int nqb = (ic + 1) % C::INFOS;
        const uint32_t nq_par = (((ic + 1) / C::INFOS) & 1) ^ 1;
        for (int c = 0; ok && c < pt.n_kv; ++c, ++gchunk) {
          const int kv0 = (pt.c0 + c) * BN;
          // pages of the chunk: one, or `boxes` of them
          const int col0 = kv0 >> s.ps_shift;
          if (q_pending && mbar_test_wait_w(smem_u32(&bar_qempty[nqb]), nq_par)) {
            issue_q(nx, pn_, ic + 1);
            q_pending = false;
          }
          if (pg_n != it.n || col0 < pg0 || col0 + boxes > pg0 + 32) {
            pg_n = it.n;
            pg0 = col0;
            const int cc = col0 + lane;
            pid = -1;
            if (cc <= (it.q.len - 1) >> s.ps_shift) {
              pid = __ldg(s.table + static_cast<int64_t>(it.n) * s.max_pages + cc);
              if (pid < 0 || pid >= s.num_pages) {
                pid = -1;
                if (s.err) atomicOr(s.err, ATTN_DEVERR_INDEX_RANGE);
              }
            }
            pg_h = -1;
          }
          if constexpr (E4M3) {
            if (pg_h != it.h) {
              pg_h = it.h;
              pks = 1.f, pvs = -INFINITY;
              if (pid >= 0) {
                pks = __ldg(a.k_scale + static_cast<int64_t>(pid) * s.heads_kv + it.h);
                pvs = __log2f(__ldg(a.v_scale + static_cast<int64_t>(pid) * s.heads_kv + it.h));
              }
            }
            // the scales of the chunk's groups of 16 keys (lanes 0..3)
            const int key0 = kv0 + 16 * (lane & 3), col = key0 >> s.ps_shift;
            const float ks = __shfl_sync(0xffffffffu, pks, col - pg0);
            const float vs = __shfl_sync(0xffffffffu, pvs, col - pg0);
            if (lane < 4) sh_scale[gchunk & 31][lane] = make_float2(ks, vs);
            __syncwarp();
          }
          // bits of the boxes that have a page; the y coordinate of lane l's box
          const uint32_t have = (__ballot_sync(0xffffffffu, pid >= 0) >> (col0 - pg0)) & ((1u << boxes) - 1);
          const int mine = __shfl_sync(0xffffffffu, pid, (col0 - pg0 + lane) & 31);
          const int y = ((mine * s.heads_kv + it.h) << s.ps_shift) + (boxes > 1 ? 0 : kv0 & ((1 << s.ps_shift) - 1));
          const bool full = have == (1u << boxes) - 1;
          const bool dirty = !full || kv0 + BN > it.q.len;
          int bad = 0;   // per 16 keys
          if (!full)
            for (int b = 0; b < boxes; ++b)
              if (!(have >> b & 1)) bad |= ((1 << (box / 16)) - 1) << (b * (box / 16));
          if (lane == 0) sh_bad[gchunk & 31] = bad;
          if constexpr (E4M3) {
            // rows that exist: those below the length, less those of missing pages
            uint64_t rows = kv0 + 64 > it.q.len ? (1ull << (it.q.len - kv0)) - 1 : ~0ull;
            for (int g = 0; g < 4; ++g)
              if (bad >> g & 1) rows &= ~(0xffffull << (16 * g));
            const int64_t at = static_cast<int64_t>(y) * D;   // of lane b's box
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const int gi = gring + 2 * c + kv, slot = gi % C::RAW;
              if (!mbar_wait_w(&bar_rempty[slot], ((gi / C::RAW) & 1) ^ 1, ac)) { ok = false; break; }
              uint64_t* bar = &bar_rfull[slot];
              if (lane == 0) {
                sh_rows[slot] = rows;
                sh_more[slot] = 1;
                mbar_arrive_expect_tx(bar, __popc(have) * box * D);
              }
              __syncwarp();
              if (lane < boxes && mine >= 0)
                bulk_load(bar, sRing + C::NSLOT * C::KV_BYTES + slot * C::RAW_BYTES + lane * box * D,
                          static_cast<const uint8_t*>(kv ? a.v_cache : a.k_cache) + at, box * D);
            }
          }
#pragma unroll
          for (int kv = 0; kv < (E4M3 ? 0 : 2); ++kv) {
            const int gi = gring + 2 * c + kv;
            const int slot = gi % C::NSLOT, use = gi / C::NSLOT;
            if (!mbar_wait_w(&bar_empty[slot], (use & 1) ^ 1, ac)) { ok = false; break; }
            uint8_t* dst = sRing + slot * C::KV_BYTES;
            const CUtensorMap* m = kv ? &a.tm_v : &a.tm_k;
            uint64_t* bar = kv && dirty ? &bar_tail : &bar_full[slot];
            if (lane == 0) mbar_arrive_expect_tx(bar, __popc(have) * box * 128 * C::PANELS);
            __syncwarp();
            if (lane < boxes && mine >= 0) {   // lane b copies box b
#pragma unroll
              for (int pn = 0; pn < C::PANELS; ++pn)
                tma_load_2d(m, bar, dst + pn * BN * 128 + lane * box * 128, pn * 64, y);
            }
            if (kv && dirty) {   // zero what no key has, then hand the chunk over
              if (!mbar_wait_w(&bar_tail, tails & 1, ac)) { ok = false; break; }
              ++tails;
              for (int x = lane; x < BN * 8 * C::PANELS; x += 32) {
                const int row = (x >> 3) % BN;
                if (kv0 + row >= it.q.len || (bad >> (row >> 4) & 1))
                  reinterpret_cast<uint4*>(dst)[x] = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar_full[slot]);
            }
          }
        }
        if (ok && q_pending) {
          ok = mbar_wait_w(&bar_qempty[nqb], nq_par, ac);
          if (ok) issue_q(nx, pn_, ic + 1);
        }
        gring += 2 * pt.n_kv;
        ++ic;
        if (!have_next) {   // no more parts
          const int qb = ic % C::INFOS;
          if (ok && mbar_wait_w(&bar_qempty[qb], ((ic / C::INFOS) & 1) ^ 1, ac) && lane == 0) {
            sh_info[qb].kind = 0;
            mbar_arrive(&bar_q[qb]);
          }
          break;
        }
        it = nx;
        pt = pn_;
        left = left_nx;
      }
      if (!ok) {   // a wait ran out: what is in flight gets a moment to land before the CTA leaves
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 2000000ull) {
        }
      }
      if constexpr (E4M3) {   // no more chunks
        const int slot = gring % C::RAW;
        if (ok && mbar_wait_w(&bar_rempty[slot], ((gring / C::RAW) & 1) ^ 1, ac) && lane == 0) {
          sh_more[slot] = 0;
          mbar_arrive(&bar_rfull[slot]);
        }
      }
    }
  } else if (warp == 9 || warp == 10) {
    // ---------------- MMA issuer of query tile t ----------------
    const int t = warp - 9;
    if (range > 0) {
      // bf16 operands, e4m3: fp16 (A and B formats, bits 7..12, 0)
      constexpr uint32_t fmt = E4M3 ? ~(0x3fu << 7) : ~0u;
      const uint32_t idS = idesc_bf16(C::BM, BN, false, false) & fmt;
      const uint32_t idO = idesc_bf16(C::BM, D, false, true) & fmt;
      const uint64_t dR_k0 = desc_kmajor_base(smem_u32(sRing));
      const uint64_t dR_mn0 = desc_mnmajor_base(smem_u32(sRing), BN);
      const uint32_t tS = tmem + (t ? C::COL_S1 : C::COL_S0);
      const uint32_t tO = tmem + (t ? C::COL_O1 : C::COL_O0);
      const uint32_t tP = tmem + (t ? C::COL_P1 : C::COL_P0);
      int ic = 0, gring = 0, cs = 0, qc = 0;   // cs, qc: S and query tiles of this tile so far
      bool ok = true;
      while (ok) {
        const int qb = ic % C::INFOS, qu = ic / C::INFOS;
        if (!mbar_wait_w(&bar_q[qb], qu & 1, ac)) break;
        if (sh_info[qb].kind == 0) break;
        const int nt = sh_info[qb].n_w[t], n_kv = sh_info[qb].n_kv;
        // tile 1 starts one softmax phase after tile 0, as in attn_fwd (only where
        // tile 0 of the first item computes something)
        if (t == 1 && ic == 0 && sh_info[qb].n_w[0] > 0 && !mbar_wait_w(&bar_stagger, 0, ac)) break;
        const uint64_t dQt = desc_kmajor_base(smem_u32(sQ + ((E4M3 ? 0 : qb) * 2 + t) * C::Q_BYTES));
        if (E4M3 && nt > 0 && !mbar_wait_w(&bar_qready[t], qc++ & 1, ac)) break;
        auto issue_s = [&](int j) -> bool {
          const int gi = gring + 2 * j, sk = gi % C::NSLOT;
          if (!mbar_wait_w(&bar_full[sk], (gi / C::NSLOT) & 1, ac)) return false;
          tc_fence_after();
          const uint64_t kd = desc_advance(dR_k0, sk * C::KV_BYTES);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_ss_w(tS, desc_advance(dQt, kmajor_step_bytes(C::BM, kk)),
                      desc_advance(kd, kmajor_step_bytes(BN, kk)), idS, kk > 0);
          umma_commit_w(&bar_s[t]);
          umma_commit_w(&bar_empty[sk]);
          return true;
        };
        auto issue_pv = [&](int j) -> bool {
          const int gi = gring + 2 * j + 1, sv = gi % C::NSLOT;
          if (!mbar_wait_w(&bar_full[sv], (gi / C::NSLOT) & 1, ac)) return false;
          if (!mbar_wait_w(&bar_p[t], (cs + j) & 1, ac)) return false;
          if (t == 0 && ic == 0 && j == 0 && lane == 0) mbar_arrive(&bar_stagger);
          tc_fence_after();
          const uint64_t vd = desc_advance(dR_mn0, sv * C::KV_BYTES);
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)   // P: 8 packed columns per 16 keys
            umma_ts_w(tO, tP + 8 * kk, desc_advance(vd, mnmajor_step_bytes(kk)), idO,
                      (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit_w(&bar_o[t]);
          umma_commit_w(&bar_empty[sv]);
          return true;
        };
        // S(j+1) as soon as the softmax has read S(j); PV(j) once P(j) is ready
        for (int j = 0; ok && j < nt; ++j) {
          if (j == 0) {
            if (cs > 0 && !mbar_wait_w(&bar_sfree[t], (cs - 1) & 1, ac)) { ok = false; break; }
            if (!issue_s(0)) { ok = false; break; }
          }
          if (j + 1 < nt) {
            if (!mbar_wait_w(&bar_sfree[t], (cs + j) & 1, ac) || !issue_s(j + 1)) {
              ok = false;
              break;
            }
          }
          if (!issue_pv(j)) ok = false;
        }
        // chunks that this tile does not reach: it still waits for each load and
        // releases the slot itself, so that it stays within one phase of it
        for (int j = nt; ok && j < n_kv; ++j) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int gi = gring + 2 * j + kv, sl = gi % C::NSLOT;
            if (!mbar_wait_w(&bar_full[sl], (gi / C::NSLOT) & 1, ac)) { ok = false; break; }
            if (lane == 0) mbar_arrive(&bar_empty[sl]);
          }
        }
        if (ok) {
          if (nt > 0) umma_commit_w(&bar_qempty[qb]);
          else if (lane == 0) mbar_arrive(&bar_qempty[qb]);
        }
        gring += 2 * n_kv;
        cs += nt;
        ++ic;
      }
    }
  } else if (E4M3 && warp > 10) {
    // ---------------- e4m3: codes to fp16, exactly ----------------
    // Warp w of four has rows 16 w .. 16 w + 15 of every chunk of keys or values; a thread
    // takes vectors of 16 codes.  The scales are left to the softmax.  (code * scale as
    // bf16, four instructions more for two codes, and per-thread copies of the codes took
    // eight warps and 712 us for 2 x 2048 tokens over 8192 keys, where this form takes 584.)
    if constexpr (E4M3) {
      if (range > 0) {
        constexpr int VR = D / 16;          // vectors of a row
        constexpr int NV = 16 * VR / 32;    // vectors of a thread
        // two 16-byte pieces of a vector: dims 16 v .. + 7 and + 8 .. + 15.  The lanes of the upper
        // half of 128 dims take the row beside (row ^ 1), whose swizzle differs in the lowest
        // bit, so that the eight lanes of a row's place meet eight banks
        const int w = warp - 11, v = lane % VR, ch = 2 * (v & 3);
        const int row0 = 16 * w + ((lane / VR) ^ (v >> 2));   // the thread's first row
        const uint8_t* raw = sRing + C::NSLOT * C::KV_BYTES + row0 * D + v * 16;
        for (int i = 0;; ++i) {
          const int rs = i % C::RAW, slot = i % C::NSLOT;
          if (!mbar_wait_w(&bar_rfull[rs], (i / C::RAW) & 1, ac)) break;
          if (!sh_more[rs]) break;
          const uint64_t rows = sh_rows[rs];
          if (!mbar_wait_w(&bar_empty[slot], ((i / C::NSLOT) & 1) ^ 1, ac)) break;
          uint4 x[NV];
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            x[k] = *reinterpret_cast<const uint4*>(raw + rs * C::RAW_BYTES + k * 512);
            if (rows != ~0ull && !(rows >> (row0 + k * (32 / VR)) & 1)) x[k] = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_rempty[rs]);
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            const int row = row0 + k * (32 / VR);
            const uint32_t xx[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                  : "=r"(y[e])
                  : "h"(static_cast<uint16_t>(xx[e >> 1] >> (16 * (e & 1)))));
            uint8_t* line = sRing + slot * C::KV_BYTES + (v >> 2) * (BN * 128) + row * 128;
            *reinterpret_cast<uint4*>(line + ((ch ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(line + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
          fence_proxy_async_smem();
          mbar_arrive(&bar_full[slot]);
        }
      }
    }
  } else if (range > 0) {
    // ---------------- softmax warpgroups ----------------
    const int t = warp >> 2;                 // query tile of this warpgroup
    const int tr = threadIdx.x & 127;        // row within the tile == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + (t ? C::COL_S1 : C::COL_S0);
    const uint32_t tO = tmem + lane_base + (t ? C::COL_O1 : C::COL_O0);
    const uint32_t tP = tmem + lane_base + (t ? C::COL_P1 : C::COL_P0);
    // a negative scale turns the logits' signs; a zero one becomes so small that
    // they vanish, but not the masks (-inf * 0)
    const bool neg = a.scale_log2 < 0.f;
    const float sl2 = fmaxf(fabsf(a.scale_log2), 1e-30f);
    const int row_tok = tr / s.group, row_head = tr - row_tok * s.group;
    const bool row_in = row_tok < a.tile_tokens;
    int ic = 0, cs = 0, gchunk = 0;
    bool ok = true;
    while (ok) {
      const int qb = ic % C::INFOS;
      if (!mbar_wait(&bar_q[qb], (ic / C::INFOS) & 1, ac)) break;
      const PartInfo& f = sh_info[qb];
      const int kind = f.kind;
      if (kind == 0) break;
      const int nt = f.n_w[t], n_kv = f.n_kv, c0 = f.c0;
      const int tok0 = (2 * f.rb + t) * a.tile_tokens, tok = tok0 + row_tok;
      const int len = f.q.len, diag = f.q.pos0 + tok0;   // diag: the first row's position
      const int lim = a.causal ? min(len - 1, f.q.pos0 + tok) : len - 1;   // last key seen
      const int row_out = row_in && tok < f.q.m ? f.q.t0 + tok : -1;      // q's and o's row
      const int hd = f.h * s.group + row_head;
      if (kind != 7 && threadIdx.x == 0)
        a.part_meta[2 * blockIdx.x + (kind >> 1 & 1)] = make_int4(kind, f.n, f.h, f.rb);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_qempty[qb]);   // (the warp has read what it needs of f)
      float m_run = -INFINITY, l_run = 0.f;
      float rowf = sl2;            // logit factor of the row
      float off = -3.4e38f;        // e4m3: R of kPHead, less m_run; O is in units of 2^(R - kPHead)
      if constexpr (E4M3) {
        // The rows as fp16 times a power of two each (kQUp).  D / 8 lanes take a row.  (The tile is
        // free: its last S of the part before has been read by this warpgroup.)
        if (nt > 0) {
          constexpr int LPR = D / 8, RPI = 32 / LPR, NI = 32 / RPI;
          const int64_t at = row_out < 0 ? -1 : static_cast<int64_t>(row_out) * a.q_stride + hd * D;
          const int sub = lane / LPR, vec = lane % LPR;
          uint4 v[NI];
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int64_t src = __shfl_sync(0xffffffffu, at, i * RPI + sub);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (src >= 0) v[i] = *reinterpret_cast<const uint4*>(a.q + src + vec * 8);
          }
          int k_row = 0;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            uint32_t w4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w4[e] << 16)),
                                       fabsf(__uint_as_float(w4[e] & 0xffff0000u))));
#pragma unroll
            for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int k = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(kQUp - k + 127) << 23);
            const int mine = __shfl_sync(0xffffffffu, k, (lane % RPI) * LPR);
            if (lane / RPI == i) k_row = mine;   // of the thread's own row
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 hh = __floats2half2_rn(__uint_as_float(w4[e] << 16) * up,
                                                   __uint_as_float(w4[e] & 0xffff0000u) * up);
              w4[e] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            const int r = (warp & 3) * 32 + i * RPI + sub;
            *reinterpret_cast<uint4*>(sQ + t * C::Q_BYTES + (vec >> 3) * C::BM * 128 + r * 128 +
                                      (((vec & 7) ^ (r & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
          rowf *= __uint_as_float(static_cast<uint32_t>(k_row - kQUp + 127) << 23);
          fence_proxy_async_smem();
          mbar_arrive(&bar_qready[t]);
        }
      }
      for (int j = 0; j < nt; ++j) {
        const int c = cs + j;
        if (!mbar_wait(&bar_s[t], c & 1, ac)) { ok = false; break; }
        tc_fence_after();
        float x[BN];
        {
          uint32_t u[BN];
#pragma unroll
          for (int cc = 0; cc < BN; cc += 32) tmem_ld32_nowait(tS + cc, u + cc);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive(&bar_sfree[t]);
#pragma unroll
          for (int cc = 0; cc < BN; ++cc) x[cc] = __uint_as_float(u[cc]);
        }
        if (neg) {
#pragma unroll
          for (int cc = 0; cc < BN; ++cc) x[cc] = -x[cc];
        }
        const int kv0 = (c0 + j) * BN;
        const int bad = sh_bad[(gchunk + j) & 31];
        if (kv0 + BN > len || (a.causal && kv0 + BN - 1 > diag)) {
#pragma unroll
          for (int cc = 0; cc < BN; ++cc)
            if (kv0 + cc > lim) x[cc] = -INFINITY;
        }
        if (bad) {
#pragma unroll
          for (int cc = 0; cc < BN; ++cc)
            if (bad >> (cc / 16) & 1) x[cc] = -INFINITY;
        }
        uint32_t pk[BN / 2];
        bool grow;
        float alpha;
        if constexpr (!E4M3) {
          float mx[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            mx[i] = x[i];
#pragma unroll
            for (int b = 1; b + 1 < BN / 8; b += 2) mx[i] = fmax3(mx[i], x[8 * b + i], x[8 * b + 8 + i]);
            if constexpr ((BN / 8) % 2 == 0) mx[i] = fmaxf(mx[i], x[BN - 8 + i]);
          }
          const float mt = fmaxf(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], fmax3(mx[5], mx[6], mx[7]))) * sl2;
          const float m_new = fmaxf(m_run, mt);
          grow = m_new > m_run + 8.0f;          // also true on the first finite max
          const float m_use = grow ? m_new : m_run;
          alpha = grow ? ex2(m_run - m_use) : 1.0f;
          const float msub = (m_use == -INFINITY) ? 0.f : m_use;
          const uint64_t nm2 = f2_pack(-msub, -msub), sl2x2 = f2_pack(sl2, sl2);
          uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int cc = 0; cc < BN; cc += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(x[cc], x[cc + 1]), sl2x2, nm2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            rs2[(cc >> 1) & 3] = f2_add(rs2[(cc >> 1) & 3], f2_pack(p0, p1));
            pk[cc / 2] = pack_bf16(p0, p1);
          }
          float r0, r1, r2, r3, r4, r5, r6, r7;
          f2_unpack(rs2[0], r0, r1);
          f2_unpack(rs2[1], r2, r3);
          f2_unpack(rs2[2], r4, r5);
          f2_unpack(rs2[3], r6, r7);
          l_run = l_run * alpha + (((r0 + r1) + (r2 + r3)) + ((r4 + r5) + (r6 + r7)));
          m_run = m_use;
        } else {
          // four groups of 16 keys with scales of their own: the logits' factor, and the summand
          // of P's exponent (log2 of the values' scale, relative to R, and kPHead), which the row
          // sum takes off again.  From -40 down nothing of it is left in fp16, P being below 2^9.
          // The logits' factor stays above zero, which would make the masks NaN.
          const float2* sc = sh_scale[(gchunk + j) & 31];
          float fg[4], lg[4], mg[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float2 kv = sc[g];
            fg[g] = fmaxf(rowf * kv.x, 1e-37f);
            lg[g] = kv.y;
            const float* xg = x + 16 * g;
            float m0 = fmax3(xg[0], xg[1], xg[2]), m1 = fmax3(xg[3], xg[4], xg[5]);
            m0 = fmax3(m0, xg[6], xg[7]);
            m1 = fmax3(m1, xg[8], xg[9]);
            m0 = fmax3(m0, xg[10], xg[11]);
            m1 = fmax3(m1, xg[12], xg[13]);
            mg[g] = fmax3(m0, m1, fmaxf(xg[14], xg[15])) * fg[g];
          }
          const float mt = fmaxf(fmaxf(mg[0], mg[1]), fmaxf(mg[2], mg[3]));
          const float m_new = fmaxf(m_run, mt);
          const bool mgrow = m_new > m_run + 8.0f;
          const float m_use = mgrow ? m_new : m_run;
          const float decay = mgrow ? ex2(m_run - m_use) : 1.0f;
          const float msub = (m_use == -INFINITY) ? 0.f : m_use;
          off = mgrow ? off - (m_use - m_run) : off;
          // log2 of the largest product, over the maximum (far below which their sum would drown)
          const float top = fmaxf(fmaxf(mg[0] - msub + lg[0], mg[1] - msub + lg[1]),
                                  fmaxf(mg[2] - msub + lg[2], mg[3] - msub + lg[3]));
          grow = __any_sync(0xffffffffu, top > off + kPSlack) && top > off;
          alpha = grow ? off - top : 0.0f;   // (log2)
          off = grow ? top : off;
          const float base = kPHead - off;
          float sum = 0.f;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float l = fmaxf(base + lg[g], -40.f);
            const uint64_t nm2 = f2_pack(l - msub, l - msub), f2 = f2_pack(fg[g], fg[g]);
            uint64_t rs2[2] = {0ull, 0ull};
#pragma unroll
            for (int cc = 16 * g; cc < 16 * g + 16; cc += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(x[cc], x[cc + 1]), f2, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              rs2[(cc >> 1) & 1] = f2_add(rs2[(cc >> 1) & 1], f2_pack(p0, p1));
              const __half2 hh = __floats2half2_rn(p0, p1);
              pk[cc / 2] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            float r0, r1;
            f2_unpack(f2_add(rs2[0], rs2[1]), r0, r1);
            sum += (r0 + r1) * ex2(-l);
          }
          l_run = l_run * decay + sum;
          m_run = m_use;
        }
        const bool warp_rescale = j > 0 && __any_sync(0xffffffffu, grow);
        if (j > 0) {
          // PV(j-1) must be done before O is rescaled and P(j) overwrites P(j-1)
          if (!mbar_wait(&bar_o[t], (c - 1) & 1, ac)) { ok = false; break; }
          tc_fence_after();
        }
        if (warp_rescale) {
          const float a_o = E4M3 ? ex2(alpha) : alpha;
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t r[32];
            tmem_ld32_nowait(tO + cc, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * a_o);
            tmem_st32(tO + cc, r);
          }
        }
#pragma unroll
        for (int cc = 0; cc < BN / 2; cc += 32) tmem_st32(tP + cc, pk + cc);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_p[t]);
      }
      // ---- the part's end: normalized rows, or a partial result ----
      if (ok && nt > 0) {
        ok = mbar_wait(&bar_o[t], (cs + nt - 1) & 1, ac);
        tc_fence_after();
      }
      if (ok) {
        const bool valid = row_out >= 0, whole = kind == 7;
        // e4m3: O's unit over the row's maximum, in two halves: it may be subnormal
        const float half = E4M3 ? ex2(0.5f * (off - kPHead)) : 1.f;
        const float unit = half * half;
        const float inv = (l_run > 0.f || l_run != l_run ? 1.0f / l_run : 0.f) * unit;
        __nv_bfloat16* orow = a.o + (static_cast<int64_t>(row_out) * s.heads_q + hd) * D;
        const int64_t at = static_cast<int64_t>(blockIdx.x) * 2 + (kind >> 1 & 1);
        float4* part = reinterpret_cast<float4*>(a.part_o) + at * (D / 4) * 2 * C::BM + t * C::BM + tr;
#pragma unroll
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t r[32];
          if (nt > 0) {
            tmem_ld32_nowait(tO + cc, r);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0u;
          }
          if (valid) {
            if (whole) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint4 v;
                v.x = pack_bf16(__uint_as_float(r[i + 0]) * inv, __uint_as_float(r[i + 1]) * inv);
                v.y = pack_bf16(__uint_as_float(r[i + 2]) * inv, __uint_as_float(r[i + 3]) * inv);
                v.z = pack_bf16(__uint_as_float(r[i + 4]) * inv, __uint_as_float(r[i + 5]) * inv);
                v.w = pack_bf16(__uint_as_float(r[i + 6]) * inv, __uint_as_float(r[i + 7]) * inv);
                *reinterpret_cast<uint4*>(orow + cc + i) = v;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                part[(cc + i) / 4 * 2 * C::BM] =
                    make_float4(__uint_as_float(r[i]) * unit, __uint_as_float(r[i + 1]) * unit,
                                __uint_as_float(r[i + 2]) * unit, __uint_as_float(r[i + 3]) * unit);
            }
          }
        }
        tc_fence_before();
        if (valid) {
          if (whole) {
            a.lse[static_cast<int64_t>(hd) * s.tokens + row_out] =
                l_run > 0.f || l_run != l_run ? (m_run + __log2f(l_run)) * kLn2 : -INFINITY;
          } else {
            a.part_ml[at * 2 * C::BM + t * C::BM + tr] = make_float2(m_run, l_run);
          }
        }
      }
      cs += nt;
      gchunk += n_kv;
      ++ic;
    }
  }

  // ---- padding rows: at or past cu_seqlens[num_seqs] ----
  const int end = a.pad ? min(max(__ldg(s.cu + s.num_seqs), 0), s.tokens) : s.tokens;
  const int64_t words = static_cast<int64_t>(s.tokens - end) * s.heads_q * (D / 8);
  uint4* o4 = reinterpret_cast<uint4*>(a.o + static_cast<int64_t>(end) * s.heads_q * D);
  const int64_t step = static_cast<int64_t>(gridDim.x) * C::THREADS;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(C::THREADS) + threadIdx.x; w < words; w += step)
    o4[w] = make_uint4(0u, 0u, 0u, 0u);
  const int64_t pad = s.tokens - end, lses = pad * s.heads_q;
  for (int64_t w = blockIdx.x * static_cast<int64_t>(C::THREADS) + threadIdx.x; w < lses; w += step)
    a.lse[w / pad * s.tokens + end + w % pad] = -INFINITY;

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
}

template <int D, bool E4M3>
cudaError_t launch(const CacheFwdArgs& a, int grid, cudaStream_t st) {
  using C = TcCfg<D, E4M3>;
  auto kern = cache_fwd_tc_kernel<D, E4M3>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  kern<<<grid, C::THREADS, C::SMEM, st>>>(a);
  e = cudaGetLastError();
  return e != cudaSuccess || grid < 2 ? e : launch_cache_join(a, D, kCacheTcRows, grid, st);
}

}  // namespace

int cache_tc_chunk(int head_dim, bool e4m3) {
  return head_dim == 128 ? TcCfg<128, false>::BN : e4m3 ? TcCfg<64, true>::BN : TcCfg<64, false>::BN;
}

cudaError_t launch_cache_fwd_tc(const CacheFwdArgs& a, int head_dim, bool e4m3, int grid,
                                cudaStream_t st) {
  if (head_dim == 64) return e4m3 ? launch<64, true>(a, grid, st) : launch<64, false>(a, grid, st);
  return e4m3 ? launch<128, true>(a, grid, st) : launch<128, false>(a, grid, st);
}

}  // namespace attn

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
  static constexpr int NSLOT = D == 128 && E4M3 ? 4 : 6;
  static constexpr int QBUFS = 2;
  // e4m3: warps 12..15 bring the keys' codes, warps 16..19 the values', into a ring of
  // RAW chunks each and convert them into the slots, after a list that warp 8 writes
  static constexpr int RAW = 2, RAW_BYTES = E4M3 ? BN * D : 0;
  static constexpr int SMEM = QBUFS * 2 * Q_BYTES + NSLOT * KV_BYTES + 2 * RAW * RAW_BYTES + 1024;
  static constexpr int THREADS = E4M3 ? 640 : 352;
  static constexpr int LIST = 8;   // chunks of the list
  // e4m3: registers of a thread, at launch and then by warpgroup (softmax, issue and
  // copy, conversion); the shares add up to what the block was launched with
  static constexpr int REGS = 96, REGS_SOFTMAX = 120, REGS_ISSUE = 80, REGS_CONVERT = 80;
  static_assert(2 * REGS_SOFTMAX + REGS_ISSUE + 2 * REGS_CONVERT <= 5 * REGS, "register shares");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_S0 = 0, COL_S1 = BN, COL_O0 = 256, COL_O1 = 256 + D;
  static constexpr uint32_t COL_P0 = D == 128 ? 2 * BN : 256 + 2 * D, COL_P1 = COL_P0 + BN / 2;
  static_assert(D != 128 || 3 * BN <= 256, "S and P of both tiles below O");
  static_assert(D == 128 || 256 + 2 * D + BN <= 512, "TMEM budget");
  static_assert(SMEM <= 227 * 1024 - 700, "shared memory");
};

// Chunks by which an item counts more in the dealing than it has: its query
// tiles, its first and last chunk and its outputs.
constexpr int kItemCost = 3;

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
template <int BN>
__device__ __forceinline__ void item_block(const CacheFwdArgs& a, TcItem& it) {
  it.seen[0] = tile_seen<BN>(a, it.q, 2 * it.rb);
  it.seen[1] = tile_seen<BN>(a, it.q, 2 * it.rb + 1);
  it.nc = max(it.seen[0], it.seen[1]) + kItemCost;
}
__device__ __forceinline__ int seq_blocks(const CacheFwdArgs& a, const StepSeq& q) {
  return (q.m + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
}
// The next item; the caller knows that there is one.
template <int BN>
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
  item_block<BN>(a, it);
}
// Chunks of one KV head of a sequence in the dealing.
template <int BN>
__device__ __forceinline__ int64_t head_chunks(const CacheFwdArgs& a, const StepSeq& q) {
  const int nb = seq_blocks(a, q);
  int64_t w = static_cast<int64_t>(nb) * kItemCost;
  for (int rb = 0; rb < nb; ++rb)
    w += max(tile_seen<BN>(a, q, 2 * rb), tile_seen<BN>(a, q, 2 * rb + 1));
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

  __shared__ uint64_t bar_q[C::QBUFS], bar_qempty[C::QBUFS];
  __shared__ uint64_t bar_full[C::NSLOT], bar_empty[C::NSLOT], bar_tail;
  __shared__ uint64_t bar_s[2], bar_p[2], bar_o[2], bar_sfree[2], bar_stagger;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ int sh_bad[32];   // by chunk: 16-key groups (bits) without a page
  // e4m3, by chunk: the pool row of each 16-key group and how many of its rows exist
  // (first group -1: the end); the scales of the groups in the raw rings
  __shared__ int2 sh_list[C::LIST][4];
  __shared__ uint64_t bar_lfull[C::LIST], bar_lempty[C::LIST];
  __shared__ float sh_scale[2][4][C::RAW];
  __shared__ int64_t sh_warp[C::THREADS / 32 + 1];
  __shared__ TcItem sh_item;
  __shared__ PartInfo sh_info[C::QBUFS];
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
    for (int b = 0; b < C::QBUFS; ++b) {
      mbar_init(&bar_q[b], 1);
      mbar_init(&bar_qempty[b], 10);     // released by both issuers and 8 softmax warps
    }
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&bar_full[i], E4M3 ? 128 : 1);
      mbar_init(&bar_empty[i], 2);       // released by both issuers
    }
    mbar_init(&bar_tail, 1);
    if constexpr (E4M3)
      for (int i = 0; i < C::LIST; ++i) {
        mbar_init(&bar_lfull[i], 1);
        mbar_init(&bar_lempty[i], 8);    // released by the converting warps
      }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&bar_s[w], 1);
      mbar_init(&bar_p[w], 128);
      mbar_init(&bar_o[w], 1);
      mbar_init(&bar_sfree[w], 128);
    }
    mbar_init(&bar_stagger, 1);
    fence_mbar_init();
    tma_prefetch_desc(&a.tm_q);
    if constexpr (!E4M3) {
      tma_prefetch_desc(&a.tm_k);
      tma_prefetch_desc(&a.tm_v);
    }
  }
  if (threadIdx.x < 2) a.part_meta[2 * blockIdx.x + threadIdx.x] = make_int4(0, 0, 0, 0);
  if (warp == 9) tmem_alloc(&tmem_base_sh, C::TMEM_COLS);

  // ---- the dealing: every thread sums a slice of the sequences, the thread whose
  // slice holds the CTA's first chunk finds its item ----
  {
    const int per = (s.num_seqs + C::THREADS - 1) / C::THREADS;
    const int n0 = threadIdx.x * per, n1 = min(s.num_seqs, n0 + per);
    int64_t mine = 0;
    int bad = 0;
    for (int n = n0; n < n1; ++n)
      mine += s.heads_kv * head_chunks<BN>(a, step_seq(s, n, &bad));
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
    if (f0 < f1 && f0 >= end - mine && f0 < end) {
      TcItem it;
      int64_t off = f0 - (end - mine);
      for (it.n = n0;; ++it.n) {
        it.q = step_seq(s, it.n);
        const int64_t w = head_chunks<BN>(a, it.q);
        if (off < s.heads_kv * w) {
          it.h = static_cast<int>(off / w);
          off -= it.h * w;
          break;
        }
        off -= s.heads_kv * w;
      }
      it.nb = seq_blocks(a, it.q);
      for (it.rb = 0;; ++it.rb) {
        item_block<BN>(a, it);
        if (off < it.nc) break;
        off -= it.nc;
      }
      sh_item = it;
      sh_c0 = static_cast<int>(off);
      sh_left = f1 - f0;
    }
    __syncthreads();
  }
  const uint32_t tmem = tmem_base_sh;
  const int64_t range = sh_left;   // chunks of the CTA

  if constexpr (E4M3) {
    if (warp < 8) setmaxnreg_inc<C::REGS_SOFTMAX>();
    else if (warp < 12) setmaxnreg_dec<C::REGS_ISSUE>();
    else setmaxnreg_dec<C::REGS_CONVERT>();
  }
  if (warp == 8) {
    // ---------------- copies (warp-uniform, lane 0 issues) ----------------
    if (range > 0) {
      const int box = min(BN, 1 << s.ps_shift), boxes = BN / box;
      const int tile_bytes = a.tile_tokens * s.group * 128 * C::PANELS;
      auto issue_q = [&](const TcItem& it, const Part& pt, int icq) {
        if (lane != 0) return;
        const int qb = icq % C::QBUFS;
        PartInfo f;
        f.n_w[0] = pt.n_w[0], f.n_w[1] = pt.n_w[1], f.n_kv = pt.n_kv, f.c0 = pt.c0;
        f.q = it.q, f.n = it.n, f.h = it.h, f.rb = it.rb;
        f.kind = 1 | (pt.c0 == 0 ? 2 : 0) | (pt.c0 + pt.span == it.nc ? 4 : 0);
        sh_info[qb] = f;
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
        item_next<BN>(a, it);
        pt = part_of(it, 0, left);
        return true;
      };
      TcItem it = sh_item, nx;
      int64_t left = range;
      Part pt = part_of(it, sh_c0, left), pn_;
      int ic = 0, gring = 0, gchunk = 0, tails = 0;
      int pg0 = -1, pg_n = -1, pid = -1;   // lane l holds the page of column pg0 + l of sequence pg_n
      bool ok = mbar_wait_w(&bar_qempty[0], 1, ac);
      if (ok) issue_q(it, pt, 0);
      while (ok) {
        nx = it;
        pn_ = pt;
        int64_t left_nx = left;
        const bool have_next = advance(nx, pn_, left_nx);
        bool q_pending = have_next;
        const int nqb = (ic + 1) % C::QBUFS;
        const uint32_t nq_par = (((ic + 1) / C::QBUFS) & 1) ^ 1;
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
          }
          if constexpr (E4M3) {
            // lanes 0..3 list the chunk's groups of 16 keys
            const int key0 = kv0 + 16 * (lane & 3), col = key0 >> s.ps_shift;
            const int page = __shfl_sync(0xffffffffu, pid, col - pg0);
            const int rows = page < 0 ? 0 : max(0, min(16, it.q.len - key0));
            const int bad = __ballot_sync(0xffffffffu, lane < 4 && page < 0 && key0 < it.q.len);
            const int at = gchunk % C::LIST;
            if (!mbar_wait_w(&bar_lempty[at], ((gchunk / C::LIST) & 1) ^ 1, ac)) { ok = false; break; }
            if (lane < 4)
              sh_list[at][lane] = make_int2(((max(page, 0) * s.heads_kv + it.h) << s.ps_shift) +
                                                (key0 & ((1 << s.ps_shift) - 1)), rows);
            if (lane == 0) sh_bad[gchunk & 31] = bad;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar_lfull[at]);
            continue;
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
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
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
          const int qb = ic % C::QBUFS;
          if (ok && mbar_wait_w(&bar_qempty[qb], ((ic / C::QBUFS) & 1) ^ 1, ac) && lane == 0) {
            sh_info[qb].kind = 0;
            mbar_arrive(&bar_q[qb]);
          }
          break;
        }
        it = nx;
        pt = pn_;
        left = left_nx;
      }
      if constexpr (E4M3) {   // the list's end
        const int at = gchunk % C::LIST;
        if (ok && mbar_wait_w(&bar_lempty[at], ((gchunk / C::LIST) & 1) ^ 1, ac)) {
          if (lane == 0) {
            sh_list[at][0].x = sh_list[at][1].x = sh_list[at][2].x = sh_list[at][3].x = -1;
            mbar_arrive(&bar_lfull[at]);
          }
        }
      }
    }
  } else if (warp == 9 || warp == 10) {
    // ---------------- MMA issuer of query tile t ----------------
    const int t = warp - 9;
    if (range > 0) {
      const uint32_t idS = idesc_bf16(C::BM, BN, false, false);
      const uint32_t idO = idesc_bf16(C::BM, D, false, true);
      const uint64_t dR_k0 = desc_kmajor_base(smem_u32(sRing));
      const uint64_t dR_mn0 = desc_mnmajor_base(smem_u32(sRing), BN);
      const uint32_t tS = tmem + (t ? C::COL_S1 : C::COL_S0);
      const uint32_t tO = tmem + (t ? C::COL_O1 : C::COL_O0);
      const uint32_t tP = tmem + (t ? C::COL_P1 : C::COL_P0);
      int ic = 0, gring = 0, cs = 0;   // cs: S tiles of this query tile so far
      bool ok = true;
      while (ok) {
        const int qb = ic % C::QBUFS, qu = ic / C::QBUFS;
        if (!mbar_wait_w(&bar_q[qb], qu & 1, ac)) break;
        if (sh_info[qb].kind == 0) break;
        const int nt = sh_info[qb].n_w[t], n_kv = sh_info[qb].n_kv;
        // tile 1 starts one softmax phase after tile 0, as in attn_fwd (only where
        // tile 0 of the first item computes something)
        if (t == 1 && ic == 0 && sh_info[qb].n_w[0] > 0 && !mbar_wait_w(&bar_stagger, 0, ac)) break;
        const uint64_t dQt = desc_kmajor_base(smem_u32(sQ + (qb * 2 + t) * C::Q_BYTES));
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
    // ---------------- e4m3: codes to bf16 values ----------------
    // Four warps for the keys, four for the values; warp w of them has keys 16 w ..
    // 16 w + 15 of every chunk, which lie in one page under one scale.  A thread copies, RAW
    // chunks ahead, the vectors of 16 codes that it converts: vector 4 j + lane % 4 of rows
    // lane / 4 and lane / 4 + 8.  Codes go through fp16 and fp32 (exactly, NaN included);
    // code * scale is rounded to bf16, which is exact for scales that are powers of two.
    // (Moving bits and one bf16 multiply, for such scales, measured 9% slower.)
    if constexpr (E4M3) {
      if (range > 0 && warp >= 12) {
        constexpr int NV = 2 * C::PANELS;   // vectors of a thread
        const int w = warp & 3, values = warp >= 16;
        const uint8_t* pool = static_cast<const uint8_t*>(values ? a.v_cache : a.k_cache);
        const float* scales = values ? a.v_scale : a.k_scale;
        uint8_t* raw = sRing + C::NSLOT * C::KV_BYTES + (values * C::RAW * 4 + w) * (C::RAW_BYTES / 4);
        float* sc_at = sh_scale[values][w];
        const int lane_row = lane >> 2;
        const int lane_off = lane_row * D + (lane & 3) * 16;
        int copied = 0;   // chunks taken from the list
        bool more = true;
        auto copy = [&]() {
          const int at = copied % C::LIST;
          more = mbar_wait_w(&bar_lfull[at], (copied / C::LIST) & 1, ac);
          if (!more) return;
          const int2 e = sh_list[at][w];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_lempty[at]);
          more = e.x >= 0;
          if (!more) return;
          const uint8_t* src = pool + static_cast<int64_t>(e.x) * D + lane_off;
          const int st = copied % C::RAW;
          const uint32_t dst = smem_u32(raw) + st * C::RAW_BYTES + lane * 16;
          const uint32_t n0 = lane_row < e.y ? 16u : 0u, n1 = lane_row + 8 < e.y ? 16u : 0u;   // else zeros
#pragma unroll
          for (int v = 0; v < NV; ++v)
            cp_async16(dst + v * 512, src + (v & 1) * 8 * D + (v >> 1) * 64, (v & 1) ? n1 : n0);
          if (lane == 0) {
            if (e.y > 0)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sc_at + st)),
                           "l"(scales + (e.x >> s.ps_shift))
                           : "memory");
            else
              sc_at[st] = 0.f;
          }
          cp_async_commit();
          ++copied;
        };
        for (int i = 0;; ++i) {
          // RAW chunks ahead, but a chunk in hand never waits for the list: what comes
          // next may depend on it (a part's query tiles on an earlier part's end)
          while (more && copied < i + C::RAW &&
                 (copied == i || mbar_test_wait_w(smem_u32(&bar_lfull[copied % C::LIST]), (copied / C::LIST) & 1)))
            copy();
          if (copied == i) break;
          static_assert(C::RAW == 2, "the waits below");
          if (copied > i + 1) cp_async_wait<1>();
          else cp_async_wait<0>();
          __syncwarp();
          const int gi = 2 * i + values, slot = gi % C::NSLOT;
          if (!mbar_wait_w(&bar_empty[slot], ((gi / C::NSLOT) & 1) ^ 1, ac)) break;
          const uint8_t* src = raw + (i % C::RAW) * C::RAW_BYTES + lane * 16;
          const float sc = sc_at[i % C::RAW];
          const uint64_t sc2 = f2_pack(sc, sc);
          uint8_t* dst = sRing + slot * C::KV_BYTES + (16 * w + lane_row) * 128;
          const int sw = lane_row & 7, ch = 2 * (lane & 3);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + v * 512);
            const uint32_t xx[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              uint32_t h;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
                  : "=r"(h)
                  : "h"(static_cast<uint16_t>(xx[e >> 1] >> (16 * (e & 1)))));
              const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
              y[e] = f2_to_bf16x2(f2_mul(f2_pack(f.x, f.y), sc2));
            }
            uint8_t* line = dst + (v >> 1) * (BN * 128) + (v & 1) * 8 * 128;
            *reinterpret_cast<uint4*>(line + ((ch ^ sw) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<uint4*>(line + (((ch + 1) ^ sw) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
          }
          fence_proxy_async_smem();
          mbar_arrive(&bar_full[slot]);
          __syncwarp();
        }
        cp_async_wait<0>();
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
      const int qb = ic % C::QBUFS;
      if (!mbar_wait(&bar_q[qb], (ic / C::QBUFS) & 1, ac)) break;
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
        const bool grow = m_new > m_run + 8.0f;          // also true on the first finite max
        const float m_use = grow ? m_new : m_run;
        const float alpha = grow ? ex2(m_run - m_use) : 1.0f;
        const float msub = (m_use == -INFINITY) ? 0.f : m_use;
        const bool warp_rescale = j > 0 && __any_sync(0xffffffffu, grow);
        const uint64_t nm2 = f2_pack(-msub, -msub), sl2x2 = f2_pack(sl2, sl2);
        uint64_t rs2[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pk[BN / 2];
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
        if (j > 0) {
          // PV(j-1) must be done before O is rescaled and P(j) overwrites P(j-1)
          if (!mbar_wait(&bar_o[t], (c - 1) & 1, ac)) { ok = false; break; }
          tc_fence_after();
        }
        if (warp_rescale) {
#pragma unroll
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t r[32];
            tmem_ld32_nowait(tO + cc, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
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
        const float inv = l_run > 0.f || l_run != l_run ? 1.0f / l_run : 0.f;
        __nv_bfloat16* orow = a.o + (static_cast<int64_t>(row_out) * s.heads_q + hd) * D;
        const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + (kind >> 1 & 1)) * 2 * C::BM + t * C::BM + tr;
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
                *reinterpret_cast<uint4*>(a.part_o + at * D + cc + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
            }
          }
        }
        tc_fence_before();
        if (valid) {
          if (whole) {
            a.lse[static_cast<int64_t>(hd) * s.tokens + row_out] =
                l_run > 0.f || l_run != l_run ? (m_run + __log2f(l_run)) * kLn2 : -INFINITY;
          } else {
            a.part_ml[at] = make_float2(m_run, l_run);
          }
        }
      }
      cs += nt;
      gchunk += n_kv;
      ++ic;
    }
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
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  if constexpr (E4M3) {
    // the warpgroups' register shares draw on what the block is launched with: a build
    // with fewer registers than they count on must not run (it would wait forever)
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs < C::REGS) return cudaErrorInvalidConfiguration;
  }
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

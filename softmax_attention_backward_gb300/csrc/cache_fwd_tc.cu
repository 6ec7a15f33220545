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
  // e4m3: warps 11..14 bring the codes into a ring of RAW chunks of their own and
  // convert them into the slots
  static constexpr int RAW = 4, RAW_BYTES = E4M3 ? BN * D : 0;
  static constexpr int SMEM = QBUFS * 2 * Q_BYTES + NSLOT * KV_BYTES + RAW * RAW_BYTES + 1024;
  static constexpr int THREADS = E4M3 ? 480 : 352;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t COL_S0 = 0, COL_S1 = BN, COL_O0 = 256, COL_O1 = 256 + D;
  static constexpr uint32_t COL_P0 = D == 128 ? 2 * BN : 256 + 2 * D, COL_P1 = COL_P0 + BN / 2;
  static_assert(D != 128 || 3 * BN <= 256, "S and P of both tiles below O");
  static_assert(D == 128 || 256 + 2 * D + BN <= 512, "TMEM budget");
  static_assert(SMEM <= 226 * 1024, "shared memory");
};

// Chunks by which an item counts more in the dealing than it has: its query
// tiles, its first and last chunk and its outputs.
constexpr int kItemCost = 3;

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
  // by chunk, which 16-key groups have no page: a bit each; e4m3: a byte each
  constexpr int BAD_SHIFT = E4M3 ? 8 : 1;
  __shared__ int sh_bad[16];
  __shared__ float sh_scale[4][C::RAW];   // e4m3: of each converting warp's 16 keys
  __shared__ int64_t sh_warp[C::THREADS / 32 + 1];
  __shared__ TcItem sh_item;
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
      mbar_init(&bar_qempty[b], 2);      // released by both issuers
    }
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&bar_full[i], E4M3 ? 128 : 1);
      mbar_init(&bar_empty[i], 2);       // released by both issuers
    }
    mbar_init(&bar_tail, 1);
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
  const TcItem first = sh_item;   // (not read when sh_left is 0)
  const int first_c0 = sh_c0;
  const int64_t range = sh_left;
  // the walk of every role: item, part, next
  auto advance = [&](TcItem& it, Part& pt, int64_t& left) -> bool {
    left -= pt.span;
    if (left <= 0) return false;
    item_next<BN>(a, it);
    pt = part_of(it, 0, left);
    return true;
  };

  if (warp == 8) {
    // ---------------- copies (warp-uniform, lane 0 issues) ----------------
    if (range > 0) {
      const int box = min(BN, 1 << s.ps_shift), boxes = BN / box;
      const int tile_bytes = a.tile_tokens * s.group * 128 * C::PANELS;
      auto issue_q = [&](const TcItem& it, int icq) {
        if (lane != 0) return;
        const int qb = icq % C::QBUFS;
        mbar_arrive_expect_tx(&bar_q[qb], 2 * tile_bytes);
        for (int t = 0; t < 2; ++t)
          for (int pn = 0; pn < C::PANELS; ++pn)
            tma_load_3d(&a.tm_q, &bar_q[qb], sQ + (qb * 2 + t) * C::Q_BYTES + pn * C::BM * 128, pn * 64,
                        it.h * s.group, it.q.t0 + (2 * it.rb + t) * a.tile_tokens);
      };
      TcItem it = first, nx;
      int64_t left = range;
      Part pt = part_of(it, first_c0, left), pn_;
      int ic = 0, gring = 0, gchunk = 0, tails = 0;
      int pg0 = -1, pg_n = -1, pid = -1;   // lane l holds the page of column pg0 + l of sequence pg_n
      bool ok = mbar_wait_w(&bar_qempty[0], 1, ac);
      if (ok) issue_q(it, 0);
      while (ok) {
        nx = it;
        pn_ = pt;
        int64_t left_nx = left;
        const bool have_next = advance(nx, pn_, left_nx);
        bool q_pending = have_next;
        const int nqb = (ic + 1) % C::QBUFS;
        const uint32_t nq_par = (((ic + 1) / C::QBUFS) & 1) ^ 1;
        for (int c = 0; ok && c < (E4M3 ? 0 : pt.n_kv); ++c, ++gchunk) {
          const int kv0 = (pt.c0 + c) * BN;
          // pages of the chunk: one, or `boxes` of them
          const int col0 = kv0 >> s.ps_shift;
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
          if (lane == 0) sh_bad[gchunk & 15] = bad;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int gi = gring + 2 * c + kv;
            const int slot = gi % C::NSLOT, use = gi / C::NSLOT;
            if (q_pending && mbar_test_wait_w(smem_u32(&bar_qempty[nqb]), nq_par)) {
              issue_q(nx, ic + 1);
              q_pending = false;
            }
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
          if (ok) issue_q(nx, ic + 1);
        }
        gring += 2 * pt.n_kv;
        ++ic;
        if (!have_next) break;
        it = nx;
        pt = pn_;
        left = left_nx;
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
      TcItem it = first;
      int64_t left = range;
      Part pt = part_of(it, first_c0, left);
      int ic = 0, gring = 0, cs = 0;   // cs: S tiles of this query tile so far
      bool ok = true, stagger = t == 1;
      while (ok) {
        const int qb = ic % C::QBUFS, qu = ic / C::QBUFS;
        const int nt = pt.n_w[t];
        if (!mbar_wait_w(&bar_q[qb], qu & 1, ac)) break;
        // tile 1 starts one softmax phase after tile 0, as in attn_fwd (only where
        // tile 0 of the first item computes something)
        if (stagger && ic == 0 && pt.n_w[0] > 0 && !mbar_wait_w(&bar_stagger, 0, ac)) break;
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
        for (int j = nt; ok && j < pt.n_kv; ++j) {
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
        gring += 2 * pt.n_kv;
        cs += nt;
        ++ic;
        if (!ok || !advance(it, pt, left)) break;
      }
    }
  } else if (E4M3 && warp > 10) {
    // ---------------- e4m3: codes to bf16 values ----------------
    // Warp w has keys 16 w .. 16 w + 15 of every chunk, which lie in one page under one
    // scale; a thread copies, four chunks of keys or values ahead, the vectors of 16 codes
    // that it converts: vector 4 j + lane % 4 of rows lane / 4 and lane / 4 + 8.  Codes go
    // through fp16 and fp32 (exactly, NaN included); code * scale is rounded to bf16,
    // which is exact for scales that are powers of two.
    if constexpr (E4M3) {
      if (range > 0) {
        constexpr int NV = 2 * C::PANELS;   // vectors of a thread
        const int w = warp - 11;
        uint8_t* raw = sRing + C::NSLOT * C::KV_BYTES + w * (C::RAW_BYTES / 4);   // + stage * RAW_BYTES
        TcItem cp = first;                  // the copies' place
        int64_t cp_left = range;
        Part cp_pt = part_of(cp, first_c0, cp_left);
        int cp_c = 0, cp_half = 0, cp_chunk = 0;
        int pg0 = -1, pg_n = -1, pid = -1;  // lane l holds the page of column pg0 + l of sequence pg_n
        bool cp_more = true;
        auto copy = [&]() {
          if (cp_more && !(cp_half & 1))
            while (cp_c >= cp_pt.n_kv) {
              cp_more = advance(cp, cp_pt, cp_left);
              cp_c = 0;
              if (!cp_more) break;
            }
          if (cp_more) {
            const int key0 = (cp_pt.c0 + cp_c) * BN + 16 * w;
            const int col = key0 >> s.ps_shift;
            if (pg_n != cp.n || col < pg0 || col >= pg0 + 32) {
              pg_n = cp.n;
              pg0 = col;
              const int cc = col + lane;
              pid = -1;
              if (cc <= (cp.q.len - 1) >> s.ps_shift) {
                pid = __ldg(s.table + static_cast<int64_t>(cp.n) * s.max_pages + cc);
                if (pid < 0 || pid >= s.num_pages) {
                  pid = -1;
                  if (s.err) atomicOr(s.err, ATTN_DEVERR_INDEX_RANGE);
                }
              }
            }
            const int page = __shfl_sync(0xffffffffu, pid, col - pg0);
            const bool values = cp_half & 1;
            const int64_t ph = static_cast<int64_t>(max(page, 0)) * s.heads_kv + cp.h;
            const uint8_t* src = static_cast<const uint8_t*>(values ? a.v_cache : a.k_cache) +
                                 ((ph << s.ps_shift) + (key0 & ((1 << s.ps_shift) - 1))) * D;
            uint8_t* dst = raw + (cp_half % C::RAW) * C::RAW_BYTES;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const int row = (v & 1) * 8 + (lane >> 2);
              const uint32_t n = page >= 0 && key0 + row < cp.q.len ? 16u : 0u;   // else zeros
              cp_async16(smem_u32(dst + (v * 32 + lane) * 16), src + row * D + (v >> 1) * 64 + (lane & 3) * 16, n);
            }
            if (lane == 0) {
              float* sc = &sh_scale[w][cp_half % C::RAW];
              if (page >= 0)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(sc)),
                             "l"((values ? a.v_scale : a.k_scale) + ph)
                             : "memory");
              else
                *sc = 0.f;
              // (missing pages; keys past the length are masked by it)
              if (!values)
                reinterpret_cast<volatile uint8_t*>(&sh_bad[cp_chunk & 15])[w] = page < 0 && key0 < cp.q.len;
            }
            if (values) {
              ++cp_c;
              ++cp_chunk;
            }
            ++cp_half;
          }
          cp_async_commit();
        };
        TcItem it = first;
        int64_t left = range;
        Part pt = part_of(it, first_c0, left);
        for (int i = 0; i < C::RAW; ++i) copy();
        int half = 0;
        bool ok = true;
        while (ok) {
          for (int i = 0; ok && i < 2 * pt.n_kv; ++i, ++half) {
            cp_async_wait<C::RAW - 1>();
            __syncwarp();
            const int slot = half % C::NSLOT;
            if (!mbar_wait_w(&bar_empty[slot], ((half / C::NSLOT) & 1) ^ 1, ac)) { ok = false; break; }
            const uint8_t* src = raw + (half % C::RAW) * C::RAW_BYTES;
            const float sc = sh_scale[w][half % C::RAW];
            const uint64_t sc2 = f2_pack(sc, sc);
            uint8_t* dst = sRing + slot * C::KV_BYTES;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const int row = 16 * w + (v & 1) * 8 + (lane >> 2);
              const uint4 x = *reinterpret_cast<const uint4*>(src + (v * 32 + lane) * 16);
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
              uint8_t* line = dst + (v >> 1) * (BN * 128) + row * 128;
              const int ch = 2 * (lane & 3);
              *reinterpret_cast<uint4*>(line + ((ch ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(line + (((ch + 1) ^ (row & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar_full[slot]);
            __syncwarp();
            copy();
          }
          if (!ok || !advance(it, pt, left)) break;
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
    TcItem it = first;
    int64_t left = range;
    Part pt = part_of(it, first_c0, left);
    int cs = 0, gchunk = 0;
    bool ok = true;
    while (ok) {
      const int nt = pt.n_w[t];
      const int tok0 = (2 * it.rb + t) * a.tile_tokens, tok = tok0 + row_tok;
      const int lim = a.causal ? min(it.q.len - 1, it.q.pos0 + tok) : it.q.len - 1;   // last key seen
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
        const int kv0 = (pt.c0 + j) * BN;
        const int bad = sh_bad[(gchunk + j) & 15];
        if (kv0 + BN > it.q.len || (a.causal && kv0 + BN - 1 > it.q.pos0 + tok0)) {
#pragma unroll
          for (int cc = 0; cc < BN; ++cc)
            if (kv0 + cc > lim) x[cc] = -INFINITY;
        }
        if (bad) {
#pragma unroll
          for (int cc = 0; cc < BN; ++cc)
            if (bad >> (BAD_SHIFT * (cc / 16)) & 1) x[cc] = -INFINITY;
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
      const bool begins = pt.c0 == 0, ends = pt.c0 + pt.span == it.nc, whole = begins && ends;
      const int which = begins ? 1 : 0;
      if (ok && nt > 0) {
        ok = mbar_wait(&bar_o[t], (cs + nt - 1) & 1, ac);
        tc_fence_after();
      }
      if (ok) {
        const bool valid = row_in && tok < it.q.m;
        const float inv = l_run > 0.f || l_run != l_run ? 1.0f / l_run : 0.f;
        const int hd = it.h * s.group + row_head;
        __nv_bfloat16* orow = a.o + (static_cast<int64_t>(it.q.t0 + tok) * s.heads_q + hd) * D;
        const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + which) * 2 * C::BM + t * C::BM + tr;
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
            a.lse[static_cast<int64_t>(hd) * s.tokens + it.q.t0 + tok] =
                l_run > 0.f || l_run != l_run ? (m_run + __log2f(l_run)) * kLn2 : -INFINITY;
          } else {
            a.part_ml[at] = make_float2(m_run, l_run);
          }
        }
        if (!whole && threadIdx.x == 0)
          a.part_meta[2 * blockIdx.x + which] = make_int4(1 | (begins ? 2 : 0) | (ends ? 4 : 0), it.n, it.h, it.rb);
      }
      cs += nt;
      gchunk += pt.n_kv;
      if (!ok || !advance(it, pt, left)) break;
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

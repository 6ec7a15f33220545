// Linear attention in chunks of C = 128 tokens on tcgen05 (linear.h; the jobs are
// those of linear.cuh).  With H the state at a chunk's near end, rows i and j of
// the chunk, and w the decays and factors of the direction,
//   out = (X Y^T o W) Z + diag(u) X H,     H <- l^C H + (diag(d) Y)^T Z
//   forwards   W_ij = scale l^(i - j), j <= i;  u_i = scale l^(i + 1);  d_j = l^(c - 1 - j)
//   backwards  W_ij = scale l^(j - i), j >= i;  u_i = l^(c - 1 - i);    d_j = scale l^(j + 1)
// (c <= C rows are the sequence's).  Decays are powers of l <= 1 with exponents of at
// least 0, so none overflows and those that underflow do not matter.
//
// A CTA walks the chunks of one (sequence, head, segment) and keeps H in the
// registers of its state warps:
//   warp 0        TMA producer: X, then Y and Z of each inner head, into a ring of tiles
//   warp 1        MMA issuer: S = X Y^T, G += (diag(d) Y)^T Z, O = X H, O += P Z
//   warp 3        bulk copies of the output
//   warps 4..7    scores: S to P = S o W as packed bf16 in TMEM, and O to diag(u) O before P Z is
//                 added to it; the output to the tile of the chunk's last Z
//   warps 8..15   state: Y to diag(d) Y in place (bf16; the second and third terms in
//                 tiles of their own), H = l^C H + G, H as bf16 to shared memory; where X has
//                 two buffers the output
// S is scaled by products of two table values below and above the diagonal block
// of 32 x 32, by a table of the 63 diagonals in it.
//
// Bound by: a chunk's tiles of 4 x 32 KB take 4700 cycles of an SM's share of the
// bandwidth where 128 SMs read (D = 128, one inner head), its products 2560 of the
// tensor cores; measured 5800 (3.1 us: 4 x 8192 tokens against 4 x 4096), as each product waits in turn for
// the warps that prepare its operands, and the warp that issues them passes one barrier after the
// other (300 to 400 cycles each).  So the order of the products is what matters: S
// of the next step goes out before P Z of this one where the ring holds both.
// 4 x 4096 tokens of 32 heads of 128: 116 us, 5 of them a graph's launch and 12 the walks' start and end;
// 79 for the bytes alone.
// Slower, same sizes: two issuing warps 8 %, one wait for several barriers 5 %, the next
// chunks' tiles fetched to L2 11 %, a ring of 3 tiles 11 %.  Products go out in fours, from loops:
// two at a time 7 % slower, all unrolled 5 % (the roles share the instruction caches).
// At D = 64 there is a second variant with two CTAs on an SM (kCtas, 64 registers a thread, one
// buffer of S; it spills 160 to 190 bytes a thread, the others none to 20), for many short walks:
// linear_api.cu has the rule.
#include "linear.cuh"

namespace attn {
namespace {

template <int D, int NS, bool kStates, int kCtas>
struct Cfg {
  static constexpr int C = kLinearChunk;
  static constexpr int TILE = C * D * 2;
  static constexpr int HTERMS = state_terms(D, NS, kCtas == 2);
  static constexpr int H_BYTES = kStates ? 0 : D * D * 2 * HTERMS;
  // second and third terms of the decayed keys; two of them where a step's are made while the step
  // before is at work (12 packed sequences of up to 2500 tokens, 16 heads of 64, their backward with
  // states 106 -> 93 us)
  static constexpr int EBUF = kStates && D == 64 && kCtas == 1 ? 2 : 1;
  static constexpr int EXTRA = EBUF * (NS - 1) * TILE;
  // the tiles that fit: 227 KB of shared memory, or 113 for each of two CTAs, 2 KB of it for the
  // alignment and what is static
  static constexpr int FIT = ((kCtas == 2 ? 113 : 227) * 1024 - 2048 - H_BYTES - EXTRA) / TILE;
  // X has buffers of its own: a chunk's X outlives the tiles of its inner heads
  static constexpr int XBUF = kStates ? 0 : FIT >= 6 ? 2 : 1;
  static constexpr int XMOD = XBUF ? XBUF : 1;
  static constexpr int NSLOT = (FIT > 8 ? 8 : FIT) - XBUF;
  static constexpr int SMEM = (XBUF + NSLOT) * TILE + H_BYTES + EXTRA + 1024;
  static constexpr int THREADS = 512;
  static constexpr int HC = D / 2;                // state columns of a thread
  // S of a step is formed while the step before is still at work, where the ring can hold both: with
  // three tiles the wait for the next Y would hold up the Z that has to leave before it
  static constexpr bool AHEAD = !kStates && kCtas == 1 && NSLOT >= 4;
  // the warps that write the output: the score warps where S of the next chunk is formed late and
  // leaves them waiting (backward of 4 x 4096 tokens of 32 heads of 128 345 -> 341 us; of 64, one CTA
  // on an SM, 226 -> 252)
  static constexpr bool OUT_BY_SCORES = XBUF == 1;
  static constexpr uint32_t COLS = 512 / kCtas;   // of TMEM
  static constexpr uint32_t COL_S = 0, S_STEP = AHEAD ? 128 : 0;   // AHEAD: two buffers
  static constexpr uint32_t COL_O = COLS / 2, COL_G = kStates ? 0 : COL_O + D;
  // without S and O there is room for two of G: a chunk's is read while the next one's is formed
  static constexpr int GBUF = kStates ? 2 : 1;
  static_assert(NSLOT >= 3, "Y and Z and one on its way");
  // (the state warps tell the products of two steps before by a slot's barrier: it must not come
  // round again until they have)
  static_assert((!kStates && EBUF == 1) || NSLOT >= 4, "a slot's turns");
};

// exp(g m) for a state that is returned: of the product and, to first order, its rounding.
__device__ __forceinline__ float decay_exact(float g, float m) {
  const float p = g * m, e = expf(p);
  return fmaf(e, fmaf(g, m, -p), e);
}

// A walk's place: sequence n, its segment `seg` of `nseg`, each of `per` chunks at most; segment
// i hands its state on at place first + i of the workspace.
struct Place {
  int n, row0, len, seg, nseg, per, first;
};

// The segment that the CTAs of a slot take, by one warp; n = -1 where there is none.  The pass over the
// states leaves out each sequence's last segment in the walk's direction.  The longer
// walks of each 32 packed sequences come first, so that no SM is left with one at the
// end (backward of 12 sequences of up to 2500 tokens, 16 heads of 64, the jobs' walks in turn, then 110
// us: 118 with each job's in the sequences' order).  The search takes n / 32 steps for n sequences, in each CTA:
// packed by the thousand they cost more than their rows (2000 of up to 16 tokens, 16 heads of 64, 2.3 ms).
template <bool kStates>
__device__ __forceinline__ Place find_place(const LinearArgs& a, const LinearJob& j, int slot) {
  constexpr int kLeft = kStates ? 1 : 0;   // segments of a sequence that have no slot
  Place p{-1, 0, 0, 0, 1, 1, 0};
  if (!a.cu) {
    p.nseg = segments_of(a.seqlen, j.seg_chunks);
    const int count = p.nseg - kLeft;
    p.n = count > 0 ? slot / count : a.num_seqs;
    p.seg = slot - p.n * count;
    p.first = p.n * (p.nseg - 1);
    if (p.n >= a.num_seqs) p.n = -1;
    else sequence_rows(a, p.n, p.row0, p.len);
  } else {
    const int lane = lane_id();
    for (int n0 = 0, before = 0, handed = 0, top = 0; n0 < a.num_seqs; n0 += 32) {
      int row0, len;
      packed_rows(a, n0, top, row0, len);
      const bool live = n0 + lane < a.num_seqs;   // (lanes past the last sequence count none)
      const int nseg = live ? segments_of(len, j.seg_chunks) : 0;
      const int count = live ? nseg - kLeft : 0;
      const int all = __reduce_add_sync(0xffffffffu, count);
      const int on = kStates ? all : all - min(32, a.num_seqs - n0);   // states handed on
      if (slot < before + all) {
        const int per = live ? (chunks_of(len) + nseg - 1) / nseg : 0;
        int turn = before;     // segments of the block's sequences with longer walks
        int prior = handed;    // states that those before hand on
#pragma unroll 4
        for (int d = 0; d < min(32, a.num_seqs - n0); ++d) {
          const int p2 = __shfl_sync(0xffffffffu, per, d), c2 = __shfl_sync(0xffffffffu, count, d);
          turn += p2 > per || (p2 == per && d < lane) ? c2 : 0;
          prior += d < lane ? c2 - (1 - kLeft) : 0;
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, slot >= turn && slot < turn + count)) - 1;
        p.n = n0 + src;
        p.row0 = __shfl_sync(0xffffffffu, row0, src);
        p.len = __shfl_sync(0xffffffffu, len, src);
        p.nseg = __shfl_sync(0xffffffffu, nseg, src);
        p.seg = slot - __shfl_sync(0xffffffffu, turn, src);
        p.first = __shfl_sync(0xffffffffu, prior, src);
        break;
      }
      before += all;
      handed += on;
    }
  }
  if (j.backwards) {   // segment 0 hands nothing on
    if (kStates) ++p.seg;
    --p.first;
  }
  p.per = (chunks_of(p.len) + p.nseg - 1) / p.nseg;
  return p;
}

// Bounded waits in few instructions: the kernel's roles have to share the instruction
// caches (at 117 KB of code the walk ran at half its speed).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const AbortCtx& c) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (uint32_t n = 0; n < (1u << 20); ++n) {
    if (mbar_try_wait_hint(addr, parity, 20000u)) return true;
    if (*reinterpret_cast<volatile int*>(c.smem_abort)) return false;
  }
  raise_error(c, ATTN_DEVERR_TIMEOUT);
  return false;
}
// The same by polling, for the warp that issues the products, with a warp-uniform result.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const AbortCtx& c) {
  const uint32_t addr = smem_u32(bar);
  bool ok = false;
#pragma unroll 1
  for (uint32_t n = 0; n < (1u << 26) && !ok; ++n) {
    ok = mbar_test_wait(addr, parity);
    if (!ok && (n & 1023) == 1023 && *reinterpret_cast<volatile int*>(c.smem_abort)) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) raise_error(c, ATTN_DEVERR_TIMEOUT);
  return ok;
}

// One arrival for a warp, behind all its lanes: 256 arrivals of a role's threads at one barrier
// take their turns.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(bar);
}

template <int D, int NS, bool kStates, int kCtas>
__global__ void __launch_bounds__(512, kCtas) linear_kernel(const __grid_constant__ LinearArgs a) {
  using C = Cfg<D, NS, kStates, kCtas>;
  constexpr int PANELS = D / 64;
  constexpr int NSLOT = C::NSLOT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sX = ring + NSLOT * C::TILE;
  uint8_t* sH = sX + C::XBUF * C::TILE;
  uint8_t* sExtra = sH + C::H_BYTES;

  // bar_out: an output's barrier comes round with its tile at the soonest, so that the warp that
  // waits is never two phases behind
  __shared__ uint64_t bar_full[NSLOT], bar_empty[NSLOT], bar_out[NSLOT];
  __shared__ uint64_t bar_xfull[2], bar_xempty[2];
  __shared__ uint64_t bar_s[2], bar_p[2], bar_y[2], bar_g[2], bar_gf[2], bar_qh, bar_o, bar_of, bar_h, bar_keep;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ Place s_place;
  __shared__ __align__(16) float s_tab[32];   // decays within a block of 32 columns
  __shared__ float s_keep[2];                 // a chunk's decay
  __shared__ float s_diag[64];                // those of its diagonal, scaled: entry 32 + j - i

  // The walks of the outputs start on SMs that the pass over the states leaves, once all of its CTAs
  // have theirs, and wait for its end where they take a state from it (2 to 4 us of each
  // call with such a pass).
  if (kStates) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = warp_id();
  AbortCtx ac{&abort_flag, a.err};

  // ---- the walk ----
  int ji = 0, item = blockIdx.x;
  while (ji + a.merged < a.jobs && item >= a.merged * a.job[ji].slots * a.job[ji].heads_x) {
    item -= a.merged * a.job[ji].slots * a.job[ji].heads_x;
    ji += a.merged;
  }
  int slot = static_cast<int>(fdiv(item, a.job[ji].fd_heads));
  const int h = item - slot * a.job[ji].heads_x;
  if (a.merged > 1) {   // the jobs' places in turn
    const int q = slot / a.merged;
    ji += slot - q * a.merged;
    slot = q;
  }
  const LinearJob& j = a.job[ji];
  item = slot * j.heads_x + h;
  const int hkv = static_cast<int>(fdiv(h, j.fd_kv));

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
      mbar_init(&bar_out[i], C::OUT_BY_SCORES ? 4 : 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_xfull[i], 1);
      mbar_init(&bar_xempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_p[i], 4);
      mbar_init(&bar_y[i], 8);
      mbar_init(&bar_g[i], 1);
      mbar_init(&bar_gf[i], 8);
    }
    mbar_init(&bar_keep, 1);
    mbar_init(&bar_qh, 1);
    mbar_init(&bar_o, 1);
    mbar_init(&bar_of, C::OUT_BY_SCORES ? 4 : 8);
    mbar_init(&bar_h, 8);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, C::COLS);
    tmem_relinquish();
  }
  const float ln = log_decay_of(a, hkv), l2 = ln * kLog2e;
  if (warp == 2) {
    const Place p = find_place<kStates>(a, j, slot);
    if (lane_id() == 0) s_place = p;
  }
  if (warp == 3) {
    const int x = lane_id();
    s_tab[x] = ex2(l2 * (j.backwards ? x : 31 - x));
    s_diag[x] = j.backwards ? 0.f : a.scale * ex2(l2 * (32 - x));
    s_diag[32 + x] = j.backwards || x == 0 ? a.scale * ex2(l2 * x) : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  const Place pl = s_place;
  const bool back = j.backwards;
  // the sequence's last segment in the walk's direction, which no state follows
  const bool is_end = pl.n >= 0 && pl.seg == (back ? 0 : pl.nseg - 1);
  const int nch = pl.n < 0 ? 0 : chunks_of(pl.len);
  const int c_lo = min(nch, pl.seg * pl.per), c_hi = min(nch, c_lo + pl.per);
  const int n_walk = c_hi - c_lo;
  const int inner = j.inner;
  // of the walk's n-th chunk: its first token, and its tokens
  auto chunk_row = [&](int n) { return (back ? c_hi - 1 - n : c_lo + n) * kLinearChunk; };
  auto chunk_len = [&](int n) { return min(kLinearChunk, pl.len - chunk_row(n)); };
  const bool want_last = kStates || (is_end && j.last && h == hkv * static_cast<int>(j.fd_kv.d));
  // bf16 terms of the decayed keys: three for a state that is returned
  const int terms = NS > 1 && want_last ? j.terms : C::HTERMS == 2 ? 1 : 2;
  // The tensor cores cut a sum off rather than round it, at each of the 8 products of a step.  Where
  // a state is returned the smaller terms are added first, and the steps of a chunk one by
  // one into H (2 sequences of 4937 tokens, 8 query heads a KV head: 3.6e-6 of the state's
  // root mean square with the leading terms first and a chunk's steps in one sum).
  const bool each = NS > 1 && terms > 2;
  const int n_grow = want_last ? n_walk : n_walk - 1;   // chunks that the state takes in
  const int steps = n_walk * inner;                     // a step: one inner head of a chunk

  // chunk n's rows, columns [c0, c0 + cols), to the place of its last Z, which the products have
  // read: rows written from registers, 16 bytes of 32 rows at a time, took 2000 cycles
  auto output = [&](int n, int c0, int cols) -> bool {
    if (!wait(&bar_o, n & 1, ac)) return false;
    tc_fence_after();
    const int wq = warp & 3, row = threadIdx.x & 127;   // (TMEM lane)
    const uint32_t tO = tmem + (static_cast<uint32_t>(wq * 32) << 16) + C::COL_O;
    uint8_t* so = ring + (2 * (n + 1) * inner - 1) % NSLOT * C::TILE;
#pragma unroll 1
    for (int cc = c0; cc < c0 + cols; cc += 32) {
      uint32_t o[32];
      tmem_ld32_nowait(tO + cc, o);
      tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 32; x += 8) {
        uint32_t w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          w[y] = pack_bf16(__uint_as_float(o[x + 2 * y]), __uint_as_float(o[x + 2 * y + 1]));
        *reinterpret_cast<uint4*>(so + sw128_offset(row, cc + x, kLinearChunk)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    tc_fence_before();
    warp_arrive(&bar_of);
    fence_proxy_async_smem();
    warp_arrive(&bar_out[n % NSLOT]);
    return true;
  };

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane_id() == 0 && n_walk > 0) {
      tma_prefetch_desc(&j.my);
      tma_prefetch_desc(&j.mz);
      const int hy = inner > 1 || kStates ? h * inner : hkv;
      int it = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* m, uint64_t* full, uint64_t* empty, uint8_t* dst, int use, int head, int row) {
        if (use > 0 && !wait(empty, (use & 1) ^ 1, ac)) {
          ok = false;
          return;
        }
        mbar_arrive_expect_tx(full, C::TILE);
        for (int pn = 0; pn < PANELS; ++pn)
          tma_load_3d(m, full, dst + pn * kLinearChunk * 128, pn * 64, head, row);
      };
      for (int n = 0; ok && n < n_walk; ++n) {
        const int row = pl.row0 + chunk_row(n);
        if constexpr (!kStates) {
          const int b = n % C::XBUF;
          load(&j.mx, &bar_xfull[b], &bar_xempty[b], sX + b * C::TILE, n / C::XBUF, h, row);
        }
        for (int t = 0; ok && t < 2 * inner; ++t, ++it) {
          const int s = it % NSLOT;
          load(t & 1 ? &j.mz : &j.my, &bar_full[s], &bar_empty[s], ring + s * C::TILE, it / NSLOT, hy + (t >> 1), row);
          // the next chunk's last Z comes to L2 before its tile, which this chunk's output holds longest
          if (!kStates && t == 2 * inner - 1 && n + 1 < n_walk)
            for (int pn = 0; pn < PANELS; ++pn)
              tma_prefetch_3d(&j.mz, pn * 64, hy + (t >> 1), pl.row0 + chunk_row(n + 1));
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    const uint32_t idS = idesc_bf16(128, 128, false, false);
    const uint32_t idO = idesc_bf16(128, D, false, true);
    const uint32_t idG = idesc_bf16(D, D, true, true);
    const uint64_t dk0 = desc_kmajor_base(smem_u32(ring));
    const uint64_t dx0 = desc_kmajor_base(smem_u32(sX));
    const uint64_t dm0 = desc_mnmajor_base(smem_u32(ring), kLinearChunk);
    const uint64_t dH = desc_mnmajor_base(smem_u32(sH), D);
    const uint64_t dE = desc_mnmajor_base(smem_u32(sExtra), kLinearChunk);
    // from one K step to the next, in a descriptor's 16 bytes: along a tile's rows, and down its columns
    constexpr int kRowStep = kmajor_step_bytes(128, 1) / 16, kColumnStep = mnmajor_step_bytes(1) / 16;
    auto slot = [](int tile) { return tile % NSLOT; };
    auto landed = [&](int tile) { return warp_wait(&bar_full[slot(tile)], (tile / NSLOT) & 1, ac); };
    // S of step t, the g-th of chunk n
    auto scores = [&](int t, int n, int g) -> bool {
      const int bx = n % C::XMOD;
      if (g == 0 && !warp_wait(&bar_xfull[bx], (n / C::XMOD) & 1, ac)) return false;
      if (!landed(2 * t)) return false;
      tc_fence_after();
      const uint64_t dx = desc_advance(dx0, bx * C::TILE), dy = desc_advance(dk0, slot(2 * t) * C::TILE);
#pragma unroll 1
      for (int k = 0; k < D / 16; k += 4)
        umma4_ss_w<kRowStep, kRowStep>(tmem + C::COL_S + C::S_STEP * (t & 1),
                                       desc_advance(dx, kmajor_step_bytes(128, k)),
                                       desc_advance(dy, kmajor_step_bytes(128, k)), idS, k > 0);
      umma_commit_w(&bar_s[t & 1]);
      return true;
    };
    // what the state takes in
    auto keys = [&](int t, int n, int g) -> bool {
      if (!landed(2 * t + 1) || (kStates && !landed(2 * t))) return false;
      const int i = each ? t : n, b = i % C::GBUF;   // G's turn and buffer
      if (n < n_grow) {
        if (!warp_wait(&bar_y[t & 1], (t >> 1) & 1, ac)) return false;
        if ((each || g == 0) && i >= C::GBUF && !warp_wait(&bar_gf[b], (i / C::GBUF - 1) & 1, ac)) return false;
        tc_fence_after();
        const uint64_t dy = desc_advance(dm0, slot(2 * t) * C::TILE), dz = desc_advance(dm0, slot(2 * t + 1) * C::TILE);
        uint32_t add = !each && g > 0;
#pragma unroll 1
        for (int e = terms - 1; e >= 0; --e)
#pragma unroll 1
          for (int k = 0; k < 8; k += 4, add = 1)
            umma4_ss_w<kColumnStep, kColumnStep>(
                tmem + C::COL_G + 128 * b,
                desc_advance(e == 0 ? dy : desc_advance(dE, (e - 1 + t % C::EBUF * (NS - 1)) * C::TILE),
                             mnmajor_step_bytes(k)),
                desc_advance(dz, mnmajor_step_bytes(k)), idG, add);
      }
      umma_commit_w(&bar_empty[slot(2 * t)]);
      if (n < n_grow && (each || g == inner - 1)) umma_commit_w(&bar_g[b]);
      return true;
    };
    // X H, at a chunk's first step; behind the S of its last step, X is free
    auto carried = [&](int n, int g) -> bool {
      const int bx = n % C::XMOD;
      if (g == 0) {
        if (!warp_wait(&bar_h, n & 1, ac) || (n > 0 && !warp_wait(&bar_of, (n - 1) & 1, ac))) return false;
        tc_fence_after();
        const uint64_t dx = desc_advance(dx0, bx * C::TILE);
#pragma unroll 1
        for (int k = 0; k < C::HTERMS * D / 16; k += 4)   // (the second term lies behind the first)
          umma4_ss_w<kRowStep, kColumnStep>(
              tmem + C::COL_O, desc_advance(dx, kmajor_step_bytes(128, k % (D / 16))),
              desc_advance(dH, (k / (D / 16)) * (D * D * 2) + mnmajor_step_bytes(k % (D / 16))), idO, k > 0);
        umma_commit_w(&bar_qh);
      }
      if (C::AHEAD ? inner == 1 : g == inner - 1) umma_commit_w(&bar_xempty[bx]);
      return true;
    };
    auto values = [&](int t, int g) -> bool {
      if (!warp_wait(&bar_p[t & 1], (t >> 1) & 1, ac)) return false;
      tc_fence_after();
      const uint64_t dz = desc_advance(dm0, slot(2 * t + 1) * C::TILE);
#pragma unroll 1
      for (int k = 0; k < 8; k += 4)
        umma4_ts_w<8, kColumnStep>(tmem + C::COL_O, tmem + C::COL_S + C::S_STEP * (t & 1) + 8 * k,
                                   desc_advance(dz, mnmajor_step_bytes(k)), idO, 1u);
      if (g == inner - 1) umma_commit_w(&bar_o);
      return true;
    };
    // AHEAD, S(t + 1) runs while the score warps scale X H of t, and they form P(t + 1) while the
    // others' products run
    int n = 0, g = 0;
    if (C::AHEAD && (steps == 0 || !scores(0, 0, 0))) n = n_walk;
    for (int t = 0; n < n_walk; ++t) {
      const bool last = g == inner - 1;
      if constexpr (kStates) {
        if (!keys(t, n, g)) break;
      } else if constexpr (C::AHEAD) {
        // (with one buffer for X the next chunk's has to wait for X H of this one)
        const bool late = C::XBUF == 1 && last;
        if (C::XBUF == 1 ? !carried(n, g) || !keys(t, n, g) : !keys(t, n, g) || !carried(n, g)) break;
        if (!late && t + 1 < steps && !scores(t + 1, n + last, last ? 0 : g + 1)) break;
        if (g + 2 == inner) umma_commit_w(&bar_xempty[n % C::XMOD]);
        if (!values(t, g)) break;
        if (late && t + 1 < steps && !scores(t + 1, n + 1, 0)) break;
      } else {
        if (!scores(t, n, g) || !carried(n, g) || !keys(t, n, g) || !values(t, g)) break;
      }
      // a chunk's last Z makes room for its output
      if (kStates || !last) umma_commit_w(&bar_empty[slot(2 * t + 1)]);
      n += last;
      g = last ? 0 : g + 1;
    }
  } else if (NS > 1 && warp == 2) {
    // A chunk's decay in two parts: an error of it would grow with every chunk that a state crosses.
    // Behind the block's barrier, for exp in fp64 is slow here (500 tokens with states 31 -> 30 us).
    if (lane_id() == 0) {
      const double keep = exp(static_cast<double>(ln) * kLinearChunk);
      s_keep[0] = static_cast<float>(keep);
      s_keep[1] = static_cast<float>(keep - s_keep[0]);
      mbar_arrive(&bar_keep);
    }
  } else if (!kStates && warp == 3) {
    // ---------------- stores ----------------
    // whole chunks leave by a bulk copy, others (rows behind the sequence are another's) by plain
    // stores; behind them the tile of the chunk's last Z, in which they lay, is free
    for (int n = 0; n < n_walk; ++n) {
      const int b = (2 * (n + 1) * inner - 1) % NSLOT, rows = chunk_len(n), row = pl.row0 + chunk_row(n);
      uint8_t* so = ring + b * C::TILE;
      if (!__all_sync(0xffffffffu, wait(&bar_out[n % NSLOT], (n / NSLOT) & 1, ac))) break;
      if (rows == kLinearChunk) {
        if (lane_id() == 0) {
          for (int pn = 0; pn < PANELS; ++pn) tma_store_3d(&j.mo, so + pn * kLinearChunk * 128, pn * 64, h, row);
          bulk_commit();
          bulk_wait_read<0>();
        }
      } else {
        __nv_bfloat16* out = j.out + (static_cast<int64_t>(row) * j.heads_x + h) * D;
#pragma unroll 4
        for (int x = lane_id(); x < rows * (D / 8); x += 32) {
          const int ro = x / (D / 8), co = x % (D / 8) * 8;
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(ro) * j.heads_x * D + co) =
              *reinterpret_cast<const uint4*>(so + sw128_offset(ro, co, kLinearChunk));
        }
        fence_proxy_async_smem();
      }
      warp_arrive(&bar_empty[b]);
    }
  } else if (!kStates && warp >= 4 && warp < 8) {
    // ---------------- scores ----------------
    const int wq = warp & 3, i = threadIdx.x & 127;   // row of the chunk, TMEM lane
    const int lane = lane_id();
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    // step t's scores, of a chunk with `rows` rows, to P
    auto convert = [&](int t, int rows) -> bool {
      if (!wait(&bar_s[t & 1], (t >> 1) & 1, ac)) return false;
      tc_fence_after();
      const uint32_t tS = lane_base + C::COL_S + C::S_STEP * (t & 1);
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        uint32_t p[16];
        if (back ? b < wq : b > wq) {
#pragma unroll
          for (int x = 0; x < 16; ++x) p[x] = 0;
        } else {
          uint32_t s[32];
          tmem_ld32_nowait(tS + 32 * b, s);
          if (b == wq) {
            const float* diag = s_diag + 32 - lane;
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              // (selects: a masked score may be infinite or NaN)
              const float f0 = diag[x], f1 = diag[x + 1];
              const float u = __uint_as_float(s[x]) * f0, v = __uint_as_float(s[x + 1]) * f1;
              p[x / 2] = pack_bf16(f0 != 0.f ? u : 0.f, f1 != 0.f ? v : 0.f);
            }
          } else {
            // the exponent left once the table's part is taken
            const float base = a.scale * ex2(l2 * (back ? 32 * b - i : i - 32 * b - 31));
            const uint64_t base2 = f2_pack(base, base);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(s_tab + x);
              const uint64_t u = f2_pack(__uint_as_float(s[x]), __uint_as_float(s[x + 1]));
              const uint64_t v = f2_pack(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3]));
              p[x / 2] = f2_to_bf16x2(f2_mul(u, f2_mul(base2, t.x)));
              p[x / 2 + 1] = f2_to_bf16x2(f2_mul(v, f2_mul(base2, t.y)));
            }
          }
          if (back && rows < 32 * b + 32) {   // columns behind the sequence
#pragma unroll
            for (int x = 0; x < 16; ++x)
              p[x] &= 32 * b + 2 * x + 1 < rows ? 0xffffffffu : 32 * b + 2 * x < rows ? 0xffffu : 0u;
          }
        }
        tmem_st16p(tS + 16 * b, p);
      }
      return true;
    };
    int n = 0, g = 0;
    bool last = false;
    for (int t = C::AHEAD ? -1 : 0; t < steps; ++t) {   // step -1: the first scores alone
      const int rows = chunk_len(n);
      if (!C::AHEAD && !convert(t, rows)) break;
      if (t >= 0) {
        last = g == inner - 1;
        if (rows < kLinearChunk && n >= n_grow) {
          // rows of Z behind the sequence may hold anything: zeros, for 0 * NaN (the state warps
          // see to it where the state takes them in)
          const int sz = (2 * t + 1) % NSLOT;
          if (!wait(&bar_full[sz], ((2 * t + 1) / NSLOT) & 1, ac)) break;
          if (i >= rows) {
            uint4* z = reinterpret_cast<uint4*>(ring + sz * C::TILE + i * 128);
#pragma unroll
            for (int x = 0; x < D / 8; ++x) z[(x >> 3) * (kLinearChunk * 8) + (x & 7)] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (g == 0) {
          // X H of the chunk, times u: what P Z adds to
          if (!wait(&bar_qh, n & 1, ac)) break;
          tc_fence_after();
          const float u = back ? ex2(l2 * max(rows - 1 - i, 0)) : a.scale * ex2(l2 * (i + 1));
          const uint64_t u2 = f2_pack(u, u);
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            uint32_t o[32];
            tmem_ld32_nowait(lane_base + C::COL_O + cc, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              float lo, hi;
              f2_unpack(f2_mul(u2, f2_pack(__uint_as_float(o[x]), __uint_as_float(o[x + 1]))), lo, hi);
              o[x] = __float_as_uint(lo);
              o[x + 1] = __float_as_uint(hi);
            }
            tmem_st32(lane_base + C::COL_O + cc, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&bar_p[t & 1]);
        if (C::OUT_BY_SCORES && last && !output(n, 0, D)) break;
      }
      if (C::AHEAD && t + 1 < steps && !convert(t + 1, chunk_len(last ? n + 1 : n))) break;
      if (t >= 0) {
        n += last;
        g = last ? 0 : g + 1;
      }
    }
  } else if (warp >= 8 && pl.n >= 0) {
    // ---------------- output and state ----------------
    const int tid = threadIdx.x - 256, half = tid >> 7, wq = warp & 3;
    // M = 64 results lie in the first 16 lanes of each warp's 32
    const bool mine = D == 128 || (lane_id() < 16);
    const int r = D == 128 ? (tid & 127) : 16 * wq + (lane_id() & 15);
    const int c0 = half * C::HC;
    const uint32_t tG = tmem + (static_cast<uint32_t>(wq * 32) << 16) + C::COL_G + c0;
    float H[C::HC];
#pragma unroll
    for (int x = 0; x < C::HC; ++x) H[x] = 0.f;
    if (!kStates) {
      // the state before the segment: the first one, then what each segment on the way adds
      if (j.first && mine) {
        const float* f = j.first + (static_cast<int64_t>(pl.n) * a.heads_kv + hkv) * D * D;
        if (j.transposed) {
#pragma unroll
          for (int x = 0; x < C::HC; ++x) H[x] = __ldg(f + (c0 + x) * D + r);
        } else {
#pragma unroll
          for (int x = 0; x < C::HC; x += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(f + r * D + c0 + x));
            H[x] = v.x, H[x + 1] = v.y, H[x + 2] = v.z, H[x + 3] = v.w;
          }
        }
      }
      const int before = back ? pl.nseg - 1 - pl.seg : pl.seg;
      if (before > 0) asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int t = 0; t < before; ++t) {
        const int sg = back ? pl.nseg - 1 - t : t;
        const int lo = sg * pl.per * kLinearChunk, hi = min(pl.len, lo + pl.per * kLinearChunk);
        const float keep = NS > 1 ? decay_exact(ln, max(hi - lo, 0)) : ex2(l2 * max(hi - lo, 0));
        const float4* g = reinterpret_cast<const float4*>(
            j.parts + (static_cast<int64_t>(pl.first + sg) * a.heads_kv + hkv) * D * D);
        if (mine)
#pragma unroll
          for (int x = 0; x < C::HC; x += 4) {
            const float4 v = __ldcg(g + ((c0 + x) >> 2) * D + r);
            H[x] = fmaf(keep, H[x], v.x);
            H[x + 1] = fmaf(keep, H[x + 1], v.y);
            H[x + 2] = fmaf(keep, H[x + 2], v.z);
            H[x + 3] = fmaf(keep, H[x + 3], v.w);
          }
      }
    }
    auto publish = [&]() {   // H as bf16, the B operand of X H
      if (mine)
#pragma unroll
        for (int x = 0; x < C::HC; x += 8) {
          uint32_t w[4], rest[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float lo = H[x + 2 * y], hi = H[x + 2 * y + 1];
            w[y] = pack_bf16(lo, hi);
            rest[y] = pack_bf16(lo - __uint_as_float(w[y] << 16), hi - __uint_as_float(w[y] & 0xffff0000u));
          }
          const uint32_t at = sw128_offset(r, c0 + x, D);
          *reinterpret_cast<uint4*>(sH + at) = make_uint4(w[0], w[1], w[2], w[3]);
          if (C::HTERMS == 2)
            *reinterpret_cast<uint4*>(sH + D * D * 2 + at) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
        }
      fence_proxy_async_smem();
      warp_arrive(&bar_h);
    };
    if (!kStates && n_walk > 0) publish();
    // what G's i-th turn holds, of chunk n, its first or its last; behind the last, the state as the
    // next chunk's operand
    auto grow = [&](int i, int n, bool first, bool last) -> bool {
      const int b = i % C::GBUF;
      if (!wait(&bar_g[b], (i / C::GBUF) & 1, ac)) return false;
      tc_fence_after();
      const int rows = chunk_len(n);
      float keep = ex2(l2 * rows), keep2 = 0.f;
      if (NS > 1) {
        if (!wait(&bar_keep, 0, ac)) return false;
        keep = !first ? 1.f : rows == kLinearChunk ? s_keep[0] : decay_exact(ln, rows);
        keep2 = first && rows == kLinearChunk ? s_keep[1] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < C::HC; x += 32) {
        uint32_t v[32];
        tmem_ld32_nowait(tG + 128 * b + x, v);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; ++y) {
          const float add = NS > 1 ? fmaf(keep2, H[x + y], __uint_as_float(v[y])) : __uint_as_float(v[y]);
          H[x + y] = fmaf(keep, H[x + y], add);
        }
      }
      tc_fence_before();
      warp_arrive(&bar_gf[b]);
      if (kStates || !last || n + 1 >= n_walk) return true;
      if (!wait(&bar_qh, n & 1, ac)) return false;   // the product that read the state before
      publish();
      return true;
    };
    const int row = tid & 127;   // row of the chunk
    int n = 0, g = 0;
    for (int t = 0; t <= steps; ++t) {
      const bool next = g == 0 && n > 0;   // a chunk is behind these warps
      // what is behind of G: a step, or the steps of a chunk
      const bool grown = each ? t > 0 && t <= n_grow * inner : next && n - 1 < n_grow;
      const int gi = each ? t - 1 : n - 1, gn = g == 0 ? n - 1 : n;
      if (!kStates && grown && !grow(gi, gn, !each || inner == 1 || g == 1, g == 0)) break;
      if (t < steps && n < n_grow) {
        const int rows = chunk_len(n);
        const int far = back ? row + 1 : max(rows - 1 - row, 0);
        const float d = (back ? a.scale : 1.f) * (NS > 1 ? decay_exact(ln, far) : ex2(l2 * far));
        const int sy = 2 * t % NSLOT;
        if (!wait(&bar_full[sy], (2 * t / NSLOT) & 1, ac)) break;
        if (!kStates && !wait(&bar_s[t & 1], (t >> 1) & 1, ac)) break;
        // the other terms' tiles: read by the products of the step before.  Where no scores hold
        // these warps back, they stay within what two barriers can tell apart.
        const int behind = terms > 1 && C::EBUF == 1 ? t - 1 : t - 2;
        if ((terms > 1 || kStates) && behind >= 0 &&
            !wait(&bar_empty[2 * behind % NSLOT], (2 * behind / NSLOT) & 1, ac))
          break;
        if (rows < kLinearChunk) {
          const int sz = (2 * t + 1) % NSLOT;
          if (!wait(&bar_full[sz], ((2 * t + 1) / NSLOT) & 1, ac)) break;
          if (row >= rows && half < PANELS) {
            uint4* z = reinterpret_cast<uint4*>(ring + sz * C::TILE + half * (kLinearChunk * 128) + row * 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) z[x] = make_uint4(0, 0, 0, 0);
          }
        }
        uint8_t* y = ring + sy * C::TILE;
        constexpr int kBatch = 4;   // pieces of 16 bytes loaded before the first is stored
#pragma unroll 1
        for (int x0 = 0; x0 < C::HC; x0 += 8 * kBatch) {
          uint4 v[kBatch];
#pragma unroll
          for (int x = 0; x < kBatch; ++x)
            v[x] = *reinterpret_cast<const uint4*>(y + sw128_offset(row, c0 + x0 + 8 * x, kLinearChunk));
          if (rows < kLinearChunk && row >= rows)
#pragma unroll
            for (int x = 0; x < kBatch; ++x) v[x] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int x = 0; x < kBatch; ++x) {
            const uint32_t at = sw128_offset(row, c0 + x0 + 8 * x, kLinearChunk);
            const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
            uint32_t term[NS][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = __uint_as_float(w[e] << 16) * d, hi = __uint_as_float(w[e] & 0xffff0000u) * d;
#pragma unroll
              for (int q = 0; q < NS; ++q) {
                term[q][e] = pack_bf16(lo, hi);
                lo -= __uint_as_float(term[q][e] << 16);
                hi -= __uint_as_float(term[q][e] & 0xffff0000u);
              }
            }
            *reinterpret_cast<uint4*>(y + at) = make_uint4(term[0][0], term[0][1], term[0][2], term[0][3]);
            if (NS > 1 && terms > 1)
#pragma unroll
              for (int q = 1; q < NS; ++q)
                *reinterpret_cast<uint4*>(sExtra + (q - 1 + t % C::EBUF * (NS - 1)) * C::TILE + at) =
                    make_uint4(term[q][0], term[q][1], term[q][2], term[q][3]);
          }
        }
        fence_proxy_async_smem();
        warp_arrive(&bar_y[t & 1]);
      }
      if (kStates && grown && !grow(gi, gn, !each || inner == 1 || g == 1, g == 0)) break;
      if (!kStates && !C::OUT_BY_SCORES && next && !output(n - 1, c0, C::HC)) break;
      if (++g == inner) {
        g = 0;
        ++n;
      }
    }
    if (kStates) {
      const int64_t at = (static_cast<int64_t>(pl.first + pl.seg) * a.heads_kv + hkv) * D * D;
      if (mine)
#pragma unroll
        for (int x = 0; x < C::HC; x += 4) {
          __stcg(reinterpret_cast<float4*>(j.parts + at) + ((c0 + x) >> 2) * D + r,
                 make_float4(H[x], H[x + 1], H[x + 2], H[x + 3]));
          if (j.parts_t)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              __stcg(j.parts_t + at + ((r >> 2) * D + c0 + x + y) * 4 + (r & 3), H[x + y]);
        }
    } else if (want_last && mine) {
      float4* f = reinterpret_cast<float4*>(j.last + ((static_cast<int64_t>(pl.n) * a.heads_kv + hkv) * D + r) * D + c0);
#pragma unroll
      for (int x = 0; x < C::HC; x += 4) f[x / 4] = make_float4(H[x], H[x + 1], H[x + 2], H[x + 3]);
    }
  }

  // ---- padding rows: at or past cu_seqlens[num_seqs] ----
  if (!kStates && a.cu) {
    const int end = min(max(__ldg(a.cu + a.num_seqs), 0), a.tokens);
    const int64_t words = static_cast<int64_t>(a.tokens - end) * j.heads_x * (D / 8);
    uint4* o4 = reinterpret_cast<uint4*>(j.out + static_cast<int64_t>(end) * j.heads_x * D);
    const int64_t step = static_cast<int64_t>(j.slots) * j.heads_x * C::THREADS;
    for (int64_t w = item * static_cast<int64_t>(C::THREADS) + threadIdx.x; w < words; w += step)
      o4[w] = make_uint4(0u, 0u, 0u, 0u);
  }

  // (no grid ends before the one that it follows)
  if (!kStates) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (*reinterpret_cast<volatile int*>(&abort_flag)) {   // a wait ran out: the copies and products in
      const uint64_t t0 = globaltimer();                   // flight get a moment to land before the CTA leaves
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
    tmem_dealloc(tmem, C::COLS);
  }
}

template <int D, int NS, bool kStates, int kCtas = 1>
cudaError_t launch(const LinearArgs& a, bool follows, cudaStream_t st) {
  using C = Cfg<D, NS, kStates, kCtas>;
  auto kern = linear_kernel<D, NS, kStates, kCtas>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  int64_t grid = 0;
  for (int i = 0; i < a.jobs; ++i) grid += static_cast<int64_t>(a.job[i].slots) * a.job[i].heads_x;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = follows ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int head_dim, bool states_only, bool pairs, bool follows,
                          cudaStream_t st) {
  int terms = 1;   // the most that a job has
  for (int i = 0; i < a.jobs; ++i) terms = a.job[i].terms > terms ? a.job[i].terms : terms;
  if (head_dim == 64) {
    if (states_only)
      return terms == 1 ? launch<64, 1, true, 2>(a, follows, st) : launch<64, 3, true>(a, follows, st);
    if (pairs) return terms == 1 ? launch<64, 1, false, 2>(a, follows, st) : launch<64, 3, false, 2>(a, follows, st);
    return terms == 1 ? launch<64, 1, false>(a, follows, st) : launch<64, 3, false>(a, follows, st);
  }
  if (states_only) return terms == 1 ? launch<128, 1, true>(a, follows, st) : launch<128, 3, true>(a, follows, st);
  return terms == 1 ? launch<128, 1, false>(a, follows, st) : launch<128, 3, false>(a, follows, st);
}

}  // namespace attn

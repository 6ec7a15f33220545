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
//   warp 1        MMA issuer: S = X Y^T, O2 = X H, O1 += P Z, G += (diag(d) Y)^T Z
//   warps 4..7    scores: S to P = S o W as packed bf16 in TMEM, then out = O1 + u O2
//   warps 8..15   state: Y to diag(d) Y in place (bf16; the second and third terms in
//                 tiles of their own), H = l^C H + G, H as bf16 to shared memory
// S is scaled by products of two table values below and above the diagonal block
// of 32 x 32, by exponentials in it.  The four products of a chunk take 2048 cycles
// of the tensor cores at D = 128, its four tiles of 32 KB 5500 cycles of an SM's share
// of the memory bandwidth: the walk is bound by memory as long as the ring holds
// the next chunk's tiles while this one's are used.
#include "linear.cuh"

namespace attn {
namespace {

template <int D, int NS, bool kStates>
struct Cfg {
  static constexpr int C = kLinearChunk;
  static constexpr int TILE = C * D * 2;
  static constexpr int H_BYTES = kStates ? 0 : D * D * 2;
  static constexpr int EXTRA = (NS - 1) * TILE;   // second and third terms of the decayed keys
  // the tiles that fit: 227 KB of shared memory, 1 KB of it for the alignment
  static constexpr int FIT = (227 * 1024 - 2048 - H_BYTES - EXTRA) / TILE;
  // X has buffers of its own: a chunk's X outlives the tiles of its inner heads
  static constexpr int XBUF = kStates ? 0 : FIT >= 6 ? 2 : 1;
  static constexpr int NSLOT = (FIT > 8 ? 8 : FIT) - XBUF;
  static constexpr int SMEM = (XBUF + NSLOT) * TILE + H_BYTES + EXTRA + 1024;
  static constexpr int THREADS = 512;
  static constexpr int HC = D / 2;                // state columns of a thread
  static constexpr uint32_t COL_S = 0, COL_O1 = 128, COL_O2 = 256, COL_G = 384;
  static_assert(NSLOT >= 3, "Y and Z and one on its way");
};

// log2 of a head's decay, at most 0.  -inf becomes a number whose products with 0
// and with token counts stay finite.
__device__ __forceinline__ float log2_decay(const LinearArgs& a, int h) {
  float g = __ldg(a.log_decay + h);
  if (!(g <= 0.f)) {
    if (a.err) atomicOr(a.err, ATTN_DEVERR_DECAY);
    g = 0.f;
  }
  return fmaxf(g * kLog2e, -1e6f);
}

// The rows of sequence n, kept within the tensors whatever cu holds.
__device__ __forceinline__ void sequence_rows(const LinearArgs& a, int n, int& row0, int& len) {
  if (!a.cu) {
    row0 = n * a.seqlen;
    len = a.seqlen;
    return;
  }
  const int b = __ldg(a.cu + n), e = __ldg(a.cu + n + 1);
  row0 = min(max(b, 0), a.tokens);
  const int end = min(max(e, row0), a.tokens);
  len = end - row0;
  if ((b != row0 || e != end) && a.err) atomicOr(a.err, ATTN_DEVERR_SEQLEN);
}

__device__ __forceinline__ int chunks_of(int len) { return (len + kLinearChunk - 1) / kLinearChunk; }
__device__ __forceinline__ int segments_of(int len, int seg_chunks) {
  return max(1, (chunks_of(len) + seg_chunks - 1) / seg_chunks);
}

// A walk's place: sequence n, its segment `seg` of `nseg`, each of `per` chunks at most.
struct Place {
  int n, row0, len, seg, nseg, per;
};

// The place of a slot, by one warp; n = -1 where the slot holds none.
__device__ __forceinline__ Place find_place(const LinearArgs& a, const LinearJob& j, int slot) {
  Place p{-1, 0, 0, 0, 1, 1};
  if (!a.cu) {
    p.nseg = segments_of(a.seqlen, j.seg_chunks);
    p.n = slot / p.nseg;
    p.seg = slot - p.n * p.nseg;
    if (p.n >= a.num_seqs) p.n = -1;
    else sequence_rows(a, p.n, p.row0, p.len);
  } else {
    const int lane = lane_id();
    for (int n0 = 0, before = 0; n0 < a.num_seqs; n0 += 32) {
      int row0 = 0, len = 0, count = 0;
      if (n0 + lane < a.num_seqs) {
        sequence_rows(a, n0 + lane, row0, len);
        count = segments_of(len, j.seg_chunks);
      }
      int sum = count;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      const bool here = slot >= before + sum - count && slot < before + sum;
      const unsigned who = __ballot_sync(0xffffffffu, here);
      if (who) {
        const int src = __ffs(who) - 1;
        p.n = n0 + src;
        p.row0 = __shfl_sync(0xffffffffu, row0, src);
        p.len = __shfl_sync(0xffffffffu, len, src);
        p.nseg = __shfl_sync(0xffffffffu, count, src);
        p.seg = slot - before - __shfl_sync(0xffffffffu, sum - count, src);
        break;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  p.per = (chunks_of(p.len) + p.nseg - 1) / p.nseg;
  return p;
}

template <int D, int NS, bool kStates>
__global__ void __launch_bounds__(512, 1) linear_kernel(const __grid_constant__ LinearArgs a) {
  using C = Cfg<D, NS, kStates>;
  constexpr int PANELS = D / 64;
  constexpr int NSLOT = C::NSLOT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sX = ring + NSLOT * C::TILE;
  uint8_t* sH = sX + C::XBUF * C::TILE;
  uint8_t* sExtra = sH + C::H_BYTES;

  __shared__ uint64_t bar_full[NSLOT], bar_empty[NSLOT];
  __shared__ uint64_t bar_xfull[2], bar_xempty[2];
  __shared__ uint64_t bar_s, bar_p, bar_o, bar_of, bar_y, bar_g, bar_h;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_flag;
  __shared__ Place s_place;
  __shared__ __align__(16) float s_tab[32];   // decays within a block of 32 columns

  const int warp = warp_id();
  AbortCtx ac{&abort_flag, a.err};

  // ---- the walk ----
  int ji = 0, item = blockIdx.x;
  while (ji + 1 < a.jobs && item >= a.job[ji].slots * a.job[ji].heads_x) {
    item -= a.job[ji].slots * a.job[ji].heads_x;
    ++ji;
  }
  const LinearJob& j = a.job[ji];
  const int slot = static_cast<int>(fdiv(item, j.fd_heads));
  const int h = item - slot * j.heads_x;
  const int hkv = static_cast<int>(fdiv(h, j.fd_kv));

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < NSLOT; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_xfull[i], 1);
      mbar_init(&bar_xempty[i], 1);
    }
    mbar_init(&bar_s, 1);
    mbar_init(&bar_p, 128);
    mbar_init(&bar_o, 1);
    mbar_init(&bar_of, 128);
    mbar_init(&bar_y, 256);
    mbar_init(&bar_g, 1);
    mbar_init(&bar_h, 256);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base_sh, 512);
  const float l2 = log2_decay(a, hkv);
  if (warp == 2) {
    const Place p = find_place(a, j, slot);
    if (lane_id() == 0) s_place = p;
  }
  if (warp == 3) s_tab[lane_id()] = ex2(l2 * (j.backwards ? lane_id() : 31 - lane_id()));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  Place pl = s_place;
  const bool back = j.backwards;
  // the sequence's last segment in the walk's direction, which no state follows
  const bool is_end = pl.n >= 0 && pl.seg == (back ? 0 : pl.nseg - 1);
  if (kStates && is_end) pl.n = -1;
  const int nch = pl.n < 0 ? 0 : chunks_of(pl.len);
  const int c_lo = min(nch, pl.seg * pl.per), c_hi = min(nch, c_lo + pl.per);
  const int n_walk = c_hi - c_lo;
  const int inner = j.inner;
  // of the walk's n-th chunk: its first token, and its tokens
  auto chunk_row = [&](int n) { return (back ? c_hi - 1 - n : c_lo + n) * kLinearChunk; };
  auto chunk_len = [&](int n) { return min(kLinearChunk, pl.len - chunk_row(n)); };
  const bool want_last = kStates || (is_end && j.last && h == hkv * static_cast<int>(j.fd_kv.d));
  const int n_grow = want_last ? n_walk : n_walk - 1;   // chunks that the state takes in

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane_id() == 0 && n_walk > 0) {
      tma_prefetch_desc(&j.my);
      tma_prefetch_desc(&j.mz);
      const int hy = inner > 1 || kStates ? h * inner : hkv;
      int it = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* m, uint64_t* full, uint64_t* empty, uint8_t* dst, int use, int head, int row) {
        if (use > 0 && !mbar_wait_spin(empty, (use & 1) ^ 1, ac)) {
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
    int tile = 0, it = 0;
    bool ok = true;
    for (int n = 0; ok && n < n_walk; ++n) {
      int bx = 0;
      if constexpr (!kStates) {
        bx = n % C::XBUF;
        if (!mbar_wait_w(&bar_xfull[bx], (n / C::XBUF) & 1, ac)) break;
      }
      for (int g = 0; ok && g < inner; ++g, ++it) {
        const int sy = tile % NSLOT, uy = (tile / NSLOT) & 1;
        const int sz = (tile + 1) % NSLOT, uz = ((tile + 1) / NSLOT) & 1;
        tile += 2;
        const bool last = g == inner - 1;
        const uint64_t dz = desc_advance(dm0, sz * C::TILE);
        if (!mbar_wait_w(&bar_full[sy], uy, ac)) { ok = false; break; }
        if (!kStates) {
          tc_fence_after();
          const uint64_t dx = desc_advance(dx0, bx * C::TILE), dy = desc_advance(dk0, sy * C::TILE);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_ss_w(tmem + C::COL_S, desc_advance(dx, kmajor_step_bytes(128, k)),
                      desc_advance(dy, kmajor_step_bytes(128, k)), idS, k > 0);
          umma_commit_w(&bar_s);
          if (g == 0) {
            if (!mbar_wait_w(&bar_h, n & 1, ac) || (n > 0 && !mbar_wait_w(&bar_of, (n - 1) & 1, ac))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              umma_ss_w(tmem + C::COL_O2, desc_advance(dx, kmajor_step_bytes(128, k)),
                        desc_advance(dH, mnmajor_step_bytes(k)), idO, k > 0);
          }
        }
        if (!mbar_wait_w(&bar_full[sz], uz, ac)) { ok = false; break; }
        if (!kStates) {
          if (!mbar_wait_w(&bar_p, it & 1, ac)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            umma_ts_w(tmem + C::COL_O1, tmem + C::COL_S + 8 * k, desc_advance(dz, mnmajor_step_bytes(k)), idO,
                      (g > 0 || k > 0) ? 1u : 0u);
          if (last) umma_commit_w(&bar_o);
        }
        if (n < n_grow) {
          if (!mbar_wait_w(&bar_y, it & 1, ac)) { ok = false; break; }
          tc_fence_after();
          const uint64_t dy = desc_advance(dm0, sy * C::TILE);
#pragma unroll
          for (int t = 0; t < NS; ++t)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              umma_ss_w(tmem + C::COL_G,
                        desc_advance(t == 0 ? dy : desc_advance(dE, (t - 1) * C::TILE), mnmajor_step_bytes(k)),
                        desc_advance(dz, mnmajor_step_bytes(k)), idG, (g > 0 || t > 0 || k > 0) ? 1u : 0u);
        }
        umma_commit_w(&bar_empty[sy]);
        umma_commit_w(&bar_empty[sz]);
        if (n < n_grow && last) umma_commit_w(&bar_g);
      }
    }
  } else if (!kStates && warp >= 4 && warp < 8) {
    // ---------------- scores and output ----------------
    const int wq = warp & 3, i = threadIdx.x & 127;   // row of the chunk, TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    int tile = 0, it = 0;
    bool ok = true;
    for (int n = 0; ok && n < n_walk; ++n) {
      const int rows = chunk_len(n), row = chunk_row(n);
      for (int g = 0; ok && g < inner; ++g, ++it, tile += 2) {
        if (!mbar_wait(&bar_s, it & 1, ac)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          uint32_t p[16];
          if (back ? b < wq : b > wq) {
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = 0;
          } else if (b == wq || (back && rows < kLinearChunk)) {
            // the diagonal block, and backwards columns behind the sequence: an exponential and a
            // comparison for each element
            uint32_t s[32];
            tmem_ld32_nowait(lane_base + C::COL_S + 32 * b, s);
            tmem_wait_ld();
            const int lead = back ? 32 * b - i : i - 32 * b, sign = back ? 1 : -1;
            const int end = back ? rows - 32 * b : 32;
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              float f[2];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int d = lead + sign * (x + y);
                f[y] = __uint_as_float(s[x + y]) * (a.scale * ex2(l2 * max(d, 0)));
                if (d < 0 || x + y >= end) f[y] = 0.f;
              }
              p[x / 2] = pack_bf16(f[0], f[1]);
            }
          } else {
            // the exponent left once the table's part is taken
            uint32_t s[32];
            tmem_ld32_nowait(lane_base + C::COL_S + 32 * b, s);
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
          tmem_st16p(lane_base + C::COL_S + 16 * b, p);
        }
        if (rows < kLinearChunk) {
          // rows of Z behind the sequence may hold anything: zeros, for 0 * NaN
          const int sz = (tile + 1) % NSLOT;
          if (!mbar_wait(&bar_full[sz], ((tile + 1) / NSLOT) & 1, ac)) { ok = false; break; }
          if (i >= rows) {
            uint4* z = reinterpret_cast<uint4*>(ring + sz * C::TILE + i * 128);
#pragma unroll
            for (int x = 0; x < D / 8; ++x) z[(x >> 3) * (kLinearChunk * 8) + (x & 7)] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bar_p);
      }
      if (!ok || !mbar_wait(&bar_o, n & 1, ac)) break;
      tc_fence_after();
      const float u = back ? ex2(l2 * max(rows - 1 - i, 0)) : a.scale * ex2(l2 * (i + 1));
      // out takes the place of X, which the products have read, and leaves by a bulk copy (by
      // plain stores where rows behind the sequence are another's): rows written from
      // registers, 16 bytes of 32 rows at a time, took 2000 cycles
      const int bx = n & (C::XBUF - 1);
      uint8_t* so = sX + bx * C::TILE;
#pragma unroll
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t o1[32], o2[32];
        tmem_ld32_nowait(lane_base + C::COL_O1 + cc, o1);
        tmem_ld32_nowait(lane_base + C::COL_O2 + cc, o2);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            w[y] = pack_bf16(fmaf(u, __uint_as_float(o2[x + 2 * y]), __uint_as_float(o1[x + 2 * y])),
                             fmaf(u, __uint_as_float(o2[x + 2 * y + 1]), __uint_as_float(o1[x + 2 * y + 1])));
          *reinterpret_cast<uint4*>(so + sw128_offset(i, cc + x, kLinearChunk)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tc_fence_before();
      mbar_arrive(&bar_of);
      if (rows == kLinearChunk) {
        fence_proxy_async_smem();
        named_bar_sync(1, 128);
        if (i == 0) {
          for (int pn = 0; pn < PANELS; ++pn)
            tma_store_3d(&j.mo, so + pn * kLinearChunk * 128, pn * 64, h, pl.row0 + row);
          bulk_commit();
          bulk_wait_read<0>();
          mbar_arrive(&bar_xempty[bx]);
        }
      } else {
        named_bar_sync(1, 128);
        __nv_bfloat16* out = j.out + (static_cast<int64_t>(pl.row0 + row) * j.heads_x + h) * D;
        for (int x = i; x < rows * (D / 8); x += 128) {
          const int ro = x / (D / 8), co = x % (D / 8) * 8;
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(ro) * j.heads_x * D + co) =
              *reinterpret_cast<const uint4*>(so + sw128_offset(ro, co, kLinearChunk));
        }
        fence_proxy_async_smem();
        named_bar_sync(1, 128);
        if (i == 0) mbar_arrive(&bar_xempty[bx]);
      }
    }
    if (i == 0) bulk_wait<0>();
  } else if (warp >= 8 && pl.n >= 0) {
    // ---------------- state ----------------
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
#pragma unroll
        for (int x = 0; x < C::HC; ++x) H[x] = __ldg(j.transposed ? f + (c0 + x) * D + r : f + r * D + c0 + x);
      }
      const int before = back ? pl.nseg - 1 - pl.seg : pl.seg;
      for (int t = 0; t < before; ++t) {
        const int sg = back ? pl.nseg - 1 - t : t;
        const int lo = sg * pl.per * kLinearChunk, hi = min(pl.len, lo + pl.per * kLinearChunk);
        const float keep = ex2(l2 * max(hi - lo, 0));
        const float4* g = reinterpret_cast<const float4*>(
            j.parts + (static_cast<int64_t>(slot + sg - pl.seg) * a.heads_kv + hkv) * D * D);
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
          const uint4 v = make_uint4(pack_bf16(H[x], H[x + 1]), pack_bf16(H[x + 2], H[x + 3]),
                                     pack_bf16(H[x + 4], H[x + 5]), pack_bf16(H[x + 6], H[x + 7]));
          *reinterpret_cast<uint4*>(sH + sw128_offset(r, c0 + x, D)) = v;
        }
      fence_proxy_async_smem();
      mbar_arrive(&bar_h);
    };
    if (!kStates && n_walk > 0) publish();
    int tile = 0, it = 0;
    bool ok = true;
    const int row = tid & 127;
    for (int n = 0; ok && n < n_grow; ++n) {
      const int rows = chunk_len(n);
      const float d = back ? a.scale * ex2(l2 * (row + 1)) : ex2(l2 * max(rows - 1 - row, 0));
      for (int g = 0; ok && g < inner; ++g, ++it, tile += 2) {
        const int sy = tile % NSLOT;
        if (!mbar_wait(&bar_full[sy], (tile / NSLOT) & 1, ac) || (!kStates && !mbar_wait(&bar_s, it & 1, ac))) {
          ok = false;
          break;
        }
        // the other terms' tiles: read by the products of the step before
        if (NS > 1 && g > 0 && !mbar_wait(&bar_empty[(tile - 2) % NSLOT], ((tile - 2) / NSLOT) & 1, ac)) {
          ok = false;
          break;
        }
        if (kStates && rows < kLinearChunk) {
          const int sz = (tile + 1) % NSLOT;
          if (!mbar_wait(&bar_full[sz], ((tile + 1) / NSLOT) & 1, ac)) { ok = false; break; }
          if (row >= rows && half < PANELS) {
            uint4* z = reinterpret_cast<uint4*>(ring + sz * C::TILE + half * (kLinearChunk * 128) + row * 128);
#pragma unroll
            for (int x = 0; x < 8; ++x) z[x] = make_uint4(0, 0, 0, 0);
          }
        }
        uint8_t* y = ring + sy * C::TILE;
#pragma unroll
        for (int x = 0; x < C::HC; x += 8) {
          const uint32_t at = sw128_offset(row, c0 + x, kLinearChunk);
          uint4 v = *reinterpret_cast<const uint4*>(y + at);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          uint32_t term[NS][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float lo = __uint_as_float(w[e] << 16) * d, hi = __uint_as_float(w[e] & 0xffff0000u) * d;
            if (row >= rows) lo = hi = 0.f;
#pragma unroll
            for (int t = 0; t < NS; ++t) {
              term[t][e] = pack_bf16(lo, hi);
              lo -= __uint_as_float(term[t][e] << 16);
              hi -= __uint_as_float(term[t][e] & 0xffff0000u);
            }
          }
          *reinterpret_cast<uint4*>(y + at) = make_uint4(term[0][0], term[0][1], term[0][2], term[0][3]);
#pragma unroll
          for (int t = 1; t < NS; ++t)
            *reinterpret_cast<uint4*>(sExtra + (t - 1) * C::TILE + at) =
                make_uint4(term[t][0], term[t][1], term[t][2], term[t][3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar_y);
      }
      if (!ok || !mbar_wait(&bar_g, n & 1, ac)) break;
      tc_fence_after();
      const float keep = ex2(l2 * rows);
#pragma unroll
      for (int x = 0; x < C::HC; x += 32) {
        uint32_t g[32];
        tmem_ld32_nowait(tG + x, g);
        tmem_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; ++y) H[x + y] = fmaf(keep, H[x + y], __uint_as_float(g[y]));
      }
      tc_fence_before();
      if (!kStates && n + 1 < n_walk) publish();
    }
    if (kStates) {
      const int64_t at = (static_cast<int64_t>(slot) * a.heads_kv + hkv) * D * D;
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

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
    tmem_relinquish();
  }
}

template <int D, int NS, bool kStates>
cudaError_t launch(const LinearArgs& a, cudaStream_t st) {
  using C = Cfg<D, NS, kStates>;
  auto kern = linear_kernel<D, NS, kStates>;
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(kern, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  int64_t grid = 0;
  for (int i = 0; i < a.jobs; ++i) grid += static_cast<int64_t>(a.job[i].slots) * a.job[i].heads_x;
  if (grid >= (int64_t(1) << 31)) return cudaErrorInvalidValue;
  kern<<<static_cast<unsigned>(grid), C::THREADS, C::SMEM, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& a, int head_dim, int terms, bool states_only,
                          cudaStream_t st) {
  if (head_dim == 64) {
    if (states_only) return terms == 1 ? launch<64, 1, true>(a, st) : launch<64, 3, true>(a, st);
    return terms == 1 ? launch<64, 1, false>(a, st) : launch<64, 3, false>(a, st);
  }
  if (states_only) return terms == 1 ? launch<128, 1, true>(a, st) : launch<128, 3, true>(a, st);
  return terms == 1 ? launch<128, 1, false>(a, st) : launch<128, 3, false>(a, st);
}

}  // namespace attn

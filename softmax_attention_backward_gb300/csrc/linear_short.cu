// Linear attention of sequences of a few tokens, token by token in fp32 (linear.h;
// the jobs are those of linear.cuh).
//
// A chunk of 128 rows on the tensor cores takes as long whether 1 or 128 of them
// are a sequence's, and its scores' rounding to bf16 does not average out over
// one or two.  Here a CTA takes 32 columns of the state of one (sequence, head) and
// walks its tokens: lanes are columns, each of four warps holds a quarter of the
// rows in registers, and an output is the sum of the warps' parts in a fixed
// order.  Bound by latency for one sequence: the loads of a batch of tokens are one
// trip to memory (4 tokens: 10.4 us, 5 of them for the launch; 12.4 with a trip for
// each token).
#include "linear.cuh"

namespace attn {
namespace {

constexpr int kSteps = 8;    // (token, inner head) pairs that are fetched together

template <int D>
__global__ void __launch_bounds__(128) linear_short_kernel(const __grid_constant__ LinearArgs a) {
  constexpr int R = D / 4;   // rows of the state in a thread
  __shared__ float s_decay[2];
  __shared__ __align__(16) float sx[kSteps][D], sy[kSteps][D], sz[kSteps][32], part[kSteps][4][32];
  const LinearJob& j = a.job[blockIdx.z / (D / 32)];
  const int n = blockIdx.x, h = blockIdx.y, c = threadIdx.x & 31, rg = threadIdx.x >> 5;
  if (h >= j.heads_x) return;
  const int col = blockIdx.z % (D / 32) * 32 + c;
  int row0, len;
  sequence_rows(a, n, row0, len);
  const int hkv = static_cast<int>(fdiv(h, j.fd_kv));
  // the decay in two parts, by one thread: exp in fp64 by all of them takes 20 us of 64 sequences' 50
  if (threadIdx.x == 0) {
    const double ld = exp(static_cast<double>(log_decay_of(a, hkv)));
    s_decay[0] = static_cast<float>(ld);
    s_decay[1] = static_cast<float>(ld - s_decay[0]);
  }
  const size_t at = (static_cast<size_t>(n) * a.heads_kv + hkv) * D * D;
  float s[R];
  if (j.first && j.transposed) {
    const float4* f = reinterpret_cast<const float4*>(j.first + at + col * D + rg * R);
#pragma unroll
    for (int i = 0; i < R; i += 4) {
      const float4 v = __ldg(f + i / 4);
      s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = j.first ? __ldg(j.first + at + (rg * R + i) * D + col) : 0.f;
  }
  const int hy = j.inner > 1 ? h * j.inner : hkv;
  const float ys = j.backwards ? a.scale : 1.f, os = j.backwards ? 1.f : a.scale;
  const int steps = len * j.inner;   // at most a few tokens' heads
  auto row = [&](int k) { return static_cast<int64_t>(row0 + (j.backwards ? len - 1 - k : k)); };
  int k = 0, g = 0;   // the token, counted along the walk, and inner head of a batch's first step
  for (int i0 = 0; i0 < steps; i0 += kSteps) {
    const int m = min(kSteps, steps - i0);
    __syncthreads();   // the batch before has been read
    // all of a batch's loads are under way together: a store between them would order them
    __nv_bfloat16 x[kSteps], y[kSteps], z[kSteps];
    int kk = k, gg = g;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i < m) {
        const int64_t t = row(kk);
        if (rg == 3) z[i] = j.z[t * j.z_stride + (hy + gg) * D + col];
        if (threadIdx.x < D) {
          y[i] = j.y[t * j.y_stride + (hy + gg) * D + threadIdx.x];
          x[i] = j.x[t * j.x_stride + h * D + threadIdx.x];
        }
        if (++gg == j.inner) gg = 0, ++kk;
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i < m) {
        if (rg == 3) sz[i][c] = __bfloat162float(z[i]);
        if (threadIdx.x < D) {
          sy[i][threadIdx.x] = __bfloat162float(y[i]) * ys;
          sx[i][threadIdx.x] = __bfloat162float(x[i]);
        }
      }
    }
    __syncthreads();
    const float l = s_decay[0], l2 = s_decay[1];
    uint32_t ends = 0;   // the steps that are a token's last
    kk = k, gg = g;
#pragma unroll 1
    for (int i = 0; i < m; ++i) {
      const float zc = sz[i][c];
      if (!j.backwards)
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = fmaf(l, s[r], l2 * s[r]);
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = fmaf(sy[i][rg * R + r], zc, s[r]);
      if (++gg < j.inner) continue;
      gg = 0, ++kk;
      ends |= 1u << i;
      float o[4] = {};
#pragma unroll
      for (int r = 0; r < R; ++r) o[r & 3] = fmaf(sx[i][rg * R + r], s[r], o[r & 3]);
      part[i][rg][c] = (o[0] + o[1]) + (o[2] + o[3]);
      if (j.backwards)
#pragma unroll
        for (int r = 0; r < R; ++r) s[r] = fmaf(l, s[r], l2 * s[r]);
    }
    __syncthreads();
    // the tokens that ended, a warp each
    for (int i = 0, t = k; i < m; ++i) {
      if (!(ends >> i & 1)) continue;
      if ((t & 3) == rg)
        j.out[(row(t) * j.heads_x + h) * D + col] = __float2bfloat16_rn(
            ((part[i][0][c] + part[i][1][c]) + (part[i][2][c] + part[i][3][c])) * os);
      ++t;
    }
    k = kk, g = gg;
  }
  if (j.last && h == hkv * static_cast<int>(j.fd_kv.d))
#pragma unroll
    for (int i = 0; i < R; ++i) j.last[at + (rg * R + i) * D + col] = s[i];
  // padding rows
  if (a.cu && rg == 0)
    for (int64_t t = min(max(__ldg(a.cu + a.num_seqs), 0), a.tokens) + n; t < a.tokens; t += a.num_seqs)
      j.out[(t * j.heads_x + h) * D + col] = __float2bfloat16_rn(0.f);
}

}  // namespace

cudaError_t launch_linear_short(const LinearArgs& a, int head_dim, cudaStream_t st) {
  int heads = 0;
  for (int i = 0; i < a.jobs; ++i) heads = a.job[i].heads_x > heads ? a.job[i].heads_x : heads;
  const dim3 grid(a.num_seqs, heads, a.jobs * (head_dim / 32));
  if (head_dim == 64) linear_short_kernel<64><<<grid, 128, 0, st>>>(a);
  else linear_short_kernel<128><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace attn

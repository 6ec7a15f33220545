// Linear attention, token by token: one CTA for each sequence, head and 32
// columns of the state.
#include "linear.cuh"

namespace attn {
namespace {

template <int D>
__global__ void __launch_bounds__(128) linear_walk_kernel(const LinearArgs a, const LinearJob j) {
  constexpr int R = D / 4;   // rows of the state in a thread
  __shared__ float sx[D], sy[D], sz[32], part[4][32];
  const int n = blockIdx.x, h = blockIdx.y, c = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const int col = blockIdx.z * 32 + c;
  int row0, len;
  linear_sequence(a, n, row0, len);
  const int hkv = fdiv(h, j.fd_kv);
  // in two parts: an error of the decay would grow with every token
  const double ld = exp2(static_cast<double>(log2_decay(a, hkv)));
  const float l = static_cast<float>(ld), l2 = static_cast<float>(ld - l);
  const size_t at = (static_cast<size_t>(n) * a.heads_kv + hkv) * D * D;
  float s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = rg * R + i;
    s[i] = !j.first ? 0.f : j.first[at + (j.transposed ? col * D + r : r * D + col)];
  }
  const int hy = j.inner > 1 ? h * j.inner : static_cast<int>(fdiv(h, j.fd_kv));
  for (int k = 0; k < len; ++k) {
    const int64_t t = row0 + (j.backwards ? len - 1 - k : k);
    if (!j.backwards)
#pragma unroll
      for (int i = 0; i < R; ++i) s[i] = fmaf(l, s[i], l2 * s[i]);
    for (int g = 0; g < j.inner; ++g) {
      __syncthreads();
      if (threadIdx.x < D) {
        if (g == 0) sx[threadIdx.x] = __bfloat162float(j.x[t * j.x_stride + h * D + threadIdx.x]);
        sy[threadIdx.x] = __bfloat162float(j.y[t * j.y_stride + (hy + g) * D + threadIdx.x]) *
                          (j.backwards ? a.scale : 1.f);
      }
      if (rg == 0) sz[c] = __bfloat162float(j.z[t * j.z_stride + (hy + g) * D + col]);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < R; ++i) s[i] = fmaf(sy[rg * R + i], sz[c], s[i]);
    }
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) o = fmaf(sx[rg * R + i], s[i], o);
    part[rg][c] = o;
    __syncthreads();
    if (rg == 0) {
      o = (part[0][c] + part[1][c]) + (part[2][c] + part[3][c]);
      j.out[(t * j.heads_x + h) * D + col] = __float2bfloat16_rn(j.backwards ? o : o * a.scale);
    }
    if (j.backwards)
#pragma unroll
      for (int i = 0; i < R; ++i) s[i] = fmaf(l, s[i], l2 * s[i]);
  }
  if (j.last && h % j.fd_kv.d == 0)
#pragma unroll
    for (int i = 0; i < R; ++i) j.last[at + (rg * R + i) * D + col] = s[i];
  // padding rows
  if (a.cu)
    for (int64_t t = max(__ldg(a.cu + a.num_seqs), 0) + n; t < a.tokens; t += a.num_seqs)
      if (rg == 0) j.out[(t * j.heads_x + h) * D + col] = __float2bfloat16_rn(0.f);
}

}  // namespace

cudaError_t launch_linear_walk(int head_dim, const LinearArgs& a, const LinearJob& j,
                               cudaStream_t st) {
  const dim3 grid(a.num_seqs, j.heads_x, head_dim / 32);
  if (head_dim == 64) linear_walk_kernel<64><<<grid, 128, 0, st>>>(a, j);
  else linear_walk_kernel<128><<<grid, 128, 0, st>>>(a, j);
  return cudaGetLastError();
}

}  // namespace attn

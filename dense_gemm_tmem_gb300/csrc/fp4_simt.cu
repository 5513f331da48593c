// fp4_simt.cu: the 4-bit product on the CUDA cores: 64 x 64 tiles, 256 threads
// of 4 x 4 sums, values times block scales widened to fp32 in shared memory.
#include "fp4.cuh"

namespace dg {
namespace {

constexpr int kT = 64, kDepth = 32, kLd = kT + 4;

__global__ void __launch_bounds__(256) fp4_simt_kernel(const Fp4Product p, int32_t tiles_n) {
  __shared__ float sa[kDepth][kLd], sb[kDepth][kLd];
  const int64_t m0 = int64_t(blockIdx.x / tiles_n) * kT, n0 = int64_t(blockIdx.x % tiles_n) * kT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t block = fp4_block(p.A.format);
  const int64_t pieces = ((p.K + block - 1) / block + 3) / 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += kDepth) {
    for (int i = threadIdx.x; i < kT * kDepth; i += 256) {
      const int k = i % kDepth, r = i / kDepth;
      const bool in = k0 + k < p.K;
      sa[k][r] = in && m0 + r < p.M ? fp4_element(p.A, m0 + r, k0 + k, pieces) : 0.f;
      sb[k][r] = in && n0 + r < p.N ? fp4_element(p.B, n0 + r, k0 + k, pieces) : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < kDepth; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      float v = acc[i][j];
      if (p.A.row_scale) v *= p.A.row_scale[m * p.A.row_scale_stride];
      if (p.B.row_scale) v *= p.B.row_scale[n * p.B.row_scale_stride];
      if (p.bias) v += p.bias[n];
      store_typed(p.C, m * p.ldc + n, v, p.out_dtype);
    }
}

}  // namespace

cudaError_t launch_fp4_simt(const Fp4Product& p, cudaStream_t stream) {
  const int64_t tm = (p.M + kT - 1) / kT, tn = (p.N + kT - 1) / kT;
  if (tm > INT32_MAX / tn) return cudaErrorInvalidValue;
  fp4_simt_kernel<<<unsigned(tm * tn), 256, 0, stream>>>(p, int32_t(tn));
  return cudaGetLastError();
}

}  // namespace dg

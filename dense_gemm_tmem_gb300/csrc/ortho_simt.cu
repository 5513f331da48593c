// ortho_simt.cu: the products of the orthogonalising call on the CUDA cores:
// 64 x 64 tiles, 256 threads of 4 x 4 sums.
#include <cuda_bf16.h>

#include "ortho.cuh"

namespace dg {
namespace {

constexpr int kT = 64, kDepth = 16, kLd = kT + 4;

struct View {  // element (i, k) of an operand
  const __half* p;
  int64_t s_i, s_k;
  __device__ float at(int64_t i, int64_t k) const { return __half2float(p[i * s_i + k * s_k]); }
};

__global__ void __launch_bounds__(256) ortho_simt_kernel(const OrthoShape s, const OrthoProduct p,
                                                         View A, View B, int64_t batch_a,
                                                         int64_t batch_b, int64_t M, int64_t N,
                                                         int64_t K) {
  __shared__ float sa[kDepth][kLd], sb[kDepth][kLd];
  const int64_t m0 = int64_t(blockIdx.x) * kT, n0 = int64_t(blockIdx.y) * kT, z = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  A.p += z * batch_a;
  B.p += z * batch_b;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += kDepth) {
    for (int i = threadIdx.x; i < kT * kDepth; i += 256) {
      const int k = i % kDepth, r = i / kDepth;
      const bool in = k0 + k < K;
      sa[k][r] = in && m0 + r < M ? A.at(m0 + r, k0 + k) : 0.f;
      sb[k][r] = in && n0 + r < N ? B.at(n0 + r, k0 + k) : 0.f;
    }
    __syncthreads();
#pragma unroll
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
      if (m >= M || n >= N) continue;
      float v = p.alpha * acc[i][j];
      if (p.kind == kApply) {
        float* x = p.x32 + z * s.rows * s.cols + m * s.cols + n;
        v = fmaf(p.beta, *x, v);
        if (p.out) {
          static_cast<__nv_bfloat16*>(p.out)[z * p.stride_out + m * p.ld_out + n] =
              __float2bfloat16_rn(v);
        } else {
          *x = v;
          p.c[z * s.stride_x + m * s.ld_x + n] = __float2half_rn(v * p.scale);
        }
      } else {
        if (p.kind == kPoly)
          v = fmaf(p.beta, __half2float(p.a[z * s.stride_a + m * s.ld_a + n]), v);
        p.c[z * s.stride_a + m * s.ld_a + n] = __float2half_rn(v);
      }
    }
}

}  // namespace

cudaError_t launch_ortho_simt(const OrthoShape& s, const OrthoProduct& p, cudaStream_t stream) {
  View A, B;
  int64_t M, N, K, ba, bb;
  if (p.kind == kGram) {
    A = B = s.tall ? View{p.a, 1, s.ld_x} : View{p.a, s.ld_x, 1};
    M = N = s.n;
    K = s.tall ? s.rows : s.cols;
    ba = bb = s.stride_x;
  } else if (p.kind == kPoly) {
    A = B = View{p.a, s.ld_a, 1};
    M = N = K = s.n;
    ba = bb = s.stride_a;
  } else {
    M = s.rows;
    N = s.cols;
    K = s.n;
    if (s.tall) {  // X·B, B symmetric
      A = View{p.x, s.ld_x, 1};
      B = View{p.a, s.ld_a, 1};
      ba = s.stride_x;
      bb = s.stride_a;
    } else {
      A = View{p.a, s.ld_a, 1};
      B = View{p.x, 1, s.ld_x};
      ba = s.stride_a;
      bb = s.stride_x;
    }
  }
  const dim3 grid(unsigned((M + kT - 1) / kT), unsigned((N + kT - 1) / kT), unsigned(s.batch));
  ortho_simt_kernel<<<grid, 256, 0, stream>>>(s, p, A, B, ba, bb, M, N, K);
  return cudaGetLastError();
}

}  // namespace dg

// fp8_simt.cu: the block-scaled product on the CUDA cores, for operands the
// TMA cannot read (base or row pitch not a multiple of 16 bytes).
//
//   C[m, n] = sum over k-blocks of sa[m, kb] sb[n, kb] (sum over k in kb of a b)
//
// 64 x 64 tiles, 4 x 4 outputs a thread; bytes are read one by one (no
// alignment to rely on), widened to fp32 in shared memory, and each k-block's
// fp32 sum is scaled into the running one.  Bound by the byte loads and the
// FMA pipe (8192^3: 48.9 ms, 22 TFLOP/s); it exists so that every stride works.
#include "fp8.cuh"

namespace dg {
namespace {

constexpr int kT = 64;   // tile edge
constexpr int kKc = 32;  // k per shared stage (divides the block of 128)

__global__ void __launch_bounds__(256) fp8_simt_kernel(const Fp8Product p, int32_t tiles_n) {
  __shared__ __align__(16) float sA[kKc][kT + 4];
  __shared__ __align__(16) float sB[kKc][kT + 4];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = int64_t(blockIdx.x / uint32_t(tiles_n)) * kT;
  const int64_t n0 = int64_t(blockIdx.x % uint32_t(tiles_n)) * kT;
  float acc[4][4] = {};
  for (int64_t kb = 0; kb * kFp8Block < p.K; ++kb) {
    float part[4][4] = {};
    const int64_t kend = min(p.K, (kb + 1) * kFp8Block);
    for (int64_t k0 = kb * kFp8Block; k0 < kend; k0 += kKc) {
      __syncthreads();
      for (int i = threadIdx.x; i < kKc * kT; i += 256) {
        // neighbouring threads along the contiguous axis
        const int ka = p.A.s_k == 1 ? i % kKc : i / kT, ma = p.A.s_k == 1 ? i / kKc : i % kT;
        const int kbx = p.B.s_k == 1 ? i % kKc : i / kT, nb = p.B.s_k == 1 ? i / kKc : i % kT;
        float a = 0.f, b = 0.f;
        if (k0 + ka < kend && m0 + ma < p.M)
          a = unpack_e4m3x2(p.A.data[(m0 + ma) * p.A.s_mn + (k0 + ka) * p.A.s_k]).x;
        if (k0 + kbx < kend && n0 + nb < p.N)
          b = unpack_e4m3x2(p.B.data[(n0 + nb) * p.B.s_mn + (k0 + kbx) * p.B.s_k]).x;
        sA[ka][ma] = a;
        sB[kbx][nb] = b;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < kKc; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(&sA[k][ty * 4]);
        const float4 b = *reinterpret_cast<const float4*>(&sB[k][tx * 4]);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(av[i], bv[j], part[i][j]);
      }
    }
    float sa[4], sb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = min(m0 + ty * 4 + i, p.M - 1), n = min(n0 + tx * 4 + i, p.N - 1);
      sa[i] = __ldg(p.A.scale + (m >> p.A.mn_shift) * p.A.c_mn + kb * p.A.c_kb);
      sb[i] = __ldg(p.B.scale + (n >> p.B.mn_shift) * p.B.c_mn + kb * p.B.c_kb);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = add_scaled(acc[i][j], part[i][j], sa[i], sb[j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= p.M) break;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + tx * 4 + j;
      if (n >= p.N) break;
      store_typed(p.C, m * p.ldc + n, acc[i][j] + (p.bias ? __ldg(p.bias + n) : 0.f),
                  p.out_dtype);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_simt(const Fp8Product& p, cudaStream_t stream) {
  const int64_t tm = (p.M + kT - 1) / kT, tn = (p.N + kT - 1) / kT;
  if (tm * tn > INT32_MAX) return cudaErrorInvalidValue;
  fp8_simt_kernel<<<unsigned(tm * tn), 256, 0, stream>>>(p, int32_t(tn));
  return cudaGetLastError();
}

}  // namespace dg

// fp8.cuh: what the block-scaled 8-bit kernels share: the scale rule, e4m3
// conversions, and the launch descriptions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm_fp8.h"
#include "internal.h"

namespace dg {

constexpr int kFp8Block = 128;          // elements that share a scale, per axis
constexpr float kE4m3Max = 448.f;       // largest e4m3 magnitude
constexpr float kAmaxMin = 0x1p-100f;   // floor of a block's maximum: 448 / it stays finite

// A block's scale and the factor its elements are multiplied by.
__device__ __forceinline__ float fp8_scale(float amax) {
  return __fdiv_rn(fmaxf(amax, kAmaxMin), kE4m3Max);
}
__device__ __forceinline__ float fp8_inverse(float amax) {
  return __fdiv_rn(kE4m3Max, fmaxf(amax, kAmaxMin));
}

// Two floats to e4m3, round to nearest even, `a` in the low byte.  |a|, |b| <=
// 448 (1 + 2^-23) from the scale rule, or NaN, which stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// Two e4m3 bytes (low 16 bits of w) to floats, exactly.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w)));
  __half2 v;
  __builtin_memcpy(&v, &h, 4);
  return __half22float2(v);
}

// A k-block's term of a product is P a b: its sum P and the two operands' scales.  |P|
// is 0 or at least 2^-18, and at most 2^25, but a b may pass fp32's range, or lose
// bits below 2^-126, where the term is an ordinary number (a block whose maximum is
// 1e30 against one of 1e14 where the other operand is zero: inf * 0).  So a b is
// formed only where it is a normal number; otherwise P meets the scale of smaller
// magnitude first, or one of the two whatever they are, which is right for scales
// between 2^-109 and 2^103.
__device__ __forceinline__ bool scale_fits(float ab) {
  return fabsf(ab) <= 0x1.fffffep127f && fabsf(ab) >= 0x1p-126f;  // NaN does not
}
__device__ __forceinline__ void scale_order(float a, float b, float& lo, float& hi) {
  const bool less = fabsf(a) < fabsf(b);  // a NaN stays one of the two
  lo = less ? a : b;
  hi = less ? b : a;
}
__device__ __forceinline__ float add_scaled(float acc, float P, float a, float b) {
  float lo, hi;
  scale_order(a, b, lo, hi);
  return fmaf(__fmul_rn(P, lo), hi, acc);
}

// An operand of a product seen as rows (the M or N axis) by K: byte (mn, k) at
// data[mn * s_mn + k * s_k], one of the strides being 1; the scale of row mn
// and k-block kb at scale[(mn >> mn_shift) * c_mn + kb * c_kb].
struct Fp8Operand {
  const uint8_t* data;
  int64_t s_mn, s_k;
  const float* scale;
  int64_t c_mn, c_kb;
  int32_t mn_shift;  // 0: a scale per row, 7: per 128 rows
};

struct Fp8Product {
  int64_t M, N, K;
  Fp8Operand A, B;
  const float* bias;
  void* C;
  int64_t ldc;
  int out_dtype;
};

cudaError_t launch_fp8_quantize(int64_t rows, int64_t cols, const void* src, int64_t ld_src,
                                int src_dtype, const gemm_fp8_matrix_t* out,
                                const gemm_fp8_matrix_t* out2, cudaStream_t stream);
// CUDA-core product: any strides, any alignment (fp8_simt.cu).
cudaError_t launch_fp8_simt(const Fp8Product& p, cudaStream_t stream);
// Tensor-core product (fp8_tc.cu), where fp8_tc_runs.
bool fp8_tc_runs(const Fp8Product& p);
cudaError_t launch_fp8_tc(gemm_ctx* h, const Fp8Product& p, cudaStream_t stream);

// Mixture-of-experts layer (fp8_moe.cu).
int64_t moe_workspace_bytes(const gemm_ctx* h, const gemm_moe_fp8_t& L);
cudaError_t launch_moe(gemm_ctx* h, const gemm_moe_fp8_t& L, void* workspace,
                       cudaStream_t stream);

// Stores v as element type `dtype`, rounded once.
__device__ __forceinline__ void store_typed(void* base, int64_t i, float v, int dtype) {
  if (dtype == GEMM_F32)
    static_cast<float*>(base)[i] = v;
  else if (dtype == GEMM_F16)
    static_cast<__half*>(base)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}

}  // namespace dg

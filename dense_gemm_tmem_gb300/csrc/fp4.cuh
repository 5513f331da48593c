// fp4.cuh: what the 4-bit kernels share: e2m1 and scale conversions, the place
// of a block's scale, and the launch descriptions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm_fp4.h"
#include "fp8.cuh"

namespace dg {

constexpr int kFp4Piece = 512;  // bytes of 128 rows x 4 blocks of scales
__host__ __device__ constexpr int fp4_block(int format) { return format == GEMM_MXFP4 ? 32 : 16; }

// Where row r's scale of block b lies; `pieces` = ceil(blocks / 4).
__host__ __device__ __forceinline__ int64_t fp4_scale_at(int64_t r, int64_t b, int64_t pieces) {
  return ((r >> 7) * pieces + (b >> 2)) * kFp4Piece + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

// Eight floats to e2m1, round to nearest even, saturating, the first in the word's
// lowest bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 p, q, s, t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 s, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %8, %7;\n\t"
      "mov.b32 %0, {p, q, s, t};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// The two values of a byte (low 8 bits of w), exactly.
__device__ __forceinline__ float2 unpack_e2m1x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 p, q, s, t;\n\t"
      "mov.b32 {p, q, s, t}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\t}"
      : "=r"(h)
      : "r"(w));
  __half2 v;
  __builtin_memcpy(&v, &h, 4);
  return __half22float2(v);
}

// A block scale's value.  e8m0 0 is 2^-127, below fp32's normal numbers.
__device__ __forceinline__ float fp4_scale_value(uint32_t byte, int format) {
  if (format == GEMM_MXFP4)
    return byte == 255 ? NAN : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
  return unpack_e4m3x2(byte).x;
}

struct Fp4Product {
  int64_t M, N, K;
  gemm_fp4_matrix_t A, B;
  const float* bias;
  void* C;
  int64_t ldc;
  int out_dtype;
};

cudaError_t launch_fp4_quantize(int64_t rows, int64_t cols, const void* src, int64_t ld_src,
                                int src_dtype, const gemm_fp4_matrix_t& out, bool pdl,
                                cudaStream_t stream);
cudaError_t launch_fp4_dequantize(int64_t rows, int64_t cols, const gemm_fp4_matrix_t& m,
                                  void* dst, int64_t ld_dst, int dst_dtype, cudaStream_t stream);
// Whether gemm_fp4_run takes one row of A on the CUDA cores.
bool fp4_one_row(const gemm_ctx* h, int64_t N);
// One row of A; where `x` is given, K elements of its type, they are quantised on the way and
// p.A is not looked at.
cudaError_t launch_fp4_row(gemm_ctx* h, const Fp4Product& p, const void* x, int x_dtype,
                           cudaStream_t stream);
cudaError_t launch_fp4(gemm_ctx* h, const Fp4Product& p, cudaStream_t stream);

}  // namespace dg

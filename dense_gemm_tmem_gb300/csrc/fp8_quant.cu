// fp8_quant.cu: a matrix to e4m3 with one fp32 scale per 1 x 128, 128 x 1 or
// 128 x 128 block (include/gemm_fp8.h), rows and columns in one pass if asked.
//
// Per block a = max |x| over its finite elements, s = max(a, 2^-100) / 448,
// q = e4m3(x * (448 / max(a, 2^-100))), each fp32 operation rounded to nearest.
// Memory is the only bound: every element is read once and written once per
// output.  A CTA therefore holds a whole 128 x 128 tile in registers (64
// elements a thread, 8 rows of 8 neighbours), takes the maxima of its rows
// (shuffles among the 16 threads of a row) and of its columns (one shuffle and
// a 4 KiB shared exchange) from the same registers, and writes both outputs
// from them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.cuh"

namespace dg {
namespace {

constexpr int kQuantThreads = 256;  // 16 across x 16 down, 8 x 8 elements each
constexpr int kRowsPer = 8;         // rows ty, ty + 16, ...
constexpr int kColsPer = 8;         // columns 8 tx ... 8 tx + 7

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// Eight consecutive elements, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      T lo, hi;
      const uint16_t l = uint16_t(w[i] & 0xffffu), h = uint16_t(w[i] >> 16);
      __builtin_memcpy(&lo, &l, 2);
      __builtin_memcpy(&hi, &h, 2);
      v[2 * i] = to_f32<T>(lo);
      v[2 * i + 1] = to_f32<T>(hi);
    }
  }
}

// Writes 8 neighbouring e4m3 values, the first `valid` of them.
__device__ __forceinline__ void store8(uint8_t* p, const float (&q)[8], int valid, bool aligned) {
  const uint32_t lo = pack_e4m3x4(q[0], q[1], q[2], q[3]);
  const uint32_t hi = pack_e4m3x4(q[4], q[5], q[6], q[7]);
  if (valid == 8 && aligned) {
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) p[j] = uint8_t((j < 4 ? lo >> (8 * j) : hi >> (8 * (j - 4))) & 0xff);
}

struct QuantOut {
  uint8_t* data;
  int64_t ld;
  float* scale;
  int64_t sr, sc;
  bool aligned;  // 8-byte stores allowed
};

struct QuantArgs {
  const void* src;
  int64_t rows, cols, ld;
  bool vec;  // 16-byte loads allowed
  int32_t tiles_c;
  QuantOut row, col, tile;
};

enum : int { kRow = 1, kCol = 2, kTile = 4 };

template <typename T, int MODE>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantArgs a) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int warp = threadIdx.x >> 5;
  const int32_t bi = int32_t(blockIdx.x / uint32_t(a.tiles_c));
  const int32_t bj = int32_t(blockIdx.x % uint32_t(a.tiles_c));
  const int64_t r0 = int64_t(bi) * kFp8Block, c0 = int64_t(bj) * kFp8Block + tx * kColsPer;
  const int valid = int(min(int64_t(kColsPer), a.cols - c0));  // <= 0: no column of this thread
  const T* src = static_cast<const T*>(a.src);

  float v[kRowsPer][kColsPer];
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    const int64_t r = r0 + ty + 16 * i;
#pragma unroll
    for (int j = 0; j < kColsPer; ++j) v[i][j] = 0.f;
    if (r < a.rows && valid > 0) {
      const T* p = src + r * a.ld + c0;
      if (a.vec && valid == kColsPer) {
        load8<T>(p, v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kColsPer; ++j)
          if (j < valid) v[i][j] = to_f32<T>(p[j]);
      }
    }
  }
  // fmaxf passes over NaN; an infinity becomes NaN here, so it is stored as
  // NaN and is in no maximum
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
    for (int j = 0; j < kColsPer; ++j) most = fmaxf(most, fabsf(v[i][j]));
  if (most == INFINITY) {
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
      for (int j = 0; j < kColsPer; ++j)
        if (fabsf(v[i][j]) == INFINITY) v[i][j] = NAN;
  }

  if constexpr ((MODE & kRow) != 0) {
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < kColsPer; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float inv = fp8_inverse(m);
      const int64_t r = r0 + ty + 16 * i;
      if (r < a.rows) {
        if (tx == 0) a.row.scale[r * a.row.sr + int64_t(bj) * a.row.sc] = fp8_scale(m);
        if (valid > 0) {
          float q[kColsPer];
#pragma unroll
          for (int j = 0; j < kColsPer; ++j) q[j] = __fmul_rn(v[i][j], inv);
          store8(a.row.data + r * a.row.ld + c0, q, valid, a.row.aligned);
        }
      }
    }
  }
  if constexpr ((MODE & kCol) != 0) {
    __shared__ float red[kQuantThreads / 32][kFp8Block];
    __shared__ float cinv[kFp8Block];
#pragma unroll
    for (int j = 0; j < kColsPer; ++j) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) m = fmaxf(m, fabsf(v[i][j]));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));  // the warp's other row
      if ((threadIdx.x & 31) < 16) red[warp][tx * kColsPer + j] = m;
    }
    __syncthreads();
    if (threadIdx.x < kFp8Block) {
      float m = 0.f;
#pragma unroll
      for (int w = 0; w < kQuantThreads / 32; ++w) m = fmaxf(m, red[w][threadIdx.x]);
      cinv[threadIdx.x] = fp8_inverse(m);
      const int64_t c = int64_t(bj) * kFp8Block + threadIdx.x;
      if (c < a.cols) a.col.scale[int64_t(bi) * a.col.sr + c * a.col.sc] = fp8_scale(m);
    }
    __syncthreads();
    float inv[kColsPer];
#pragma unroll
    for (int j = 0; j < kColsPer; ++j) inv[j] = cinv[tx * kColsPer + j];
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const int64_t r = r0 + ty + 16 * i;
      if (r < a.rows && valid > 0) {
        float q[kColsPer];
#pragma unroll
        for (int j = 0; j < kColsPer; ++j) q[j] = __fmul_rn(v[i][j], inv[j]);
        store8(a.col.data + r * a.col.ld + c0, q, valid, a.col.aligned);
      }
    }
  }
  if constexpr ((MODE & kTile) != 0) {
    __shared__ float wmax[kQuantThreads / 32];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
      for (int j = 0; j < kColsPer; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) wmax[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) m = fmaxf(m, wmax[w]);
    const float inv = fp8_inverse(m);
    if (threadIdx.x == 0)
      a.tile.scale[int64_t(bi) * a.tile.sr + int64_t(bj) * a.tile.sc] = fp8_scale(m);
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const int64_t r = r0 + ty + 16 * i;
      if (r < a.rows && valid > 0) {
        float q[kColsPer];
#pragma unroll
        for (int j = 0; j < kColsPer; ++j) q[j] = __fmul_rn(v[i][j], inv);
        store8(a.tile.data + r * a.tile.ld + c0, q, valid, a.tile.aligned);
      }
    }
  }
}

QuantOut out_of(const gemm_fp8_matrix_t* m) {
  QuantOut o{};
  if (!m) return o;
  o.data = static_cast<uint8_t*>(m->data);
  o.ld = m->ld;
  o.scale = m->scale;
  o.sr = m->scale_stride_r;
  o.sc = m->scale_stride_c;
  o.aligned = ((reinterpret_cast<uintptr_t>(m->data) | uintptr_t(m->ld)) & 7) == 0;
  return o;
}

template <typename T>
cudaError_t launch_typed(const QuantArgs& a, int mode, unsigned grid, cudaStream_t s) {
  switch (mode) {
    case kRow: quantize_kernel<T, kRow><<<grid, kQuantThreads, 0, s>>>(a); break;
    case kCol: quantize_kernel<T, kCol><<<grid, kQuantThreads, 0, s>>>(a); break;
    case kRow | kCol: quantize_kernel<T, kRow | kCol><<<grid, kQuantThreads, 0, s>>>(a); break;
    case kTile: quantize_kernel<T, kTile><<<grid, kQuantThreads, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp8_quantize(int64_t rows, int64_t cols, const void* src, int64_t ld_src,
                                int src_dtype, const gemm_fp8_matrix_t* out,
                                const gemm_fp8_matrix_t* out2, cudaStream_t stream) {
  QuantArgs a{};
  a.src = src;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld_src;
  const int64_t size = src_dtype == GEMM_F32 ? 4 : 2;
  a.vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0 && (ld_src * size) % 16 == 0;
  const int64_t tr = (rows + kFp8Block - 1) / kFp8Block, tc = (cols + kFp8Block - 1) / kFp8Block;
  a.tiles_c = int32_t(tc);
  int mode = 0;
  for (const gemm_fp8_matrix_t* m : {out, out2}) {
    if (!m) continue;
    if (m->blocks == GEMM_FP8_ROW) { a.row = out_of(m); mode |= kRow; }
    if (m->blocks == GEMM_FP8_COL) { a.col = out_of(m); mode |= kCol; }
    if (m->blocks == GEMM_FP8_TILE) { a.tile = out_of(m); mode |= kTile; }
  }
  const unsigned grid = unsigned(tr * tc);
  if (src_dtype == GEMM_F32) return launch_typed<float>(a, mode, grid, stream);
  if (src_dtype == GEMM_F16) return launch_typed<__half>(a, mode, grid, stream);
  return launch_typed<__nv_bfloat16>(a, mode, grid, stream);
}

}  // namespace dg

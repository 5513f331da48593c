// fp4_quant.cu: a matrix to e2m1 with a scale per 1 x 32 (mxfp4) or 1 x 16
// (nvfp4) block, and back (include/gemm_fp4.h).
//
// Memory is the bound: an element is read once and 9/16 of a byte written for
// it.  A thread takes 16 neighbours of a row (an nvfp4 block; half an mxfp4
// block, whose two threads share their maxima by a shuffle), so that it writes 8
// bytes of values, and 4 neighbouring blocks' threads put their scales into one
// 4-byte word.  nvfp4 needs the row's maximum first: the threads of a row (a warp,
// or the whole CTA) keep their elements in registers across that reduction; rows
// too long for that are read twice.
#include <type_traits>

#include "fp4.cuh"

namespace dg {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kUnit = 16;  // elements a thread takes at a time

// 16 neighbouring elements as loaded.
template <typename T>
struct Unit16 {
  static constexpr int kWords = sizeof(T) * kUnit / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p, int valid, bool vec) {
    if (vec && valid >= kUnit) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      if (j >= valid) continue;
      if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(float(p[j]));
      else w[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[j]);
    } else {
      const uint16_t h = uint16_t(w[j / 2] >> (16 * (j & 1)));
      T v;
      __builtin_memcpy(&v, &h, 2);
      if constexpr (std::is_same<T, __half>::value) return __half2float(v);
      else return __bfloat162float(v);
    }
  }
  // The largest finite magnitude; `odd`: there is a non-finite element.
  __device__ __forceinline__ float amax(bool& odd) const {
    float m = 0.f;
    odd = false;
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      const float a = fabsf(get(j));
      const bool fine = a < INFINITY;
      odd |= !fine;
      m = fmaxf(m, fine ? a : 0.f);
    }
    return m;
  }
};

struct QuantArgs {
  const void* src;
  int64_t rows, cols, ld;
  bool vec;
  gemm_fp4_matrix_t out;
  int64_t pieces;
};

// One unit's block: its scale byte and the factor of its elements.
template <int FMT>
__device__ __forceinline__ void block_scale(float amax, bool odd, float a448, float a2688,
                                            uint32_t& byte, float& factor) {
  if constexpr (FMT == GEMM_MXFP4) {
    const int e = int(__float_as_uint(amax) >> 23);
    byte = uint32_t(max(e - 2, 0));
    factor = __uint_as_float((254u - byte) << 23);
    if (odd) byte = 255;
  } else {
    byte = pack_e4m3x2(__fmul_rn(amax, a448), 0.f) & 0xffu;
    const float s = unpack_e4m3x2(byte).x;
    factor = s > 0.f ? __fdiv_rn(a2688, s) : 0.f;
    if (odd) byte = 0x7f;
  }
}

// A row per TPR threads (32: a warp, or the whole CTA), U units a thread in
// registers.
template <typename T, int FMT, int TPR, int U>
__global__ void __launch_bounds__(kQuantThreads) fp4_quantize_kernel(const QuantArgs a) {
  constexpr int kRowsPer = kQuantThreads / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t r = int64_t(blockIdx.x) * kRowsPer + threadIdx.x / TPR;
  const int64_t units = a.pieces * (fp4_block(FMT) * 4 / kUnit);  // whole pieces
  uint8_t* const scale = static_cast<uint8_t*>(a.out.scale);
  constexpr int kPer = FMT == GEMM_MXFP4 ? 8 : 4;  // threads of a piece's four blocks
  if (r >= (a.rows + 127) / 128 * 128) return;     // (whole warps, or the whole CTA)
  if (r >= a.rows) {                               // a row that only fills up a piece
    for (int64_t p = t; p < a.pieces; p += TPR)
      *reinterpret_cast<uint32_t*>(scale + fp4_scale_at(r, 4 * p, a.pieces)) = 0;
    return;
  }
  const T* const src = static_cast<const T*>(a.src) + r * a.ld;
  uint8_t* const data = static_cast<uint8_t*>(a.out.data) + r * a.out.ld;
  Unit16<T> x[U];
  auto load = [&](int64_t u0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = (u0 + t + i * TPR) * kUnit;
      x[i].load(src + c, int(max(int64_t(0), min(int64_t(kUnit), a.cols - c))), a.vec);
    }
  };
  load(0);
  float a448 = 0.f, a2688 = 0.f;
  if constexpr (FMT == GEMM_NVFP4) {
    float most = 0.f;
    bool odd;
    for (int64_t u0 = 0;;) {
#pragma unroll
      for (int i = 0; i < U; ++i) most = fmaxf(most, x[i].amax(odd));
      u0 += TPR * U;
      if (u0 >= units) break;
      load(u0);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    if constexpr (TPR > 32) {
      __shared__ float red[kQuantThreads / 32];
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQuantThreads / 32; ++w) most = fmaxf(most, red[w]);
    }
    most = fmaxf(most, kAmaxMin);
    a448 = __fdiv_rn(448.f, most);
    a2688 = __fdiv_rn(2688.f, most);
    if (t == 0) a.out.row_scale[r * a.out.row_scale_stride] = __fdiv_rn(most, 2688.f);
    if (units > TPR * U) load(0);
  }
  for (int64_t u0 = 0; u0 < units; u0 += TPR * U) {
    if (u0 > 0) load(u0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = u0 + t + i * TPR, c = u * kUnit;
      bool odd;
      float m = x[i].amax(odd);
      if constexpr (FMT == GEMM_MXFP4) {  // the block's other half
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        odd |= __shfl_xor_sync(0xffffffffu, int(odd), 1) != 0;
      }
      uint32_t byte;
      float f;
      block_scale<FMT>(m, odd, a448, a2688, byte, f);
      // blocks past the matrix have scale 0
      if (c >= (a.cols + fp4_block(FMT) - 1) / fp4_block(FMT) * fp4_block(FMT)) byte = 0;
      float q[kUnit];
#pragma unroll
      for (int j = 0; j < kUnit; ++j) q[j] = odd ? 0.f : __fmul_rn(x[i].get(j), f);
      const uint2 v = make_uint2(pack_e2m1x8(q), pack_e2m1x8(q + 8));
      // the four blocks' scales to the first of their threads
      constexpr int kStep = kPer / 4;
      uint32_t word = byte << (8 * ((threadIdx.x % kPer) / kStep));
      word |= __shfl_xor_sync(0xffffffffu, word, kStep);
      word |= __shfl_xor_sync(0xffffffffu, word, 2 * kStep);
      if (u >= units) continue;
      if (threadIdx.x % kPer == 0)
        *reinterpret_cast<uint32_t*>(scale + fp4_scale_at(r, c / fp4_block(FMT), a.pieces)) = word;
      const int64_t left = (a.cols - c + 1) / 2;  // bytes
      if (left >= 8) {
        *reinterpret_cast<uint2*>(data + c / 2) = v;
      } else {
        for (int j = 0; j < left; ++j)
          data[c / 2 + j] = uint8_t((j < 4 ? v.x >> (8 * j) : v.y >> (8 * (j - 4))) & 0xff);
      }
    }
  }
}

template <typename T, int FMT>
cudaError_t launch_format(const QuantArgs& a, cudaStream_t s) {
  const int64_t rows = (a.rows + 127) / 128 * 128;
  if (a.cols <= 2 * 32 * kUnit) {
    constexpr int kPer = kQuantThreads / 32;
    fp4_quantize_kernel<T, FMT, 32, 2>
        <<<unsigned((rows + kPer - 1) / kPer), kQuantThreads, 0, s>>>(a);
  } else {
    fp4_quantize_kernel<T, FMT, kQuantThreads, 2><<<unsigned(rows), kQuantThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const QuantArgs& a, cudaStream_t s) {
  return a.out.format == GEMM_MXFP4 ? launch_format<T, GEMM_MXFP4>(a, s)
                                    : launch_format<T, GEMM_NVFP4>(a, s);
}

// ---------------------------------------------------------------- reading back --
struct BackArgs {
  gemm_fp4_matrix_t m;
  int64_t rows, cols, ld, pieces;
  int64_t units;  // 16 elements each, a row
  void* dst;
  int dtype;
  bool vec;
};

__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const BackArgs a) {
  const int64_t total = a.rows * a.units;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / a.units, c = (i - r * a.units) * kUnit;
    const int64_t b = c / fp4_block(a.m.format);
    const float s = fp4_scale_value(
        static_cast<const uint8_t*>(a.m.scale)[fp4_scale_at(r, b, a.pieces)], a.m.format);
    const uint8_t* p = static_cast<const uint8_t*>(a.m.data) + r * a.m.ld + c / 2;
    uint2 q = make_uint2(0, 0);
    const int64_t bytes = (a.cols - c + 1) / 2;
    if (bytes >= 8) {
      q = __ldg(reinterpret_cast<const uint2*>(p));
    } else {
      for (int j = 0; j < bytes; ++j) (j < 4 ? q.x : q.y) |= uint32_t(p[j]) << (8 * (j & 3));
    }
    const bool has = a.m.row_scale != nullptr;
    const float g = has ? a.m.row_scale[r * a.m.row_scale_stride] : 1.f;
    float v[kUnit];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 x = unpack_e2m1x2((j < 4 ? q.x >> (8 * j) : q.y >> (8 * (j - 4))) & 0xff);
      v[2 * j] = __fmul_rn(x.x, s) * g;
      v[2 * j + 1] = __fmul_rn(x.y, s) * g;
    }
    const int64_t at = r * a.ld + c;
    if (a.vec && c + kUnit <= a.cols) {
      if (a.dtype == GEMM_F32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.dst) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (a.dtype == GEMM_F16) {
            const __half2 x = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
            __builtin_memcpy(&w[j], &x, 4);
          } else {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            __builtin_memcpy(&w[j], &x, 4);
          }
        }
        uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dst) + at);
        d[0] = make_uint4(w[0], w[1], w[2], w[3]);
        d[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kUnit; ++j)
        if (c + j < a.cols) store_typed(a.dst, at + j, v[j], a.dtype);
    }
  }
}

int64_t pieces_of(int64_t cols, int format) {
  const int64_t per = 4 * fp4_block(format);
  return (cols + per - 1) / per;
}

}  // namespace

cudaError_t launch_fp4_quantize(int64_t rows, int64_t cols, const void* src, int64_t ld_src,
                                int src_dtype, const gemm_fp4_matrix_t& out,
                                cudaStream_t stream) {
  const int64_t size = src_dtype == GEMM_F32 ? 4 : 2;
  const bool vec = (reinterpret_cast<uintptr_t>(src) & 15) == 0 &&
                   (rows == 1 || (ld_src * size) % 16 == 0);
  const QuantArgs a{src, rows, cols, ld_src, vec, out, pieces_of(cols, out.format)};
  if (src_dtype == GEMM_F32) return launch_typed<float>(a, stream);
  if (src_dtype == GEMM_F16) return launch_typed<__half>(a, stream);
  return launch_typed<__nv_bfloat16>(a, stream);
}

cudaError_t launch_fp4_dequantize(int64_t rows, int64_t cols, const gemm_fp4_matrix_t& m,
                                  void* dst, int64_t ld_dst, int dst_dtype, cudaStream_t stream) {
  const int64_t size = dst_dtype == GEMM_F32 ? 4 : 2;
  const int64_t units = (cols + kUnit - 1) / kUnit;
  const bool vec = (reinterpret_cast<uintptr_t>(dst) & 15) == 0 &&
                   (rows == 1 || (ld_dst * size) % 16 == 0);
  const BackArgs a{m,     rows, cols,      ld_dst, pieces_of(cols, m.format),
                   units, dst,  dst_dtype, vec};
  const int64_t ctas = (rows * units + 255) / 256;
  fp4_dequantize_kernel<<<unsigned(ctas < (1 << 20) ? ctas : (1 << 20)), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dg

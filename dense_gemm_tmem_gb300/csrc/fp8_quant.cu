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
// from them.  What is left to keep short is the instruction count: 16-bit
// elements stay packed and their maxima are taken two at a time as integers
// (magnitudes order like their bits), and the divisions of a thread's 8 rows
// are shared out among the 16 threads that need them.  Four CTAs an SM for
// 16-bit sources (8192 x 8192 bf16 both ways: 53 us with three, 48 with four,
// 5.7 TB/s of the 6.8 a copy reaches here).  For fp32 ones the tile alone takes 64
// registers: three CTAs for 128 x 128 and 128 x 1 blocks (2050 x 5000 tiles 10.6 us
// with two, 9.6 with three; 8192 x 8192 columns 53.3 and 51.3, though they spill 60
// bytes: 2050 x 5000 11.8 and 12.0, 2048 x 4101, which 16-byte loads cannot read, 13.7
// and 16.1), two where rows are kept as well (8192 x 8192 both ways 69.6 us, 79.6 with
// three, which spill; 4096 x 4096 rows 18.1 and 19.3).
// Rows that 16-byte loads cannot read (an odd pitch, an unaligned base) are read element
// by element: 8192 x 8191 bf16 rows 70 us, 8192 x 8192 36; 2048 x 4101 11.7, 2048 x 4096
// 8.2.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8.cuh"

namespace dg {
namespace {

constexpr int kQuantThreads = 256;  // 16 across x 16 down, 8 x 8 elements each
constexpr int kRowsPer = 8;         // rows ty, ty + 16, ...
constexpr int kColsPer = 8;         // columns 8 tx ... 8 tx + 7

// Eight neighbouring elements of a row: fp32 values, or 16-bit ones in pairs.
template <typename T>
struct Row8 {
  uint32_t w[4];
  static constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;

  __device__ __forceinline__ void load(const T* p) {  // 16-byte aligned
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ __forceinline__ void load(const T* p, int valid) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = 0;
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) w[j / 2] |= uint32_t(h[j]) << (16 * (j & 1));
  }
  __device__ __forceinline__ float get(int j) const {
    const uint16_t h = uint16_t(w[j / 2] >> (16 * (j & 1)));
    T v;
    __builtin_memcpy(&v, &h, 2);
    if constexpr (std::is_same<T, __half>::value) return __half2float(v);
    else return __bfloat162float(v);
  }
  // Magnitudes of pair k; `clean`: non-finite ones count as 0.
  template <bool clean>
  __device__ __forceinline__ uint32_t mag(int k) const {
    uint32_t a = w[k] & 0x7fff7fffu;
    if constexpr (clean) {
      if ((a & 0xffffu) >= kInf) a &= 0xffff0000u;
      if ((a >> 16) >= kInf) a &= 0xffffu;
    }
    return a;
  }
  // Infinities become NaN.
  __device__ __forceinline__ void poison() {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if ((w[k] & 0x7fffu) == kInf) w[k] |= 1u;
      if ((w[k] >> 16 & 0x7fffu) == kInf) w[k] |= 0x10000u;
    }
  }
};
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
// The larger of a pair's two magnitudes, as fp32.
template <typename T>
__device__ __forceinline__ float wide(uint32_t pair) {
  const uint16_t h = uint16_t(max(pair & 0xffffu, pair >> 16));
  T v;
  __builtin_memcpy(&v, &h, 2);
  if constexpr (std::is_same<T, __half>::value) return __half2float(v);
  else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ float half_of(uint32_t pair, int i) {
  return wide<T>(i ? pair >> 16 : pair & 0xffffu);
}

template <>
struct Row8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void load(const float* p, int valid) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? p[j] : 0.f;
  }
  __device__ __forceinline__ float get(int j) const { return v[j]; }
};

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

// CTAs an SM that the registers are cut for.
constexpr int quant_ctas(size_t size, int mode) {
  return size == 2 ? 4 : mode == kTile || mode == kCol ? 3 : 1;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kQuantThreads, quant_ctas(sizeof(T), MODE))
    quantize_kernel(const QuantArgs a) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int warp = threadIdx.x >> 5;
  const int32_t bi = int32_t(blockIdx.x / uint32_t(a.tiles_c));
  const int32_t bj = int32_t(blockIdx.x % uint32_t(a.tiles_c));
  const int64_t r0 = int64_t(bi) * kFp8Block, c0 = int64_t(bj) * kFp8Block + tx * kColsPer;
  const int valid = int(min(int64_t(kColsPer), a.cols - c0));  // <= 0: no column of this thread
  const T* src = static_cast<const T*>(a.src);

  Row8<T> x[kRowsPer];
  if (a.vec && r0 + kFp8Block <= a.rows && int64_t(bj + 1) * kFp8Block <= a.cols) {
    // a whole tile: no condition between the loads, so that all are in flight
    // together (with one per row, 8192 x 8192 bf16 both ways took 125 us)
    const T* p = src + (r0 + ty) * a.ld + c0;
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i, p += 16 * a.ld) x[i].load(p);
  } else {
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const int64_t r = r0 + ty + 16 * i;
      const T* p = src + (r < a.rows ? r * a.ld : 0) + c0;
      if (r < a.rows && a.vec && valid >= kColsPer) x[i].load(p);
      else x[i].load(p, r < a.rows ? valid : 0);
    }
  }

  // maxima of this thread's rows and columns over their finite elements
  constexpr bool kRows = (MODE & (kRow | kTile)) != 0, kCols = (MODE & kCol) != 0;
  float rmax[kRowsPer], cmax[kColsPer];
  if constexpr (sizeof(T) == 4) {
    auto maxima = [&]() {
      float most = 0.f;
#pragma unroll
      for (int j = 0; j < kColsPer; ++j) cmax[j] = 0.f;
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) {
        rmax[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kColsPer; ++j) {  // fmaxf passes over NaN
          const float m = fabsf(x[i].v[j]);
          if (kRows || !kCols) rmax[i] = fmaxf(rmax[i], m);
          if (kCols) cmax[j] = fmaxf(cmax[j], m);
        }
        most = fmaxf(most, rmax[i]);
      }
#pragma unroll
      for (int j = 0; j < kColsPer; ++j) most = fmaxf(most, cmax[j]);
      return most;
    };
    if (maxima() == INFINITY) {  // infinities become NaN: stored as such, in no maximum
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i)
#pragma unroll
        for (int j = 0; j < kColsPer; ++j)
          if (fabsf(x[i].v[j]) == INFINITY) x[i].v[j] = NAN;
      maxima();
    }
  } else {
    uint32_t cp[4], rp[kRowsPer];
    auto maxima = [&](auto clean) {
      uint32_t most = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) cp[k] = 0;
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) {
        uint32_t m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m[k] = x[i].template mag<decltype(clean)::value>(k);
          if (kCols) cp[k] = max2(cp[k], m[k]);
        }
        if (kRows || !kCols) {
          rp[i] = max2(max2(m[0], m[1]), max2(m[2], m[3]));
          most = max2(most, rp[i]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) most = max2(most, cp[k]);
      return max(most & 0xffffu, most >> 16);
    };
    if (maxima(std::false_type()) >= Row8<T>::kInf) {
      maxima(std::true_type());
#pragma unroll
      for (int i = 0; i < kRowsPer; ++i) x[i].poison();
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i)
      if (kRows) rmax[i] = wide<T>(rp[i]);
#pragma unroll
    for (int j = 0; j < kColsPer; ++j)
      if (kCols) cmax[j] = half_of<T>(cp[j / 2], j & 1);
  }

  if constexpr ((MODE & kRow) != 0) {
    // the 16 threads of a row share its maximum; each divides for one of the
    // thread's 8 rows (every row twice), and hands the factor round
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
#pragma unroll
      for (int d = 1; d < 16; d <<= 1)
        rmax[i] = fmaxf(rmax[i], __shfl_xor_sync(0xffffffffu, rmax[i], d));
      if ((tx & 7) == i) mine = rmax[i];
    }
    const float my_inv = fp8_inverse(mine), my_scale = fp8_scale(mine);
    {
      const int64_t r = r0 + ty + 16 * (tx & 7);
      if (tx < 8 && r < a.rows) a.row.scale[r * a.row.sr + int64_t(bj) * a.row.sc] = my_scale;
    }
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const float inv = __shfl_sync(0xffffffffu, my_inv, (threadIdx.x & 16) + i);
      const int64_t r = r0 + ty + 16 * i;
      if (r < a.rows && valid > 0) {
        float q[kColsPer];
#pragma unroll
        for (int j = 0; j < kColsPer; ++j) q[j] = __fmul_rn(x[i].get(j), inv);
        store8(a.row.data + r * a.row.ld + c0, q, valid, a.row.aligned);
      }
    }
  }
  if constexpr ((MODE & kCol) != 0) {
    __shared__ float red[kQuantThreads / 32][kFp8Block];
    __shared__ float cinv[kFp8Block];
#pragma unroll
    for (int j = 0; j < kColsPer; ++j) {
      cmax[j] = fmaxf(cmax[j], __shfl_xor_sync(0xffffffffu, cmax[j], 16));  // the other row
      if ((threadIdx.x & 31) < 16) red[warp][tx * kColsPer + j] = cmax[j];
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
        for (int j = 0; j < kColsPer; ++j) q[j] = __fmul_rn(x[i].get(j), inv[j]);
        store8(a.col.data + r * a.col.ld + c0, q, valid, a.col.aligned);
      }
    }
  }
  if constexpr ((MODE & kTile) != 0) {
    __shared__ float wmax[kQuantThreads / 32];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) m = fmaxf(m, rmax[i]);
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
        for (int j = 0; j < kColsPer; ++j) q[j] = __fmul_rn(x[i].get(j), inv);
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

// fp4_quant.cu: a matrix to e2m1 with a scale per 1 x 32 (mxfp4) or 1 x 16
// (nvfp4) block, and back (include/gemm_fp4.h).
//
// Memory is the bound: an element is read once and 9/16 of a byte written for
// it.  A thread takes 16 neighbours of a row (an nvfp4 block; half an mxfp4
// block, whose two threads share their maxima by a shuffle), so that it writes 8
// bytes of values, and 4 neighbouring blocks' threads put their scales into one
// 4-byte word.  nvfp4 needs the row's maximum first: the threads of a row (a warp,
// or the whole CTA) keep their elements in registers across that reduction; rows
// too long for that are read twice.  What is left to keep short is the instruction
// count: 16-bit elements stay packed and maxima are taken of magnitudes as integers
// (which order like the numbers), and a row's division by its blocks' scales, which
// have 8 different mantissas, is made once for each of those (8192^2 bf16 nvfp4 54 us
// before, 32 now, 5.4 TB/s; mxfp4, which waits for no row, 30; graph replay, as below).
// Reading back is bound by its stores: 8192^2 bf16 38 us (mxfp4 39), where filling as many
// bytes takes 35.4; streaming stores, 2 or 8 rows a thread instead of 4: 3 to 10 % more.
#include "fp4_quant.cuh"

namespace dg {
namespace {

constexpr int kQuantThreads = 128;
constexpr int kBackThreads = 256;

// Launches of up to so many CTAs let the next kernel's CTAs in beside them (and enter
// beside the last kernel's): of longer ones they would take room.
constexpr int64_t kEarlyCtas = 256;

struct QuantArgs {
  const void* src;
  int64_t rows, cols, ld;
  Span span;
  gemm_fp4_matrix_t out;
  int64_t pieces;
  bool early;  // the next kernel may start beside this one (GEMM_OPT_PDL)
};

// CTAs an SM that the registers are cut for.
constexpr int quant_ctas(size_t size, int units) {
  return size == 2 ? (units > 2 ? 8 : 10) : (units > 2 ? 5 : 8);
}

// A row per TPR threads (32: a warp, or the whole CTA), U units a thread in
// registers.
template <typename T, int FMT, int TPR, int U>
__global__ void __launch_bounds__(kQuantThreads, quant_ctas(sizeof(T), U))
    fp4_quantize_kernel(const QuantArgs a) {
  constexpr int kRowsPer = kQuantThreads / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t r = int64_t(blockIdx.x) * kRowsPer + threadIdx.x / TPR;
  const int64_t units = a.pieces * (fp4_block(FMT) * 4 / kUnit);  // whole pieces
  uint8_t* const scale = static_cast<uint8_t*>(a.out.scale);
  constexpr int kPer = FMT == GEMM_MXFP4 ? 8 : 4;  // threads of a piece's four blocks
  if (a.early) pdl_launch_dependents();
  pdl_wait_prerequisites();
  if (r >= (a.rows + 127) / 128 * 128) return;     // (whole warps, or the whole CTA)
  if (r >= a.rows) {                               // a row that only fills up a piece
    for (int64_t p = t; p < a.pieces; p += TPR)
      *reinterpret_cast<uint32_t*>(scale + fp4_scale_at(r, 4 * p, a.pieces)) = 0;
    return;
  }
  const T* const src = static_cast<const T*>(a.src) + r * a.ld;
  uint8_t* const data = static_cast<uint8_t*>(a.out.data) + r * a.out.ld;
  // the row's place among the scales; piece p is p * kFp4Piece further on
  uint8_t* const scale_row = scale + fp4_scale_at(r, 0, a.pieces);
  Unit16<T> x[U];
  float m[U];
  bool odd[U];
  auto load = [&](int64_t u0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t c = (u0 + t + i * TPR) * kUnit;
      x[i].load(src + c, int(max(int64_t(0), min(int64_t(kUnit), a.cols - c))), a.span);
    }
  };
  auto maxima = [&]() {
#pragma unroll
    for (int i = 0; i < U; ++i) m[i] = x[i].amax(odd[i]);
  };
  load(0);
  maxima();
  float a448 = 0.f, quotient = 0.f;
  if constexpr (FMT == GEMM_NVFP4) {
    float most = 0.f;
    for (int64_t u0 = 0;;) {
#pragma unroll
      for (int i = 0; i < U; ++i) most = fmaxf(most, m[i]);
      u0 += TPR * U;
      if (u0 >= units) break;
      load(u0);
      maxima();
    }
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    if constexpr (TPR > 32) {
      __shared__ float red[kQuantThreads / 32];
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = most;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kQuantThreads / 32; ++w) most = fmaxf(most, red[w]);
    }
    most = fmaxf(most, kAmaxMin);
    a448 = __fdiv_rn(448.f, most);
    // 2688 / a by each mantissa of an e4m3 number; its exponent then shifts exactly
    quotient = __fdiv_rn(__fdiv_rn(2688.f, most), 1.f + 0.125f * float(threadIdx.x & 7));
    if (t == 0) a.out.row_scale[r * a.out.row_scale_stride] = __fdiv_rn(most, 2688.f);
    if (units > TPR * U) {
      load(0);
      maxima();
    }
  }
  for (int64_t u0 = 0; u0 < units; u0 += TPR * U) {
    if (u0 > 0) {
      load(u0);
      maxima();
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = u0 + t + i * TPR, c = u * kUnit;
      uint32_t byte;
      float f;
      bool bad = odd[i];
      if constexpr (FMT == GEMM_MXFP4) {
        // the block's other half; 2^e with e = floor(log2 amax) - 2
        const float most = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
        bad |= __shfl_xor_sync(0xffffffffu, int(bad), 1) != 0;
        byte = uint32_t(max(int(__float_as_uint(most) >> 23) - 2, 0));
        f = __uint_as_float((254u - byte) << 23);
        if (bad) byte = 255;
      } else {
        byte = pack_e4m3x2(__fmul_rn(m[i], a448), 0.f) & 0xffu;
        const uint32_t s = __float_as_uint(unpack_e4m3x2(byte).x);
        f = __shfl_sync(0xffffffffu, quotient, (s >> 20) & 7) *
            __uint_as_float((254u << 23) - (s & 0x7f800000u));
        if (s == 0) f = 0.f;
        if (bad) byte = 0x7f;
      }
      // blocks past the matrix have scale 0
      if (c >= (a.cols + fp4_block(FMT) - 1) / fp4_block(FMT) * fp4_block(FMT)) byte = 0;
      float q[kUnit];
#pragma unroll
      for (int j = 0; j < kUnit / 2; ++j) {
        const float2 y = mul2(x[i].pair(j), f);
        q[2 * j] = y.x;
        q[2 * j + 1] = y.y;
      }
      uint2 v = make_uint2(pack_e2m1x8(q), pack_e2m1x8(q + 8));
      if (bad) v = make_uint2(0, 0);
      // the four blocks' scales to the first of their threads
      constexpr int kStep = kPer / 4;
      uint32_t word = byte << (8 * ((threadIdx.x % kPer) / kStep));
      word |= __shfl_xor_sync(0xffffffffu, word, kStep);
      word |= __shfl_xor_sync(0xffffffffu, word, 2 * kStep);
      if (u >= units) continue;
      if (threadIdx.x % kPer == 0)
        *reinterpret_cast<uint32_t*>(scale_row + u / kPer * kFp4Piece) = word;
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
cudaError_t launch_format(QuantArgs a, cudaStream_t s) {
  const int64_t rows = (a.rows + 127) / 128 * 128;
  const int64_t units = a.pieces * (fp4_block(FMT) * 4 / kUnit);
  constexpr int kPer = kQuantThreads / 32;
  // a warp a row up to 2 units a lane, else the CTA with as few units a thread as hold
  // the row, 4 at most
  const bool warps = units <= 2 * 32;
  const int64_t grid = warps ? rows / kPer : rows;
  a.early = a.early && grid <= kEarlyCtas;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(kQuantThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.early ? 1 : 0;
  if (warps) return cudaLaunchKernelEx(&cfg, fp4_quantize_kernel<T, FMT, 32, 2>, a);
  switch (units <= kQuantThreads ? 1 : units <= 2 * kQuantThreads ? 2
                                   : units <= 3 * kQuantThreads   ? 3
                                                                  : 4) {
    case 1: return cudaLaunchKernelEx(&cfg, fp4_quantize_kernel<T, FMT, kQuantThreads, 1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, fp4_quantize_kernel<T, FMT, kQuantThreads, 2>, a);
    case 3: return cudaLaunchKernelEx(&cfg, fp4_quantize_kernel<T, FMT, kQuantThreads, 3>, a);
    default: return cudaLaunchKernelEx(&cfg, fp4_quantize_kernel<T, FMT, kQuantThreads, 4>, a);
  }
}

template <typename T>
cudaError_t launch_typed(const QuantArgs& a, cudaStream_t s) {
  return a.out.format == GEMM_MXFP4 ? launch_format<T, GEMM_MXFP4>(a, s)
                                    : launch_format<T, GEMM_NVFP4>(a, s);
}

// ---------------------------------------------------------------- reading back --
// Bytes in 9/16, out 2 or 4 an element.  A thread writes an aligned 16 bytes of a row (8 or
// 4 neighbours, which may lie in two blocks where the row does not start on 16 bytes), so
// that a warp's stores are contiguous, for kBackRows rows at once, whose loads are in
// flight together.
constexpr int kBackRows = 4;

struct BackArgs {
  gemm_fp4_matrix_t m;
  int64_t rows, cols, ld, pieces;
  void* dst;
  int32_t tpr_log2;  // threads of a row
  int32_t chunks;    // CTAs along a row
};

// The largest e8m0 scales take values of 4 and 6 out of fp32, from where a row scale below 1
// may bring them back: 3 of the block scale's powers of two then go with the row scale,
// exactly, so that value times block scale stays exact.  FAR below: mxfp4 with a row scale
// (as a test of the pointer in the kernel it cost mxfp4 without one 1.4 of 39.3 us).
__device__ __forceinline__ void far_scale(float& block, float& row) {
  if (block >= 0x1p126f && fabsf(row) < 1.f) {
    block *= 0.125f;
    row *= 8.f;
  }
}

// ALIGNED: every row of dst starts on 16 bytes.  (8192^2 bf16 38 us, through the general
// way twice that; 1000 x 8191, which has to take it, 14, element by element 26.)
template <typename T, int FMT, bool ALIGNED, bool FAR>
__global__ void __launch_bounds__(kBackThreads) fp4_dequantize_kernel(const BackArgs a) {
  constexpr int kPer = 16 / sizeof(T);  // elements a thread
  const int tpr = 1 << a.tpr_log2, lanes = kBackThreads >> a.tpr_log2;
  const int64_t group = blockIdx.x / uint32_t(a.chunks);
  const int64_t place =
      int64_t(blockIdx.x - group * a.chunks) * tpr + (threadIdx.x & (tpr - 1));
  const int64_t r0 = group * (lanes * kBackRows) + (threadIdx.x >> a.tpr_log2);
  uint32_t q[kBackRows], s[kBackRows][2];
  float g[kBackRows];
  int64_t first[kBackRows];  // this thread's first element, below 0 where the row starts later
#pragma unroll
  for (int i = 0; i < kBackRows; ++i) {
    const int64_t r = r0 + i * lanes;
    q[i] = s[i][0] = s[i][1] = 0;
    g[i] = 1.f;
    first[i] = a.cols;
    if (r >= a.rows) continue;
    const uint32_t off =
        ALIGNED ? 0u
                : uint32_t(reinterpret_cast<uintptr_t>(static_cast<T*>(a.dst) + r * a.ld)) & 15u;
    const int64_t c = place * kPer - int64_t(off / sizeof(T));
    first[i] = c;
    if (c >= a.cols || c + kPer <= 0) continue;
    // the values from element c on, out of the two words that hold them
    const uint8_t* const row = static_cast<const uint8_t*>(a.m.data) + r * a.m.ld;
    if constexpr (ALIGNED) {
      const int64_t bytes = min(int64_t(kPer / 2), (a.cols - c + 1) / 2);
      if (bytes == kPer / 2) {
        if constexpr (kPer == 8) q[i] = __ldg(reinterpret_cast<const uint32_t*>(row + c / 2));
        else q[i] = __ldg(reinterpret_cast<const uint16_t*>(row + c / 2));
      } else {
        for (int j = 0; j < bytes; ++j) q[i] |= uint32_t(row[c / 2 + j]) << (8 * j);
      }
      s[i][0] = __ldg(static_cast<const uint8_t*>(a.m.scale) +
                      fp4_scale_at(r, c / fp4_block(FMT), a.pieces));
      if (a.m.row_scale) g[i] = __ldg(a.m.row_scale + r * a.m.row_scale_stride);
      continue;
    }
    const int64_t word = c >= 0 ? c >> 3 : -1, last = (a.cols - 1) >> 3;
    auto word_at = [&](int64_t k) -> uint32_t {
      if (k < 0 || k > last) return 0;
      const int64_t bytes = (a.cols + 1) / 2 - 4 * k;
      if (bytes >= 4) return __ldg(reinterpret_cast<const uint32_t*>(row) + k);
      uint32_t v = 0;
      for (int j = 0; j < bytes; ++j) v |= uint32_t(row[4 * k + j]) << (8 * j);
      return v;
    };
    const uint32_t shift = uint32_t(c & 7) * 4;
    const uint32_t lo = word_at(word);
    q[i] = lo;
    if (shift + 4 * kPer > 32) q[i] = __funnelshift_r(lo, word_at(word + 1), shift);
    else q[i] >>= shift;
    const int64_t b0 = (c > 0 ? c : 0) / fp4_block(FMT);
    const int64_t b1 = min(c + kPer, a.cols) - 1 >= 0 ? (min(c + kPer, a.cols) - 1) / fp4_block(FMT)
                                                      : 0;
    const uint8_t* const scale = static_cast<const uint8_t*>(a.m.scale);
    s[i][0] = __ldg(scale + fp4_scale_at(r, b0, a.pieces));
    s[i][1] = b1 == b0 ? s[i][0] : uint32_t(__ldg(scale + fp4_scale_at(r, b1, a.pieces)));
    if (a.m.row_scale) g[i] = __ldg(a.m.row_scale + r * a.m.row_scale_stride);
  }
#pragma unroll
  for (int i = 0; i < kBackRows; ++i) {
    const int64_t r = r0 + i * lanes, c = first[i];
    if (r >= a.rows || c >= a.cols || c + kPer <= 0) continue;
    float f0 = fp4_scale_value(s[i][0], FMT), g0 = g[i];
    float f1 = ALIGNED ? f0 : fp4_scale_value(s[i][1], FMT), g1 = g0;
    if constexpr (FAR) {
      far_scale(f0, g0);
      if constexpr (!ALIGNED) far_scale(f1, g1);
    }
    // how many of the elements lie in the first of the two blocks
    const int in0 = ALIGNED ? kPer
                            : int(fp4_block(FMT) - (c > 0 ? c : 0) % fp4_block(FMT)) +
                                  (c < 0 ? int(-c) : 0);
    T out[kPer];
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) {
      const float2 x = unpack_e2m1x2((q[i] >> (8 * j)) & 0xff);
      const bool a0 = ALIGNED || 2 * j < in0, a1 = ALIGNED || 2 * j + 1 < in0;
      const float v[2] = {__fmul_rn(x.x, a0 ? f0 : f1) * (a0 ? g0 : g1),
                          __fmul_rn(x.y, a1 ? f0 : f1) * (a1 ? g0 : g1)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (sizeof(T) == 4) out[2 * j + k] = v[k];
        else if constexpr (std::is_same<T, __half>::value) out[2 * j + k] = __float2half_rn(v[k]);
        else out[2 * j + k] = __float2bfloat16_rn(v[k]);
      }
    }
    T* const d = static_cast<T*>(a.dst) + r * a.ld + c;
    if ((ALIGNED || c >= 0) && c + kPer <= a.cols) {
      uint4 w;
      __builtin_memcpy(&w, out, 16);
      *reinterpret_cast<uint4*>(d) = w;
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (c + j >= 0 && c + j < a.cols) d[j] = out[j];
    }
  }
}

template <typename T>
cudaError_t launch_back(BackArgs a, cudaStream_t s) {
  constexpr int kPer = 16 / sizeof(T);
  const bool aligned = (reinterpret_cast<uintptr_t>(a.dst) & 15) == 0 &&
                       (a.rows == 1 || a.ld * int64_t(sizeof(T)) % 16 == 0);
  const int64_t places = (a.cols + kPer - 1) / kPer + (aligned ? 0 : 1);
  a.tpr_log2 = 5;
  while (a.tpr_log2 < 8 && (int64_t(1) << a.tpr_log2) < places) ++a.tpr_log2;
  const int64_t tpr = int64_t(1) << a.tpr_log2, rows = (kBackThreads / tpr) * kBackRows;
  const int64_t chunks = (places + tpr - 1) / tpr, groups = (a.rows + rows - 1) / rows;
  if (groups > INT32_MAX / chunks) return cudaErrorInvalidValue;
  a.chunks = int32_t(chunks);
  const unsigned grid = unsigned(groups * chunks);
  auto launch = [&](auto kern) {
    kern<<<grid, kBackThreads, 0, s>>>(a);
    return cudaGetLastError();
  };
  if (a.m.format == GEMM_MXFP4 && a.m.row_scale)
    return aligned ? launch(fp4_dequantize_kernel<T, GEMM_MXFP4, true, true>)
                   : launch(fp4_dequantize_kernel<T, GEMM_MXFP4, false, true>);
  if (a.m.format == GEMM_MXFP4)
    return aligned ? launch(fp4_dequantize_kernel<T, GEMM_MXFP4, true, false>)
                   : launch(fp4_dequantize_kernel<T, GEMM_MXFP4, false, false>);
  return aligned ? launch(fp4_dequantize_kernel<T, GEMM_NVFP4, true, false>)
                 : launch(fp4_dequantize_kernel<T, GEMM_NVFP4, false, false>);
}

int64_t pieces_of(int64_t cols, int format) {
  const int64_t per = 4 * fp4_block(format);
  return (cols + per - 1) / per;
}

}  // namespace

cudaError_t launch_fp4_quantize(int64_t rows, int64_t cols, const void* src, int64_t ld_src,
                                int src_dtype, const gemm_fp4_matrix_t& out, bool pdl,
                                cudaStream_t stream) {
  const int64_t size = src_dtype == GEMM_F32 ? 4 : 2;
  const uint8_t* const begin = static_cast<const uint8_t*>(src);
  const Span span{begin, begin + ((rows - 1) * ld_src + cols) * size};
  const QuantArgs a{src, rows, cols, ld_src, span, out, pieces_of(cols, out.format), pdl};
  if (src_dtype == GEMM_F32) return launch_typed<float>(a, stream);
  if (src_dtype == GEMM_F16) return launch_typed<__half>(a, stream);
  return launch_typed<__nv_bfloat16>(a, stream);
}

cudaError_t launch_fp4_dequantize(int64_t rows, int64_t cols, const gemm_fp4_matrix_t& m,
                                  void* dst, int64_t ld_dst, int dst_dtype, cudaStream_t stream) {
  const BackArgs a{m, rows, cols, ld_dst, pieces_of(cols, m.format), dst, 0, 0};
  if (dst_dtype == GEMM_F32) return launch_back<float>(a, stream);
  if (dst_dtype == GEMM_F16) return launch_back<__half>(a, stream);
  return launch_back<__nv_bfloat16>(a, stream);
}

}  // namespace dg

// fp4_row.cu: the 4-bit product of one row of A (a decode step of one token), without the
// tensor cores.
//
//   C[n] = ra rb[n] sum over blocks j of sa[j] sb[n, j] (sum over k in j of a[k] b[n, k])
//
// B is read once and an element of it used once, so that its bytes are the bound (9/16 of one
// an element, 17/32 in mxfp4) and, with a few MB of them, latency: launch, one trip to
// memory, the sums' way together.  A warp takes four rows of B, 32 apart, whose scales lie
// in the same 16 bytes, and 1024 neighbours of K at a time, 32 a lane: 16 bytes of each row.
// As many of a CTA's warps share its rows' K as keep all warps resident together, so that
// with a few MB each has one such piece and all loads are in flight at once.  What the first
// piece reads is sent for to L2 before the kernel ahead in the stream is done: that is no
// read, so that it may be B's writer.
//
// Values are widened to fp16 and multiplied there, two at a time: products of e2m1 numbers
// are multiples of 1/4 up to 36, so that the 8 that one half of a word sums are exact
// (288 in steps of 1/4, 1152 of the 2048 that fp16 holds).  The sum of a block of 16 is then
// exact in fp32, and its scale and the sum along K are applied there.
//
// Measured (graph replay, cold B, us, N x K, nvfp4 / mxfp4; in brackets on the tensor cores,
// fp4_tc_kernel.cuh): 4096 x 4096 3.7 / 3.7 (6.2 / 5.9), 1024 x 1024 2.2 / 2.3 (3.7 / 3.5), 1024 x
// 8192 3.2 / 3.2 (5.5 / 5.2), 8192 x 1024 3.3 / 3.3 (4.4 / 4.3), 8192 x 8192 9.9 / 9.8 (11.2 /
// 10.7), 4100 x 4100 5.1 / 5.2 (6.7 / 6.4); more, and where the tensor cores take over, in
// fp4_tc.cu.  An almost empty launch takes 1.8; over that, 4096 x 4096 moves 5.0 TB/s and 8192 x
// 8192 4.7.  The loads' latency bounds it: 32 warps an SM, each of which first loads and then
// computes, use 21 % of the issue slots and 17 % of DRAM's time at 4096 x 4096, 34 and 37 % at
// 8192 x 8192 (of a profiled launch with cold caches, 7.0 and 12.8 us).
// Dropped: the next piece's loads ahead of this one's sums, in more registers and
// so with fewer warps (4.5 and 10.7), nothing sent for ahead of the stream (4.5 and 10.3, both
// before the row's scales were read at the start), every next piece sent for to L2 too (3.8
// and 10.4), integer dot products of values taken from
// a table by byte permutes (5.0), two rows of A (5.2; 14.2 at 8192 x 8192, where the tensor
// cores take 11).
// A layer's row, quantised on the way: every CTA quantises all of it for itself, the steps of
// fp4_quant.cu, into shared memory, which spares a launch and its latency.  One launch / two
// (us, bf16 in and out, nvfp4, mxfp4): 4096 x 4096 4.5 / 5.3, 4.3 / 5.0, 1024 x 1024 2.9 / 4.1, 2.6 /
// 3.9, 8192 x 8192 12.1 / 12.8, 11.0 / 12.0, 1024 x 65536 27 / 29, 23 / 25, and 3.8 of the host's
// time instead of 6.5.  (Quantised by every warp in registers: they spill.)
#include "context.h"
#include "fp4_quant.cuh"
#include "ptx.cuh"

namespace dg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kWarpsPerSm = 32;  // resident: 4 CTAs of 64 registers a thread
constexpr int kRows = 4;         // of B, a warp's
constexpr int kLaneBytes = 16;   // of a row, 32 values
constexpr int kChunk = 32 * kLaneBytes;

struct RowArgs {
  gemm_fp4_matrix_t A, B;
  const float* bias;
  void* C;
  int64_t pieces;
  int32_t N, bytes;    // bytes of a row
  int32_t chunks;      // ceil(bytes / kChunk)
  int32_t split_log2;  // warps that share a row
  int32_t out_dtype;
  // or A as it is, quantised on the way (by every CTA for itself, into shared memory)
  const void* x;
  Span span;
  int32_t K;
};

// The eight values of a word as fp16 pairs, exactly.
__device__ __forceinline__ void widen(uint32_t w, __half2* h) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 p, q, s, t;\n\t"
      "mov.b32 {p, q, s, t}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, s;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, t;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) __builtin_memcpy(&h[i], &r[i], 4);
}

// 16 bytes of a row of `bytes` from byte c on, zeros past its end.
__device__ __forceinline__ uint4 load_row(const uint8_t* row, int c, int bytes) {
  if (c + kLaneBytes <= bytes) return __ldg(reinterpret_cast<const uint4*>(row + c));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < kLaneBytes; ++j)
    if (c + j < bytes) w[j / 4] |= uint32_t(row[c + j]) << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// x of `chunks` * 1024 elements, zeros from K on, to shared memory as the quantiser stores it
// (fp4_quant.cu): a unit's 8 bytes of values, 2 bytes of scales for each 32 elements.  By the
// whole CTA; returns the row's scale.
template <class X, int FMT>
__device__ __forceinline__ float quantize_row(const X* x, int K, int chunks, const Span& span,
                                              uint2* values, uint8_t* scales) {
  const int units = chunks * (2 * kChunk / kUnit);  // a multiple of 64
  Unit16<X> v;
  float m;
  bool odd;
  auto take = [&](int u) {
    v.load(x + u * kUnit, max(0, min(kUnit, K - u * kUnit)), span);
    m = v.amax(odd);
  };
  float a448 = 0.f, a2688 = 0.f, scale = 1.f;
  if constexpr (FMT == GEMM_NVFP4) {
    float most = 0.f;
    for (int u = threadIdx.x; u < units; u += kThreads) {
      take(u);
      most = fmaxf(most, m);
    }
    __shared__ uint32_t red[kWarps];
    const uint32_t all = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = all;
    __syncthreads();
    most = kAmaxMin;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) most = fmaxf(most, __uint_as_float(red[i]));
    a448 = __fdiv_rn(448.f, most);
    a2688 = __fdiv_rn(2688.f, most);
    scale = __fdiv_rn(most, 2688.f);
  }
  for (int u = threadIdx.x; u < units; u += kThreads) {
    if (FMT == GEMM_MXFP4 || units > kThreads) take(u);  // else it has its only one
    uint32_t byte;
    float f;
    if constexpr (FMT == GEMM_MXFP4) {  // the block's other half
      const float most = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      odd = __shfl_xor_sync(0xffffffffu, int(odd), 1) != 0 || odd;
      byte = uint32_t(max(int(__float_as_uint(most) >> 23) - 2, 0));
      f = __uint_as_float((254u - byte) << 23);
      if (odd) byte = 255;
    } else {
      byte = pack_e4m3x2(__fmul_rn(m, a448), 0.f) & 0xffu;
      const float s = unpack_e4m3x2(byte).x;
      f = s == 0.f ? 0.f : __fdiv_rn(a2688, s);
      if (odd) byte = 0x7f;
    }
    float q[kUnit];
#pragma unroll
    for (int j = 0; j < kUnit / 2; ++j) {
      const float2 y = mul2(v.pair(j), f);
      q[2 * j] = y.x;
      q[2 * j + 1] = y.y;
    }
    values[u] = odd ? make_uint2(0, 0) : make_uint2(pack_e2m1x8(q), pack_e2m1x8(q + 8));
    if (FMT == GEMM_NVFP4 || u % 2 == 0) scales[u] = uint8_t(byte);
  }
  __syncthreads();
  return scale;
}

// X: the type of A as it is, or void where it is in 4 bits.
template <int FMT, class X>
__global__ void __launch_bounds__(kThreads, kWarpsPerSm / kWarps)
    fp4_row_kernel(const RowArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = 1 << a.split_log2, places = kWarps >> a.split_log2;
  // this warp's rows are group * 128 + rr + 32 j of B, its part of K is warp / places
  const int place = int(blockIdx.x) * places + warp % places, rr = place & 31;
  const int64_t group = place >> 5, n0 = group * 128 + rr;
  const uint8_t* const row = static_cast<const uint8_t*>(a.B.data) + n0 * a.B.ld;
  pdl_launch_dependents();
  {
    const int c = warp / places * kChunk + lane * kLaneBytes;
    if (c < a.bytes && lane % 2 == 0) {  // 32 bytes each
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (n0 + 32 * j < a.N)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 32 * j * a.B.ld + c));
    }
  }
  pdl_wait_prerequisites();
  // the element that this thread writes, and its scales: the first places * kRows threads
  const int at = int(blockIdx.x) * places + int(threadIdx.x) / kRows;
  const int64_t n = int64_t(at >> 5) * 128 + (at & 31) + 32 * (threadIdx.x % kRows);
  const bool writes = int(threadIdx.x) < places * kRows && n < a.N;
  float ra = 1.f, rb = 1.f, bias = 0.f;
  if (writes) {
    if (std::is_void<X>::value && a.A.row_scale) ra = __ldg(a.A.row_scale);
    if (a.B.row_scale) rb = __ldg(a.B.row_scale + n * a.B.row_scale_stride);
    if (a.bias) bias = __ldg(a.bias + n);
  }
  extern __shared__ uint4 x_values[];
  const uint16_t* const x_scales = reinterpret_cast<const uint16_t*>(x_values + a.chunks * 32);
  if constexpr (!std::is_void<X>::value)
    ra = quantize_row<X, FMT>(static_cast<const X*>(a.x), a.K, a.chunks, a.span,
                              reinterpret_cast<uint2*>(x_values),
                              reinterpret_cast<uint8_t*>(x_values + a.chunks * 32));
  float acc[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) acc[j] = 0.f;
  if (n0 < a.N) {
    const uint8_t* const scale_b = static_cast<const uint8_t*>(a.B.scale) +
                                   group * a.pieces * kFp4Piece + rr * 16;
    constexpr int kPieceBytes = 2 * fp4_block(FMT);  // values of four blocks
    // of a lane's first block in the four
    const int shift = lane * kLaneBytes % kPieceBytes / kLaneBytes * (FMT == GEMM_MXFP4 ? 8 : 16);
    for (int ch = warp / places; ch < a.chunks; ch += splits) {
      const int c = ch * kChunk + lane * kLaneBytes;
      if (c >= a.bytes) continue;
      const int64_t piece = int64_t(c / kPieceBytes) * kFp4Piece;
      uint4 b[kRows];
      // rows past B's last are read as its row n0, and their sums dropped
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        b[j] = load_row(row + (n0 + 32 * j < a.N ? 32 * j : 0) * a.B.ld, c, a.bytes);
      const uint4 sb4 = __ldg(reinterpret_cast<const uint4*>(scale_b + piece));
      uint4 x;
      uint32_t sa;
      if constexpr (std::is_void<X>::value) {
        x = load_row(static_cast<const uint8_t*>(a.A.data), c, a.bytes);
        sa = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.A.scale) +
                                                     piece)) >> shift;
      } else {
        x = x_values[ch * 32 + lane];
        sa = x_scales[ch * 32 + lane];
      }
      const uint32_t sb[kRows] = {sb4.x >> shift, sb4.y >> shift, sb4.z >> shift, sb4.w >> shift};
      float sum[kRows][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // 16 values each
        __half2 xa[8];
        widen(i == 0 ? x.x : x.z, xa);
        widen(i == 0 ? x.y : x.w, xa + 4);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          __half2 xb[8];
          widen(i == 0 ? b[j].x : b[j].z, xb);
          widen(i == 0 ? b[j].y : b[j].w, xb + 4);
          __half2 s = __hmul2(xb[0], xa[0]);
#pragma unroll
          for (int k = 1; k < 8; ++k) s = __hfma2(xb[k], xa[k], s);
          const float2 t = __half22float2(s);
          sum[j][i] = t.x + t.y;
        }
      }
      if constexpr (FMT == GEMM_MXFP4) {
        // the two scales' product may lie outside fp32's range: A's first where it is below
        // 1, which is exact (a sum is a multiple of 1/4, and 2^-129 is above fp32's least
        // number), else B's
        const float fa = fp4_scale_value(sa & 0xff, FMT);
        const float first = fa < 1.f ? fa : 1.f, last = fa < 1.f ? 1.f : fa;
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          acc[j] = fmaf((sum[j][0] + sum[j][1]) * first * fp4_scale_value(sb[j] & 0xff, FMT), last,
                        acc[j]);
      } else {
        const float2 fa = unpack_e4m3x2(sa & 0xffff);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
          const float2 fb = unpack_e4m3x2(sb[j] & 0xffff);
          acc[j] = fmaf(sum[j][0], fa.x * fb.x, acc[j]);
          acc[j] = fmaf(sum[j][1], fa.y * fb.y, acc[j]);
        }
      }
    }
  }
  // over the lanes: two exchanges leave each with one row's sum
  const bool hi = lane & 16, odd = lane & 8;
  float u[2], v;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    u[i] = (hi ? acc[i + 2] : acc[i]) +
           __shfl_xor_sync(0xffffffffu, hi ? acc[i] : acc[i + 2], 16);
  v = (odd ? u[1] : u[0]) + __shfl_xor_sync(0xffffffffu, odd ? u[0] : u[1], 8);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  // and over the parts of K, in their order
  __shared__ float part[kWarps][kRows];
  if (lane % 8 == 0) part[warp][lane / 8] = v;
  __syncthreads();
  if (!writes) return;
  float s = 0.f;
  for (int k = 0; k < splits; ++k)
    s += part[k * places + int(threadIdx.x) / kRows][threadIdx.x % kRows];
  s = scale_fits(ra * rb) ? fmaf(s, ra * rb, bias) : add_scaled(bias, s, ra, rb);
  store_typed(a.C, n, s, a.out_dtype);
}

}  // namespace

cudaError_t launch_fp4_row(gemm_ctx* h, const Fp4Product& p, const void* x, int x_dtype,
                           cudaStream_t stream) {
  const int format = p.B.format;
  RowArgs a{};
  a.A = p.A;
  a.B = p.B;
  a.bias = p.bias;
  a.C = p.C;
  const int64_t per = 4 * fp4_block(format);
  a.pieces = (p.K + per - 1) / per;
  a.N = int32_t(p.N);
  a.bytes = int32_t((p.K + 1) / 2);
  a.chunks = (a.bytes + kChunk - 1) / kChunk;
  a.out_dtype = p.out_dtype;
  a.x = x;
  a.K = int32_t(p.K);
  const uint8_t* const begin = static_cast<const uint8_t*>(x);
  a.span = Span{begin, x ? begin + p.K * (x_dtype == GEMM_F32 ? 4 : 2) : begin};
  const int64_t places = (p.N + 127) / 128 * 32;  // of a warp's four rows
  while ((2 << a.split_log2) <= kWarps && (1 << a.split_log2) < a.chunks &&
         (places << (a.split_log2 + 1)) <= int64_t(h->num_sms) * kWarpsPerSm)
    ++a.split_log2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(places / (kWarps >> a.split_log2)), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = x ? unsigned(a.chunks) * 32 * (kLaneBytes + 2) : 0;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = h->opt.pdl != 0 ? 1 : 0;
  auto launch = [&](auto mx, auto nv) {
    return format == GEMM_MXFP4 ? cudaLaunchKernelEx(&cfg, mx, a) : cudaLaunchKernelEx(&cfg, nv, a);
  };
  if (!x) return launch(fp4_row_kernel<GEMM_MXFP4, void>, fp4_row_kernel<GEMM_NVFP4, void>);
  if (x_dtype == GEMM_F32)
    return launch(fp4_row_kernel<GEMM_MXFP4, float>, fp4_row_kernel<GEMM_NVFP4, float>);
  if (x_dtype == GEMM_F16)
    return launch(fp4_row_kernel<GEMM_MXFP4, __half>, fp4_row_kernel<GEMM_NVFP4, __half>);
  return launch(fp4_row_kernel<GEMM_MXFP4, __nv_bfloat16>,
                fp4_row_kernel<GEMM_NVFP4, __nv_bfloat16>);
}

}  // namespace dg

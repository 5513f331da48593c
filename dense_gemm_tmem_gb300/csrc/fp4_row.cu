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
// fp4_tc_kernel.cuh): 4096 x 4096 3.7 / 3.6 (6.4 / 6.1), 1024 x 1024 1.9 / 1.9 (3.7 / 3.5), 1024 x
// 8192 3.3 / 3.3 (5.6 / 5.4), 8192 x 1024 3.3 / 3.3 (4.4 / 4.3), 8192 x 8192 9.9 / 10.0 (10.8 /
// 10.5), 4100 x 4100 5.2 / 5.3 (6.7 / 6.4).  An almost empty launch takes 1.8; over that, 4096 x
// 4096 moves 5.0 TB/s and 8192 x 8192 4.7.  The loads' latency bounds it: 32 warps an SM, each
// of which first loads and then computes, fill half of the issue slots, and DRAM a third.
// Dropped: the next piece's loads ahead of this one's sums, in more registers and
// so with fewer warps (4.5 and 10.7), nothing sent for ahead of the stream (4.5 and 10.3, both
// before the row's scales were read at the start), every next piece sent for to L2 too (3.8
// and 10.4), integer dot products of values taken from
// a table by byte permutes (5.0), two rows of A (5.2; 14.2 at 8192 x 8192, where the tensor
// cores take 11).
#include "context.h"
#include "fp4.cuh"
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

template <int FMT>
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
    if (a.A.row_scale) ra = __ldg(a.A.row_scale);
    if (a.B.row_scale) rb = __ldg(a.B.row_scale + n * a.B.row_scale_stride);
    if (a.bias) bias = __ldg(a.bias + n);
  }
  float acc[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) acc[j] = 0.f;
  if (n0 < a.N) {
    const uint8_t* const data_a = static_cast<const uint8_t*>(a.A.data);
    const uint8_t* const scale_a = static_cast<const uint8_t*>(a.A.scale);
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
      const uint4 x = load_row(data_a, c, a.bytes);
      const uint32_t sa = __ldg(reinterpret_cast<const uint32_t*>(scale_a + piece)) >> shift;
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

cudaError_t launch_fp4_row(gemm_ctx* h, const Fp4Product& p, cudaStream_t stream) {
  RowArgs a{};
  a.A = p.A;
  a.B = p.B;
  a.bias = p.bias;
  a.C = p.C;
  const int64_t per = 4 * fp4_block(p.A.format);
  a.pieces = (p.K + per - 1) / per;
  a.N = int32_t(p.N);
  a.bytes = int32_t((p.K + 1) / 2);
  a.chunks = (a.bytes + kChunk - 1) / kChunk;
  a.out_dtype = p.out_dtype;
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
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = h->opt.pdl != 0 ? 1 : 0;
  return p.A.format == GEMM_MXFP4 ? cudaLaunchKernelEx(&cfg, fp4_row_kernel<GEMM_MXFP4>, a)
                                  : cudaLaunchKernelEx(&cfg, fp4_row_kernel<GEMM_NVFP4>, a);
}

}  // namespace dg

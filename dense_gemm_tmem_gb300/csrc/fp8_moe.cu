// fp8_moe.cu: the mixture-of-experts layer for a few tokens, on the CUDA cores.
//
// Four launches: router (logits, choice, gates, x quantised), gate and up
// products with silu, the quantised hidden values, down products with the
// weighted sum.  One warp per output row; every weight row is read once per
// token that chose its expert.
#include "fp8.cuh"

namespace dg {
namespace {

constexpr int kMoeThreads = 256;

__device__ __forceinline__ float load_x(const void* p, int64_t i, int dtype) {
  return dtype == GEMM_F16 ? __half2float(static_cast<const __half*>(p)[i])
                           : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Floats in a total order as integers: NaN above +inf, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct MoeArgs {
  gemm_moe_fp8_t L;
  uint8_t* xq;    // tokens x hidden
  float* xs;      // tokens x ceil(hidden / 128)
  float* h;       // picks x inner
  uint8_t* hq;
  float* hs;
};

// One block of 128 values of a row, quantised by one warp (4 per lane).
__device__ __forceinline__ void quant_block(const float (&v)[4], int lane, int64_t c0, int64_t cols,
                                            uint8_t* q, float* s) {
  float m = 0.f;
  float w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = fabsf(v[j]) == INFINITY ? NAN : v[j];
    m = fmaxf(m, fabsf(w[j]));
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float inv = fp8_inverse(m);
  const uint32_t pk = pack_e4m3x4(__fmul_rn(w[0], inv), __fmul_rn(w[1], inv),
                                  __fmul_rn(w[2], inv), __fmul_rn(w[3], inv));
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c0 + lane * 4 + j < cols) q[c0 + lane * 4 + j] = uint8_t(pk >> (8 * j));
  if (lane == 0) *s = fp8_scale(m);
}

__global__ void __launch_bounds__(kMoeThreads) moe_router_kernel(const MoeArgs a) {
  __shared__ float logit[GEMM_MOE_MAX_EXPERTS];
  __shared__ uint32_t key[GEMM_MOE_MAX_EXPERTS];
  __shared__ int chosen[GEMM_MOE_MAX_TOP_K];
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t H = a.L.hidden, kbs = (H + 127) / 128;
  for (int64_t kb = warp; kb < kbs; kb += kMoeThreads / 32) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = kb * 128 + lane * 4 + j;
      v[j] = c < H ? load_x(a.L.x, t * a.L.ld_x + c, a.L.dtype) : 0.f;
    }
    quant_block(v, lane, kb * 128, H, a.xq + t * H, a.xs + t * kbs + kb);
  }
  for (int64_t e = warp; e < a.L.experts; e += kMoeThreads / 32) {
    float s = 0.f;
    for (int64_t c = lane; c < H; c += 32)
      s = fmaf(load_x(a.L.x, t * a.L.ld_x + c, a.L.dtype),
               load_x(a.L.router, e * a.L.ld_router + c, a.L.dtype), s);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) {
      logit[e] = s;
      key[e] = order_key(s);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.L.experts; e += kMoeThreads) {
    int rank = 0;
    for (int j = 0; j < a.L.experts; ++j) rank += key[j] > key[e] || (key[j] == key[e] && j < e);
    if (rank < a.L.top_k) chosen[rank] = e;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const float top = logit[chosen[0]];
    float sum = 0.f;
    if (a.L.renormalize)
      for (int j = 0; j < a.L.top_k; ++j) sum += expf(logit[chosen[j]] - top);
    else
      for (int j = 0; j < a.L.experts; ++j) sum += expf(logit[j] - top);
    for (int j = 0; j < a.L.top_k; ++j) {
      a.L.ids[t * a.L.top_k + j] = chosen[j];
      a.L.gates[t * a.L.top_k + j] = expf(logit[chosen[j]] - top) / sum;
    }
  }
}

// One weight row times one quantised vector, by a warp.
__device__ __forceinline__ float row_dot(const gemm_fp8_experts_t& w, int64_t e, int64_t row,
                                         const uint8_t* q, const float* s, int64_t K, int lane) {
  const uint8_t* p = static_cast<const uint8_t*>(w.data) + e * w.expert_stride + row * w.ld;
  const float* ws = w.scale + e * w.scale_stride_e + (row >> 7) * w.scale_stride_r;
  float acc = 0.f;
  for (int64_t kb = 0; kb * 128 < K; ++kb) {
    float part = 0.f;
    for (int64_t k = kb * 128 + lane; k < min(K, kb * 128 + 128); k += 32)
      part = fmaf(unpack_e4m3x2(p[k]).x, unpack_e4m3x2(q[k]).x, part);
    acc = fmaf(part, ws[kb * w.scale_stride_c] * s[kb], acc);
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  return acc;
}

__global__ void __launch_bounds__(kMoeThreads) moe_gate_up_kernel(const MoeArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t i = int64_t(blockIdx.x) * (kMoeThreads / 32) + warp, pick = blockIdx.y;
  if (i >= a.L.inner) return;
  const int64_t t = pick / a.L.top_k, e = a.L.ids[pick], H = a.L.hidden;
  const uint8_t* q = a.xq + t * H;
  const float* s = a.xs + t * ((H + 127) / 128);
  const float g = row_dot(a.L.gate, e, i, q, s, H, lane);
  const float u = row_dot(a.L.up, e, i, q, s, H, lane);
  if (lane == 0) a.h[pick * a.L.inner + i] = g / (1.f + expf(-g)) * u;
}

__global__ void __launch_bounds__(kMoeThreads) moe_hidden_kernel(const MoeArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t I = a.L.inner, kbs = (I + 127) / 128, pick = blockIdx.x;
  for (int64_t kb = warp; kb < kbs; kb += kMoeThreads / 32) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = kb * 128 + lane * 4 + j;
      v[j] = c < I ? a.h[pick * I + c] : 0.f;
    }
    quant_block(v, lane, kb * 128, I, a.hq + pick * I, a.hs + pick * kbs + kb);
  }
}

__global__ void __launch_bounds__(kMoeThreads) moe_down_kernel(const MoeArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * (kMoeThreads / 32) + warp, t = blockIdx.y;
  if (r >= a.L.hidden) return;
  const int64_t I = a.L.inner;
  float acc = 0.f;
  for (int j = 0; j < a.L.top_k; ++j) {
    const int64_t pick = t * a.L.top_k + j;
    acc = fmaf(a.L.gates[pick], row_dot(a.L.down, a.L.ids[pick], r, a.hq + pick * I,
                                        a.hs + pick * ((I + 127) / 128), I, lane), acc);
  }
  if (lane == 0) store_typed(a.L.out, t * a.L.ld_out + r, acc, a.L.dtype);
}

int64_t up256(int64_t b) { return (b + 255) & ~int64_t(255); }

}  // namespace

int64_t moe_workspace_bytes(const gemm_moe_fp8_t& L) {
  const int64_t P = L.tokens * L.top_k;
  return up256(L.tokens * L.hidden) + up256(L.tokens * ((L.hidden + 127) / 128) * 4) +
         up256(P * L.inner * 4) + up256(P * L.inner) + up256(P * ((L.inner + 127) / 128) * 4);
}

cudaError_t launch_moe(const gemm_moe_fp8_t& L, void* workspace, cudaStream_t stream) {
  MoeArgs a{};
  a.L = L;
  const int64_t P = L.tokens * L.top_k;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.xq = w;
  w += up256(L.tokens * L.hidden);
  a.xs = reinterpret_cast<float*>(w);
  w += up256(L.tokens * ((L.hidden + 127) / 128) * 4);
  a.h = reinterpret_cast<float*>(w);
  w += up256(P * L.inner * 4);
  a.hq = w;
  w += up256(P * L.inner);
  a.hs = reinterpret_cast<float*>(w);
  const unsigned rows = kMoeThreads / 32;
  moe_router_kernel<<<unsigned(L.tokens), kMoeThreads, 0, stream>>>(a);
  moe_gate_up_kernel<<<dim3(unsigned((L.inner + rows - 1) / rows), unsigned(P)), kMoeThreads, 0,
                       stream>>>(a);
  moe_hidden_kernel<<<unsigned(P), kMoeThreads, 0, stream>>>(a);
  moe_down_kernel<<<dim3(unsigned((L.hidden + rows - 1) / rows), unsigned(L.tokens)), kMoeThreads,
                    0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace dg

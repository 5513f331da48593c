// ortho.cu: the orthogonalising call (include/gemm_ortho.h): argument checks, the
// scales of the 16-bit copies, the norm and the launches.
//
// Precision.  A product needs 16-bit operands to run on the tensor cores at their rate.
// They are fp16, not bfloat16, because everything in a step is bounded (singular values
// start below 1, the coefficients say how far they grow), so that a power of two per
// step keeps each copy in fp16's range and 11 bits of each number.  The iterate itself
// stays in fp32: small singular values grow by up to 3.4445^5 = 485 in five steps, and what
// rounding X adds to them would grow alike.  Simulated, error of the result relative to
// doubles, all in bfloat16 / all in fp16 / X in fp32: Gaussian matrix 1.1e-2 / 1.3e-3 / 1.5e-3,
// a gradient of 64 falling directions over noise 4.7e-2 / 6e-3 / 3e-4, of 16 over less noise
// 18e-2 / 2.2e-2 / 3e-4.
//
// The norm and the scaling read G twice and write 6 bytes an element.
#include <algorithm>
#include <cmath>

#include "context.h"
#include "ortho.cuh"

namespace dg {
namespace {

constexpr int kPrepThreads = 256;
constexpr int kNormParts = 1024;  // CTAs that sum one matrix, at most
constexpr int kUnit = 8;         // neighbours that a thread takes at a time

// Sums of squares as three numbers, so that no element's square leaves fp32's range
// (J. L. Blue, "A portable Fortran program to find the Euclidean norm of a vector",
// 1978): magnitudes above 2^40 are taken down by 2^96 first (squares up to 2^64, which
// any sum of 2^40 holds), those below 2^-50 up by 2^64.
struct Squares {
  float big = 0.f, mid = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float a = fabsf(x);
    if (a > 0x1p40f) {
      const float t = a * 0x1p-96f;
      big = fmaf(t, t, big);
    } else if (a < 0x1p-50f) {
      const float t = a * 0x1p64f;
      small = fmaf(t, t, small);
    } else {  // NaN too
      mid = fmaf(a, a, mid);
    }
  }
  // A unit at once where its largest magnitude is an ordinary one: what then underflows
  // is 2^-26 of its sum at most.
  __device__ __forceinline__ void add(const float (&x)[kUnit]) {
    float most = 0.f, sum = 0.f;
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      most = fmaxf(most, fabsf(x[j]));
      sum = fmaf(x[j], x[j], sum);
    }
    if (most <= 0x1p40f && most >= 0x1p-50f) {
      mid += sum;
    } else {
#pragma unroll
      for (int j = 0; j < kUnit; ++j) add(x[j]);
    }
  }
  // 1 / max(norm, eps) as two factors, since it may lie outside fp32's range.
  __device__ __forceinline__ void inverse(float eps, float& p1, float& p2) const {
    float m, down;  // norm = sqrt(m) / down
    if (big > 0.f || !(mid + small < INFINITY)) {
      m = big + mid * 0x1p-96f * 0x1p-96f;
      down = 0x1p-96f;
      if (!(mid + small < INFINITY)) m = NAN;
    } else if (mid > 0.f) {
      m = mid + small * 0x1p-64f * 0x1p-64f;
      down = 1.f;
    } else {
      m = small;
      down = 0x1p64f;
    }
    float root = sqrtf(m);
    if (root < eps * down) {
      root = eps;
      down = 1.f;
    }
    p1 = down;
    p2 = m < INFINITY ? __fdiv_rn(1.f, root) : NAN;
  }
};

struct PrepArgs {
  const void* g;
  int64_t rows, cols, ld_g, stride_g;
  int dtype;
  bool vec;      // 16-byte loads of g
  int32_t parts; // CTAs of the norm
  float* sums;   // batch x parts x 3
  float eps;
  float* x32;
  __half* x16;
  int64_t ld_x, stride_x;
  float scale;   // of the 16-bit copy
  uint32_t* done;  // the products' counters, set to 0
  int64_t counters;
};

// Elements c ... c + 7 of a row of g, zeros past its end.
__device__ __forceinline__ void load_unit(const PrepArgs& a, int64_t row_at, int32_t c,
                                          float (&x)[kUnit]) {
  const int64_t at = row_at + c;
  if (a.vec && c + kUnit <= a.cols) {
    if (a.dtype == GEMM_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.g) + at);
      const float4 u = __ldg(p), v = __ldg(p + 1);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
      x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
      const uint4 u =
          __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.g) + at));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if (a.dtype == GEMM_F16) {
          __half2 h;
          __builtin_memcpy(&h, &w[j], 4);
          f = __half22float2(h);
        } else {
          f = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
        }
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kUnit; ++j) {
    x[j] = 0.f;
    if (c + j >= a.cols) continue;
    if (a.dtype == GEMM_F32) x[j] = static_cast<const float*>(a.g)[at + j];
    else if (a.dtype == GEMM_F16) x[j] = __half2float(static_cast<const __half*>(a.g)[at + j]);
    else x[j] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.g)[at + j]);
  }
}

// Walks the units of a matrix, `step` threads apart, without a division a unit.
struct UnitWalk {
  int32_t r, c, dr, dc, per;  // row and unit, their steps, units a row
  __device__ __forceinline__ UnitWalk(int64_t start, int64_t step, int32_t per) : per(per) {
    r = int32_t(start / per);
    c = int32_t(start - int64_t(r) * per);
    dr = int32_t(step / per);
    dc = int32_t(step - int64_t(dr) * per);
  }
  __device__ __forceinline__ void next() {
    r += dr;
    c += dc;
    if (c >= per) {
      c -= per;
      ++r;
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The squares of a CTA's threads, added in a fixed order; every thread has the sum.
__device__ __forceinline__ Squares block_sum(Squares s) {
  constexpr int kWarps = kPrepThreads / 32;
  __shared__ float red[3][kWarps];
  s.big = warp_sum(s.big);
  s.mid = warp_sum(s.mid);
  s.small = warp_sum(s.small);
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = s.big;
    red[1][threadIdx.x >> 5] = s.mid;
    red[2][threadIdx.x >> 5] = s.small;
  }
  __syncthreads();
  s = Squares();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    s.big += red[0][w];
    s.mid += red[1][w];
    s.small += red[2][w];
  }
  return s;
}

__global__ void __launch_bounds__(kPrepThreads) ortho_norm_kernel(const PrepArgs a) {
  const int64_t z = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  Squares s;
  const int32_t per = int32_t((a.cols + kUnit - 1) / kUnit);
  UnitWalk u(int64_t(blockIdx.x) * kPrepThreads + threadIdx.x, int64_t(a.parts) * kPrepThreads,
             per);
#pragma unroll 4
  for (; u.r < a.rows; u.next()) {
    float x[kUnit];
    load_unit(a, z * a.stride_g + int64_t(u.r) * a.ld_g, u.c * kUnit, x);
    s.add(x);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) {
    float* p = a.sums + (z * a.parts + blockIdx.x) * 3;
    p[0] = s.big;
    p[1] = s.mid;
    p[2] = s.small;
  }
}

// X = G / max(norm, eps) and its 16-bit copy, with zeros up to the rows' padded ends.
__global__ void __launch_bounds__(kPrepThreads) ortho_scale_kernel(const PrepArgs a) {
  const int64_t z = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait_prerequisites();
  Squares s;
  for (int i = threadIdx.x; i < a.parts; i += kPrepThreads) {
    const float* p = a.sums + (z * a.parts + i) * 3;
    s.big += p[0];
    s.mid += p[1];
    s.small += p[2];
  }
  for (int64_t i = (z * gridDim.x + blockIdx.x) * kPrepThreads + threadIdx.x; i < a.counters;
       i += int64_t(gridDim.x) * gridDim.y * kPrepThreads)
    a.done[i] = 0;
  s = block_sum(s);
  float p1, p2;
  s.inverse(a.eps, p1, p2);
  UnitWalk u(int64_t(blockIdx.x) * kPrepThreads + threadIdx.x,
             int64_t(gridDim.x) * kPrepThreads, int32_t(a.ld_x / kUnit));
#pragma unroll 2
  for (; u.r < a.rows; u.next()) {
    float x[kUnit];
    load_unit(a, z * a.stride_g + int64_t(u.r) * a.ld_g, u.c * kUnit, x);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) x[j] = x[j] * p1 * p2;
    const int64_t at = z * a.stride_x + int64_t(u.r) * a.ld_x + u.c * kUnit;
    float4* to = reinterpret_cast<float4*>(a.x32 + at);
    to[0] = make_float4(x[0], x[1], x[2], x[3]);
    to[1] = make_float4(x[4], x[5], x[6], x[7]);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 h = __floats2half2_rn(x[2 * j] * a.scale, x[2 * j + 1] * a.scale);
      __builtin_memcpy(&w[j], &h, 4);
    }
    *reinterpret_cast<uint4*>(a.x16 + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

cudaError_t launch_prep(void (*kern)(PrepArgs), const PrepArgs& a, unsigned ctas, int64_t batch,
                        bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(ctas, unsigned(batch), 1);
  cfg.blockDim = dim3(kPrepThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1u : 0u;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

OrthoShape shape_of(const gemm_orthogonalize_t& p) {
  OrthoShape s{};
  s.batch = p.batch;
  s.rows = p.rows;
  s.cols = p.cols;
  s.n = std::min(p.rows, p.cols);
  s.tall = p.rows > p.cols;
  s.ld_x = round_up(p.cols, 64);
  s.ld_a = round_up(s.n, 64);
  s.stride_x = s.rows * s.ld_x;
  s.stride_a = s.n * s.ld_a;
  return s;
}

// Workspace: the norm's parts, the products' counters, the iterate in fp32, two 16-bit copies of it, A and B.
struct Space {
  int64_t parts, done, x32, x16, a16, b16, total;
};
Space space_of(const OrthoShape& s, int32_t steps) {
  Space w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  w.parts = take(s.batch * kNormParts * 3 * 4);
  w.done = take(ortho_counters(s, steps) * 4);
  w.x32 = take(s.batch * s.stride_x * 4);
  w.x16 = take(2 * round_up(s.batch * s.stride_x * 2, 256));
  w.a16 = take(s.batch * s.stride_a * 2);
  w.b16 = take(s.batch * s.stride_a * 2);
  w.total = at;
  return w;
}

// Largest |c1 t + c2 t^2| on [0, m].
double most_quadratic(double c1, double c2, double m) {
  double most = std::fabs(m * (c1 + c2 * m));
  const double t = c2 != 0 ? -c1 / (2 * c2) : -1;
  if (t > 0 && t < m) most = std::max(most, std::fabs(t * (c1 + c2 * t)));
  return most;
}
// Largest |s (a + b s^2 + c s^4)| on [0, m]: at m or where the derivative
// a + 3 b y + 5 c y^2 vanishes, y = s^2.
double most_quintic(double a, double b, double c, double m) {
  auto at = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
  double most = at(m);
  auto try_y = [&](double y) {
    if (y > 0 && y < m * m) most = std::max(most, at(std::sqrt(y)));
  };
  if (c == 0) {
    if (b != 0) try_y(-a / (3 * b));
  } else {
    const double d = 9 * b * b - 20 * a * c;
    if (d >= 0) {
      try_y((-3 * b + std::sqrt(d)) / (10 * c));
      try_y((-3 * b - std::sqrt(d)) / (10 * c));
    }
  }
  return most;
}

// The power of two that takes magnitudes up to `most` to at most 2^14: fp16 goes to
// 65504, and what rounding adds to a bound is far less than the factor of 4 left.
int scale_for(double most) {
  if (!(most > 0)) return 0;
  int e;
  std::frexp(most, &e);  // most <= 2^e
  return std::min(14 - e, 100);
}

struct Plan {
  int x[GEMM_ORTHO_MAX_STEPS], a[GEMM_ORTHO_MAX_STEPS], b[GEMM_ORTHO_MAX_STEPS];
};

// Exponents of the 16-bit copies from bounds on the singular values before each step.
int plan_scales(const gemm_orthogonalize_t& p, Plan* plan) {
  double u = 1.0;  // the Frobenius norm bounds them
  for (int i = 0; i < p.steps; ++i) {
    const double a = p.coefficients[3 * i], b = p.coefficients[3 * i + 1],
                 c = p.coefficients[3 * i + 2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return GEMM_ERR_INVALID_ARG;
    const double most_b = most_quadratic(b, c, u * u);
    plan->x[i] = scale_for(u);
    plan->a[i] = scale_for(u * u);
    plan->b[i] = scale_for(most_b);
    u = most_quintic(a, b, c, u);
    if (!(u <= 1e4) || !(most_b <= 1e8)) return GEMM_ERR_INVALID_ARG;
    // below, the factors between the copies' scales would leave fp32's range
    if (i + 1 < p.steps && u > 0 && u < 0x1p-20) return GEMM_ERR_INVALID_ARG;
  }
  return GEMM_OK;
}

int check_sizes(const gemm_orthogonalize_t* p) {
  if (!p || p->batch < 0 || p->rows < 0 || p->cols < 0 || p->steps < 1 ||
      p->steps > GEMM_ORTHO_MAX_STEPS)
    return GEMM_ERR_INVALID_ARG;
  if (p->rows >= (1 << 20) || p->cols >= (1 << 20) || p->batch >= (1 << 16))
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

cudaError_t enqueue(gemm_ctx* h, const gemm_orthogonalize_t& p, const Plan& plan, uint8_t* w,
                    cudaStream_t stream) {
  const OrthoShape s = shape_of(p);
  const Space at = space_of(s, p.steps);
  float* x32 = reinterpret_cast<float*>(w + at.x32);
  __half* x16[2] = {reinterpret_cast<__half*>(w + at.x16),
                    reinterpret_cast<__half*>(w + at.x16 +
                                              round_up(s.batch * s.stride_x * 2, 256))};
  auto two = [](int e) { return std::ldexp(1.f, e); };
  PrepArgs prep{};
  prep.g = p.g;
  prep.rows = s.rows;
  prep.cols = s.cols;
  prep.ld_g = p.ld_g;
  prep.stride_g = p.stride_g;
  prep.dtype = p.dtype;
  const int64_t size = p.dtype == GEMM_F32 ? 4 : 2;
  prep.vec = (reinterpret_cast<uintptr_t>(p.g) & 15) == 0 &&
             (s.rows == 1 || p.ld_g * size % 16 == 0) &&
             (s.batch == 1 || p.stride_g * size % 16 == 0);
  // the CTAs that are resident together share the batch; 2 units a thread at least
  const int64_t units = s.rows * (s.ld_x / kUnit);
  const int64_t ctas = std::max<int64_t>(
      1, std::min((units + 2 * kPrepThreads - 1) / (2 * kPrepThreads),
                  (int64_t(h->num_sms) * 6 + s.batch - 1) / s.batch));
  prep.parts = int32_t(std::min<int64_t>(ctas, kNormParts));
  prep.sums = reinterpret_cast<float*>(w + at.parts);
  prep.eps = float(p.eps);
  prep.x32 = x32;
  prep.x16 = x16[0];
  prep.ld_x = s.ld_x;
  prep.stride_x = s.stride_x;
  prep.scale = two(plan.x[0]);
  prep.done = reinterpret_cast<uint32_t*>(w + at.done);
  prep.counters = ortho_counters(s, p.steps);
  const bool pdl = h->opt.pdl != 0;
  cudaError_t e =
      launch_prep(ortho_norm_kernel, prep, unsigned(prep.parts), s.batch, pdl, stream);
  if (e == cudaSuccess)
    e = launch_prep(ortho_scale_kernel, prep, unsigned(ctas), s.batch, pdl, stream);
  if (e != cudaSuccess) return e;
  OrthoCall c{};
  c.shape = s;
  c.steps = p.steps;
  for (int i = 0; i < p.steps; ++i) {
    OrthoStep& q = c.step[i];
    q.gram_alpha = two(plan.a[i] - 2 * plan.x[i]);
    q.poly_alpha = std::ldexp(p.coefficients[3 * i + 2], plan.b[i] - 2 * plan.a[i]);
    q.poly_beta = std::ldexp(p.coefficients[3 * i + 1], plan.b[i] - plan.a[i]);
    q.apply_alpha = two(-plan.b[i] - plan.x[i]);
    q.apply_beta = p.coefficients[3 * i];
    q.scale = i + 1 < p.steps ? two(plan.x[i + 1]) : 0.f;
  }
  c.x32 = x32;
  c.x16[0] = x16[0];
  c.x16[1] = x16[1];
  c.a16 = reinterpret_cast<__half*>(w + at.a16);
  c.b16 = reinterpret_cast<__half*>(w + at.b16);
  c.done = prep.done;
  c.out = p.out;
  c.ld_out = p.ld_out;
  c.stride_out = p.stride_out;
  return launch_ortho_products(h, c, stream);
}

}  // namespace
}  // namespace dg

extern "C" {

int gemm_orthogonalize_workspace(gemm_handle_t h, const gemm_orthogonalize_t* p, int64_t* bytes) {
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (!h) return GEMM_ERR_INVALID_ARG;
  const int rc = dg::check_sizes(p);
  if (rc != GEMM_OK) return rc;
  *bytes = dg::space_of(dg::shape_of(*p), p->steps).total;
  return GEMM_OK;
}

int gemm_orthogonalize(gemm_handle_t h, const gemm_orthogonalize_t* p, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  if (!h) return GEMM_ERR_INVALID_ARG;
  int rc = dg::check_sizes(p);
  if (rc != GEMM_OK) return rc;
  if ((p->dtype != GEMM_F16 && p->dtype != GEMM_BF16 && p->dtype != GEMM_F32) ||
      !p->coefficients || !(p->eps >= 0x1p-100 && p->eps <= 0x1p100) || p->ld_g < p->cols ||
      p->ld_out < p->cols)
    return GEMM_ERR_INVALID_ARG;
  if (p->batch > 1 && (p->stride_g < 0 || p->stride_out < p->rows * p->ld_out - (p->ld_out - p->cols)))
    return GEMM_ERR_INVALID_ARG;
  dg::Plan plan;
  if ((rc = dg::plan_scales(*p, &plan)) != GEMM_OK) return rc;
  if (p->batch == 0 || p->rows == 0 || p->cols == 0) return GEMM_OK;
  if ((reinterpret_cast<uintptr_t>(p->g) % (p->dtype == GEMM_F32 ? 4 : 2)) != 0 ||
      reinterpret_cast<uintptr_t>(p->out) % 2 != 0)
    return GEMM_ERR_UNSUPPORTED;
  if (!p->g || !p->out || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      workspace_bytes < dg::space_of(dg::shape_of(*p), p->steps).total)
    return GEMM_ERR_INVALID_ARG;
  return dg::on_device(h->device, [&]() -> int {
    return dg::enqueue(h, *p, plan, static_cast<uint8_t*>(workspace),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
  });
}

}  // extern "C"

// ortho.cu: the orthogonalising call (include/gemm_ortho.h): argument checks, the
// scales of the 16-bit copies, the norm and the sequence of launches.
#include <algorithm>
#include <cmath>

#include "context.h"
#include "ortho.cuh"

namespace dg {
namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 128;  // CTAs that sum one matrix

// Sums of squares as three numbers, so that no element's square leaves fp32's range
// (J. L. Blue, "A portable Fortran program to find the Euclidean norm of a vector",
// 1978): magnitudes above 2^50 are taken down by 2^96 first (squares up to 2^64, which any sum of
// 2^40 holds), those below 2^-50 up by 2^64.
struct Squares {
  float big = 0.f, mid = 0.f, small = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float a = fabsf(x);
    if (a > 0x1p50f) {
      const float t = a * 0x1p-96f;
      big = fmaf(t, t, big);
    } else if (a < 0x1p-50f) {
      const float t = a * 0x1p64f;
      small = fmaf(t, t, small);
    } else {  // NaN too
      mid = fmaf(a, a, mid);
    }
  }
  __device__ __forceinline__ double norm() const {
    return sqrt(double(big) * 0x1p192 + double(mid) + double(small) * 0x1p-128);
  }
};

__device__ __forceinline__ float load_typed(const void* p, int64_t i, int dtype) {
  if (dtype == GEMM_F32) return static_cast<const float*>(p)[i];
  if (dtype == GEMM_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float red[kNormThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < kNormThreads / 32; ++w) v += red[w];
  __syncthreads();
  return v;
}

struct PrepArgs {
  const void* g;
  int64_t rows, cols, ld_g, stride_g;
  int dtype;
  float* parts;  // batch x kNormParts x 3
  double eps;
  float* x32;
  __half* x16;
  int64_t ld_x, stride_x;
  float scale;   // of the 16-bit copy
};

__global__ void __launch_bounds__(kNormThreads) ortho_norm_kernel(const PrepArgs a) {
  const int64_t z = blockIdx.y, n = a.rows * a.cols;
  Squares s;
  for (int64_t i = int64_t(blockIdx.x) * kNormThreads + threadIdx.x; i < n;
       i += int64_t(kNormParts) * kNormThreads) {
    const int64_t r = i / a.cols, c = i - r * a.cols;
    s.add(load_typed(a.g, z * a.stride_g + r * a.ld_g + c, a.dtype));
  }
  const float big = block_sum(s.big), mid = block_sum(s.mid), small = block_sum(s.small);
  if (threadIdx.x == 0) {
    float* p = a.parts + (z * kNormParts + blockIdx.x) * 3;
    p[0] = big;
    p[1] = mid;
    p[2] = small;
  }
}

// X = G / max(norm, eps) and its 16-bit copy.
__global__ void __launch_bounds__(kNormThreads) ortho_scale_kernel(const PrepArgs a) {
  const int64_t z = blockIdx.y;
  Squares s;
  if (threadIdx.x < kNormParts) {
    const float* p = a.parts + (z * kNormParts + threadIdx.x) * 3;
    s.big = p[0];
    s.mid = p[1];
    s.small = p[2];
  }
  s.big = block_sum(s.big);
  s.mid = block_sum(s.mid);
  s.small = block_sum(s.small);
  const double norm = s.norm();
  const double inv = 1.0 / fmax(norm, a.eps);
  // 1 / norm may lie outside fp32's range: a factor in [1, 2) and two powers of two
  const bool fine = norm < INFINITY;
  const int e = fine ? ilogb(inv) : 0;
  const float p1 = fine ? float(scalbn(1.0, e / 2)) : NAN;
  const float p2 = fine ? float(scalbn(inv, -e) * scalbn(1.0, e - e / 2)) : NAN;
  for (int64_t i = int64_t(blockIdx.x) * kNormThreads + threadIdx.x; i < a.stride_x;
       i += int64_t(gridDim.x) * kNormThreads) {
    const int64_t r = i / a.ld_x, c = i - r * a.ld_x;
    const float x =
        c < a.cols ? load_typed(a.g, z * a.stride_g + r * a.ld_g + c, a.dtype) * p1 * p2 : 0.f;
    a.x32[z * a.stride_x + i] = x;
    a.x16[z * a.stride_x + i] = __float2half_rn(x * a.scale);
  }
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

// Workspace: the norm's parts, the iterate in fp32, two 16-bit copies of it, A and B.
struct Space {
  int64_t parts, x32, x16, a16, b16, total;
};
Space space_of(const OrthoShape& s) {
  Space w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  w.parts = take(s.batch * kNormParts * 3 * 4);
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
  return std::min(14 - e, 40);
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
  const Space at = space_of(s);
  float* x32 = reinterpret_cast<float*>(w + at.x32);
  __half* x16[2] = {reinterpret_cast<__half*>(w + at.x16),
                    reinterpret_cast<__half*>(w + at.x16 +
                                              round_up(s.batch * s.stride_x * 2, 256))};
  __half* a16 = reinterpret_cast<__half*>(w + at.a16);
  __half* b16 = reinterpret_cast<__half*>(w + at.b16);
  auto two = [](int e) { return std::ldexp(1.f, e); };
  const PrepArgs prep{p.g,    s.rows, s.cols,  p.ld_g, p.stride_g,
                      p.dtype, reinterpret_cast<float*>(w + at.parts), p.eps, x32,
                      x16[0], s.ld_x, s.stride_x, two(plan.x[0])};
  ortho_norm_kernel<<<dim3(kNormParts, unsigned(s.batch)), kNormThreads, 0, stream>>>(prep);
  const int64_t per = (s.rows * s.cols + kNormThreads - 1) / kNormThreads;
  ortho_scale_kernel<<<dim3(unsigned(std::min<int64_t>(per, 1024)), unsigned(s.batch)),
                       kNormThreads, 0, stream>>>(prep);
  cudaError_t e = cudaGetLastError();
  for (int i = 0; i < p.steps && e == cudaSuccess; ++i) {
    const float a = p.coefficients[3 * i], b = p.coefficients[3 * i + 1],
                c = p.coefficients[3 * i + 2];
    const bool last = i + 1 == p.steps;
    OrthoProduct q{};
    q.kind = kGram;
    q.alpha = two(plan.a[i] - 2 * plan.x[i]);
    q.a = x16[i & 1];
    q.c = a16;
    e = launch_ortho_product(h, s, q, stream);
    if (e != cudaSuccess) break;
    q = {};
    q.kind = kPoly;
    q.alpha = std::ldexp(c, plan.b[i] - 2 * plan.a[i]);
    q.beta = std::ldexp(b, plan.b[i] - plan.a[i]);
    q.a = a16;
    q.c = b16;
    e = launch_ortho_product(h, s, q, stream);
    if (e != cudaSuccess) break;
    q = {};
    q.kind = kApply;
    q.alpha = two(-plan.b[i] - plan.x[i]);
    q.beta = a;
    q.a = b16;
    q.x = x16[i & 1];
    q.x32 = x32;
    if (last) {
      q.out = p.out;
      q.ld_out = p.ld_out;
      q.stride_out = p.stride_out;
    } else {
      q.scale = two(plan.x[i + 1]);
      q.c = x16[(i + 1) & 1];
    }
    e = launch_ortho_product(h, s, q, stream);
  }
  return e;
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
  *bytes = dg::space_of(dg::shape_of(*p)).total;
  return GEMM_OK;
}

int gemm_orthogonalize(gemm_handle_t h, const gemm_orthogonalize_t* p, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  if (!h) return GEMM_ERR_INVALID_ARG;
  int rc = dg::check_sizes(p);
  if (rc != GEMM_OK) return rc;
  if ((p->dtype != GEMM_F16 && p->dtype != GEMM_BF16 && p->dtype != GEMM_F32) ||
      !p->coefficients || !(p->eps >= 0x1p-100) || !std::isfinite(p->eps) || p->ld_g < p->cols ||
      p->ld_out < p->cols)
    return GEMM_ERR_INVALID_ARG;
  if (p->batch > 1 && (p->stride_g < 0 || p->stride_out < p->rows * p->ld_out - (p->ld_out - p->cols)))
    return GEMM_ERR_INVALID_ARG;
  dg::Plan plan;
  if ((rc = dg::plan_scales(*p, &plan)) != GEMM_OK) return rc;
  if (p->batch == 0 || p->rows == 0 || p->cols == 0) return GEMM_OK;
  if (!p->g || !p->out || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      workspace_bytes < dg::space_of(dg::shape_of(*p)).total)
    return GEMM_ERR_INVALID_ARG;
  return dg::on_device(h->device, [&]() -> int {
    return dg::enqueue(h, *p, plan, static_cast<uint8_t*>(workspace),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
  });
}

}  // extern "C"

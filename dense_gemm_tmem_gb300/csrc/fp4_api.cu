// fp4_api.cu: the C-ABI of include/gemm_fp4.h: argument checks and dispatch.
#include "context.h"
#include "fp4.cuh"

namespace dg {
namespace {

bool bad_type(int t) { return t != GEMM_F16 && t != GEMM_F32 && t != GEMM_BF16; }
bool bad_format(int f) { return f != GEMM_MXFP4 && f != GEMM_NVFP4; }

int check_matrix(const gemm_fp4_matrix_t* m, int64_t rows, int64_t cols) {
  if (!m || bad_format(m->format) || m->ld < (cols + 1) / 2) return GEMM_ERR_INVALID_ARG;
  if (rows > 0 && cols > 0 && (!m->data || !m->scale)) return GEMM_ERR_INVALID_ARG;
  if (rows >= kMaxCoord || cols >= kMaxCoord || m->ld >= (int64_t(1) << 40) || m->ld % 16 != 0 ||
      ((reinterpret_cast<uintptr_t>(m->data) | reinterpret_cast<uintptr_t>(m->scale)) & 15) ||
      reinterpret_cast<uintptr_t>(m->row_scale) % 4 != 0)
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

// Elements of `type` that do not start on a multiple of their size, which no load or store
// may touch.
bool misaligned(const void* p, int type) {
  return reinterpret_cast<uintptr_t>(p) % (type == GEMM_F32 ? 4 : 2) != 0;
}

int done(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA; }

}  // namespace
}  // namespace dg

extern "C" {

int64_t gemm_fp4_scale_bytes(int64_t rows, int64_t cols, int format) {
  if (rows < 0 || cols < 0 || rows >= dg::kMaxCoord || cols >= dg::kMaxCoord ||
      dg::bad_format(format))
    return GEMM_ERR_INVALID_ARG;
  const int64_t per = 4 * dg::fp4_block(format);
  return (rows + 127) / 128 * ((cols + per - 1) / per) * dg::kFp4Piece;
}

int gemm_fp4_quantize(gemm_handle_t h, int64_t rows, int64_t cols, const void* src,
                      int64_t ld_src, int src_dtype, const gemm_fp4_matrix_t* out, void* stream) {
  if (!h || rows < 0 || cols < 0 || ld_src < cols || dg::bad_type(src_dtype))
    return GEMM_ERR_INVALID_ARG;
  const int rc = dg::check_matrix(out, rows, cols);
  if (rc != GEMM_OK) return rc;
  if ((out->format == GEMM_MXFP4) != (out->row_scale == nullptr) && rows > 0 && cols > 0)
    return GEMM_ERR_INVALID_ARG;
  if (out->format == GEMM_NVFP4 && rows > 1 && out->row_scale_stride == 0)
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!src) return GEMM_ERR_INVALID_ARG;
  if (dg::misaligned(src, src_dtype)) return GEMM_ERR_UNSUPPORTED;
  return dg::on_device(h->device, [&]() -> int {
    return dg::done(dg::launch_fp4_quantize(rows, cols, src, ld_src, src_dtype, *out,
                                            h->opt.pdl != 0, static_cast<cudaStream_t>(stream)));
  });
}

int gemm_fp4_dequantize(gemm_handle_t h, int64_t rows, int64_t cols, const gemm_fp4_matrix_t* m,
                        void* dst, int64_t ld_dst, int dst_dtype, void* stream) {
  if (!h || rows < 0 || cols < 0 || ld_dst < cols || dg::bad_type(dst_dtype))
    return GEMM_ERR_INVALID_ARG;
  const int rc = dg::check_matrix(m, rows, cols);
  if (rc != GEMM_OK) return rc;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!dst) return GEMM_ERR_INVALID_ARG;
  if (dg::misaligned(dst, dst_dtype)) return GEMM_ERR_UNSUPPORTED;
  return dg::on_device(h->device, [&]() -> int {
    return dg::done(dg::launch_fp4_dequantize(rows, cols, *m, dst, ld_dst, dst_dtype,
                                              static_cast<cudaStream_t>(stream)));
  });
}

int gemm_fp4_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const gemm_fp4_matrix_t* A,
                 const gemm_fp4_matrix_t* B, const float* bias, void* C, int64_t ldc,
                 int out_dtype, void* stream) {
  if (!h || M < 0 || N < 0 || K < 0 || ldc < N || dg::bad_type(out_dtype))
    return GEMM_ERR_INVALID_ARG;
  int rc = dg::check_matrix(A, M, K);
  if (rc != GEMM_OK) return rc;
  rc = dg::check_matrix(B, N, K);
  if (rc != GEMM_OK) return rc;
  if (A->format != B->format) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  if (!C) return GEMM_ERR_INVALID_ARG;
  if (dg::misaligned(C, out_dtype) || dg::misaligned(bias, GEMM_F32)) return GEMM_ERR_UNSUPPORTED;
  const dg::Fp4Product p{M, N, K, *A, *B, bias, C, ldc, out_dtype};
  return dg::on_device(h->device, [&]() -> int {
    return dg::done(dg::launch_fp4(h, p, static_cast<cudaStream_t>(stream)));
  });
}

int gemm_fp4_one_row(gemm_handle_t h, int64_t N, int64_t K) {
  return h && N >= 0 && K >= 0 && dg::fp4_one_row(h, N);
}

int gemm_fp4_linear_row(gemm_handle_t h, int64_t N, int64_t K, const void* x, int x_dtype,
                        const gemm_fp4_matrix_t* W, const float* bias, void* y, int y_dtype,
                        void* stream) {
  if (!h || N < 0 || K < 0 || dg::bad_type(x_dtype) || dg::bad_type(y_dtype))
    return GEMM_ERR_INVALID_ARG;
  const int rc = dg::check_matrix(W, N, K);
  if (rc != GEMM_OK) return rc;
  if (N == 0) return GEMM_OK;
  if (!y || (K > 0 && !x)) return GEMM_ERR_INVALID_ARG;
  if (K > GEMM_FP4_ROW_MOST || dg::misaligned(x, x_dtype) || dg::misaligned(y, y_dtype) ||
      dg::misaligned(bias, GEMM_F32))
    return GEMM_ERR_UNSUPPORTED;
  const dg::Fp4Product p{1, N, K, *W, *W, bias, y, N, y_dtype};
  return dg::on_device(h->device, [&]() -> int {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return dg::done(K == 0 ? dg::launch_fp4(h, p, s) : dg::launch_fp4_row(h, p, x, x_dtype, s));
  });
}

}  // extern "C"

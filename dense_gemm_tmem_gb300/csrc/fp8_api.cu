// fp8_api.cu: the C-ABI of include/gemm_fp8.h: argument checks and dispatch.
#include "context.h"
#include "fp8.cuh"

namespace dg {
namespace {

bool bad_blocks(int32_t b) { return b < GEMM_FP8_ROW || b > GEMM_FP8_TILE; }
bool bad_type(int t) { return t != GEMM_F16 && t != GEMM_F32 && t != GEMM_BF16; }

// The operand's view as rows by K, or an error.  `mn` by `K` elements, stored
// with K along the rows (k_rows) or down the columns.
int operand_view(const gemm_fp8_matrix_t* m, int64_t mn, int64_t K, bool k_rows, Fp8Operand* o) {
  if (!m || bad_blocks(m->blocks)) return GEMM_ERR_INVALID_ARG;
  if (m->blocks == (k_rows ? GEMM_FP8_COL : GEMM_FP8_ROW)) return GEMM_ERR_INVALID_ARG;
  if (m->ld < (k_rows ? K : mn)) return GEMM_ERR_INVALID_ARG;
  if (mn > 0 && K > 0 && (!m->data || !m->scale)) return GEMM_ERR_INVALID_ARG;
  o->data = static_cast<const uint8_t*>(m->data);
  o->s_mn = k_rows ? m->ld : 1;
  o->s_k = k_rows ? 1 : m->ld;
  o->scale = m->scale;
  o->c_mn = k_rows ? m->scale_stride_r : m->scale_stride_c;
  o->c_kb = k_rows ? m->scale_stride_c : m->scale_stride_r;
  o->mn_shift = m->blocks == GEMM_FP8_TILE ? 7 : 0;
  return GEMM_OK;
}

int check_moe_sizes(const gemm_moe_fp8_t* L) {
  if (!L) return GEMM_ERR_INVALID_ARG;
  if (L->tokens < 0 || L->hidden <= 0 || L->inner <= 0 || L->experts <= 0 || L->top_k < 1 ||
      L->top_k > L->experts || (L->dtype != GEMM_F16 && L->dtype != GEMM_BF16))
    return GEMM_ERR_INVALID_ARG;
  if (L->tokens > GEMM_MOE_MAX_TOKENS || L->experts > GEMM_MOE_MAX_EXPERTS ||
      L->top_k > GEMM_MOE_MAX_TOP_K || L->hidden >= (1 << 20) || L->inner >= (1 << 20))
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

int check_experts(const gemm_fp8_experts_t& w, int64_t rows, int64_t cols, int64_t experts) {
  if (!w.data || !w.scale || w.ld < cols) return GEMM_ERR_INVALID_ARG;
  if (experts > 1 && w.expert_stride < rows * w.ld - (w.ld - cols)) return GEMM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(w.data) & 15) || w.ld % 16 != 0 ||
      (experts > 1 && w.expert_stride % 16 != 0))
    return GEMM_ERR_UNSUPPORTED;
  return GEMM_OK;
}

}  // namespace
}  // namespace dg

extern "C" {

int gemm_fp8_quantize(gemm_handle_t h, int64_t rows, int64_t cols, const void* src,
                      int64_t ld_src, int src_dtype, const gemm_fp8_matrix_t* out,
                      const gemm_fp8_matrix_t* out2, void* stream) {
  if (!h || !out || rows < 0 || cols < 0 || ld_src < cols || dg::bad_type(src_dtype))
    return GEMM_ERR_INVALID_ARG;
  for (const gemm_fp8_matrix_t* m : {out, out2}) {
    if (!m) continue;
    if (dg::bad_blocks(m->blocks) || m->ld < cols) return GEMM_ERR_INVALID_ARG;
    if (rows > 0 && cols > 0 && (!m->data || !m->scale)) return GEMM_ERR_INVALID_ARG;
  }
  if (out2 && !((out->blocks == GEMM_FP8_ROW && out2->blocks == GEMM_FP8_COL) ||
                (out->blocks == GEMM_FP8_COL && out2->blocks == GEMM_FP8_ROW)))
    return GEMM_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (!src) return GEMM_ERR_INVALID_ARG;
  const int64_t tr = (rows + 127) / 128, tc = (cols + 127) / 128;
  if (tr > INT32_MAX / tc) return GEMM_ERR_UNSUPPORTED;
  return dg::on_device(h->device, [&]() -> int {
    return dg::launch_fp8_quantize(rows, cols, src, ld_src, src_dtype, out, out2,
                                   static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
  });
}

int gemm_fp8_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const gemm_fp8_matrix_t* A,
                 const gemm_fp8_matrix_t* B, const float* bias, void* C, int64_t ldc,
                 int a_major, int b_major, int out_dtype, void* stream) {
  if (!h || M < 0 || N < 0 || K < 0 || a_major < 0 || a_major > 1 || b_major < 0 || b_major > 1 ||
      dg::bad_type(out_dtype) || ldc < N)
    return GEMM_ERR_INVALID_ARG;
  dg::Fp8Product p{};
  int rc = dg::operand_view(A, M, K, a_major == GEMM_ROW_MAJOR, &p.A);
  if (rc != GEMM_OK) return rc;
  rc = dg::operand_view(B, N, K, b_major == GEMM_COL_MAJOR, &p.B);
  if (rc != GEMM_OK) return rc;
  if (M > INT32_MAX || N > INT32_MAX || K > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return GEMM_OK;
  if (!C) return GEMM_ERR_INVALID_ARG;
  p.M = M;
  p.N = N;
  p.K = K;
  p.bias = bias;
  p.C = C;
  p.ldc = ldc;
  p.out_dtype = out_dtype;
  return dg::on_device(h->device, [&]() -> int {
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dg::fp8_tc_runs(p) ? dg::launch_fp8_tc(h, p, s) : dg::launch_fp8_simt(p, s);
    return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
  });
}

int gemm_moe_fp8_workspace(gemm_handle_t h, const gemm_moe_fp8_t* L, int64_t* bytes) {
  if (!bytes) return GEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (!h) return GEMM_ERR_INVALID_ARG;
  const int rc = dg::check_moe_sizes(L);
  if (rc != GEMM_OK) return rc;
  *bytes = dg::moe_workspace_bytes(h, *L);
  return GEMM_OK;
}

int gemm_moe_fp8(gemm_handle_t h, const gemm_moe_fp8_t* L, void* workspace,
                 int64_t workspace_bytes, void* stream) {
  if (!h) return GEMM_ERR_INVALID_ARG;
  int rc = dg::check_moe_sizes(L);
  if (rc != GEMM_OK) return rc;
  if (L->ld_x < L->hidden || L->ld_router < L->hidden || L->ld_out < L->hidden)
    return GEMM_ERR_INVALID_ARG;
  if (L->tokens == 0) return GEMM_OK;
  if (!L->x || !L->router || !L->out || !L->ids || !L->gates) return GEMM_ERR_INVALID_ARG;
  if ((rc = dg::check_experts(L->gate, L->inner, L->hidden, L->experts)) != GEMM_OK) return rc;
  if ((rc = dg::check_experts(L->up, L->inner, L->hidden, L->experts)) != GEMM_OK) return rc;
  if ((rc = dg::check_experts(L->down, L->hidden, L->inner, L->experts)) != GEMM_OK) return rc;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      workspace_bytes < dg::moe_workspace_bytes(h, *L))
    return GEMM_ERR_INVALID_ARG;
  return dg::on_device(h->device, [&]() -> int {
    return dg::launch_moe(h, *L, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_CUDA;
  });
}

}  // extern "C"

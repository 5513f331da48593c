/*
 * gemm_ortho.h: orthogonalising a matrix (an optimiser's update of a linear
 * layer's weight) by Newton-Schulz steps on the GB300 (sm_103a) GEMM library.
 *
 * For each matrix G (rows x cols) of a batch:
 *     X = G / max(|G|, eps),   |G| the Frobenius norm,
 *     for each step's (a, b, c):  A = X·Xᵀ,  X = a X + (b A + c A·A)·X
 * (with Xᵀ·X and the products from the right where rows > cols, which is the
 * same).  Each singular value s becomes a s + b s^3 + c s^5, so that the result
 * has G's singular vectors and singular values near 1.
 *
 * X is kept in fp32 between the steps; the products read 16-bit copies of X, A
 * and bA + cA·A (fp16, scaled by powers of two that keep them within its
 * range) and sum in fp32.
 *
 * Conventions are those of gemm.h: device pointers owned by the caller, work
 * enqueued on `stream` without waiting, a gemm_status_t returned, one handle
 * not to be run on two unordered streams at once.  Device-side wait timeouts
 * are reported by gemm_status.
 */
#ifndef DGEMM_GB300_GEMM_ORTHO_H_
#define DGEMM_GB300_GEMM_ORTHO_H_

#include "gemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GEMM_ORTHO_MAX_STEPS = 64 };

typedef struct {
  int64_t batch, rows, cols;
  int32_t steps;              /* 1 ... GEMM_ORTHO_MAX_STEPS */
  int32_t dtype;              /* of g: GEMM_F16, GEMM_BF16 or GEMM_F32 */
  const float *coefficients;  /* HOST memory: a, b, c of each step, read during the call */
  double eps;                 /* 2^-100 ... 2^100 */
  const void *g;              /* matrix i at g + i * stride_g elements */
  int64_t ld_g, stride_g;
  void *out;                  /* bfloat16; may be g itself, which is read before it is written */
  int64_t ld_out, stride_out;
} gemm_orthogonalize_t;

/* Device bytes of scratch that gemm_orthogonalize needs (pointers and strides
 * are not looked at).  Errors as gemm_orthogonalize's checks of sizes; *bytes
 * is then 0. */
int gemm_orthogonalize_workspace(gemm_handle_t h, const gemm_orthogonalize_t *p, int64_t *bytes);

/* Enqueues the steps.  workspace: at least gemm_orthogonalize_workspace bytes
 * of device memory, 256-byte aligned, owned by the caller and in use until the
 * stream has passed this call; its contents are unspecified before and after.
 * A matrix with a non-finite element becomes NaN throughout.
 * batch, rows or cols == 0: nothing is launched.
 * Errors: INVALID_ARG (negative size, steps out of range, ld < cols, matrices
 * of a batch that overlap in out, NULL pointer, workspace too small or
 * misaligned, unknown enum, eps out of range, coefficients that are not finite,
 * let singular values of [0, 1] grow beyond 10^4 or b A + c A·A beyond 10^8, or
 * take all of them below 2^-20, but not to 0, before the last step),
 * UNSUPPORTED (rows or cols of 2^20 or more, batch of 2^16 or more, g or out not
 * on a multiple of its elements' size), CUDA. */
int gemm_orthogonalize(gemm_handle_t h, const gemm_orthogonalize_t *p, void *workspace,
                       int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DGEMM_GB300_GEMM_ORTHO_H_ */

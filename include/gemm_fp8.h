/*
 * gemm_fp8.h: the block-scaled 8-bit operators of the GB300 (sm_103a) GEMM
 * library: quantising a matrix to e4m3 with one fp32 scale for each block of
 * 128, the product of two such matrices, and a whole mixture-of-experts layer
 * for a few tokens on such weights.
 *
 * A block-scaled matrix X (rows x cols) is a grid of blocks, each of 1 x 128,
 * 128 x 1 or 128 x 128 elements (the last ones ragged), with one fp32 scale s
 * per block and one e4m3 value q per element: X = q * s.  Quantising sets, for
 * a block whose largest finite magnitude is a,
 *     s = max(a, 2^-100) / 448,    q = e4m3(x * (448 / max(a, 2^-100))),
 * in fp32, each operation rounded to nearest even.  A non-finite element is
 * stored as NaN and does not touch its block's scale.
 *
 * Conventions are those of gemm.h: device pointers owned by the caller, work
 * enqueued on `stream` without waiting, a gemm_status_t returned, one handle
 * not to be run on two unordered streams at once (gemm_fp8_quantize uses
 * nothing of the handle but its device and may run on any stream).
 * Device-side wait timeouts are reported by gemm_status.
 */
#ifndef DGEMM_GB300_GEMM_FP8_H_
#define DGEMM_GB300_GEMM_FP8_H_

#include "gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A third element type, next to GEMM_F16 and GEMM_F32; the calls of this file
 * take it, those of gemm.h do not. */
enum { GEMM_BF16 = 2 };

/* Block shapes: which elements share a scale. */
enum {
  GEMM_FP8_ROW = 0,  /* 1 x 128: along a row */
  GEMM_FP8_COL = 1,  /* 128 x 1: down a column */
  GEMM_FP8_TILE = 2  /* 128 x 128 */
};

/* A block-scaled matrix in row-major storage: value (r, c) is the e4m3 byte
 * data[r * ld + c], its block (i, j) has scale[i * scale_stride_r + j *
 * scale_stride_c].  No alignment is required; the tensor-core path of
 * gemm_fp8_run reads data that is 16-byte aligned with ld a multiple of 16. */
typedef struct {
  void *data;
  int64_t ld;              /* bytes from row to row, >= cols */
  float *scale;
  int64_t scale_stride_r;  /* floats from one block row to the next */
  int64_t scale_stride_c;  /* floats from one block column to the next */
  int32_t blocks;          /* GEMM_FP8_ROW, _COL or _TILE */
  int32_t reserved;        /* 0 */
} gemm_fp8_matrix_t;

/* Quantises src (rows x cols, row-major with ld_src elements from row to row,
 * of type GEMM_F16, GEMM_BF16 or GEMM_F32) into *out, and, when out2 is not
 * NULL, in the same pass over src into *out2: one of the two then has
 * GEMM_FP8_ROW and the other GEMM_FP8_COL blocks.  Bytes between cols and ld
 * are left as they are.  rows == 0 or cols == 0: nothing is launched.
 * Errors: INVALID_ARG (negative size, ld_src < cols, ld < cols, NULL pointer
 * of a non-empty matrix, unknown enum), UNSUPPORTED (out2 with other block
 * shapes; more than 2^31 - 1 blocks of 128 x 128), CUDA. */
int gemm_fp8_quantize(gemm_handle_t h, int64_t rows, int64_t cols, const void *src,
                      int64_t ld_src, int src_dtype, const gemm_fp8_matrix_t *out,
                      const gemm_fp8_matrix_t *out2, void *stream);

/* C = A·B (+bias) of block-scaled A (M x K) and B (K x N), summed in fp32 and
 * rounded once to C's type (GEMM_F16, GEMM_BF16 or GEMM_F32).
 * a_major GEMM_ROW_MAJOR: A is the stored matrix M x K; GEMM_COL_MAJOR: the
 * stored matrix is K x M.  b_major GEMM_ROW_MAJOR: stored K x N;
 * GEMM_COL_MAJOR: stored N x K.  Scales must be constant along 128 elements of
 * K: an operand stored with K along its rows has ROW or TILE blocks, one stored
 * with K down its columns COL or TILE blocks.
 * The sum of 128 of K is multiplied by its two scales in an order that keeps it
 * within fp32's range wherever the result is, for scales down to 2^-109 (the least
 * that quantising makes), unless both operands have scales above 2^103 (block maxima
 * above 4.5e33) within 512 of K.
 * bias: NULL or N fp32 values added in fp32 before the rounding.  C is
 * row-major with ldc >= N elements from row to row.
 * The three products of a linear layer: forward y = x·Wᵀ (x ROW row-major, W
 * TILE col-major), input gradient dx = dy·W (dy ROW row-major, W TILE
 * row-major), weight gradient dW = dyᵀ·x (dy COL col-major, x COL row-major).
 * Operands that are 16-byte aligned with ld a multiple of 16 run on the tensor
 * cores, others on a CUDA-core kernel, which is much slower.
 * M == 0 or N == 0: nothing is launched.  K == 0: C = bias (or 0).
 * Errors: INVALID_ARG (negative size, ld < the stored row, ldc < N, NULL
 * pointer of a non-empty operand, unknown enum, blocks that do not run along
 * K), UNSUPPORTED (M, N or K of 2^31 or more), CUDA. */
int gemm_fp8_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const gemm_fp8_matrix_t *A,
                 const gemm_fp8_matrix_t *B, const float *bias, void *C, int64_t ldc,
                 int a_major, int b_major, int out_dtype, void *stream);

/* One weight of every expert: expert e's matrix (rows x cols as the layer
 * says, 128 x 128 blocks) starts at data + e * expert_stride, its scales at
 * scale + e * scale_stride_e. */
typedef struct {
  const void *data;
  int64_t ld;
  int64_t expert_stride;
  const float *scale;
  int64_t scale_stride_e, scale_stride_r, scale_stride_c;
} gemm_fp8_experts_t;

/* A mixture-of-experts layer on a few tokens.  With x (tokens x hidden) and
 * router (experts x hidden) of type `dtype` (GEMM_F16 or GEMM_BF16):
 *     l = x · routerᵀ (fp32),  p = softmax(l) over the experts,
 *     ids[t][0 .. top_k-1] = the experts of token t with the largest l, in
 *       descending order (of equal ones the lower index first; a NaN counts
 *       as the largest),
 *     gates[t][j] = p at ids[t][j], divided by their sum if renormalize,
 *     h = silu(gate_e · x̂) * (up_e · x̂),   x̂ = x quantised with ROW blocks,
 *     out[t] = sum_j gates[t][j] * (down_e · ĥ), ĥ = h quantised with ROW blocks,
 * products and sums in fp32, out rounded once to `dtype`.  gate and up are
 * inner x hidden, down is hidden x inner.  Weight scales lie between 2^-109 and
 * 2^103, x̂'s and ĥ's may be any.
 * ids (tokens x top_k int32) and gates (tokens x top_k fp32) are outputs too.
 * The same call gives the same bits every time; with other tokens beside it a
 * token's sums may be cut differently, which moves their last bits. */
typedef struct {
  int64_t tokens, hidden, inner, experts;
  int32_t top_k;
  int32_t renormalize;
  int32_t dtype;
  int32_t reserved;          /* 0 */
  const void *x;
  int64_t ld_x;
  const void *router;
  int64_t ld_router;
  gemm_fp8_experts_t gate, up, down;
  void *out;
  int64_t ld_out;
  int32_t *ids;
  float *gates;
} gemm_moe_fp8_t;

enum { GEMM_MOE_MAX_TOKENS = 64, GEMM_MOE_MAX_EXPERTS = 512, GEMM_MOE_MAX_TOP_K = 16 };

/* Device bytes of scratch that gemm_moe_fp8 needs for this layer (its
 * pointers and strides are not looked at).  Errors as gemm_moe_fp8's size
 * checks; *bytes is then 0. */
int gemm_moe_fp8_workspace(gemm_handle_t h, const gemm_moe_fp8_t *layer, int64_t *bytes);

/* Enqueues the layer.  workspace: at least gemm_moe_fp8_workspace bytes of
 * device memory, 256-byte aligned, owned by the caller and in use until the
 * stream has passed this call; its contents are unspecified before and after.
 * tokens == 0: nothing is launched.
 * Errors: INVALID_ARG (negative or zero sizes other than tokens, top_k outside
 * 1 ... experts, leading dimension shorter than the row, NULL pointer,
 * workspace too small or misaligned, unknown enum), UNSUPPORTED (more than
 * GEMM_MOE_MAX_TOKENS tokens, _MAX_EXPERTS experts or _MAX_TOP_K choices;
 * expert weights that are not 16-byte aligned with ld and expert_stride
 * multiples of 16; hidden or inner of 2^20 or more), CUDA. */
int gemm_moe_fp8(gemm_handle_t h, const gemm_moe_fp8_t *layer, void *workspace,
                 int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* DGEMM_GB300_GEMM_FP8_H_ */

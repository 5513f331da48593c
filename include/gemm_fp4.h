/*
 * gemm_fp4.h: the 4-bit operators of the GB300 (sm_103a) GEMM library:
 * quantising a matrix to microscaled 4-bit floating point, reading one back,
 * and the product of two such matrices.
 *
 * A 4-bit matrix X (rows x cols) holds one e2m1 value per element (0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 with a sign; code 8 is the sign), a scale for each block of
 * neighbours along its rows and, where row_scale is given, one fp32 scale per
 * row: X = value * block scale * row scale.  The formats, with what quantising
 * does (in fp32, each operation rounded to nearest even):
 *   GEMM_MXFP4  1 x 32 blocks, e8m0 scale 2^e stored as e + 127,
 *               e = floor(log2(amax)) - 2 within -127 ... 127,
 *               value = e2m1(x * 2^-e), saturating.  No row scale.
 *   GEMM_NVFP4  1 x 16 blocks, e4m3 scale s, row scale g = a / 2688 with
 *               a = max(largest magnitude of the row, 2^-100),
 *               s = e4m3(amax * (448 / a)), value = e2m1(x * ((2688 / a) / s)),
 *               0 where s is 0.
 * amax is over a block's finite elements.  A block with a non-finite element is
 * stored as zeros with a scale of NaN (0xff in mxfp4, 0x7f in nvfp4).
 *
 * Conventions are those of gemm.h: device pointers owned by the caller, work
 * enqueued on `stream` without waiting, a gemm_status_t returned, one handle
 * not to be run on two unordered streams at once (quantising and reading back
 * use nothing of the handle but its device and may run on any stream).
 * Device-side wait timeouts are reported by gemm_status.
 */
#ifndef DGEMM_GB300_GEMM_FP4_H_
#define DGEMM_GB300_GEMM_FP4_H_

#include "gemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GEMM_MXFP4 = 0, GEMM_NVFP4 = 1 };

/* Storage.  Row r's values are ceil(cols / 2) bytes at data + r * ld, the even
 * column in the low half of a byte; the high half of an odd row's last byte is
 * 0.  Block scales lie in pieces of 128 rows x 4 blocks, 512 bytes each, as the
 * tensor cores read them: the scale of row r, block b is
 *   scale[((r / 128) * ceil(blocks / 4) + b / 4) * 512
 *         + (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4],
 * blocks = ceil(cols / 32 or 16); bytes of a piece past the matrix are 0
 * (gemm_fp4_scale_bytes gives the size).  A product's e4m3 scales have a sign
 * bit of 0: the tensor cores have no sign there (reading back takes either).  data and scale are 16-byte aligned
 * and ld is a multiple of 16. */
typedef struct {
  void *data;
  int64_t ld;                /* bytes from row to row, >= ceil(cols / 2) */
  void *scale;
  float *row_scale;          /* NULL: 1 for every row */
  int64_t row_scale_stride;  /* floats from one row to the next; 0: one for all */
  int32_t format;            /* GEMM_MXFP4 or GEMM_NVFP4 */
  int32_t reserved;          /* 0 */
} gemm_fp4_matrix_t;

/* Bytes of the block scales of a rows x cols matrix; GEMM_ERR_INVALID_ARG for a
 * negative size or an unknown format. */
int64_t gemm_fp4_scale_bytes(int64_t rows, int64_t cols, int format);

/* Quantises src (rows x cols, row-major with ld_src elements from row to row,
 * of type GEMM_F16, GEMM_BF16 or GEMM_F32) into *out; in nvfp4 out->row_scale
 * (one float per row, any stride but 0) is written too, in mxfp4 it is NULL.
 * Bytes of data between ceil(cols / 2) and ld are left as they are.
 * rows == 0 or cols == 0: nothing is launched.
 * Errors: INVALID_ARG (negative size, ld_src < cols, ld < ceil(cols / 2), NULL
 * pointer of a non-empty matrix, a row scale that the format does not have or
 * lacks, unknown enum), UNSUPPORTED (misaligned data, scale or ld; src or
 * row_scale not on a multiple of its elements' size; rows or cols of 2^31 -
 * 1024 or more), CUDA. */
int gemm_fp4_quantize(gemm_handle_t h, int64_t rows, int64_t cols, const void *src,
                      int64_t ld_src, int src_dtype, const gemm_fp4_matrix_t *out, void *stream);

/* Writes the values that *m stands for into dst (rows x cols, row-major, ld_dst
 * elements from row to row), value * block scale exactly, times the row scale
 * in fp32, rounded once more to dst_dtype.
 * Errors: as gemm_fp4_quantize; a row scale is optional in both formats. */
int gemm_fp4_dequantize(gemm_handle_t h, int64_t rows, int64_t cols, const gemm_fp4_matrix_t *m,
                        void *dst, int64_t ld_dst, int dst_dtype, void *stream);

/* C = A·Bᵀ (+bias) of 4-bit matrices A (M x K) and B (N x K) of one format,
 * summed in fp32, times the two row scales, rounded once to C's type
 * (GEMM_F16, GEMM_BF16 or GEMM_F32).  bias: NULL or N fp32 values added in
 * fp32 before the rounding.  C is row-major with ldc >= N elements from row to
 * row.  This is y = x·Wᵀ of a linear layer with W stored outputs x inputs.
 * M == 0 or N == 0: nothing is launched.  K == 0: C = bias (or 0).
 * Errors: INVALID_ARG (negative size, ld < ceil(K / 2), ldc < N, NULL pointer
 * of a non-empty operand, unknown enum, two formats), UNSUPPORTED (misaligned
 * data, scale or ld; C, bias or row_scale not on a multiple of its elements'
 * size; M, N or K of 2^31 - 1024 or more), CUDA. */
int gemm_fp4_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K, const gemm_fp4_matrix_t *A,
                 const gemm_fp4_matrix_t *B, const float *bias, void *C, int64_t ldc,
                 int out_dtype, void *stream);

/* 1 where gemm_fp4_run takes one row of A on the CUDA cores, whose bits
 * gemm_fp4_linear_row gives; 0 where it takes it on the tensor cores: N is 2^15
 * or more, or an option asks for one of their forms (GEMM_OPT_FORCE_SWAP_AB,
 * _FORCE_TILE_N, _CLUSTER_SPLIT).  Also 0 for no handle or a negative size. */
int gemm_fp4_one_row(gemm_handle_t h, int64_t N, int64_t K);

/* y = x·Wᵀ (+bias) for one row x of K elements (GEMM_F16, GEMM_BF16 or GEMM_F32),
 * quantised to W's format on the way, in one launch on the CUDA cores whatever
 * the options: the bits of gemm_fp4_quantize and gemm_fp4_run where
 * gemm_fp4_one_row is 1.
 * y: N elements of y_dtype, apart from x.  N == 0: nothing is launched.  K == 0: y = bias (or 0).
 * Errors: as theirs; UNSUPPORTED also for K above GEMM_FP4_ROW_MOST. */
enum { GEMM_FP4_ROW_MOST = 65536 };
int gemm_fp4_linear_row(gemm_handle_t h, int64_t N, int64_t K, const void* x, int x_dtype,
                        const gemm_fp4_matrix_t* W, const float* bias, void* y, int y_dtype,
                        void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DGEMM_GB300_GEMM_FP4_H_ */

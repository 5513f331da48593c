// ortho.cuh: what the parts of the orthogonalising call share.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gemm_ortho.h"
#include "fp8.cuh"

namespace dg {

// The smaller side n of the iterate is the side of A = X·Xᵀ (or Xᵀ·X).  16-bit
// copies are stored times a power of two, the product undoes it.
struct OrthoShape {
  int64_t batch, rows, cols;
  int64_t n;                // min(rows, cols)
  bool tall;                // rows > cols
  // elements from row to row of the iterate and its 16-bit copies, and of A and B:
  // multiples of 64, zeros past the matrix
  int64_t ld_x, ld_a;
  int64_t stride_x, stride_a;
};

// The products of a step.  kGram: A16 = half(gram_alpha · X16·X16ᵀ); kPoly: B16 =
// half(poly_alpha · A16·A16ᵀ + poly_beta · A16); kApply: X = apply_alpha · (B16·X16) +
// apply_beta · X, in fp32 (and X16 = half(X · scale)), or, in the last step, `out` =
// bfloat16 of it.
enum OrthoKind : int { kGram = 0, kPoly = 1, kApply = 2 };
struct OrthoStep {
  float gram_alpha, poly_alpha, poly_beta, apply_alpha, apply_beta, scale;
};

struct OrthoCall {
  OrthoShape shape;
  int32_t steps;
  OrthoStep step[GEMM_ORTHO_MAX_STEPS];
  float* x32;          // the iterate (laid out as its 16-bit copies)
  __half* x16[2];      // step i reads x16[i & 1] and writes the other
  __half *a16, *b16;
  uint32_t* done;      // ortho_counters of them, 0 at the start
  void* out;           // bfloat16
  int64_t ld_out, stride_out;
};

// Counters that launch_ortho_products needs: one per tile of each product.
int64_t ortho_counters(const OrthoShape& s, int32_t steps);
cudaError_t launch_ortho_products(gemm_ctx* h, const OrthoCall& c, cudaStream_t stream);

}  // namespace dg

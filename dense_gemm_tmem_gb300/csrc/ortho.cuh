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

// One product of a step.  kGram: A16 = half(alpha · X16·X16ᵀ); kPoly: B16 = half(alpha
// · A16·A16ᵀ + beta · A16); kApply: X = alpha · (B16·X16) + beta · X, in fp32 (and
// X16 = half(X · scale)), or, in the last step, `out` = bfloat16 of it.
enum OrthoKind : int { kGram = 0, kPoly = 1, kApply = 2 };

struct OrthoProduct {
  int kind;
  float alpha, beta, scale;
  const __half* a;   // X16, A16, B16
  const __half* x;   // kApply: X16
  __half* c;         // A16, B16, X16 (not the one that is read)
  float* x32;        // kApply: the iterate, read and written (laid out as X16)
  void* out;         // kApply, last step: bfloat16, else NULL
  int64_t ld_out, stride_out;
};

cudaError_t launch_ortho_product(gemm_ctx* h, const OrthoShape& s, const OrthoProduct& p,
                                 cudaStream_t stream);

}  // namespace dg

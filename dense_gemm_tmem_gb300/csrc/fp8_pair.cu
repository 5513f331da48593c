// fp8_pair.cu: plan, tensor maps and launch of the two-SM block-scaled product.
#include <algorithm>

#include "context.h"
#include "fp8_pair_kernel.cuh"

namespace dg {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row-to-row pitch of an operand's storage; one row needs none, so any will do.
int64_t pitch_of(const Fp8Operand& o, int64_t mn, int64_t K) {
  const int64_t pitch = o.s_k == 1 ? o.s_mn : o.s_k;
  const int64_t rows = o.s_k == 1 ? mn : K;
  return rows == 1 ? (pitch + 15) & ~int64_t(15) : pitch;
}

bool tma_readable(const Fp8Operand& o, int64_t mn, int64_t K) {
  const int64_t pitch = pitch_of(o, mn, K);
  return (reinterpret_cast<uintptr_t>(o.data) & 15) == 0 && pitch % 16 == 0 &&
         pitch < (int64_t(1) << 40);
}

// The operand in 128-byte-swizzled boxes of one k-block: K-major {128 k, rows},
// MN-major {128 rows, 128 k}; outside the matrix reads as zero.  Encoded anew
// on every call.
bool encode_fp8(CUtensorMap* map, const Fp8Operand& o, int64_t mn, int64_t K, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const bool k_major = o.s_k == 1;
  const cuuint64_t dims[2] = {cuuint64_t(k_major ? K : mn), cuuint64_t(k_major ? mn : K)};
  const cuuint64_t strides[1] = {cuuint64_t(pitch_of(o, mn, K))};
  const cuuint32_t box[2] = {kFp8Block, k_major ? cuuint32_t(box_rows) : cuuint32_t(kFp8Block)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(o.data), dims, strides,
            box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool TRANS, bool COLVEC>
cudaError_t launch_inst(const CUtensorMap& tmA, const CUtensorMap& tmB, const Fp8PairArgs& args,
                        bool pdl, cudaStream_t stream) {
  auto kern = fp8_pair_kernel<BN, TRANS, COLVEC>;
  constexpr int smem = Fp8PairConfig<BN>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(unsigned(2 * args.work.grid), 1, 1);
  cfg.blockDim = dim3(kF8Threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1u : 0u;
  return cudaLaunchKernelEx(&cfg, kern, tmA, tmB, args);
}

}  // namespace

// Whether the tensor cores can run the product: operands the TMA can read and
// int32 coordinates.
bool fp8_pair_runs(const Fp8Product& p) {
  return p.K > 0 && p.M <= kMaxCoord && p.N <= kMaxCoord && p.K <= kMaxCoord &&
         tma_readable(p.A, p.M, p.K) && tma_readable(p.B, p.N, p.K);
}

cudaError_t launch_fp8_pair(gemm_ctx* h, const Fp8Product& p, cudaStream_t stream) {
  // Few rows of A (K-major): operands swapped, so that the other side fills the
  // 256 MMA rows and A's rows are the MMA's columns, 32, 64 or 128 of them.
  const bool trans = p.M <= 128 && p.N > p.M && p.A.s_k == 1;
  const Fp8Operand& opA = trans ? p.B : p.A;
  const Fp8Operand& opB = trans ? p.A : p.B;
  const int64_t Mm = trans ? p.N : p.M, Nm = trans ? p.M : p.N;
  const bool b_mn = opB.s_k != 1;  // needs the whole 128-wide swizzle row per CTA
  const int64_t pairs = std::max(1, h->opt.pair_clusters);
  const int64_t tiles_m = ceil_div(Mm, kPairBM), I = ceil_div(p.K, kFp8Block);
  int bn;
  if (trans)
    bn = Nm <= 32 ? 32 : Nm <= 64 ? 64 : 128;
  else
    bn = b_mn || tiles_m * ceil_div(Nm, 256) >= pairs / 2 ? 256 : 128;
  const int64_t tiles_n = ceil_div(Nm, bn), T = tiles_m * tiles_n;
  if (T > INT32_MAX / 2) return cudaErrorInvalidValue;
  // Fewer tiles than half the pairs: every tile's k-blocks split evenly over
  // the pairs, at least kMinSplit k-blocks each.
  constexpr int64_t kMinSplit = 2;
  int64_t grid = std::min(pairs, T), sk = 0;
  if (2 * T < pairs) {
    const int64_t g = std::min(pairs, std::max(T, T * I / kMinSplit));
    if (g > T) {
      grid = g;
      sk = T;
    }
  }
  Fp8PairArgs a{};
  a.work.tiles_m = int32_t(tiles_m);
  a.work.tiles_n = int32_t(tiles_n);
  a.work.k_iters = int32_t(I);
  a.work.dp_tiles = int32_t(T - sk);
  a.work.sk_tiles = int32_t(sk);
  a.work.grid = int32_t(grid);
  a.work.group_m = 16;
  a.work.csplit = 0;
  a.Mm = int32_t(Mm);
  a.Nm = int32_t(Nm);
  a.row = Fp8Scales{opA.scale, opA.c_mn, opA.c_kb, opA.mn_shift};
  a.col = Fp8Scales{opB.scale, opB.c_mn, opB.c_kb, opB.mn_shift};
  a.C = p.C;
  a.ldc = p.ldc;
  a.bias = p.bias;
  a.out_dtype = p.out_dtype;
  const int64_t pitch = p.ldc * (p.out_dtype == GEMM_F32 ? 4 : 2);
  a.c_vec = (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 && pitch % 16 == 0 ? 1 : 0;
  a.a_mn = opA.s_k != 1;
  a.b_mn = b_mn;
  a.workspace = h->workspace;
  a.tickets = h->tickets;
  a.status = h->status;
  a.wait_limit_ns = h->opt.wait_limit_ns;
  // e4m3 is type code 0 of kind::f8f6f4, as fp16 is of kind::f16
  a.idesc = make_idesc_f16(kPairBM, bn, a.a_mn, a.b_mn);
  CUtensorMap tmA, tmB;
  if (!encode_fp8(&tmA, opA, Mm, p.K, kBM) || !encode_fp8(&tmB, opB, Nm, p.K, bn / 2))
    return cudaErrorInvalidValue;
  const bool pdl = h->opt.pdl != 0;
  const bool colvec = trans || opB.mn_shift == 0;
  if (trans) {
    if (bn == 32) return launch_inst<32, true, true>(tmA, tmB, a, pdl, stream);
    if (bn == 64) return launch_inst<64, true, true>(tmA, tmB, a, pdl, stream);
    return launch_inst<128, true, true>(tmA, tmB, a, pdl, stream);
  }
  if (bn == 256)
    return colvec ? launch_inst<256, false, true>(tmA, tmB, a, pdl, stream)
                  : launch_inst<256, false, false>(tmA, tmB, a, pdl, stream);
  return colvec ? launch_inst<128, false, true>(tmA, tmB, a, pdl, stream)
                : launch_inst<128, false, false>(tmA, tmB, a, pdl, stream);
}

}  // namespace dg

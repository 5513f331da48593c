// fp8_tc.cu: plan, tensor maps and launch of the tensor-core block-scaled product.
#include <algorithm>

#include "context.h"
#include "fp8_tc_kernel.cuh"

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

// The operand's maps (Fp8Maps), 128-byte swizzle; outside the matrix reads as
// zero.  Encoded anew on every call.
bool encode_fp8(Fp8Maps* m, const Fp8Operand& o, int64_t mn, int64_t K, int box_rows,
                int group) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t pitch = cuuint64_t(pitch_of(o, mn, K));
  const cuuint32_t estr[3] = {1, 1, 1};
  auto encode = [&](CUtensorMap* map, cuuint32_t rank, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<uint8_t*>(o.data), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (o.s_k != 1) {
    const cuuint64_t dims[2] = {cuuint64_t(mn), cuuint64_t(K)};
    const cuuint32_t box[2] = {kFp8Block, cuuint32_t(kFp8Block * group)};
    if (!encode(&m->group, 2, dims, &pitch, box)) return false;
    m->one = m->group;  // never used
    return true;
  }
  const cuuint64_t dims2[2] = {cuuint64_t(K), cuuint64_t(mn)};
  const cuuint32_t box2[2] = {kFp8Block, cuuint32_t(box_rows)};
  if (!encode(&m->one, 2, dims2, &pitch, box2)) return false;
  m->group = m->one;
  if (group == 1 || K < kFp8Block * group) return true;  // no whole group: never used
  const cuuint64_t dims3[3] = {kFp8Block, cuuint64_t(mn), cuuint64_t(K / kFp8Block)};
  const cuuint64_t strides3[2] = {pitch, kFp8Block};
  const cuuint32_t box3[3] = {kFp8Block, cuuint32_t(box_rows), cuuint32_t(group)};
  return encode(&m->group, 3, dims3, strides3, box3);
}

// Row-major C for the epilogue's TMA stores: boxes of 32 rows of 128 bytes,
// 128-byte swizzle.  Only rows of whole 16-byte pieces: a store cut off by the
// matrix's edge inside a piece writes the rest of it (seen: zeros past N).
bool encode_c(CUtensorMap* map, const Fp8Product& p) {
  EncodeTiledFn fn = encode_fn();
  const int size = p.out_dtype == GEMM_F32 ? 4 : 2;
  const cuuint64_t dims[2] = {cuuint64_t(p.N), cuuint64_t(p.M)};
  const cuuint64_t pitch = cuuint64_t(p.ldc) * size;
  const cuuint32_t box[2] = {cuuint32_t(128 / size), 32}, estr[2] = {1, 1};
  if (!fn || pitch >= (cuuint64_t(1) << 40) || p.N * size % 16 != 0) return false;
  return fn(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
            p.C, dims, &pitch, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool TRANS, bool COLVEC, bool OUT32>
cudaError_t launch_inst(const Fp8Maps& mA, const Fp8Maps& mB, const CUtensorMap& mC,
                        const Fp8TcArgs& args, int device, bool pdl, cudaStream_t stream) {
  auto kern = fp8_tc_kernel<BN, TRANS, COLVEC, OUT32>;
  constexpr int smem = Fp8TcConfig<BN>::kSmemBytes;
  static SharedMemoryOnce once;
  cudaError_t e = once.allow(kern, smem, device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (args.work.csplit > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(args.work.csplit);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(unsigned(args.work.grid), 1, 1);
  cfg.blockDim = dim3(kF8Threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(n);
  return cudaLaunchKernelEx(&cfg, kern, mA, mB, mC, args);
}

}  // namespace

// Whether the tensor cores can run the product: operands the TMA can read and
// int32 coordinates.
bool fp8_tc_runs(const Fp8Product& p) {
  return p.K > 0 && p.M <= kMaxCoord && p.N <= kMaxCoord && p.K <= kMaxCoord &&
         tma_readable(p.A, p.M, p.K) && tma_readable(p.B, p.N, p.K);
}

cudaError_t launch_fp8_tc(gemm_ctx* h, const Fp8Product& p, cudaStream_t stream) {
  // Few rows of A (K-major): operands swapped, so that the other side fills the
  // 128 MMA rows and A's rows are the MMA's columns, 32, 64 or 128 of them.
  const bool trans = p.M <= 128 && p.N > p.M && p.A.s_k == 1;
  const Fp8Operand& opA = trans ? p.B : p.A;
  const Fp8Operand& opB = trans ? p.A : p.B;
  const int64_t Mm = trans ? p.N : p.M, Nm = trans ? p.M : p.N;
  const int64_t sms = h->num_sms;
  const int64_t tiles_m = ceil_div(Mm, kBM), I = ceil_div(p.K, kFp8Block);
  // Fewer tiles than half the SMs: each tile's k-blocks over a cluster, the
  // largest whose clusters are all resident at once, if that takes more than
  // kSplitGain k-blocks off each CTA: adding the partials costs about as long as
  // 8 k-blocks (2 us of 0.28 at 32 columns, 3 of 0.35 at 64, 4.3 of 0.51 at 128).
  // Measured (graph replay, cold inputs, us, split / whole): 1 x 4096 x 4096 8.4
  // / 12.4, 64 x 4096 x 4096 9.9 / 14.2, 128 x 1024 x 8192 11.0 / 31.9, 512 x 512
  // x 2048 7.4 / 7.8; not taken: 515 x 1000 x 2056 15.7 / 9.2, 1024^3 14.0 / 6.0,
  // 32 x 2048 x 1024 5.3 / 5.2.
  constexpr int64_t kSplitGain = 8;
  const int forced = h->opt.csplit;  // GEMM_OPT_CLUSTER_SPLIT
  auto split_of = [&](int64_t T) -> int64_t {
    if (forced < 2 && (forced >= 0 || 2 * T >= sms)) return 1;
    for (int s : {8, 4, 2}) {
      if (forced >= 2 ? s == forced && I >= s && T * s <= INT32_MAX
                      : T <= h->opt.csplit_clusters[s] && T * s <= sms &&
                            I - ceil_div(I, s) > kSplitGain)
        return s;
    }
    return 1;
  };
  // Tiles of 64 columns instead of 128 where both leave SMs idle (B K-major, whose
  // boxes may have 64 rows): 515 x 1000 x 2056 9.2 us instead of 10.8, 1024^3 6.0
  // instead of 7.0, 256 x 1024 x 4096 8.7 instead of 9.4; but over a deep K, where
  // the wider tiles can be split further, 512 x 1024 x 8192 15.2 instead of 13.0.
  constexpr int64_t kDeepK = 48;  // k-blocks
  int bn;
  if (trans) {
    bn = Nm <= 32 ? 32 : Nm <= 64 ? 64 : 128;
  } else if (Nm > 128 && tiles_m * ceil_div(Nm, 256) >= sms / 2) {
    bn = 256;
  } else {
    const int64_t wide = tiles_m * ceil_div(Nm, 128), narrow = tiles_m * ceil_div(Nm, 64);
    bn = opB.s_k == 1 && 2 * wide <= sms && (I < kDeepK || split_of(wide) == split_of(narrow))
             ? 64 : 128;
  }
  const int64_t tiles_n = ceil_div(Nm, bn), T = tiles_m * tiles_n;
  if (T > INT32_MAX / 2) return cudaErrorInvalidValue;
  const int64_t split = bn <= 128 ? split_of(T) : 1;
  const int64_t grid = split > 1 ? T * split : std::min(sms, T);
  Fp8TcArgs a{};
  a.work.tiles_m = int32_t(tiles_m);
  a.work.tiles_n = int32_t(tiles_n);
  a.work.k_iters = int32_t(I);
  a.work.dp_tiles = int32_t(split > 1 ? 0 : T);
  a.work.sk_tiles = int32_t(split > 1 ? T : 0);
  a.work.grid = int32_t(grid);
  a.work.group_m = 16;
  a.work.csplit = int32_t(split);
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
  a.b_mn = opB.s_k != 1;
  a.k_full = int32_t(p.K / kFp8Block);
  a.status = h->status;
  a.wait_limit_ns = h->opt.wait_limit_ns;
  // e4m3 is type code 0 of kind::f8f6f4, as fp16 is of kind::f16
  a.idesc = make_idesc_f16(kBM, bn, a.a_mn, a.b_mn);
  Fp8Maps mA, mB;
  const int group = bn == 256 ? Fp8TcConfig<256>::kGroup : Fp8TcConfig<128>::kGroup;
  if (!encode_fp8(&mA, opA, Mm, p.K, kBM, group) || !encode_fp8(&mB, opB, Nm, p.K, bn, group))
    return cudaErrorInvalidValue;
  CUtensorMap mC{};
  a.c_tma = bn == 256 && a.c_vec && encode_c(&mC, p);
  const bool pdl = h->opt.pdl != 0;
  const bool colvec = trans || opB.mn_shift == 0;
  const bool out32 = p.out_dtype == GEMM_F32;
  auto launch = [&](auto inst) { return inst(mA, mB, mC, a, h->device, pdl, stream); };
  if (trans) {
    if (bn == 32) return launch(launch_inst<32, true, true, false>);
    if (bn == 64) return launch(launch_inst<64, true, true, false>);
    return launch(launch_inst<128, true, true, false>);
  }
  if (bn == 256) {
    if (colvec)
      return out32 ? launch(launch_inst<256, false, true, true>)
                   : launch(launch_inst<256, false, true, false>);
    return out32 ? launch(launch_inst<256, false, false, true>)
                 : launch(launch_inst<256, false, false, false>);
  }
  if (bn == 64) {
    if (colvec)
      return out32 ? launch(launch_inst<64, false, true, true>)
                   : launch(launch_inst<64, false, true, false>);
    return out32 ? launch(launch_inst<64, false, false, true>)
                 : launch(launch_inst<64, false, false, false>);
  }
  if (colvec)
    return out32 ? launch(launch_inst<128, false, true, true>)
                 : launch(launch_inst<128, false, true, false>);
  return out32 ? launch(launch_inst<128, false, false, true>)
               : launch(launch_inst<128, false, false, false>);
}

}  // namespace dg

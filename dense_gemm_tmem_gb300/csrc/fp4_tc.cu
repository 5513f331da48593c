// fp4_tc.cu: plan, tensor maps and launch of the 4-bit product.
#include <algorithm>

#include "context.h"
#include "fp4_tc_kernel.cuh"

namespace dg {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* p, cuuint64_t inner,
            cuuint64_t outer, cuuint64_t pitch, cuuint32_t box_inner, cuuint32_t box_outer,
            CUtensorMapSwizzle swizzle) {
  EncodeTiledFn fn = encode_fn();
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint32_t box[2] = {box_inner, box_outer}, estr[2] = {1, 1};
  return fn && fn(map, type, 2, const_cast<void*>(p), dims, &pitch, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Values: rows of ceil(K / 2) bytes in boxes of box_rows x 128, zeros outside.  Scales:
// groups of 128 rows in boxes of box_groups x a k-block's pieces (8-byte elements, as a
// box has at most 256), zeros past the last piece.
bool encode_operand(CUtensorMap* values, CUtensorMap* scales, const gemm_fp4_matrix_t& m,
                    int64_t rows, int64_t K, int box_rows, int box_groups) {
  const int64_t pieces = ceil_div(K, 4 * fp4_block(m.format));
  const int per = kF4BlockK / (4 * fp4_block(m.format));
  return encode(values, CU_TENSOR_MAP_DATA_TYPE_UINT8, m.data, cuuint64_t(ceil_div(K, 2)),
                cuuint64_t(rows), cuuint64_t(rows > 1 ? m.ld : (m.ld + 15) & ~int64_t(15)), 128,
                cuuint32_t(box_rows), CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode(scales, CU_TENSOR_MAP_DATA_TYPE_UINT64, m.scale,
                cuuint64_t(pieces * (kFp4Piece / 8)), cuuint64_t(ceil_div(rows, 128)),
                cuuint64_t(pieces * kFp4Piece), cuuint32_t(per * kFp4Piece / 8),
                cuuint32_t(box_groups), CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Row-major C for the epilogue's TMA stores, as the 8-bit product's: boxes of 32 rows
// of 128 bytes, only for rows of whole 16-byte pieces.
bool encode_c(CUtensorMap* map, const Fp4Product& p) {
  const int size = p.out_dtype == GEMM_F32 ? 4 : 2;
  const cuuint64_t pitch = cuuint64_t(p.ldc) * size;
  return pitch < (cuuint64_t(1) << 40) && p.N * size % 16 == 0 &&
         encode(map, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                p.C, cuuint64_t(p.N), cuuint64_t(p.M), pitch, cuuint32_t(128 / size), 32,
                CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int BN, bool PAIR, bool TRANS, int FMT, bool OUT32>
cudaError_t launch_inst(const Fp4Maps& maps, const CUtensorMap& mC, const Fp4TcArgs& args,
                        int device, bool pdl, cudaStream_t stream) {
  auto kern = fp4_tc_kernel<BN, PAIR, TRANS, FMT, OUT32>;
  constexpr int smem = Fp4TcConfig<BN, PAIR, FMT>::kSmemBytes;
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
  const int cluster = PAIR ? 2 : args.work.csplit;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = unsigned(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(unsigned(args.work.grid * (PAIR ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(kF4Threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(n);
  return cudaLaunchKernelEx(&cfg, kern, maps, mC, args);
}

template <int FMT, class Launch>
cudaError_t launch_format(int bn, bool trans, bool out32, Launch&& launch) {
  if (trans)  // stores any type
    return bn == 32 ? launch(launch_inst<32, false, true, FMT, false>)
                    : launch(launch_inst<64, false, true, FMT, false>);
  if (bn == 256)
    return out32 ? launch(launch_inst<256, true, false, FMT, true>)
                 : launch(launch_inst<256, true, false, FMT, false>);
  if (bn == 64)
    return out32 ? launch(launch_inst<64, false, false, FMT, true>)
                 : launch(launch_inst<64, false, false, FMT, false>);
  return out32 ? launch(launch_inst<128, false, false, FMT, true>)
               : launch(launch_inst<128, false, false, FMT, false>);
}

// K == 0: C = bias (or 0).
__global__ void fp4_fill_kernel(int64_t M, int64_t N, const float* bias, void* C, int64_t ldc,
                                int dtype) {
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < M * N;
       i += int64_t(gridDim.x) * blockDim.x)
    store_typed(C, i / N * ldc + i % N, bias ? bias[i % N] : 0.f, dtype);
}

}  // namespace

// One row: a kernel of its own, unless an option asks for a form of the tensor cores' or B has
// so many rows that its warps, four rows each, come in 1.7 rounds or more. Measured (graph
// replay, cold B, us, own kernel / tensor cores, nvfp4, mxfp4; in brackets a layer, one launch
// / quantising and tensor cores).  N x K, its own: 4096 x 4096 3.7 / 6.2, 3.7 / 5.9 [4.5 /
// 7.2, 4.3 / 6.7], 16 x 4096 1.8 / 4.0, 1.9 / 3.8, 64 x 65536 9.4 / 12.4, 9.5 / 11.5, 8192 x
// 8192 9.9 / 11.2, 9.8 / 10.7 [12.1 / 13.3, 11.0 / 11.8], 14336 x 4096 9.1 / 9.0, 9.3 / 8.6
// [10.0 / 10.5, 10.0 / 10.0], 24576 x 4096 15.5 / 15.7, 15.9 / 14.6 [16.0 / 17.6, 16.2 /
// 16.5], 2048 x 65536 17 / 24, 18 / 22.  The tensor cores': 32768 x 4096 18.2 / 16.4, 18.2 /
// 15.7 [18.7 / 18.6, 18.7 / 17.6], 65536 x 1024 11.7 / 11.1, 11.8 / 10.1 [14.0 / 13.2, 12.2 /
// 12.1], 128256 x 4096 53 / 48, 55 / 45 [57 / 50, 59 / 47].  Between them the rule misses up
// to a quarter where the warps leave half of the SMs' places empty (10240 x 8192 15.4 / 13.6,
// 16.2 / 12.8 [17.4 / 16.5, 17.4 / 14.4]) and where K is deep (1024 x 100000 20.7 / 19.6, 21.8
// / 18.6).
bool fp4_one_row(const gemm_ctx* h, int64_t N) {
  constexpr int64_t kRowMostN = int64_t(1) << 15;
  return N < kRowMostN && h->opt.force_swap < 0 && h->opt.csplit < 0 && h->opt.force_tile_n <= 0;
}

cudaError_t launch_fp4(gemm_ctx* h, const Fp4Product& p, cudaStream_t stream) {
  if (p.K == 0) {
    fp4_fill_kernel<<<1024, 256, 0, stream>>>(p.M, p.N, p.bias, p.C, p.ldc, p.out_dtype);
    return cudaGetLastError();
  }
  if (p.M == 1 && fp4_one_row(h, p.N)) return launch_fp4_row(h, p, nullptr, 0, stream);
  const int64_t I = ceil_div(p.K, kF4BlockK);
  // Few rows of A: operands swapped, so that the other side fills the 128 MMA rows and
  // A's rows are the MMA's columns, 32 or 64 of them.  Measured (mxfp4, graph replay, cold
  // inputs, us, swapped / not), N x K 4096 x 4096: 6.4 / 8.0 for 16 rows, 6.7 / 7.7 for 32;
  // 8192 x 1024: 4.4 / 4.9, 4.5 / 4.8.  33 to 63 rows where K is deep and N wide: 48 rows
  // 4096 x 4096 7.1 / 7.8, 4096 x 2816 6.6 / 7.0, 14336 x 4096 10.1 / 12.1, but 4096 x 2048
  // 6.2 / 5.4 and 1024 x 2816 5.6 / 5.3; 64 rows, which fill their boxes, 7.3 / 7.2.
  constexpr int64_t kSwapRows = 32, kSwapMost = 64, kSwapDepth = 8, kSwapWidth = 2048;
  const int swap = h->opt.force_swap;  // GEMM_OPT_FORCE_SWAP_AB
  const bool few = p.M <= kSwapRows ||
                   (p.M < kSwapMost && I > kSwapDepth && p.N >= kSwapWidth);
  const bool trans = swap == 1 ? p.M <= kSwapMost : swap != 0 && few && p.N > p.M;
  const gemm_fp4_matrix_t& opA = trans ? p.B : p.A;
  const gemm_fp4_matrix_t& opB = trans ? p.A : p.B;
  const int64_t Mm = trans ? p.N : p.M, Nm = trans ? p.M : p.N;
  const int64_t sms = h->num_sms;
  const int64_t pairs = h->opt.pair_clusters > 0 ? h->opt.pair_clusters : sms / 2;
  // Fewer tiles than half the SMs: each tile's k-blocks over a cluster, the largest
  // whose clusters are all resident at once, if that takes more than kSplitGain
  // k-blocks off each CTA (adding the partials costs about as long; one more where the tiles
  // have 64 columns instead of 32).  Measured (nvfp4, us, split / whole), 32 columns: 1 x
  // 4096 x 4096 6.4 / 7.6, 1 x 1024 x 8192 5.6 / 11.8 (rows forced here), 16 x 512 x 2048 4.6 / 5.0, 20 x 4096 x 2816
  // 6.2 / 6.4; not taken 20 x 4096 x 2048 5.8 / 5.5, 20 x 1024 x 1792 4.8 / 4.8.  64 columns: 256
  // x 1024 x 4096 7.0 / 7.7, 512 x 512 x 8192 8.0 / 12.0, 64 x 4096 x 4096 7.6 / 7.8; not taken
  // 128 x 1024 x 2048 5.6 / 5.1, 64 x 2048 x 2560 6.5 / 6.0, 64 x 4096 x 3328 7.6 / 7.1.  More
  // CTAs than SMs: 64 x 8192 x 8192 by 4 18.3, by 2, which fit, 12.4, whole 14.4.
  constexpr int64_t kSplitGain = 6;
  const int forced = h->opt.csplit;  // GEMM_OPT_CLUSTER_SPLIT
  auto split_of = [&](int64_t T, int64_t gain) -> int64_t {
    if (forced < 2 && (forced >= 0 || 2 * T >= sms)) return 1;
    for (int s : {8, 4, 2}) {
      if (I < s) continue;  // a CTA without a k-block has no partial to add
      if (forced >= 2 ? s == forced && T * s <= INT32_MAX
                      : T <= h->opt.csplit_clusters[s] && T * s <= sms &&
                            I - ceil_div(I, s) > gain)
        return s;
    }
    return 1;
  };
  int64_t tiles_m = ceil_div(Mm, kBM);
  int bn;
  // Tiles of 256 x 256 of a pair where there are more than 5/4 of them for each pair and K
  // is deep enough for what the pair loses between tiles, its one accumulator being read
  // out (1.2 us): nvfp4, us, 256 / 128: 4096^3 37.4 / 39.5, 8192^3 182 / 253, 4096 x 2048 x
  // 8192 32 / 41, 6000 x 6000 x 2000 55 / 60, but 2048^3 12.2 / 9.4, 1024 x 4096 x 4096 15.1
  // / 14.0, 4096 x 4096 x 1024 22.5 / 19.2, 8192 x 8192 x 1024 64 / 58.  Tiles of 64 columns
  // instead of 128 where both leave half of the SMs idle: 515 x 1000 x 2056 6.4 / 7.6, 1024^3
  // 4.6 / 5.3, but 1001 x 2050 x 4100 14.7 / 12.0, 1536 x 1536 x 1024 6.2 / 5.3.
  constexpr int64_t kPairDepth = 8;  // k-blocks
  const int tile_n = h->opt.force_tile_n;  // GEMM_OPT_FORCE_TILE_N: 64, 128 or 256 (pairs)
  const int64_t wide = ceil_div(Mm, 256) * ceil_div(Nm, 256);
  if (trans) {
    bn = Nm <= 32 ? 32 : 64;
  } else if (tile_n > 0 ? tile_n >= 256 : 4 * wide >= 5 * pairs && I >= kPairDepth) {
    bn = 256;
    tiles_m = ceil_div(Mm, 256);
  } else {
    const bool narrow = tile_n > 0 ? tile_n <= 64 : 2 * tiles_m * ceil_div(Nm, 128) <= sms;
    bn = narrow ? 64 : 128;
  }
  const int64_t tiles_n = ceil_div(Nm, bn), T = tiles_m * tiles_n;
  if (T > INT32_MAX / 2) return cudaErrorInvalidValue;
  const int64_t split = bn <= 128 ? split_of(T, bn == 32 ? kSplitGain : kSplitGain + 1) : 1;
  Fp4TcArgs a{};
  a.work.tiles_m = int32_t(tiles_m);
  a.work.tiles_n = int32_t(tiles_n);
  a.work.k_iters = int32_t(I);
  a.work.dp_tiles = int32_t(split > 1 ? 0 : T);
  a.work.sk_tiles = int32_t(split > 1 ? T : 0);
  a.work.grid = int32_t(split > 1 ? T * split : std::min(bn == 256 ? pairs : sms, T));
  a.work.group_m = bn == 256 ? 8 : 16;
  a.work.csplit = int32_t(split);
  a.Mm = int32_t(Mm);
  a.Nm = int32_t(Nm);
  a.row_scale = opA.row_scale;
  a.row_stride = opA.row_scale_stride;
  a.col_scale = opB.row_scale;
  a.col_stride = opB.row_scale_stride;
  a.C = p.C;
  a.ldc = p.ldc;
  a.bias = p.bias;
  a.out_dtype = p.out_dtype;
  const int64_t pitch = p.ldc * (p.out_dtype == GEMM_F32 ? 4 : 2);
  a.c_vec = (reinterpret_cast<uintptr_t>(p.C) & 15) == 0 && pitch % 16 == 0 ? 1 : 0;
  a.steps = int32_t(ceil_div(p.K, 64));
  a.status = h->status;
  a.wait_limit_ns = h->opt.wait_limit_ns;
  a.idesc = make_idesc_f4(bn == 256 ? 256 : kBM, bn, p.A.format);
  Fp4Maps m;
  if (!encode_operand(&m.a, &m.sa, opA, Mm, p.K, kBM, 1) ||
      !encode_operand(&m.b, &m.sb, opB, Nm, p.K, bn == 256 ? 128 : bn, bn == 256 ? 2 : 1))
    return cudaErrorInvalidValue;
  CUtensorMap mC{};
  a.c_tma = bn == 256 && a.c_vec && encode_c(&mC, p);
  const bool pdl = h->opt.pdl != 0, out32 = p.out_dtype == GEMM_F32;
  auto launch = [&](auto inst) { return inst(m, mC, a, h->device, pdl, stream); };
  return p.A.format == GEMM_MXFP4 ? launch_format<GEMM_MXFP4>(bn, trans, out32, launch)
                                  : launch_format<GEMM_NVFP4>(bn, trans, out32, launch);
}

}  // namespace dg

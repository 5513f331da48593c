// ortho_tc.cu: tensor maps and launch of the orthogonalising call's products.
#include <algorithm>

#include "context.h"
#include "ortho_tc_kernel.cuh"

namespace dg {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An operand stored in rows of `ld` fp16 elements, `batch` matrices of `stride`: K along
// the rows (zeros from `k` to the next multiple of 64) or down them (mn_major).
bool encode(CUtensorMap* map, const __half* p, int64_t mn, int64_t k, int64_t ld, int64_t batch,
            int64_t stride, bool mn_major) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const cuuint64_t row = cuuint64_t(ld) * 2, matrix = cuuint64_t(stride) * 2;
  const cuuint64_t dk[4] = {64, cuuint64_t(mn), cuuint64_t(ceil_div(k, 64)), cuuint64_t(batch)};
  const cuuint64_t sk[3] = {row, 128, matrix};
  const cuuint32_t bk[4] = {64, 128, kOrGroup, 1};
  const cuuint64_t dm[3] = {cuuint64_t(mn), cuuint64_t(k), cuuint64_t(batch)};
  const cuuint64_t sm[2] = {row, matrix};
  const cuuint32_t bm[3] = {64, 64 * kOrGroup, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, mn_major ? 3 : 4, const_cast<__half*>(p),
            mn_major ? dm : dk, mn_major ? sm : sk, mn_major ? bm : bk, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAIR>
cudaError_t launch(const CUtensorMap& mA, const CUtensorMap& mB, const OrTcArgs& args,
                   gemm_ctx* h, cudaStream_t stream) {
  auto kern = ortho_tc_kernel<PAIR>;
  constexpr int smem = OrConfig<PAIR>::kSmemBytes;
  static SharedMemoryOnce once;
  cudaError_t e = once.allow(kern, smem, h->device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (h->opt.pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (PAIR) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(unsigned(args.owners * (PAIR ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(kOrThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(n);
  return cudaLaunchKernelEx(&cfg, kern, mA, mB, args);
}

}  // namespace

cudaError_t launch_ortho_product(gemm_ctx* h, const OrthoShape& s, const OrthoProduct& p,
                                 cudaStream_t stream) {
  OrTcArgs a{};
  a.batch = int32_t(s.batch);
  a.rows = int32_t(s.rows);
  a.cols = int32_t(s.cols);
  a.n = int32_t(s.n);
  a.ld_x = s.ld_x;
  a.ld_a = s.ld_a;
  a.stride_x = s.stride_x;
  a.stride_a = s.stride_a;
  a.p = p;
  a.out_vec = (reinterpret_cast<uintptr_t>(p.out) & 7) == 0 && p.ld_out % 4 == 0 &&
              (s.batch == 1 || p.stride_out % 4 == 0);
  a.status = h->status;
  a.wait_limit_ns = h->opt.wait_limit_ns;
  const bool symmetric = p.kind != kApply;
  const int64_t M = symmetric ? s.n : s.rows, N = symmetric ? s.n : s.cols;
  const int64_t K = p.kind == kGram ? (s.tall ? s.rows : s.cols) : s.n;
  auto tiles = [&](int64_t tile) {
    const int64_t m = ceil_div(M, tile), n = ceil_div(N, tile);
    return symmetric ? m * (m + 1) / 2 : m * n;
  };
  // Pairs' tiles where they occupy half of the SMs, else four times as many small ones.
  const int64_t pairs = h->opt.pair_clusters > 0 ? h->opt.pair_clusters : h->num_sms / 2;
  const bool pair = h->opt.pair >= 0 ? h->opt.pair == 1 : 2 * tiles(256) * s.batch > pairs;
  const int64_t tile = pair ? 256 : 128;
  a.tiles_m = int32_t(ceil_div(M, tile));
  a.tiles_n = int32_t(ceil_div(N, tile));
  const int64_t per = tiles(tile);
  if (per * s.batch > INT32_MAX / 2) return cudaErrorInvalidValue;
  a.per = int32_t(per);
  a.group_m = 8;
  a.k_blocks = int32_t(ceil_div(K, 64));
  a.owners = int32_t(std::min<int64_t>(pair ? pairs : h->num_sms, per * s.batch));
  CUtensorMap mA, mB;
  bool ok;
  if (p.kind == kGram) {
    a.a_mn = a.b_mn = s.tall;
    ok = encode(&mA, p.a, s.n, K, s.ld_x, s.batch, s.stride_x, s.tall);
    mB = mA;
  } else if (p.kind == kPoly) {
    ok = encode(&mA, p.a, s.n, s.n, s.ld_a, s.batch, s.stride_a, false);
    mB = mA;
  } else if (s.tall) {  // X·B, B symmetric
    ok = encode(&mA, p.x, s.rows, s.n, s.ld_x, s.batch, s.stride_x, false) &&
         encode(&mB, p.a, s.n, s.n, s.ld_a, s.batch, s.stride_a, false);
  } else {              // B·X, X's rows along K
    a.b_mn = 1;
    ok = encode(&mA, p.a, s.n, s.n, s.ld_a, s.batch, s.stride_a, false) &&
         encode(&mB, p.x, s.cols, s.n, s.ld_x, s.batch, s.stride_x, true);
  }
  if (!ok) return cudaErrorInvalidValue;
  a.idesc = make_idesc_f16(int(tile), int(tile), a.a_mn, a.b_mn);
  return pair ? launch<true>(mA, mB, a, h, stream) : launch<false>(mA, mB, a, h, stream);
}

}  // namespace dg

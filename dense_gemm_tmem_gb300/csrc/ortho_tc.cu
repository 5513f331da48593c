// ortho_tc.cu: tensor maps and launch of the orthogonalising call's products.
#include <algorithm>

#include "context.h"
#include "ortho_tc_kernel.cuh"

namespace dg {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The maps of matrices stored in rows of `ld` fp16 elements (zeros from `cols` to the next
// multiple of 64), `batch` of them `stride` apart: with K along the rows, and down them.
bool encode(OrOperand* m, const __half* p, int64_t rows, int64_t cols, int64_t ld, int64_t batch,
            int64_t stride, int b_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const cuuint64_t row = cuuint64_t(ld) * 2, matrix = cuuint64_t(stride) * 2;
  auto tiled = [&](CUtensorMap* map, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<__half*>(p), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t dk[4] = {64, cuuint64_t(rows), cuuint64_t(ceil_div(cols, 64)),
                            cuuint64_t(batch)};
  const cuuint64_t sk[3] = {row, 128, matrix};
  const cuuint32_t ba[4] = {64, 128, kOrGroup, 1}, bb[4] = {64, cuuint32_t(b_rows), kOrGroup, 1};
  const cuuint64_t dm[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(batch)};
  const cuuint64_t sm[2] = {row, matrix};
  const cuuint32_t bm[3] = {64, 64 * kOrGroup, 1};
  return tiled(&m->ka, 4, dk, sk, ba) && tiled(&m->kb, 4, dk, sk, bb) &&
         tiled(&m->mn, 3, dm, sm, bm);
}

template <class Cfg>
cudaError_t launch(const OrMaps& maps, const OrTcArgs& args, gemm_ctx* h, cudaStream_t stream) {
  auto kern = ortho_tc_kernel<Cfg>;
  constexpr int smem = Cfg::kSmemBytes;
  static SharedMemoryOnce once;
  cudaError_t e = once.allow(kern, smem, h->device);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  attr[n].id = cudaLaunchAttributeCooperative;  // tiles wait for tiles of other CTAs
  attr[n].val.cooperative = 1;
  ++n;
  if (Cfg::kPair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.gridDim = dim3(unsigned(args.owners * (Cfg::kPair ? 2 : 1)), 1, 1);
  cfg.blockDim = dim3(kOrThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(n);
  return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

using Wide = OrConfig<true, 256>;
using Narrow = OrConfig<true, 128>;
using Small = OrConfig<false, 64>;

struct Tiles {
  int64_t r, c, sym, apply;  // of X's rows and columns, and in all of a matrix
};
template <class Cfg>
Tiles tiles_of(const OrthoShape& s) {
  Tiles t{};
  t.r = ceil_div(s.rows, Cfg::kTileM);
  t.c = ceil_div(s.cols, Cfg::kTileN);
  const int64_t n = ceil_div(s.n, Cfg::kTileM);
  t.sym = Cfg::kRatio * (n * (n + 1) / 2);
  t.apply = t.r * t.c;
  return t;
}

}  // namespace

int64_t ortho_counters(const OrthoShape& s, int32_t steps) {
  const Tiles t = tiles_of<Small>(s);
  return 3 * int64_t(steps) * s.batch * std::max(t.sym, t.apply);
}

cudaError_t launch_ortho_products(gemm_ctx* h, const OrthoCall& c, cudaStream_t stream) {
  const OrthoShape& s = c.shape;
  // Which tiles.  256 x 256: 640 cycles a k-block, 8 flops a loaded byte and cycle more
  // than the others, but each ends with 4 us of epilogue before another product's tile
  // can start; 256 x 128: 480 cycles and 2 us; 128 x 64 of one CTA: 545 cycles, 1 us.
  // So the widest ones where kApply has more than 5/3 of them for each pair, the small
  // ones where it has one for each SM at most and K is so short that its loads take less
  // than an epilogue.  Measured (us, 256 / 128 / 64, each forced, one after the other):
  // 4096^2 1023 / 1504 / 3799 (by itself 988), 8 x 1024^2 286 / 286 / 596, 10 x 700 x 1000
  // 234 / 224 / 433, 2048^2 293 / 284 / 532, 1000 x 4096 282 / 252 / 352, 1024^2 196 / 157
  // / 166, 700 x 1000 180 / 140 / 147, 4 x 512^2 159 / 123 / 117, 512^2 151 / 114 / 111,
  // 128^2 112 / 83 / 67, 64 x 4096 193 / 165 / 189, 4096 x 128 212 / 172 / 179, 16 x 16384
  // 476 / 433 / 566.
  constexpr int64_t kShortK = 8;  // k-blocks
  const int64_t pairs = h->opt.pair_clusters > 0 ? h->opt.pair_clusters : h->num_sms / 2;
  const Tiles wide = tiles_of<Wide>(s), narrow = tiles_of<Narrow>(s), small = tiles_of<Small>(s);
  const int64_t kb = ceil_div(std::max(s.rows, s.cols), 64);
  enum { kWide, kNarrow, kSmall } kind;
  if (h->opt.pair == 0) kind = kSmall;  // GEMM_OPT_PAIR and _FORCE_TILE_N force them
  else if (h->opt.pair == 1) kind = h->opt.force_tile_n == 128 ? kNarrow : kWide;
  else if (3 * wide.apply * s.batch > 5 * pairs) kind = kWide;
  else kind = kb <= kShortK && small.apply * s.batch <= h->num_sms ? kSmall : kNarrow;
  const Tiles t = kind == kWide ? wide : kind == kNarrow ? narrow : small;
  const bool pair = kind != kSmall;
  if (t.sym > INT32_MAX / 16 || t.apply > INT32_MAX / 16) return cudaErrorInvalidValue;
  OrTcArgs a{};
  a.batch = int32_t(s.batch);
  a.steps = c.steps;
  a.owners = int32_t(std::min<int64_t>(pair ? pairs : h->num_sms,
                                       std::max(t.sym, t.apply) * s.batch));
  a.tall = s.tall;
  a.tiles_r = int32_t(t.r);
  a.tiles_c = int32_t(t.c);
  a.per_sym = int32_t(t.sym);
  a.per_apply = int32_t(t.apply);
  a.kb_gram = int32_t(ceil_div(s.tall ? s.rows : s.cols, 64));
  a.kb_n = int32_t(ceil_div(s.n, 64));
  a.rows = int32_t(s.rows);
  a.cols = int32_t(s.cols);
  a.n = int32_t(s.n);
  a.ld_x = s.ld_x;
  a.ld_a = s.ld_a;
  a.stride_x = s.stride_x;
  a.stride_a = s.stride_a;
  a.x16[0] = c.x16[0];
  a.x16[1] = c.x16[1];
  a.a16 = c.a16;
  a.b16 = c.b16;
  a.x32 = c.x32;
  a.out = c.out;
  a.ld_out = c.ld_out;
  a.stride_out = c.stride_out;
  a.out_vec = (reinterpret_cast<uintptr_t>(c.out) & 7) == 0 && c.ld_out % 4 == 0 &&
              (s.batch == 1 || c.stride_out % 4 == 0);
  a.done = c.done;
  a.done_stride = std::max(t.sym, t.apply) * s.batch;
  a.status = h->status;
  a.wait_limit_ns = h->opt.wait_limit_ns;
  std::copy(c.step, c.step + c.steps, a.step);
  OrMaps m{};
  const int b_rows = kind == kWide ? Wide::kBRows : kind == kNarrow ? Narrow::kBRows
                                                                     : Small::kBRows;
  bool ok = encode(&m.a, c.a16, s.n, s.n, s.ld_a, s.batch, s.stride_a, b_rows) &&
            encode(&m.b, c.b16, s.n, s.n, s.ld_a, s.batch, s.stride_a, b_rows);
  for (int i = 0; ok && i < 2; ++i)
    ok = encode(&m.x[i], c.x16[i], s.rows, s.cols, s.ld_x, s.batch, s.stride_x, b_rows);
  if (!ok) return cudaErrorInvalidValue;
  if (kind == kWide) return launch<Wide>(m, a, h, stream);
  return kind == kNarrow ? launch<Narrow>(m, a, h, stream) : launch<Small>(m, a, h, stream);
}

}  // namespace dg

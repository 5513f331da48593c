// fp4_tc_kernel.cuh: the 4-bit product on the tensor cores
// (tcgen05.mma.kind::mxf4 and kind::mxf4nvf4, block_scale).
//
//   C[m, n] = ra[m] rb[n] sum over k of a[m, k] sa[m, k / n_s] b[n, k] sb[n, k / n_s]
//
// with a scale for each n_s = 32 or 16 neighbours along K, which the tensor core
// applies itself: the scales lie in TMEM beside the accumulator, and a whole tile is
// one MMA chain.  256 values of K are 128 bytes, one swizzle row, and 4 MMAs of K =
// 64; their scales are 4 (nvfp4) or 2 (mxfp4) pieces of 128 rows x 4 blocks, stored
// in memory as the 32 x 16-byte boxes that tcgen05.cp takes.  Per CTA:
//   warp 0, one lane   TMA producer: 128 rows of A, this CTA's rows of B and the
//                      pieces of their scales into an S-stage ring.
//   warp 1             per stage, copies its scales into the TMEM columns that
//                      belong to the stage (the ring's own barriers so keep a
//                      stage's scales until its MMAs are done), then 4 MMAs.
//   warps 4-11         epilogue, two warpgroups of BN / 2 columns: TMEM to
//                      registers, the buffer goes back, row scales, bias, store.
// PAIR: two CTAs on two SMs own a 256 x 256 tile (cta_group::2), each with its 128
// rows of A and half of B's rows, both with all of B's scales.
//
// What bounds it, 8192^3 nvfp4 in 182 us (6.0 PFLOP/s; mxfp4 172, 6.4): a k-block's MMAs
// take 512 cycles, a tile's 32 of them 16400 of the 22900 that it takes.  1750 are copies
// of scales (mxfp4 half of that), 2250 pass between two tiles, because 512 columns of
// TMEM hold one accumulator and the scales (its 256 columns are read in 1550), and some
// 4000 are waits for loads, whose latency of 2500 cycles under load five stages do not
// cover.  Left out in copies made for the purpose: A's and B's loads 169 us, the scales'
// 177, the stores 166.  Measured and dropped: tiles of 192 columns with two accumulators
// (mxfp4 178 against 173; in nvfp4 TMEM then holds two k-blocks' scales, 223), the scales
// copied a k-block ahead (226 and 321), one more thread to send for the scales' loads
// (188 against 184), polling instead of suspended waits (191), all of the accumulator's
// reads in flight together (no change), 128 columns (230).
// tcgen05.mma reads scales from even TMEM columns only: tiles start at multiples of 64
// rows of B (160-wide ones, whose scales start at odd columns, fault).
// Small products are bound by latency: launch, first loads, the cluster's exchange; one row
// of A has a kernel of its own (fp4_row.cu).
#pragma once

#include "fp4.cuh"
#include "fp8_tc_kernel.cuh"
#include "tc2_kernel.cuh"

namespace dg {

constexpr int kF4RoleWarps = 4;  // producer, MMA issuer, two idle: one warpgroup
constexpr int kF4EpiWarps = 8;
constexpr int kF4Threads = 32 * (kF4RoleWarps + kF4EpiWarps);
constexpr int kF4BlockK = 256;  // values of K per k-block: 128 bytes
// Registers: 3 warpgroups launch with 168 each.  A pair's epilogue holds 128 sums a
// thread: the role warpgroup gives up all but 40, the epilogue's two take 232 (40 + 2 *
// 232 = 504 = 3 * 168).  A pair's kernel is still compiled for the 168 of the launch and
// spills (-Xptxas -v: 324 bytes stored and 360 loaded where C has 16 bits, 76 and 200 in
// fp32); the other tiles do not.
constexpr int kF4RoleRegs = 40, kF4EpiRegs = 232;

template <int BN, bool PAIR, int FMT>
struct Fp4TcConfig {
  static constexpr int kPieces = FMT == GEMM_MXFP4 ? 2 : 4;        // per k-block and 128 rows
  static constexpr int kGroups = BN > 128 ? BN / 128 : 1;          // of 128 rows, B's scales
  static constexpr int kBRows = PAIR ? BN / 2 : BN;                // that this CTA loads
  static constexpr int kABytes = kBM * 128;
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kSaBytes = kPieces * kFp4Piece;
  static constexpr int kSbBytes = kGroups * kPieces * kFp4Piece;
  static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
  static constexpr int kStages = PAIR ? 5 : BN == 128 ? 5 : 6;
  static constexpr int kBuffers = BN == 256 ? 1 : 2;               // TMEM accumulators
  // TMEM columns of a stage's scales: 4 per piece and 128 rows
  static constexpr int kSaCols = 4 * kPieces, kSbCols = 4 * kPieces * kGroups;
  static constexpr int kAccCols = BN * kBuffers;
  static constexpr int kUsedCols = kAccCols + kStages * (kSaCols + kSbCols);
  static constexpr int kTmemCols = kUsedCols <= 256 ? 256 : 512;
  static_assert(kUsedCols <= 512 && (BN % 64 == 0 || BN == 32), "TMEM columns");
  static constexpr int kHalf = BN / 2;
  static constexpr int kWarpStage = BN == 256 ? 4096 : 32 * 20 * 4;  // a store box, or staged rows
  static constexpr int kEpiBytes = kF4EpiWarps * kWarpStage;
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiBytes + kBarBytes;
  static_assert(2 * kHalf * 4 <= kWarpStage, "a warp's column scales and biases");
  static constexpr int kParkRow = BN + 4, kParkCol = kBM + 4;
  static_assert(BN == 256 || (kBM * kParkRow * 4 <= kStages * kStageBytes &&
                              BN * kParkCol * 4 <= kStages * kStageBytes), "the ring holds it");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static_assert((2 * kStages + 2 * kBuffers + 1) * 8 + 16 <= kBarBytes, "barrier area");
};

struct Fp4TcArgs {
  WorkSpec work;
  int32_t Mm, Nm;          // MMA-view extents
  const float* row_scale;  // of the MMA-view A and B operands; NULL: 1
  int64_t row_stride;
  const float* col_scale;
  int64_t col_stride;
  void* C;                 // row-major in the problem's view
  int64_t ldc;
  const float* bias;       // NULL or one per column of C
  int32_t out_dtype;
  int32_t c_vec;           // 1: C's base is 16-byte aligned, its pitch a multiple of 16 bytes
  int32_t c_tma;           // 1: C leaves by TMA (256-wide tiles)
  int32_t steps;           // MMAs of K = 64 in all
  int* status;
  uint64_t wait_limit_ns;
  uint32_t idesc;
};

struct Fp4Maps {
  CUtensorMap a, b, sa, sb;  // values (boxes of rows x 128 bytes, swizzled), scale pieces
};

// 32 rows of 16 bytes of shared memory to 4 TMEM columns, the same in all four lane
// quarters: a piece of 128 rows x 4 blocks.
template <bool PAIR>
__device__ __forceinline__ void f4_copy_scales(uint32_t tmem, uint64_t desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
                 : "memory");
}

// D[tmem] (+)= (A sa) · (B sb)ᵀ, 64 of K.
#define DG_F4_MMA(GROUP, KIND)                                                                  \
  asm volatile(                                                                                 \
      "{\n\t.reg .pred p;\n\t"                                                                  \
      "setp.ne.b32 p, %6, 0;\n\t"                                                               \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"   \
      ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)           \
      : "memory")
template <bool PAIR, int FMT>
__device__ __forceinline__ void f4_mma_issue(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t sa, uint32_t sb,
                                             uint32_t accumulate) {
  if constexpr (FMT == GEMM_MXFP4) {
    if constexpr (PAIR) DG_F4_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else DG_F4_MMA("1", "mxf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (PAIR) DG_F4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else DG_F4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
  }
}
#undef DG_F4_MMA

// Instruction descriptor of the two kinds: bits 4-5 / 29-30 which scales of a 32-bit
// word B / A take (0 or 2), 7-9 / 10-11 A / B type (1 = e2m1), 17-22 N >> 3, 23 scale
// type (0 = e4m3, 1 = e8m0), 27-28 M >> 7.
__host__ __device__ constexpr uint32_t make_idesc_f4(int m, int n, int format) {
  return (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) |
         (uint32_t(format == GEMM_MXFP4) << 23) | (uint32_t(m >> 7) << 27);
}

// Shared-memory descriptor of unswizzled 16-byte rows, 8 of them (128 bytes) together.
__device__ __forceinline__ uint64_t make_sdesc_rows16(uint32_t saddr) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}

// TMA producer (one thread).  Returns how many stages it filled.
template <int BN, bool PAIR, bool TRANS, int FMT>
__device__ __forceinline__ uint32_t f4_producer(const Fp4Maps& m, const Fp4TcArgs& args,
                                                uint8_t* ring, uint64_t* full, uint64_t* empty,
                                                const WaitCtl& wc, uint32_t rank, int32_t owner) {
  using Cfg = Fp4TcConfig<BN, PAIR, FMT>;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init_tc(W, owner);
  Unit u;
  int s = 0;
  uint32_t ph = 0, filled = 0;
  // Swapped operands: what the first stages load of A, the weight, is sent for to L2 before
  // the kernels ahead in the stream are done: that is no read, so that they may write it.
  // (A layer of 4096 x 4096 for 16 rows 8.0 us instead of 8.8, the product alone 6.7 / 6.9.
  // Other tiles, whose loads then follow at once, lose half a microsecond.)
  if constexpr (TRANS) {
    WorkIter first = it;
    if (first.next(W, u)) {
      int32_t tm, tn;
      tile_coords(W, u.tile, tm, tn);
      for (int32_t kb = u.kb0; kb < u.kb1 && kb < u.kb0 + Cfg::kStages; ++kb) {
        tma_prefetch_2d(&m.a, kb * 128, tm * kBM);
        tma_prefetch_2d(&m.sa, kb * (Cfg::kPieces * kFp4Piece / 8), tm);
      }
    }
  }
  pdl_wait_prerequisites();
  while (it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    const int32_t a_row = tm * (PAIR ? 2 * kBM : kBM) + int32_t(rank) * kBM;
    const int32_t b_row = tn * BN + (PAIR ? int32_t(rank) * Cfg::kBRows : 0);
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      if (!wait_bounded(smem_u32(&empty[s]), ph ^ 1, wc, kSiteProducer)) return filled;
      const uint32_t own = smem_u32(&full[s]);
      if (rank == 0) mbar_arrive_expect_tx(own, (PAIR ? 2 : 1) * Cfg::kStageBytes);
      const uint32_t a = smem_u32(ring) + uint32_t(s) * Cfg::kStageBytes;
      const uint32_t b = a + Cfg::kABytes, sa = b + Cfg::kBBytes, sb = sa + Cfg::kSaBytes;
      const int32_t sc = kb * (Cfg::kPieces * kFp4Piece / 8);  // the map's elements have 8 bytes
      if constexpr (PAIR) {
        const uint32_t bar = map_to_rank(own, 0);
        tma_load_2d_pair(a, &m.a, bar, kb * 128, a_row);
        tma_load_2d_pair(b, &m.b, bar, kb * 128, b_row);
        tma_load_2d_pair(sa, &m.sa, bar, sc, a_row / 128);
        tma_load_2d_pair(sb, &m.sb, bar, sc, tn * BN / 128);
      } else {
        tma_load_2d(a, &m.a, own, kb * 128, a_row);
        tma_load_2d(b, &m.b, own, kb * 128, b_row);
        tma_load_2d(sa, &m.sa, own, sc, a_row / 128);
        tma_load_2d(sb, &m.sb, own, sc, tn * BN / 128);
      }
      ++filled;
      if (++s == Cfg::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  return filled;
}

// MMA issuer: the whole warp runs the loop, one lane issues.  Whether it issued anything.
template <int BN, bool PAIR, int FMT>
__device__ __forceinline__ bool f4_mma(const Fp4TcArgs& args, uint32_t ring, uint32_t full,
                                       uint32_t empty, uint32_t acc_full, uint32_t acc_empty,
                                       const WaitCtl& wc, uint32_t tmem_base, int32_t owner) {
  using Cfg = Fp4TcConfig<BN, PAIR, FMT>;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init_tc(W, owner);
  Unit u;
  uint32_t s = 0, ph = 0, b = 0, bph = 1;
  bool ok = true, any = false;
  const bool leader = f8_elect();
  auto commit = [&](uint32_t bar) {
    if constexpr (PAIR) tc_commit_pair_both(bar);
    else tc_commit(bar);
  };
  while (ok && it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    // where this tile's rows of B start within their 128 rows of scales
    const uint32_t sb_off = BN < 128 ? uint32_t(tn * BN % 128 / 32) : 0;
    ok = __all_sync(0xffffffffu, wait_bounded(acc_empty + 8 * b, bph, wc, kSiteMmaAccum));
    if (!ok) break;
    tc_fence_after();
    const uint32_t d = tmem_base + b * BN;
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      if (!mbar_test(full + 8 * s, ph)) ok = wait_bounded(full + 8 * s, ph, wc, kSiteMmaFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      if (leader) {
        const uint32_t a = ring + s * Cfg::kStageBytes;
        const uint32_t sa = a + Cfg::kABytes + Cfg::kBBytes, sb = sa + Cfg::kSaBytes;
        const uint32_t ta = tmem_base + Cfg::kAccCols + s * (Cfg::kSaCols + Cfg::kSbCols);
        const uint32_t tb = ta + Cfg::kSaCols;
        const int left = args.steps - 4 * kb;
        const uint64_t sadesc = make_sdesc_rows16(sa), sbdesc = make_sdesc_rows16(sb);
#pragma unroll
        for (int p = 0; p < Cfg::kPieces; ++p) {
          f4_copy_scales<PAIR>(ta + 4 * p, sadesc + uint64_t(p * (kFp4Piece >> 4)));
#pragma unroll
          for (int i = 0; i < Cfg::kGroups; ++i)
            f4_copy_scales<PAIR>(tb + 4 * (p * Cfg::kGroups + i),
                                 sbdesc + uint64_t((i * Cfg::kPieces + p) * (kFp4Piece >> 4)));
        }
        const uint64_t adesc = make_sdesc_sw128(a, 16, 1024);
        const uint64_t bdesc = make_sdesc_sw128(a + Cfg::kABytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk >= left) break;
          const int p = FMT == GEMM_MXFP4 ? kk / 2 : kk;
          const uint32_t id = FMT == GEMM_MXFP4 && (kk & 1) ? (2u << 4) | (2u << 29) : 0u;
          f4_mma_issue<PAIR, FMT>(d, adesc + uint64_t(kk * 2), bdesc + uint64_t(kk * 2),
                                  args.idesc | id, ta + 4 * p,
                                  tb + 4 * p * Cfg::kGroups + sb_off,
                                  kb > u.kb0 || kk > 0 ? 1u : 0u);
        }
        commit(empty + 8 * s);
        if (kb + 1 == u.kb1) commit(acc_full + 8 * b);
      }
      __syncwarp();
      any = true;
      if (++s == uint32_t(Cfg::kStages)) {
        s = 0;
        ph ^= 1;
      }
    }
    if (++b == uint32_t(Cfg::kBuffers)) {
      b = 0;
      bph ^= 1;
    }
  }
  return any;
}

// A warp's column scales and biases, HC of each, in its staging memory until the tile is
// staged there.
template <int HC>
struct F4Columns {
  static constexpr int kPer = (HC + 31) / 32;  // a lane's
  float s[kPer], b[kPer];
  bool fits;  // every column's scale times this lane's row scale is a number fp32 holds

  // Sent for before the wait for the tile's sum; columns outside the matrix have 1 and 0.
  __device__ __forceinline__ void load(const float* scale, int64_t stride, const float* bias,
                                       int32_t n0, int32_t N, int lane) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = lane + i * 32;
      const bool in = j < HC && n0 + j < N;
      s[i] = scale && in ? __ldg(scale + int64_t(n0 + j) * stride) : 1.f;
      b[i] = bias && in ? __ldg(bias + n0 + j) : 0.f;
    }
  }
  __device__ __forceinline__ void share(float* to, float row, int lane) {
    float most = 0.f, least = INFINITY;
    bool nan = false;
    __syncwarp();  // the last tile's have been read
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (lane + i * 32 < HC) {
        to[lane + i * 32] = s[i];
        to[HC + lane + i * 32] = b[i];
      }
      const float a = fabsf(s[i]);
      most = fmaxf(most, a);
      least = fminf(least, a);
      nan |= !(a == a);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
      least = fminf(least, __shfl_xor_sync(0xffffffffu, least, d));
    }
    fits = __all_sync(0xffffffffu, !nan && scale_fits(row * most) && scale_fits(row * least));
    __syncwarp();
  }
};

template <int BN, bool PAIR, bool TRANS, int FMT, bool OUT32>
__device__ __forceinline__ void f4_epilogue(const Fp4TcArgs& args, const CUtensorMap* tmC,
                                            uint32_t acc_full, uint32_t acc_empty,
                                            const WaitCtl& wc, uint32_t tmem_base, float* stage,
                                            float* park, uint32_t rank, int32_t owner) {
  using Cfg = Fp4TcConfig<BN, PAIR, FMT>;
  constexpr int HC = Cfg::kHalf, CW = HC < 32 ? 16 : 32;
  const WorkSpec& W = args.work;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;                          // TMEM lane quarter this warp may access
  const int wg = (warp - kF4RoleWarps) >> 2;       // which half of the columns
  const int row = q * 32 + lane;
  float* stage_w = stage + (warp - kF4RoleWarps) * (Cfg::kWarpStage / 4);
  WorkIter it;
  it.init_tc(W, owner);
  pdl_wait_prerequisites();
  Unit u;
  uint32_t b = 0, bph = 0;
  const uint32_t tlane = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(wg * HC);
  // the bias joins the scales, but for a split tile's (added after the partials) and for
  // a transposed one's (a lane's own)
  const float* const bias = TRANS || (BN <= 128 && W.csplit > 1) ? nullptr : args.bias;
  const bool columns = args.row_scale != nullptr || args.col_scale != nullptr || bias != nullptr;
  F4Columns<HC> C;
  Fp4TcArgs plain = args;
  plain.bias = nullptr;
  while (it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    const int32_t mrow0 = tm * (PAIR ? 2 * kBM : kBM) + int32_t(rank) * kBM;
    const int32_t mm = mrow0 + row;
    const int32_t nn0 = tn * BN + wg * HC;
    const float rs = args.row_scale && mm < args.Mm
                         ? __ldg(args.row_scale + int64_t(mm) * args.row_stride) : 1.f;
    if (columns) {
      C.load(args.col_scale, args.col_stride, bias, nn0, args.Nm, lane);
      if (BN == 256 && lane == 0) bulk_wait_read_all();  // the last tile's store has left
      C.share(stage_w, rs, lane);
    }
    const bool ok = wait_bounded(acc_full + 8 * b, bph, wc, kSiteEpilogue);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after();
    float acc[HC];
#pragma unroll
    for (int c = 0; c < HC / CW; ++c) {
      uint32_t v[CW];
      tmem_issue<CW>(tlane + uint32_t(b * BN + c * CW), v);
      if constexpr (CW == 32) {
        tmem_wait_ld32(v);
      } else {
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                       "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                       "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
      }
#pragma unroll
      for (int j = 0; j < CW; ++j) acc[c * CW + j] = __uint_as_float(v[j]);
    }
    // the buffer's last read is done: back to the MMA issuer
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if constexpr (PAIR) mbar_arrive_cluster(map_to_rank(acc_empty + 8 * b, 0));
      else mbar_arrive(acc_empty + 8 * b);
    }
    if (++b == uint32_t(Cfg::kBuffers)) {
      b = 0;
      bph ^= 1;
    }
    if (columns) {
      // the product of the two scales where fp32 holds it, else the smaller first
      const uint32_t cs = smem_u32(stage_w), cb = cs + 4 * HC;
      if (C.fits) {
#pragma unroll
        for (int j = 0; j < HC; j += 4) {
          const float4 s4 = lds4(cs + 4 * j);
          const float4 b4 = lds4(cb + 4 * j);
          acc[j] = fmaf(acc[j], s4.x * rs, b4.x);
          acc[j + 1] = fmaf(acc[j + 1], s4.y * rs, b4.y);
          acc[j + 2] = fmaf(acc[j + 2], s4.z * rs, b4.z);
          acc[j + 3] = fmaf(acc[j + 3], s4.w * rs, b4.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < HC; ++j) {
          float lo, hi;
          scale_order(rs, stage_w[j], lo, hi);
          acc[j] = fmaf(__fmul_rn(acc[j], lo), hi, stage_w[HC + j]);
        }
      }
    }
    if (BN <= 128 && W.csplit > 1) {
      // The CTA's only unit: its MMAs have read the ring and every copy into it has
      // landed, so the partial tile may take its place.
      fence_proxy_async_smem();
#pragma unroll
      for (int j = 0; j < HC / 4; ++j) {
        const float4 x = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
        const int c = wg * HC + 4 * j;
        if constexpr (TRANS) {
          park[(c + 0) * Cfg::kParkCol + row] = x.x;
          park[(c + 1) * Cfg::kParkCol + row] = x.y;
          park[(c + 2) * Cfg::kParkCol + row] = x.z;
          park[(c + 3) * Cfg::kParkCol + row] = x.w;
        } else {
          *reinterpret_cast<float4*>(park + row * Cfg::kParkRow + c) = x;
        }
      }
      return;
    }
    if constexpr (TRANS) {
      if (mm < args.Mm) {
        const float bv = args.bias ? __ldg(args.bias + mm) : 0.f;
#pragma unroll
        for (int j = 0; j < HC; ++j)
          if (nn0 + j < args.Nm)
            store_typed(args.C, int64_t(nn0 + j) * args.ldc + mm, acc[j] + bv, args.out_dtype);
      }
    } else {
      constexpr int SIZE = OUT32 ? 4 : 2;
      if (BN == 256 && args.c_tma)
        f8_store_tma<HC, SIZE, 1>(plain, tmC, acc, smem_u32(stage_w), mrow0 + q * 32, lane, nn0);
      else
        f8_store_rows<HC, SIZE>(plain, acc, stage_w, mrow0 + q * 32, lane, nn0);
    }
  }
  // every store this warp issued has landed before the CTA moves on
  if (BN == 256 && lane == 0) bulk_wait_all();
}

// args.work counts tiles (128 x BN, or 256 x 256 for a pair) and CTAs (or pairs).
template <int BN, bool PAIR, bool TRANS, int FMT, bool OUT32>
__global__ void __launch_bounds__(kF4Threads, 1)
    fp4_tc_kernel(const __grid_constant__ Fp4Maps maps, const __grid_constant__ CUtensorMap tmC,
                  const Fp4TcArgs args) {
  using Cfg = Fp4TcConfig<BN, PAIR, FMT>;
  constexpr int S = Cfg::kStages, NB = Cfg::kBuffers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  static_assert(Cfg::kStageBytes % 1024 == 0, "stages and staging boxes 1024-byte aligned");
  float* stage = reinterpret_cast<float*>(ring + S * Cfg::kStageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(stage) + Cfg::kEpiBytes);
  uint64_t* full = bars;                // S: a stage's bytes have landed (the leader's)
  uint64_t* empty = bars + S;           // S: its MMAs are done
  uint64_t* acc_full = empty + S;       // NB: a unit's sum is in TMEM
  uint64_t* acc_empty = acc_full + NB;  // NB: all epilogue warps have read it (the leader's)
  uint64_t* drain = acc_empty + NB;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* peer_filled = tmem_slot + 2;  // leader: stages that the peer's producer filled

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const int32_t owner = PAIR ? int32_t(blockIdx.x >> 1) : int32_t(blockIdx.x);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), kF4EpiWarps * (PAIR ? 2 : 1));
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *peer_filled = 0;
    fence_barrier_init();
    tma_prefetch_map(&maps.a);
    tma_prefetch_map(&maps.b);
    tma_prefetch_map(&maps.sa);
    tma_prefetch_map(&maps.sb);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), Cfg::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  const WaitCtl wc{args.wait_limit_ns, args.status, abort_flag};

  uint32_t filled = 0;
  bool issued = false;
  if (warp >= kF4RoleWarps) {
    if constexpr (PAIR) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF4EpiRegs));
    f4_epilogue<BN, PAIR, TRANS, FMT, OUT32>(args, &tmC, smem_u32(acc_full), smem_u32(acc_empty),
                                             wc, tmem_base, stage,
                                             reinterpret_cast<float*>(ring), rank, owner);
  } else {
    if constexpr (PAIR) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF4RoleRegs));
    if (warp == 0 && lane == 0) {
      filled = f4_producer<BN, PAIR, TRANS, FMT>(maps, args, ring, full, empty, wc, rank, owner);
      if (PAIR && rank != 0) st_dsmem_u32(map_to_rank(smem_u32(peer_filled), 0), filled);
    } else {
      pdl_wait_prerequisites();
      if (warp == 1 && rank == 0)
        issued = f4_mma<BN, PAIR, FMT>(args, smem_u32(ring), smem_u32(full), smem_u32(empty),
                                       smem_u32(acc_full), smem_u32(acc_empty), wc, tmem_base,
                                       owner);
    }
  }
  // after an abort, copies and MMAs may still be in flight
  if constexpr (!PAIR) {
    if (threadIdx.x == 0)
      for (uint32_t s = 0; s < uint32_t(S) && s < filled; ++s)
        wait_drain(smem_u32(&full[s]), ((filled - 1 - s) / S) & 1, wc);
  }
  tc_fence_before();
  __syncthreads();
  // (a pair's: whichever of the two CTAs gave up)
  if (warp == 1 && issued && (PAIR || *abort_flag != 0)) {
    if (f8_elect()) {
      if constexpr (PAIR) tc_commit_pair_self(smem_u32(drain));
      else tc_commit(smem_u32(drain));
      wait_drain(smem_u32(drain), 0, wc);
    }
    __syncwarp();
  }
  if constexpr (PAIR) {
    // both CTAs' roles are done; the leader waits for the loads of both, then the
    // peer may leave (see tc2_drain_loads)
    __syncthreads();
    cluster_sync_all();
    if (rank == 0 && threadIdx.x == 0) {
      const uint32_t n0 = filled, n1 = *peer_filled, n = n0 > n1 ? n0 : n1;
      for (uint32_t s = 0; s < uint32_t(S) && s < n; ++s) {
        const uint32_t at = s + ((n - 1 - s) / S) * S;  // the stage's last filled slot
        const uint32_t bar = smem_u32(&full[s]);
        if (at >= n0) mbar_arrive_expect_tx(bar, Cfg::kStageBytes);
        else if (at >= n1) mbar_complete_tx(bar, Cfg::kStageBytes);
        wait_drain(bar, (at / S) & 1, wc);
      }
    }
    cluster_sync_all();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
  if constexpr (BN <= 128) {
    if (args.work.csplit > 1) {
      cluster_sync_all();  // every partial of the cluster is parked
      if (warp >= kF4RoleWarps) {
        const uint32_t park = smem_u32(ring);
        if (args.work.csplit == 2) f8_cluster_reduce<BN, TRANS, 2, kF4RoleWarps>(args, park);
        else if (args.work.csplit == 4) f8_cluster_reduce<BN, TRANS, 4, kF4RoleWarps>(args, park);
        else f8_cluster_reduce<BN, TRANS, 8, kF4RoleWarps>(args, park);
      }
      cluster_sync_all();  // no CTA leaves while another reads its partial
    }
  }
}

}  // namespace dg

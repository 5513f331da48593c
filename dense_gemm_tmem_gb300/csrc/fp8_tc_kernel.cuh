// fp8_tc_kernel.cuh: the block-scaled product on the tensor cores
// (tcgen05.mma.kind::f8f6f4).
//
//   C[m, n] = sum over kb of sa[m, kb] sb[n, kb] P_kb[m, n],
//   P_kb[m, n] = sum over the 128 k of block kb of a[m, k] b[n, k]
//
// The scales change every 128 k, so no accumulator may run past a block: each
// k-block's P is its own short MMA chain (4 x K = 32) into a TMEM buffer, and
// the sum over k-blocks is kept in fp32 registers.  A k-block of 128 bytes is
// one 128-byte swizzle row, so the ring is that of the 16-bit kernel with twice
// the k per block.  Per CTA (persistent, one per SM, 128 x BN tiles):
//   warp 0, one lane   TMA producer: 128 rows of A and BN rows of B, kGroup
//                      k-blocks per stage, into an S-stage ring.
//   warp 1, one lane   4 MMAs of 128 x BN x 32 per k-block into the next of the
//                      TMEM buffers; commits free the stage and hand the buffer
//                      to the epilogue.
//   warps 2-3          the scales of the k-blocks ahead, by 4-byte asynchronous
//                      copies (any stride) into a ring of two slots of
//                      kScaleGroup k-blocks each: read straight from global memory
//                      by the epilogue, two k-blocks ahead, their latency cost 180
//                      of 656 us at 8192^3.
//   warps 4-11         epilogue, two warpgroups of BN / 2 columns: TMEM ->
//                      registers, acc += (sa sb) P, or, with a scale per column,
//                      (P sb) sa, and the buffer goes back (fp8.cuh says why in
//                      this order).  A 128 x 256 tile keeps 128 fp32 sums a thread.
//                      (C of 256-wide tiles leaves by TMA from staged boxes, so
//                      that the next tile is summed meanwhile.)
// What bounds it: nothing alone.  A k-block of a 128 x 256 tile takes the tensor
// pipe 512 cycles, the epilogue 256 issue slots of FMAs a scheduler and as many
// cycles of TMEM reads, and two buffers of 256 columns are all the TMEM there is
// to overlap them: 1015 cycles a k-block, 8192^3 in 471 us (2334 TFLOP/s).  With
// a sixteenth of the FMAs 396, a quarter of the MMAs 417, one TMEM read of eight
// 451, a third of the loads 478 of the 487 it then was.  The tile belongs to one
// SM because on CTA pairs (cta_group::2, 256 x 256) each hand-over crosses SMs
// (727 against 656 us with the same, slower epilogue), and the loads that a pair
// would save are not the bound.
// For skinny problems (TRANS: operands swapped, C stored transposed) the bound
// is the stream of the weights.
// Small problems split each tile's k-blocks over a cluster of 2, 4 or 8 CTAs,
// which park their fp32 partial tiles in shared memory and add them through
// distributed shared memory in rank order (a split through global memory with a
// ticket took 16.1 us for 1 x 4096 x 4096, clusters of 4 take 7.5).
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "tc_kernel.cuh"

namespace dg {

constexpr int kF8EpiWarps = 8;
constexpr int kF8RoleWarps = 4;  // producer, MMA issuer, two scale loaders: one warpgroup
constexpr int kF8ScaleThreads = 64;
constexpr int kF8Threads = 32 * (kF8RoleWarps + kF8EpiWarps);
// Registers a thread: 3 warpgroups launch with 168 each (504 in all).  Where the
// epilogue needs more, the role warpgroup gives up all but 40 (its scale loaders then
// spill some 100 bytes, beside the main loop) and the epilogue's two take 232 each (40
// + 2 * 232 = 504): for 256-wide tiles, 128 sums a thread, and for 128-wide ones with a
// scale per column.  Measured, with / without, us: 128-wide with columns' scales, dW of
// 1024^3 8.8 / 11.7, of 1000 x 2000 x 4096 23.2 / 33.7, transposed 128 x 1024 x 8192
// 11.0 / 11.2 but 100 x 4096 x 4096 12.2 / 11.7; with tile scales, which take no part,
// 1001 x 2050 x 4100 18.9 / 18.5, 700 x 2048 x 2048 10.3 / 9.9.
constexpr int kF8RoleRegs = 40, kF8EpiRegs = 232;
template <int BN, bool COLVEC>
constexpr bool kF8SplitRegs = BN == 256 || (BN == 128 && COLVEC);

template <int BN>
struct Fp8TcConfig {
  // k-blocks per stage and TMA copy: an SM's TMA unit takes about as long for a
  // copy of 32 KiB as for one of 16
  static constexpr int kGroup = BN == 256 ? 1 : 2;
  static constexpr int kABytes = kBM * kFp8Block;  // per k-block
  static constexpr int kBBytes = BN * kFp8Block;
  static constexpr int kStageBytes = kGroup * (kABytes + kBBytes);
  // (a fourth stage of 256-wide tiles would take the room of the stores' boxes)
  static constexpr int kStages = BN == 256 ? 3 : BN == 128 ? 3 : BN == 64 ? 4 : 5;
  static constexpr int kBuffers = BN == 256 ? 2 : 4;      // TMEM accumulators
  static constexpr int kTmemCols = BN * kBuffers;         // a power of two >= 32
  static constexpr int kHalf = BN / 2;                    // columns per warpgroup
  // columns per TMEM load (two loads' registers beside 128 sums leave room for 16)
  static constexpr int kChunk = BN == 256 || kHalf < 32 ? 16 : 32;
  static constexpr int kStoreLd = 16 + 4;                 // staged store: 64 bytes a row, in floats
  // a warp's staging: rows of kStoreLd, or two boxes of 32 rows of 128 bytes
  static constexpr int kWarpStage = BN == 256 ? 8192 : 32 * kStoreLd * 4;
  static constexpr int kEpiBytes = kF8EpiWarps * kWarpStage;
  // scales of one k-block: the tile's rows, then its columns
  static constexpr int kScaleGroup = 4;  // k-blocks per ring slot
  static constexpr int kScaleRing = 2;
  static constexpr int kScaleFloats = kBM + BN;
  // a slot: its k-blocks' scales, then a factor for each warpgroup's rows (f8_scales)
  static constexpr int kSlotFloats = kScaleGroup * kScaleFloats + 4;
  static constexpr int kScaleBytes = kScaleRing * kSlotFloats * 4;
  static constexpr int kBarBytes = 384;
  static constexpr int kSmemBytes =
      1024 + kStages * kStageBytes + kEpiBytes + kScaleBytes + kBarBytes;
  // a parked partial tile (BN <= 128): rows (or, transposed, columns) padded by 4 floats
  static constexpr int kParkRow = BN + 4, kParkCol = kBM + 4;
  static_assert(kBM * kParkRow * 4 <= kStages * kStageBytes &&
                BN * kParkCol * 4 <= kStages * kStageBytes, "the ring holds it");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static_assert((2 * kStages + 2 * kBuffers + 1 + 2 * kScaleRing) * 8 + 16 <= kBarBytes,
                "barrier area");
};

// One operand's scales in the MMA view: row (or column) r of k-block kb at
// p[(r >> shift) * stride + kb * kb_stride].
struct Fp8Scales {
  const float* p;
  int64_t stride, kb_stride;
  int32_t shift;
};

struct Fp8TcArgs {
  WorkSpec work;
  int32_t Mm, Nm;      // MMA-view extents
  Fp8Scales row, col;  // of the MMA-view A and B operands
  void* C;             // row-major in the problem's view
  int64_t ldc;
  const float* bias;   // NULL or one per column of C
  int32_t out_dtype;
  int32_t c_vec;       // 1: C's base is 16-byte aligned, its pitch a multiple of 16 bytes
  int32_t c_tma;       // 1: C leaves by TMA (256-wide tiles)
  int32_t a_mn, b_mn;  // 1: the operand is MN-major (b_mn: BN a multiple of 128)
  int32_t k_full;      // whole k-blocks of K
  int* status;
  uint64_t wait_limit_ns;
  uint32_t idesc;
};

// Whether the phase has completed, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One lane of the warp, the same on every call.
__device__ __forceinline__ bool f8_elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[smem desc] · B[smem desc]ᵀ, e4m3 x e4m3 -> fp32, one CTA.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// d += a * b with b straight from a TMEM load.  Volatile, so that it stays
// behind the (volatile) wait for that load, which need not name the registers.
__device__ __forceinline__ void fma_tmem(float& d, float a, uint32_t b) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(d) : "f"(a), "f"(__uint_as_float(b)));
}

// d += (b lo) hi, likewise (scale_order).
__device__ __forceinline__ void fma_tmem2(float& d, float lo, float hi, uint32_t b) {
  asm volatile(
      "{\n\t.reg .f32 t;\n\t"
      "mul.rn.f32 t, %3, %1;\n\t"
      "fma.rn.f32 %0, t, %2, %0;\n\t}"
      : "+f"(d)
      : "f"(lo), "f"(hi), "f"(__uint_as_float(b)));
}

// (x a, y b) with a and b likewise, one instruction.  (A scale per column is a
// product per element on top of the FMA: 104 us instead of 74 at 4096^3.)
__device__ __forceinline__ float2 mul2_tmem(float x, float y, uint32_t a, uint32_t b) {
  float2 r;
  asm volatile(
      "{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%2, %3};\n\t"
      "mov.b64 q, {%4, %5};\n\t"
      "mul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x), "f"(y), "r"(a), "r"(b));
  return r;
}

// Four floats of shared memory, read here and not earlier: loads that the
// compiler moves up cost the registers of the sums.
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// An operand's two tensor maps: `group` brings kGroup whole k-blocks in one
// box (K-major: {128 k, rows}, or for kGroup > 1 the view {128 k, rows,
// k-block}; MN-major: {128 rows, 128 k x kGroup}), `one` a single k-block of a
// K-major operand, zeros past K.
struct Fp8Maps {
  CUtensorMap group, one;
};

// One operand's part of a stage.  A K-major group that reaches into the ragged
// last k-block comes block by block; blocks past K read as zeros.  An MN-major
// operand comes in boxes of 128 rows.
template <int ROWS, int G>
__device__ __forceinline__ void f8_load(const Fp8Maps& m, uint32_t dst, uint32_t bar, int32_t mn,
                                        int32_t row, int32_t kb, int32_t k_full) {
  if (mn) {
#pragma unroll
    for (int i = 0; i < ROWS / 128; ++i)
      tma_load_2d(dst + i * G * 128 * kFp8Block, &m.group, bar, row + i * 128, kb * kFp8Block);
  } else if (G > 1 && kb + G <= k_full) {
    tma_load_3d(dst, &m.group, bar, 0, row, kb);
  } else {
#pragma unroll
    for (int j = 0; j < G; ++j)
      tma_load_2d(dst + j * ROWS * kFp8Block, &m.one, bar, (kb + j) * kFp8Block, row);
  }
}

// TMA producer (one thread).  Returns how many stages it filled.
template <int BN>
__device__ __forceinline__ uint32_t f8_producer(const Fp8Maps& mA, const Fp8Maps& mB,
                                                const Fp8TcArgs& args, uint8_t* sA, uint8_t* sB,
                                                uint64_t* full, uint64_t* empty,
                                                const WaitCtl& wc) {
  using Cfg = Fp8TcConfig<BN>;
  constexpr int G = Cfg::kGroup;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init(W, int32_t(blockIdx.x));
  Unit u;
  int s = 0;
  uint32_t ph = 0, filled = 0;
  pdl_wait_prerequisites();
  while (it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    for (int32_t kb = u.kb0; kb < u.kb1; kb += G) {
      if (!wait_bounded(smem_u32(&empty[s]), ph ^ 1, wc, kSiteProducer)) return filled;
      const uint32_t fb = smem_u32(&full[s]);
      mbar_arrive_expect_tx(fb, Cfg::kStageBytes);
      f8_load<kBM, G>(mA, smem_u32(sA + s * G * Cfg::kABytes), fb, args.a_mn, tm * kBM, kb,
                      args.k_full);
      f8_load<BN, G>(mB, smem_u32(sB + s * G * Cfg::kBBytes), fb, args.b_mn, tn * BN, kb,
                     args.k_full);
      ++filled;
      if (++s == Cfg::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  return filled;
}

// 4 bytes global -> shared, asynchronously.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Scale loaders (64 threads): rows t and t + 64 of the tile and, a warp for each
// warpgroup of the epilogue, its half's columns; rows and columns past the matrix
// clamped to its last, and k-blocks past the unit to its last, so that a slot is
// always whole.  Where 128 columns share a scale only one a warp is needed, and the
// copies' landing arrives on the ring slot's barrier.
// With a scale per column a warp looks its columns over first.  The epilogue
// multiplies a block's sum (up to 2^25) by the column's scale before the row's, so
// columns above 2^103 are taken down by 2^25 and the warpgroup told to take its rows
// up by as much.  (Row times column, whose range takes a look at every pair, cost a
// linear step of 4096^3 326 us instead of 315, 64 x 4096 x 4096 9.0 instead of 8.85.)
constexpr float kColumnMost = 0x1p103f, kColumnDown = 0x1p-25f, kRowUp = 0x1p25f;

template <int BN, bool COLVEC>
__device__ __forceinline__ void f8_scales(const Fp8TcArgs& args, float* ring, uint64_t* sc_full,
                                          uint64_t* sc_empty, const WaitCtl& wc) {
  using Cfg = Fp8TcConfig<BN>;
  constexpr int HC = Cfg::kHalf, kCols = COLVEC ? (HC + 31) / 32 : 1;
  const int t = int(threadIdx.x) - 64, w = t >> 5, lane = t & 31;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init(W, int32_t(blockIdx.x));
  Unit u;
  uint32_t slot = 0, ph = 0;
  bool ok = true;
  pdl_wait_prerequisites();
  // this thread's column i of the tile and its place behind the rows
  auto column = [&](int i) { return w * HC + (COLVEC ? lane + i * 32 : 0); };
  auto place = [&](int i) { return kBM + (COLVEC ? column(i) : w); };
  auto mine = [&](int i) { return COLVEC ? lane + i * 32 < HC : lane == 0; };
  while (ok && it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    // addresses are worked out for every copy: registers are short here
    auto row_at = [&](int i, int32_t kb) {
      const int32_t r = min(tm * kBM + t + i * kF8ScaleThreads, args.Mm - 1);
      return args.row.p + int64_t(r >> args.row.shift) * args.row.stride +
             kb * args.row.kb_stride;
    };
    auto col_at = [&](int i, int32_t kb) {
      const int32_t n = min(tn * BN + column(i), args.Nm - 1);
      return args.col.p + int64_t(n >> args.col.shift) * args.col.stride +
             kb * args.col.kb_stride;
    };
    for (int32_t kb = u.kb0; kb < u.kb1; kb += Cfg::kScaleGroup) {
      // the warp's lanes together: they look the slot over together
      ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(&sc_empty[slot]), ph ^ 1, wc,
                                                kSiteProducer));
      if (!ok) break;
      float* to = ring + slot * Cfg::kSlotFloats;
      uint32_t dst = smem_u32(to);
#pragma unroll 1
      for (int j = 0; j < Cfg::kScaleGroup; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          cp_async4(dst + (t + i * kF8ScaleThreads) * 4, row_at(i, min(kb + j, u.kb1 - 1)));
        }
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if (mine(i)) cp_async4(dst + place(i) * 4, col_at(i, min(kb + j, u.kb1 - 1)));
        dst += Cfg::kScaleFloats * 4;
      }
      if constexpr (COLVEC) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        bool big = false;
#pragma unroll 1
        for (int j = 0; j < Cfg::kScaleGroup; ++j)
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (mine(i)) big |= fabsf(to[j * Cfg::kScaleFloats + place(i)]) > kColumnMost;
        big = __any_sync(0xffffffffu, big);
        if (big) {
#pragma unroll 1
          for (int j = 0; j < Cfg::kScaleGroup; ++j)
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (mine(i)) to[j * Cfg::kScaleFloats + place(i)] *= kColumnDown;
        }
        if (lane == 0) to[Cfg::kScaleGroup * Cfg::kScaleFloats + w] = big ? kRowUp : 1.f;
        mbar_arrive(smem_u32(&sc_full[slot]));
      } else {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&sc_full[slot]))
                     : "memory");
      }
      if (++slot == uint32_t(Cfg::kScaleRing)) {
        slot = 0;
        ph ^= 1;
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// After an abort the MMAs in flight must finish before their TMEM is freed.  Called
// by the issuing warp when every role has ended: the wait that gave up may have been
// a reader's, after the issuer's own last one.
__device__ __forceinline__ void f8_drain(uint32_t drain, const WaitCtl& wc) {
  if (*wc.abort == 0) return;
  if (f8_elect()) {
    tc_commit(drain);
    wait_drain(drain, 0, wc);
  }
  __syncwarp();
}

// MMA issuer: the whole warp runs the loop, so that addresses and descriptors
// stay in uniform registers; one lane issues.  Buffer j of a unit's k-block j
// modulo kBuffers; `phases` holds each buffer's parity.  Whether it issued anything.
template <int BN>
__device__ __forceinline__ bool f8_mma(const Fp8TcArgs& args, uint32_t sA, uint32_t sB,
                                       uint32_t full, uint32_t empty, uint32_t acc_full,
                                       uint32_t acc_empty, const WaitCtl& wc,
                                       uint32_t tmem_base) {
  using Cfg = Fp8TcConfig<BN>;
  constexpr int G = Cfg::kGroup, NB = Cfg::kBuffers;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init(W, int32_t(blockIdx.x));
  Unit u;
  uint32_t s = 0, ph = 0, phases = (1u << NB) - 1;
  bool ok = true, any = false;
  const bool leader = f8_elect();
  // K = 32 steps: 32 bytes along a K-major row, 32 rows of 128 bytes MN-major;
  // k-block j of a group: a block of rows K-major, 128 rows of k MN-major; the
  // 128-row boxes of an MN-major B of 256 rows lie kGroup k-blocks apart
  const uint32_t a_step = args.a_mn ? (4096u >> 4) : (32u >> 4);
  const uint32_t b_step = args.b_mn ? (4096u >> 4) : (32u >> 4);
  const uint32_t b_blk = args.b_mn ? 128u * kFp8Block : uint32_t(Cfg::kBBytes);
  const uint32_t b_lbo = args.b_mn ? uint32_t(G) * 128u * kFp8Block : 16u;
  const uint64_t adesc0 = make_sdesc_sw128(sA, 16, 1024);
  const uint64_t bdesc0 = make_sdesc_sw128(sB, b_lbo, 1024);
  while (ok && it.next(W, u)) {
    uint32_t b = 0;
    for (int32_t kb = u.kb0; ok && kb < u.kb1; kb += G) {
      if (!mbar_test(full + 8 * s, ph)) ok = wait_bounded(full + 8 * s, ph, wc, kSiteMmaFull);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        if (kb + j >= u.kb1) break;  // the unit ends inside the group
        if (!mbar_test(acc_empty + 8 * b, (phases >> b) & 1))
          ok = ok && wait_bounded(acc_empty + 8 * b, (phases >> b) & 1, wc, kSiteMmaAccum);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const uint64_t adesc = adesc0 + ((s * G * Cfg::kABytes + j * Cfg::kABytes) >> 4);
          const uint64_t bdesc = bdesc0 + ((s * G * Cfg::kBBytes + j * b_blk) >> 4);
          const uint32_t d = tmem_base + b * BN;
#pragma unroll
          for (int kk = 0; kk < kFp8Block / 32; ++kk)
            tc_mma_f8(d, adesc + uint64_t(kk * a_step), bdesc + uint64_t(kk * b_step),
                      args.idesc, kk > 0 ? 1u : 0u);
          // the stage's commit first: the epilogue's last wait then covers it
          if (j == G - 1 || kb + j + 1 >= u.kb1) tc_commit(empty + 8 * s);
          tc_commit(acc_full + 8 * b);
        }
        __syncwarp();
        any = true;
        phases ^= 1u << b;
        b = b + 1 == NB ? 0 : b + 1;
      }
      if (++s == uint32_t(Cfg::kStages)) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  return any;
}

// Row-major store of a warp's 32 rows x HC columns (lane i holds row mrow0 + i),
// 64 bytes of each row at a time through the warp's shared rows, so that 4 lanes
// store a row's 64 bytes and an instruction 8 rows.  SIZE: bytes an element.
// The bias is added in fp32 before the one rounding.
template <int HC, int SIZE>
__device__ __forceinline__ void f8_store_rows(const Fp8TcArgs& a, const float (&acc)[HC],
                                              float* stage_w, int32_t mrow0, int lane,
                                              int32_t nn0) {
  constexpr int PER = 64 / SIZE;               // columns a pass
  constexpr int VEC = 16 / SIZE;               // columns a lane stores
  constexpr int LD = 20;                       // floats a staged row
  static_assert(HC % PER == 0, "whole passes");
  const bool f16 = a.out_dtype == GEMM_F16;
  const int piece = lane & 3, rs = lane >> 2;
#pragma unroll
  for (int c = 0; c < HC; c += PER) {
    __syncwarp();                              // the previous pass has been read
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if constexpr (SIZE == 4) {
        const float b = a.bias && nn0 + c + j < a.Nm ? __ldg(a.bias + nn0 + c + j) : 0.f;
        w[j] = __float_as_uint(acc[c + j] + b);
      } else {
        float2 x = make_float2(acc[c + 2 * j], acc[c + 2 * j + 1]);
        if (a.bias) {
          const int32_t n = nn0 + c + 2 * j;
          if (n < a.Nm) x.x += __ldg(a.bias + n);
          if (n + 1 < a.Nm) x.y += __ldg(a.bias + n + 1);
        }
        if (f16) {
          const __half2 h = __floats2half2_rn(x.x, x.y);
          __builtin_memcpy(&w[j], &h, 4);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
          __builtin_memcpy(&w[j], &h, 4);
        }
      }
    }
    uint4* own = reinterpret_cast<uint4*>(stage_w + lane * LD);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      own[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    __syncwarp();
    if (a.c_vec && nn0 + c + PER <= a.Nm) {
      uint4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = *reinterpret_cast<const uint4*>(stage_w + (i * 8 + rs) * LD + 4 * piece);
      const int32_t r0 = mrow0 + rs;
      uint8_t* p = static_cast<uint8_t*>(a.C) +
                   (int64_t(r0) * a.ldc + nn0 + c + piece * VEC) * SIZE;
      const int64_t step = a.ldc * (8 * SIZE);
#pragma unroll
      for (int i = 0; i < 4; ++i, p += step)
        if (r0 + 8 * i < a.Mm) *reinterpret_cast<uint4*>(p) = x[i];
    } else {
      // unaligned rows or the matrix's edge: element by element, neighbouring
      // lanes still on neighbouring columns (16-byte pieces taken apart by one
      // lane each cost 1001 x 2050 x 4100 9 of its 26 us)
      using E = typename std::conditional<SIZE == 4, uint32_t, uint16_t>::type;
      const int col = lane % PER, r0 = lane / PER;
      const E* from = reinterpret_cast<const E*>(stage_w + r0 * LD) + col;
      const bool in = nn0 + c + col < a.Nm;
      E* p = static_cast<E*>(a.C) + int64_t(mrow0 + r0) * a.ldc + nn0 + c + col;
      constexpr int kStep = 32 / PER;          // rows an instruction
#pragma unroll 4
      for (int i = 0; i < 32; i += kStep)
        if (in && mrow0 + r0 + i < a.Mm) p[int64_t(i) * a.ldc] = from[i * (LD * 4 / SIZE)];
    }
  }
}

// The same by TMA, 128 bytes of the 32 rows (a swizzled box) at a time through two
// boxes a warp: the stores drain while the next tile is summed (4096^3 73.2 against
// 76.7 us with f8_store_rows, a linear step of three such products 317 against 327).
// Outside the matrix nothing is stored.
template <int HC, int SIZE>
__device__ __forceinline__ void f8_store_tma(const Fp8TcArgs& a, const CUtensorMap* map,
                                             const float (&acc)[HC], uint32_t stage,
                                             int32_t mrow0, int lane, int32_t nn0) {
  constexpr int PER = 128 / SIZE;              // columns a box
  const bool f16 = a.out_dtype == GEMM_F16;
#pragma unroll
  for (int c = 0; c < HC; c += PER) {
    if (mrow0 >= a.Mm || nn0 + c >= a.Nm) break;
    if (lane == 0) {                           // the box's last store has been read
      if (c == 0) bulk_wait_read_all();
      else if (c >= 2 * PER) bulk_wait_read_1();
    }
    __syncwarp();
    const uint32_t box = stage + uint32_t((c / PER) & 1) * 4096u, row = box + uint32_t(lane) * 128u;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        constexpr int E = 4 / SIZE;            // elements a word
        const int at = c + (4 * k + j) * E;
        float x[2] = {acc[at], E == 2 ? acc[at + E - 1] : 0.f};
        if (a.bias) {
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (nn0 + at + e < a.Nm) x[e] += __ldg(a.bias + nn0 + at + e);
        }
        if constexpr (SIZE == 4) {
          w[j] = __float_as_uint(x[0]);
        } else if (f16) {
          const __half2 h = __floats2half2_rn(x[0], x[1]);
          __builtin_memcpy(&w[j], &h, 4);
        } else {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[0], x[1]);
          __builtin_memcpy(&w[j], &h, 4);
        }
      }
      st_shared_v4(row + uint32_t((k ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, box, nn0 + c, mrow0);
      bulk_commit_group();
    }
  }
}

// CW consecutive fp32 columns of this thread's TMEM lane; the registers may be
// read, by volatile statements, after tmem_wait.
template <int CW>
__device__ __forceinline__ void tmem_issue(uint32_t taddr, uint32_t (&r)[CW]) {
  if constexpr (CW == 32) {
    tmem_ld32(taddr, r);
  } else {
    static_assert(CW == 16, "chunk width");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}
__device__ __forceinline__ void tmem_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

template <int BN, bool TRANS, bool COLVEC, bool OUT32>
__device__ __forceinline__ void f8_epilogue(const Fp8TcArgs& args, const CUtensorMap* tmC,
                                            uint32_t acc_full,
                                            uint32_t acc_empty, uint32_t sc_full,
                                            uint32_t sc_empty, const WaitCtl& wc,
                                            uint32_t tmem_base, float* stage, const float* ring,
                                            float* park) {
  using Cfg = Fp8TcConfig<BN>;
  constexpr int HC = Cfg::kHalf, CW = Cfg::kChunk;
  const WorkSpec& W = args.work;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;               // TMEM lane quarter this warp may access
  const int wg = (warp - kF8RoleWarps) >> 2;       // which half of the columns
  const int row = q * 32 + lane;
  float* stage_w = stage + (warp - kF8RoleWarps) * (Cfg::kWarpStage / 4);
  WorkIter it;
  const int32_t cta = int32_t(blockIdx.x);
  it.init(W, cta);
  pdl_wait_prerequisites();
  Unit u;
  // buffer j % kBuffers holds the unit's k-block j; `phases`: each buffer's parity
  uint32_t phases = 0, slot = 0, sph = 0;
  bool ok = true;
  const uint32_t tlane = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(wg * HC);
  while (it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    const int32_t mrow0 = tm * kBM;
    const int32_t mm = mrow0 + row;
    const int32_t nn0 = tn * BN + wg * HC;
    float acc[HC];
#pragma unroll
    for (int j = 0; j < HC; ++j) acc[j] = 0.f;
    // kScaleGroup k-blocks a turn, unrolled, so that buffers and chunks are
    // constants.  Chunk c + 1 of a buffer is loaded while chunk c is added (NV = 2),
    // but not where 128 sums and one scale for all columns leave it to the other
    // warp to fill the wait (8192^3 476 against 484 us).
    // (Asking for the next buffer a chunk ahead, to load its first chunk early,
    // was slower: 561 against 520 us at 8192^3, all else equal.)  After a wait gave up the loop
    // runs on to its end on whatever it reads, each further wait returning at
    // once; the tile is then not stored.
    constexpr int NV = BN == 256 && !COLVEC ? 1 : 2;
    constexpr int NC = HC / CW, NB = Cfg::kBuffers, SG = Cfg::kScaleGroup;
    static_assert(SG % NB == 0 && (NC == 1 || NC % 2 == 0), "constant buffers and chunks");
    uint32_t v[NV][CW];
    // waits for buffer i's product and sends its first chunk on its way
    auto begin = [&](int i) {
      ok &= wait_bounded(acc_full + 8 * i, (phases >> i) & 1, wc, kSiteEpilogue);
      tc_fence_after();
      if (NV == 2) tmem_issue<CW>(tlane + uint32_t(i * BN), v[0]);
    };
    begin(0);
    int32_t kb = u.kb0;
    bool odd = false;
    for (; kb < u.kb1; kb += SG) {
      ok &= wait_bounded(sc_full + 8 * slot, sph, wc, kSiteEpilogue);
      const float* sc = ring + slot * Cfg::kSlotFloats;
      const uint32_t sc_at = smem_u32(sc + wg * HC);
      float rs[SG];
      const float up = COLVEC ? sc[SG * Cfg::kScaleFloats + wg] : 1.f;
#pragma unroll
      for (int j = 0; j < SG; ++j) {
        rs[j] = sc[j * Cfg::kScaleFloats + row];
        if (COLVEC) {
          rs[j] *= up;
        } else {
          rs[j] *= sc[j * Cfg::kScaleFloats + kBM + wg];
        }
      }
      if constexpr (!COLVEC) {
        static_assert(SG == 4, "the four of a slot");
        const float a0 = fabsf(rs[0]), a1 = fabsf(rs[1]), a2 = fabsf(rs[2]), a3 = fabsf(rs[3]);
        const float most = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3));
        const float least = fminf(fminf(a0, a1), fminf(a2, a3));
        odd = __any_sync(0xffffffffu, !(scale_fits(most) && scale_fits(least)));
        if (__builtin_expect(odd, 0)) break;
      }
#pragma unroll
      for (int j = 0; j < SG; ++j) {
        if (kb + j >= u.kb1) break;
        const int i = j % NB, next = (j + 1) % NB;
        phases ^= 1u << i;
        if (NV == 2) tmem_wait();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (NV == 1) {
            tmem_issue<CW>(tlane + uint32_t(i * BN + c * CW), v[0]);
            tmem_wait();
          }
          if (NV == 2 && c + 1 < NC) {
            tmem_issue<CW>(tlane + uint32_t(i * BN + (c + 1) * CW), v[(c + 1) & (NV - 1)]);
          } else if (c + 1 == NC) {  // the buffer's last read is done: back to the MMA issuer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8 * i);
          }
          float* d = acc + c * CW;
          const uint32_t* x = v[c & (NV - 1)];
          if constexpr (COLVEC) {
            const uint32_t cs = sc_at + uint32_t(j * Cfg::kScaleFloats + kBM + c * CW) * 4;
#pragma unroll
            for (int e = 0; e < CW; e += 4) {
              const float4 s4 = lds4(cs + e * 4);
              const float2 lo = mul2_tmem(s4.x, s4.y, x[e], x[e + 1]);
              const float2 hi = mul2_tmem(s4.z, s4.w, x[e + 2], x[e + 3]);
              d[e] = fmaf(lo.x, rs[j], d[e]);
              d[e + 1] = fmaf(lo.y, rs[j], d[e + 1]);
              d[e + 2] = fmaf(hi.x, rs[j], d[e + 2]);
              d[e + 3] = fmaf(hi.y, rs[j], d[e + 3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < CW; ++e) fma_tmem(d[e], rs[j], x[e]);
          }
          if (NV == 2 && c + 1 < NC) tmem_wait();
        }
        if (kb + j + 1 < u.kb1) begin(next);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(sc_empty + 8 * slot);
      if (++slot == uint32_t(Cfg::kScaleRing)) {
        slot = 0;
        sph ^= 1;
      }
    }
    if constexpr (!COLVEC) {
      if (__builtin_expect(odd, 0)) {
        // From a slot on with scale products that fp32 cannot hold: the scale of smaller
        // magnitude first.  (A loop of its own: a branch in the one above cost it 30 of
        // 470 us.)
        if (NV == 2) tmem_wait();  // the chunk under way is read again
        const int32_t odd0 = kb;
#pragma unroll 1
        for (; kb < u.kb1; ++kb) {
          const int j = (kb - odd0) % SG, i = j % NB;
          if (kb > odd0) {
            if (j == 0) ok &= wait_bounded(sc_full + 8 * slot, sph, wc, kSiteEpilogue);
            ok &= wait_bounded(acc_full + 8 * i, (phases >> i) & 1, wc, kSiteEpilogue);
            tc_fence_after();
          }
          phases ^= 1u << i;
          const float* s = ring + slot * Cfg::kSlotFloats + j * Cfg::kScaleFloats;
          float lo, hi;
          scale_order(s[row], s[kBM + wg], lo, hi);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            tmem_issue<CW>(tlane + uint32_t(i * BN + c * CW), v[0]);
            tmem_wait();
#pragma unroll
            for (int e = 0; e < CW; ++e) fma_tmem2(acc[c * CW + e], lo, hi, v[0][e]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty + 8 * i);
          if (j == SG - 1 || kb + 1 == u.kb1) {
            if (lane == 0) mbar_arrive(sc_empty + 8 * slot);
            if (++slot == uint32_t(Cfg::kScaleRing)) {
              slot = 0;
              sph ^= 1;
            }
          }
        }
      }
    }

    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const float* bias = args.bias;
    if (BN <= 128 && W.csplit > 1) {
      // The CTA's only unit: its MMAs have read the ring and every copy into it
      // has landed, so the partial tile may take its place.  Columns are kept
      // together for the transposed store, rows otherwise.
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
        const float bv = bias ? __ldg(bias + mm) : 0.f;
#pragma unroll
        for (int j = 0; j < HC; ++j)
          if (nn0 + j < args.Nm)
            store_typed(args.C, int64_t(nn0 + j) * args.ldc + mm,
                        acc[j] + bv, args.out_dtype);
      }
    } else {
      constexpr int SIZE = OUT32 ? 4 : 2;
      if (BN == 256 && args.c_tma)
        f8_store_tma<HC, SIZE>(args, tmC, acc, smem_u32(stage_w), mrow0 + q * 32, lane, nn0);
      else
        f8_store_rows<HC, SIZE>(args, acc, stage_w, mrow0 + q * 32, lane, nn0);
    }
  }
  // every store this warp issued has landed before the CTA moves on
  if (BN == 256 && lane == 0) bulk_wait_all();
}

// Four neighbouring outputs of a row of C, `valid` of them inside the matrix.
__device__ __forceinline__ void f8_store4(const Fp8TcArgs& a, int64_t off, const float (&v)[4],
                                          int valid) {
  if (valid >= 4 && a.c_vec) {
    if (a.out_dtype == GEMM_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.C) + off) =
          make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint2 pk;
      if (a.out_dtype == GEMM_F16) {
        const __half2 x = __floats2half2_rn(v[0], v[1]), y = __floats2half2_rn(v[2], v[3]);
        __builtin_memcpy(&pk.x, &x, 4);
        __builtin_memcpy(&pk.y, &y, 4);
      } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]);
        const __nv_bfloat162 y = __floats2bfloat162_rn(v[2], v[3]);
        __builtin_memcpy(&pk.x, &x, 4);
        __builtin_memcpy(&pk.y, &y, 4);
      }
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.C) + off) = pk;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < valid) store_typed(a.C, off + j, v[j], a.out_dtype);
}

// Cluster split, after every CTA of the cluster has parked its partial: the
// tile's valid outputs, four neighbours at a time, are dealt to the cluster's
// threads; each adds the partials in rank order and stores.  8 remote loads a
// thread are in flight (one quad at a time cost 6 us of a 128 x 128 tile split
// in two).
template <int BN, bool TRANS, int SPLIT>
__device__ __forceinline__ void f8_cluster_reduce(const Fp8TcArgs& a, uint32_t park) {
  using Cfg = Fp8TcConfig<BN>;
  constexpr int kThreads = 32 * kF8EpiWarps, U = 8 / SPLIT;
  const int32_t tile = int32_t(blockIdx.x) / SPLIT;
  const int rank = int(blockIdx.x) % SPLIT;
  int32_t tm, tn;
  tile_coords(a.work, tile, tm, tn);
  const int rows = min(kBM, a.Mm - tm * kBM), cols = min(BN, a.Nm - tn * BN);
  // quads run along C's rows: the tile's columns, or its rows when transposed
  const int per = TRANS ? (rows + 3) / 4 : (cols + 3) / 4;
  const int total = per * (TRANS ? cols : rows);
  uint32_t peer[SPLIT];
#pragma unroll
  for (int r = 0; r < SPLIT; ++r) peer[r] = map_to_rank(park, uint32_t(r));
  for (int i0 = rank * kThreads + int(threadIdx.x) - 32 * kF8RoleWarps; i0 < total;
       i0 += U * SPLIT * kThreads) {
    float4 x[U][SPLIT];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = min(i0 + k * SPLIT * kThreads, total - 1);
      const int line = i / per, q = (i - line * per) * 4;
      const uint32_t at = uint32_t(line * (TRANS ? Cfg::kParkCol : Cfg::kParkRow) + q) * 4;
#pragma unroll
      for (int r = 0; r < SPLIT; ++r) x[k][r] = ld_dsmem_f32x4(peer[r] + at);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * SPLIT * kThreads;
      if (i >= total) break;
      const int line = i / per, q = (i - line * per) * 4;
      float v[4] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w};
#pragma unroll
      for (int r = 1; r < SPLIT; ++r) {
        v[0] += x[k][r].x; v[1] += x[k][r].y; v[2] += x[k][r].z; v[3] += x[k][r].w;
      }
      // C row and first column in the problem's view
      const int64_t crow = TRANS ? tn * BN + line : tm * kBM + line;
      const int32_t c0 = TRANS ? tm * kBM + q : tn * BN + q;
      const int valid = (TRANS ? a.Mm : a.Nm) - c0;
      if (a.bias)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < valid) v[j] += __ldg(a.bias + c0 + j);
      f8_store4(a, crow * a.ldc + c0, v, valid);
    }
  }
}

// args.work counts 128 x BN tiles and CTAs.  COLVEC: a scale per column, not per
// 128; OUT32: fp32 output (the transposed store takes any type).
template <int BN, bool TRANS, bool COLVEC, bool OUT32>
__global__ void __launch_bounds__(kF8Threads, 1)
    fp8_tc_kernel(const __grid_constant__ Fp8Maps mA, const __grid_constant__ Fp8Maps mB,
                  const __grid_constant__ CUtensorMap tmC, const Fp8TcArgs args) {
  using Cfg = Fp8TcConfig<BN>;
  constexpr int S = Cfg::kStages, NB = Cfg::kBuffers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * Cfg::kGroup * Cfg::kABytes;
  float* stage = reinterpret_cast<float*>(sB + S * Cfg::kGroup * Cfg::kBBytes);
  float* ring = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(stage) + Cfg::kEpiBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(ring) +
                                               Cfg::kScaleBytes);
  uint64_t* full = bars;                // S: a stage's bytes have landed
  uint64_t* empty = bars + S;           // S: its MMAs are done
  uint64_t* acc_full = empty + S;       // NB: a k-block's product is in TMEM
  uint64_t* acc_empty = acc_full + NB;  // NB: all epilogue warps have read it
  uint64_t* sc_full = acc_empty + NB;   // kScaleRing: a k-block's scales have landed
  uint64_t* sc_empty = sc_full + Cfg::kScaleRing;  // kScaleRing: all epilogue warps used them
  uint64_t* drain = sc_empty + Cfg::kScaleRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // uniform
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), kF8EpiWarps);
    }
    for (int i = 0; i < Cfg::kScaleRing; ++i) {
      mbar_init(smem_u32(&sc_full[i]), kF8ScaleThreads);
      mbar_init(smem_u32(&sc_empty[i]), kF8EpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_map(&mA.group);
    tma_prefetch_map(&mB.group);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  const WaitCtl wc{args.wait_limit_ns, args.status, abort_flag};

  uint32_t filled = 0;
  bool issued = false;
  if (warp >= kF8RoleWarps) {
    if constexpr (kF8SplitRegs<BN, COLVEC>)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8EpiRegs));
    f8_epilogue<BN, TRANS, COLVEC, OUT32>(args, &tmC, smem_u32(acc_full), smem_u32(acc_empty),
                                   smem_u32(sc_full), smem_u32(sc_empty), wc, tmem_base, stage,
                                   ring, reinterpret_cast<float*>(smem));
  } else {
    if constexpr (kF8SplitRegs<BN, COLVEC>)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RoleRegs));
    if (warp == 0 && lane == 0) {
      filled = f8_producer<BN>(mA, mB, args, sA, sB, full, empty, wc);
    } else if (warp == 1) {
      pdl_wait_prerequisites();
      issued = f8_mma<BN>(args, smem_u32(sA), smem_u32(sB), smem_u32(full), smem_u32(empty),
                          smem_u32(acc_full), smem_u32(acc_empty), wc, tmem_base);
    } else if (warp >= 2) {
      f8_scales<BN, COLVEC>(args, ring, sc_full, sc_empty, wc);
    } else {
      pdl_wait_prerequisites();
    }
  }
  // after an abort, copies may still be in flight: each stage's last one
  if (threadIdx.x == 0)
    for (uint32_t s = 0; s < uint32_t(S) && s < filled; ++s)
      wait_drain(smem_u32(&full[s]), ((filled - 1 - s) / S) & 1, wc);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (issued) f8_drain(smem_u32(drain), wc);
    tc_fence_after();
    tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
  if (BN <= 128 && args.work.csplit > 1) {
    cluster_sync_all();  // every partial of the cluster is parked
    if (warp >= kF8RoleWarps) {
      const uint32_t park = smem_u32(smem);
      if (args.work.csplit == 2) f8_cluster_reduce<BN, TRANS, 2>(args, park);
      else if (args.work.csplit == 4) f8_cluster_reduce<BN, TRANS, 4>(args, park);
      else f8_cluster_reduce<BN, TRANS, 8>(args, park);
    }
    cluster_sync_all();  // no CTA leaves while another reads its partial
  }
}

}  // namespace dg

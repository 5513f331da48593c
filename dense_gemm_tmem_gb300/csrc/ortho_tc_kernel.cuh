// ortho_tc_kernel.cuh: all products of the orthogonalising call in one launch, on the
// tensor cores (tcgen05.mma.kind::f16, fp32 sums in TMEM).  Each step is
//   kGram   A16 = half(alpha X·Xᵀ)               symmetric
//   kPoly   B16 = half(alpha A·Aᵀ + beta A)      symmetric
//   kApply  X   = alpha B·X + beta X             (or X·B), fp32, and its 16-bit copy
// for every matrix of the batch.  Of a symmetric result only the tiles on and below the
// diagonal blocks are computed, which takes the step from 4 to 3 m^2 n + m^3 flops, and
// stored: where a product reads A above the diagonal, it loads the mirrored block and the
// MMAs take that operand MN-major.  (Stored twice, a tile's epilogue took twice as long.)
// X lies as it lies too: Xᵀ is never formed.  Rows are padded with zeros to 64 elements,
// so a k-block is always whole.
//
// The tiles of all products are laid end to end (step, product, matrix, row by row) and
// dealt to the CTAs in turn.  A tile waits only for the tiles it reads: each tile has a
// counter that its epilogue warps raise, and a tile's loads along K go as far as the
// counters allow, so that the next product starts while the last tiles of this one are
// computed and stored.
// A tile's counters belong to tiles before it in the order and all CTAs are resident
// (cooperative launch), so every wait ends.  What a tile overwrites has no reader left by
// then: A(i, j) was read by tiles of kPoly in rows i and j, which all of X's rows i and j
// have waited for; all of B by kApply tiles that all of A has waited for; the 16-bit copy
// of X that kApply writes is not the one it reads, and the step that read it is over.
//   warp 0, one lane   TMA producer, two k-blocks per stage (an SM's TMA unit takes
//                      about as long for a copy of 32 KiB as for one of 16)
//   warp 1, one lane   MMAs into one of two accumulators
//   warp 2             watches the counters of what the next loads read
//   warps 4-11         epilogue, two warpgroups of half the columns each, beside the
//                      next tile's MMAs
// Two CTAs on two SMs own a 256 x 256 or a 256 x 128 tile (cta_group::2), or one CTA a
// 128 x 64 tile: ortho_tc.cu says which when.
//
// What bounds it.  4096^2 (988 us, 1.39 PFLOP/s of the flops counted): the MMAs, 640 cycles
// a k-block of 256 x 256 as in the library's other products, 23 to 26 us a tile beside the
// last one's epilogue; 528 tiles a step on 76 pairs are 6.95 each, 8 us a step are waits.
// Smaller matrices: the chain of 15 products, each of which costs, after its MMAs, the
// epilogue (1.1 us for 32 columns a warp), 0.8 to 1.7 us until its stores are acknowledged,
// 0.9 until another SM has seen the counter and 0.9 for the first loads: 7 us a product for
// 512^2, 15 for 2048^2.  With one short side kGram has a tile or a few, each of which
// walks all of the long side alone: 64 x 4096 165 us, 128 x 4096 176, 16 x 16384 433.  (A
// launch a product took 8 and 17, 4096^2 1030.)  Measured and dropped: results stored
// twice instead of read mirrored (512^2 149 us against 113), 16 bytes a lane straight from
// registers (10 x 700 x 1000 251 against 228), TMA stores (235), two copies for an
// MN-major operand (228 against 225), a fence after relaxed polls (225 against 223).
#pragma once

#include "fp8_tc_kernel.cuh"
#include "ortho.cuh"
#include "tc2_kernel.cuh"

namespace dg {

constexpr int kOrRoleWarps = 4, kOrEpiWarps = 8;
constexpr int kOrThreads = 32 * (kOrRoleWarps + kOrEpiWarps);
// Registers a thread: 3 warpgroups launch with 168 each (504 in all); the roles keep 56,
// the epilogue's two take 224 each, for the chunk that is sent for ahead.  (Compiled for
// 168, the kernels spill a little, -Xptxas -v: 88 bytes stored and 72 loaded in 256-wide
// tiles, 32 and 56 in 128-wide, 24 and 48 in 64-wide ones.)
constexpr int kOrRoleRegs = 56, kOrEpiRegs = 224;
constexpr int kOrGroup = 2;   // k-blocks of 64 per stage

template <bool PAIR_, int TN>
struct OrConfig {
  static constexpr bool kPair = PAIR_;
  static constexpr int kTileM = kPair ? 256 : 128, kTileN = TN;
  static constexpr int kRatio = kTileM / kTileN;          // tiles along a diagonal block's row
  static constexpr int kBRows = kPair ? TN / 2 : TN;      // of B that a CTA loads
  static constexpr int kABlock = 128 * 128;               // bytes of a k-block of A
  static constexpr int kBBlock = kBRows * 128;
  static constexpr int kABytes = kOrGroup * kABlock;
  static constexpr int kStageBytes = kABytes + kOrGroup * kBBlock;
  static constexpr int kStages = kBRows > 64 ? 3 : 4;
  static constexpr int kTmemCols = 2 * kTileN;
  static constexpr int kHalf = kTileN / 2;                // columns per warpgroup
  static constexpr int kPieceBlocks = kTileM / kBK;       // k-blocks of a piece of K
  static constexpr int kEpiBytes = kOrEpiWarps * 4096;    // 32 x 32 floats a warp
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiBytes + kBarBytes;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static_assert(kPieceBlocks % kOrGroup == 0, "a stage's k-blocks lie in one piece");
};

struct OrTcArgs {
  int32_t batch, steps, owners, tall;
  int32_t tiles_r, tiles_c;   // of X
  int32_t per_sym, per_apply; // tiles of one matrix that are computed
  int32_t kb_gram, kb_n;      // k-blocks of 64: of kGram, and of n
  int32_t rows, cols, n;
  int64_t ld_x, ld_a, stride_x, stride_a;
  __half *x16[2], *a16, *b16; // step i reads x16[i & 1]
  float* x32;
  void* out;
  int64_t ld_out, stride_out;
  int32_t out_vec;            // 8-byte stores of `out`
  uint32_t* done;             // a counter per tile, kApply's per_apply apart
  int64_t done_stride;        // counters of one product (all matrices)
  int* status;
  uint64_t wait_limit_ns;
  OrthoStep step[GEMM_ORTHO_MAX_STEPS];
};

// An operand's maps: boxes of 128 rows (the MMA's A) and of OrConfig's kBRows (its B) by two
// blocks of 64 columns, and of 128 rows by one.
struct OrOperand {
  CUtensorMap ka, kb, mn;
};
struct OrMaps {
  OrOperand x[2], a, b;
};

// One tile: where it is in the order.
struct OrTile {
  int32_t step, kind, z, tm, tn;
};
template <class Cfg>
__device__ __forceinline__ OrTile or_tile(const OrTcArgs& a, int64_t t) {
  constexpr int R = Cfg::kRatio;
  OrTile o;
  const int64_t sym = int64_t(a.per_sym) * a.batch, per = 2 * sym + int64_t(a.per_apply) * a.batch;
  o.step = int32_t(t / per);
  int64_t r = t - o.step * per;
  o.kind = r < sym ? kGram : r < 2 * sym ? kPoly : kApply;
  r -= o.kind * sym;
  const int32_t count = o.kind == kApply ? a.per_apply : a.per_sym;
  o.z = int32_t(r / count);
  const int32_t x = int32_t(r - int64_t(o.z) * count);
  if (o.kind != kApply) {  // row by row: R (i + 1) tiles in row i
    int32_t i = int32_t((sqrtf((8.f / R) * float(x) + 1.f) - 1.f) * 0.5f);
    while (R * (i * (i + 1) / 2) > x) --i;
    while (R * ((i + 1) * (i + 2) / 2) <= x) ++i;
    o.tm = i;
    o.tn = x - R * (i * (i + 1) / 2);
  } else if (!a.tall) {    // the order in which the next kGram wants X
    o.tm = x / a.tiles_c;
    o.tn = x - o.tm * a.tiles_c;
  } else {
    o.tn = x / a.tiles_r;
    o.tm = x - o.tn * a.tiles_r;
  }
  return o;
}
__device__ __forceinline__ int64_t or_total(const OrTcArgs& a) {
  return (2 * int64_t(a.per_sym) + a.per_apply) * a.batch * a.steps;
}
template <class Cfg>
__device__ __forceinline__ int32_t or_pieces(const OrTcArgs& a, int32_t kind) {
  constexpr int P = Cfg::kPieceBlocks;
  return ((kind == kGram ? a.kb_gram : a.kb_n) + P - 1) / P;
}
__device__ __forceinline__ int32_t or_k_blocks(const OrTcArgs& a, int32_t kind) {
  return kind == kGram ? a.kb_gram : a.kb_n;
}
// The counters of one product of one matrix.
__device__ __forceinline__ uint32_t* or_counters(const OrTcArgs& a, int32_t step, int32_t kind,
                                                 int32_t z) {
  return a.done + (int64_t(step) * 3 + kind) * a.done_stride +
         int64_t(z) * (kind == kApply ? a.per_apply : a.per_sym);
}
// Tile (tm, tn)'s place among them.
template <class Cfg>
__device__ __forceinline__ int32_t or_index(const OrTcArgs& a, int32_t kind, int32_t tm,
                                            int32_t tn) {
  if (kind != kApply) return Cfg::kRatio * (tm * (tm + 1) / 2) + tn;
  return a.tall ? tn * a.tiles_r + tm : tm * a.tiles_c + tn;
}
// Which way the MMA's operands of a piece lie: bit 0 A MN-major, bit 1 B.  Block (i, p) of
// A16 or B16 above the diagonal is the mirrored (p, i).
template <class Cfg>
__device__ __forceinline__ int or_majors(const OrTcArgs& a, const OrTile& o, int32_t p) {
  constexpr int R = Cfg::kRatio;
  if (o.kind == kGram) return a.tall ? 3 : 0;
  const int i = p > o.tm, j = p > o.tn / R;
  if (o.kind == kPoly) return i | (j << 1);
  return a.tall ? j << 1 : i | 2;
}
__device__ __forceinline__ uint32_t ld_acquire_gpu(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release_gpu(uint32_t* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
// Between the epilogues' stores of global memory and the copies that read it.
__device__ __forceinline__ void fence_proxy_async_all() {
  asm volatile("fence.proxy.async;" ::: "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t c0, int32_t c1,
                                                 int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Whether block (i, p) of a symmetric result, or the mirrored one, is stored.
template <class Cfg>
__device__ __forceinline__ bool or_block_done(const OrTcArgs& a, const uint32_t* counters,
                                              int32_t i, int32_t p) {
  constexpr int R = Cfg::kRatio;
  constexpr uint32_t kFull = kOrEpiWarps * (Cfg::kPair ? 2 : 1);
  const uint32_t* c = counters + or_index<Cfg>(a, kPoly, max(i, p), R * min(i, p));
  bool have = true;
#pragma unroll
  for (int r = 0; r < R; ++r) have &= ld_acquire_gpu(c + r) >= kFull;
  return have;
}
// Whether X's tiles in row tm, or R of them from column R j on (those there are), are.
template <class Cfg>
__device__ __forceinline__ bool or_x_done(const OrTcArgs& a, const uint32_t* counters, int32_t tm,
                                          int32_t tn, int32_t count) {
  constexpr uint32_t kFull = kOrEpiWarps * (Cfg::kPair ? 2 : 1);
  bool have = true;
  for (int r = 0; r < count; ++r)
    have &= ld_acquire_gpu(counters + or_index<Cfg>(a, kApply, tm, tn + r)) >= kFull;
  return have;
}

// Watches the counters of what this CTA's tiles read (one warp): `ready` counts the tiles'
// K in pieces of kTileM, as far as they may be loaded.
template <class Cfg>
__device__ __forceinline__ void or_watch(const OrTcArgs& args, volatile uint32_t* ready,
                                         const WaitCtl& wc, int32_t owner) {
  constexpr int R = Cfg::kRatio;
  const int lane = threadIdx.x & 31;
  uint32_t passed = 0;
  pdl_wait_prerequisites();
  for (int64_t t = owner; t < or_total(args); t += args.owners) {
    const OrTile o = or_tile<Cfg>(args, t);
    const int32_t pieces = or_pieces<Cfg>(args, o.kind);
    if (o.kind == kGram && o.step == 0) {
      passed += pieces;
      if (lane == 0) *ready = passed;
      continue;
    }
    const uint32_t* const counters =
        o.kind == kGram ? or_counters(args, o.step - 1, kApply, o.z)
                        : or_counters(args, o.step, o.kind - 1, o.z);
    for (int32_t p0 = 0; p0 < pieces; p0 += 32) {
      const int32_t p = min(p0 + lane, pieces - 1), count = min(32, pieces - p0);
      auto look = [&]() {
        if (o.kind == kGram) {  // the rows (or columns) of X that the tile multiplies
          if (args.tall)
            return or_x_done<Cfg>(args, counters, p, R * o.tm,
                                   min(R, args.tiles_c - R * o.tm)) &&
                   or_x_done<Cfg>(args, counters, p, o.tn, o.tn < args.tiles_c);
          const int32_t there = min(R, args.tiles_c - R * p);
          return or_x_done<Cfg>(args, counters, o.tm, R * p, there) &&
                 or_x_done<Cfg>(args, counters, o.tn / R, R * p, there);
        }
        if (o.kind == kPoly)    // the rows of A
          return or_block_done<Cfg>(args, counters, o.tm, p) &&
                 or_block_done<Cfg>(args, counters, o.tn / R, p);
        // the rows of B; X is complete where B is
        return or_block_done<Cfg>(args, counters, args.tall ? o.tn / R : o.tm, p);
      };
      bool have = false;
      int32_t seen = 0;
      uint64_t t0 = 0;
      while (seen < count) {
        if (!have) have = look();
        const uint32_t all = __ballot_sync(0xffffffffu, have);
        const int32_t now = all == 0xffffffffu ? count : min(count, __ffs(~all) - 1);
        if (now > seen) {
          seen = now;
          __syncwarp();  // every lane's acquire before the count is published
          __threadfence_block();
          if (lane == 0) *ready = passed + uint32_t(seen);
          t0 = 0;
        } else if (t0 == 0) {
          t0 = globaltimer_ns();
        } else {
          bool stop = *wc.abort != 0;
          if (globaltimer_ns() - t0 > wc.limit_ns) {
            if (lane == 0) {
              *wc.abort = 1;
              atomicCAS(wc.status, 0, 1 + kSiteProducer);
            }
            stop = true;
          }
          if (__any_sync(0xffffffffu, stop)) return;
        }
      }
      passed += uint32_t(count);
    }
  }
}

// Until `ready` reaches `want` (bounded).
__device__ __forceinline__ bool or_wait_ready(const volatile uint32_t* ready, uint32_t want,
                                              const WaitCtl& wc) {
  if (int32_t(*ready - want) < 0) {
    const uint64_t t0 = globaltimer_ns();
    while (int32_t(*ready - want) < 0) {
      if (*wc.abort) return false;
      if (globaltimer_ns() - t0 > wc.limit_ns) {
        *wc.abort = 1;
        atomicCAS(wc.status, 0, 1 + kSiteProducer);
        return false;
      }
    }
  }
  __threadfence_block();
  return true;
}

// TMA producer (one thread).  Returns how many stages it filled.
template <class Cfg>
__device__ __forceinline__ uint32_t or_producer(const OrMaps& maps, const OrTcArgs& args,
                                                uint32_t ring, uint64_t* full, uint64_t* empty,
                                                const volatile uint32_t* ready,
                                                const WaitCtl& wc, uint32_t rank, int32_t owner) {
  int s = 0;
  uint32_t ph = 0, filled = 0, passed = 0;
  pdl_wait_prerequisites();
  for (int64_t t = owner; t < or_total(args); t += args.owners) {
    const OrTile o = or_tile<Cfg>(args, t);
    const int32_t a_row = o.tm * Cfg::kTileM + int32_t(rank) * 128;
    const int32_t b_row = o.tn * Cfg::kTileN + int32_t(rank) * Cfg::kBRows;
    const int32_t k_blocks = or_k_blocks(args, o.kind);
    const OrOperand& x = maps.x[o.step & 1];
    const OrOperand& mA = o.kind == kGram ? x : o.kind == kPoly ? maps.a : args.tall ? x : maps.b;
    const OrOperand& mB = o.kind == kGram ? x : o.kind == kPoly ? maps.a : args.tall ? maps.b : x;
    int majors = 0;
    for (int32_t kb = 0; kb < k_blocks; kb += kOrGroup) {
      if (kb % Cfg::kPieceBlocks == 0) {
        if (!or_wait_ready(ready, ++passed, wc)) return filled;
        fence_proxy_async_all();
        majors = or_majors<Cfg>(args, o, kb / Cfg::kPieceBlocks);
      }
      if (!wait_bounded(smem_u32(&empty[s]), ph ^ 1, wc, kSiteProducer)) return filled;
      const uint32_t own = smem_u32(&full[s]);
      if (rank == 0) mbar_arrive_expect_tx(own, (Cfg::kPair ? 2 : 1) * Cfg::kStageBytes);
      // K-major: 128 (or kBRows) rows of two k-blocks; MN-major: two blocks of 64 columns,
      // 128 rows of K deep, which is the same box, or one block where kBRows is 64
      auto load4 = [&](uint32_t dst, const CUtensorMap* map, int32_t row, int32_t block) {
        if constexpr (Cfg::kPair)
          tma_load_4d_pair(dst, map, map_to_rank(own, 0), 0, row, block, o.z);
        else
          tma_load_4d(dst, map, own, 0, row, block, o.z);
      };
      auto load3 = [&](uint32_t dst, const CUtensorMap* map, int32_t row) {
        if constexpr (Cfg::kPair) tma_load_3d_pair(dst, map, map_to_rank(own, 0), row, kb * kBK, o.z);
        else tma_load_3d(dst, map, own, row, kb * kBK, o.z);
      };
      const uint32_t a_dst = ring + uint32_t(s) * Cfg::kStageBytes, b_dst = a_dst + Cfg::kABytes;
      if (majors & 1) load4(a_dst, &mA.ka, kb * kBK, a_row / 64);
      else load4(a_dst, &mA.ka, a_row, kb);
      if (!(majors & 2)) load4(b_dst, &mB.kb, b_row, kb);
      else if (Cfg::kBRows > 64) load4(b_dst, &mB.kb, kb * kBK, b_row / 64);
      else load3(b_dst, &mB.mn, b_row);
      ++filled;
      if (++s == Cfg::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  return filled;
}

// MMA issuer (one thread).  Whether it issued anything.
template <class Cfg>
__device__ __forceinline__ bool or_mma(const OrTcArgs& args, uint32_t ring, uint64_t* full,
                                       uint64_t* empty, uint64_t* acc_full, uint64_t* acc_empty,
                                       const WaitCtl& wc, uint32_t tmem_base, int32_t owner) {
  int s = 0, b = 0;
  uint32_t ph = 0, aph = 1;
  bool any = false;
  auto commit = [&](uint64_t* bar) {
    if constexpr (Cfg::kPair) tc_commit_pair_both(smem_u32(bar));
    else tc_commit(smem_u32(bar));
  };
  for (int64_t t = owner; t < or_total(args); t += args.owners) {
    const OrTile o = or_tile<Cfg>(args, t);
    const int32_t k_blocks = or_k_blocks(args, o.kind);
    if (!wait_bounded(smem_u32(&acc_empty[b]), aph, wc, kSiteMmaAccum)) return any;
    tc_fence_after();
    const uint32_t d = tmem_base + uint32_t(b * Cfg::kTileN);
    for (int32_t kb = 0; kb < k_blocks; kb += kOrGroup) {
      const int majors = or_majors<Cfg>(args, o, kb / Cfg::kPieceBlocks);
      const int a_mn = majors & 1, b_mn = majors >> 1;
      const uint32_t idesc = make_idesc_f16(Cfg::kTileM, Cfg::kTileN, a_mn, b_mn);
      // MN-major: 64-wide halves two k-blocks apart, 16 of K 2 KiB apart, a k-block 8
      const uint32_t a_lbo = a_mn ? uint32_t(kOrGroup) * 8192u : 16u;
      const uint32_t b_lbo = b_mn ? uint32_t(kOrGroup) * 8192u : 16u;
      const uint32_t a_step = a_mn ? (2048u >> 4) : (32u >> 4);
      const uint32_t b_step = b_mn ? (2048u >> 4) : (32u >> 4);
      const uint32_t a_blk = a_mn ? 8192u : uint32_t(Cfg::kABlock);
      const uint32_t b_blk = b_mn ? 8192u : uint32_t(Cfg::kBBlock);
      if (!wait_bounded(smem_u32(&full[s]), ph, wc, kSiteMmaFull)) return any;
      tc_fence_after();
      const uint32_t a0 = ring + uint32_t(s) * Cfg::kStageBytes, b0 = a0 + Cfg::kABytes;
#pragma unroll
      for (int j = 0; j < kOrGroup; ++j) {
        if (kb + j >= k_blocks) break;
        const uint64_t adesc = make_sdesc_sw128(a0 + uint32_t(j) * a_blk, a_lbo, 1024);
        const uint64_t bdesc = make_sdesc_sw128(b0 + uint32_t(j) * b_blk, b_lbo, 1024);
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
          const uint32_t acc = kb > 0 || j > 0 || kk > 0 ? 1u : 0u;
          if constexpr (Cfg::kPair)
            tc_mma_f16_pair(d, adesc + uint64_t(kk * a_step), bdesc + uint64_t(kk * b_step), idesc,
                            acc);
          else
            tc_mma_f16(d, adesc + uint64_t(kk * a_step), bdesc + uint64_t(kk * b_step), idesc,
                       acc);
        }
      }
      any = true;
      commit(&empty[s]);
      if (++s == Cfg::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
    commit(&acc_full[b]);
    if (++b == 2) {
      b = 0;
      aph ^= 1;
    }
  }
  return any;
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  uint32_t w;
  __builtin_memcpy(&w, &h, 4);
  return w;
}

// A warp's 32 x 32 floats (lane i holds row i) turned, through shared memory, so that 8
// lanes hold a row: x[i] is floats 4 (lane % 8) ... + 3 of row 4 i + lane / 8.  16-byte
// pieces are swapped about by row, so that neither side meets a bank twice.  `at` is 128-byte
// aligned: an address is a register and a constant.
__device__ __forceinline__ void or_turn(uint32_t at, const float (&v)[32], float4 (&x)[8],
                                        int lane) {
  __syncwarp();  // the last chunk has been read
  const uint32_t to = at + lane * 128 + ((lane & 7) << 4);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st_shared_v4(to ^ (c << 4), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
                 __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
  __syncwarp();
  const uint32_t even = at + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
  const uint32_t odd = (even ^ 64u) + 512u;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = lds4((i & 1 ? odd : even) + (i / 2) * 1024);
}

// Where a lane's 4 neighbours lie in rows of `ld` elements: row 4 i + lane / 8 from row0 on
// at p + i * step.  `whole`: all 32 rows and columns are inside.
template <class T>
struct OrPlace {
  T* p;
  int64_t step;
  __device__ __forceinline__ OrPlace(T* base, int64_t ld, int32_t row0, int32_t col0, int lane)
      : p(base + (row0 + (lane >> 3)) * ld + col0 + (lane & 7) * 4), step(4 * ld) {}
  __device__ __forceinline__ T* at(int i) const { return p + i * step; }
};

// What a chunk adds: 8 x 4 neighbours of the iterate, or of A as halves in x and y.
struct OrOld {
  float4 v[8];
};

// A chunk's place in the matrix: 32 rows from row0, 32 columns from col0, of which those
// below row_end and col_end count.
struct OrChunk {
  int32_t row0, col0, row_end, col_end;
  __device__ __forceinline__ bool whole() const {
    return row0 + 32 <= row_end && col0 + 32 <= col_end;
  }
  __device__ __forceinline__ bool has(int i, int lane) const {
    return row0 + 4 * i + (lane >> 3) < row_end && col0 + (lane & 7) * 4 < col_end;
  }
};

// One chunk of a symmetric result.  `old`: what or_read_symmetric brought of A.
__device__ __forceinline__ void or_read_symmetric(const OrTcArgs& a, OrOld& old, int32_t z,
                                                  const OrChunk& k, int lane) {
  const OrPlace<const __half> from(a.a16 + z * a.stride_a, a.ld_a, k.row0, k.col0, lane);
  const bool whole = k.whole();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint2 x = make_uint2(0, 0);
    if (whole || k.has(i, lane)) x = __ldcg(reinterpret_cast<const uint2*>(from.at(i)));
    old.v[i].x = __uint_as_float(x.x);
    old.v[i].y = __uint_as_float(x.y);
  }
}
__device__ __forceinline__ float2 half2_floats(float bits) {
  __half2 h;
  __builtin_memcpy(&h, &bits, 4);
  return __half22float2(h);
}
__device__ __forceinline__ void or_store_symmetric(const OrTcArgs& a, const float (&v)[32],
                                                   const OrOld& old, uint32_t stage,
                                                   const OrTile& o, float alpha, float beta,
                                                   const OrChunk& k, int lane) {
  float4 x[8];
  or_turn(stage, v, x, lane);
  const bool poly = o.kind == kPoly;
  __half* const base = (poly ? a.b16 : a.a16) + o.z * a.stride_a;
  const OrPlace<__half> to(base, a.ld_a, k.row0, k.col0, lane);
  const bool whole = k.whole();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i].x *= alpha;
    x[i].y *= alpha;
    x[i].z *= alpha;
    x[i].w *= alpha;
    if (poly) {
      const float2 l = half2_floats(old.v[i].x), u = half2_floats(old.v[i].y);
      x[i].x = fmaf(beta, l.x, x[i].x);
      x[i].y = fmaf(beta, l.y, x[i].y);
      x[i].z = fmaf(beta, u.x, x[i].z);
      x[i].w = fmaf(beta, u.y, x[i].w);
    }
    if (whole || k.has(i, lane))
      *reinterpret_cast<uint2*>(to.at(i)) =
          make_uint2(pack_half2(x[i].x, x[i].y), pack_half2(x[i].z, x[i].w));
  }
}

// One chunk of the new iterate; `old`: what or_read_iterate brought.
__device__ __forceinline__ void or_read_iterate(const OrTcArgs& a, OrOld& old, int32_t z,
                                                const OrChunk& k, int lane) {
  const OrPlace<const float> from(a.x32 + z * a.stride_x, a.ld_x, k.row0, k.col0, lane);
  const bool whole = k.whole();
#pragma unroll
  for (int i = 0; i < 8; ++i)
    old.v[i] = whole || k.has(i, lane) ? __ldcg(reinterpret_cast<const float4*>(from.at(i)))
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ void or_store_iterate(const OrTcArgs& a, const float (&v)[32],
                                                 const OrOld& old, uint32_t stage,
                                                 const OrTile& o, float alpha, float beta,
                                                 float scale, const OrChunk& k, int lane) {
  float4 x[8];
  or_turn(stage, v, x, lane);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i].x = fmaf(alpha, x[i].x, beta * old.v[i].x);
    x[i].y = fmaf(alpha, x[i].y, beta * old.v[i].y);
    x[i].z = fmaf(alpha, x[i].z, beta * old.v[i].z);
    x[i].w = fmaf(alpha, x[i].w, beta * old.v[i].w);
  }
  const bool whole = k.whole();
  if (o.step + 1 < a.steps) {
    const OrPlace<float> to(a.x32 + o.z * a.stride_x, a.ld_x, k.row0, k.col0, lane);
    const OrPlace<__half> to16(a.x16[(o.step + 1) & 1] + o.z * a.stride_x, a.ld_x, k.row0, k.col0,
                               lane);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (whole || k.has(i, lane)) {
        *reinterpret_cast<float4*>(to.at(i)) = x[i];
        *reinterpret_cast<uint2*>(to16.at(i)) = make_uint2(
            pack_half2(x[i].x * scale, x[i].y * scale), pack_half2(x[i].z * scale, x[i].w * scale));
      }
    return;
  }
  const OrPlace<__nv_bfloat16> to(static_cast<__nv_bfloat16*>(a.out) + o.z * a.stride_out,
                                  a.ld_out, k.row0, k.col0, lane);
  const int32_t left = a.cols - k.col0 - (lane & 7) * 4;  // columns from this lane's first on
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (!whole && !k.has(i, lane)) continue;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[i].x, x[i].y);
    const __nv_bfloat162 hi = __floats2bfloat162_rn(x[i].z, x[i].w);
    if (a.out_vec && left >= 4) {
      uint2 w;
      __builtin_memcpy(&w.x, &lo, 4);
      __builtin_memcpy(&w.y, &hi, 4);
      *reinterpret_cast<uint2*>(to.at(i)) = w;
    } else {
      if (left > 0) to.at(i)[0] = lo.x;
      if (left > 1) to.at(i)[1] = lo.y;
      if (left > 2) to.at(i)[2] = hi.x;
      if (left > 3) to.at(i)[3] = hi.y;
    }
  }
}

template <class Cfg>
__device__ __forceinline__ void or_epilogue(const OrTcArgs& args, uint64_t* acc_full,
                                            uint64_t* acc_empty, const volatile uint32_t* ready,
                                            const WaitCtl& wc,
                                            uint32_t tmem_base, uint8_t* stage, uint32_t rank,
                                            int32_t owner) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, wg = (warp - kOrRoleWarps) >> 2;
  const uint32_t stage_w = smem_u32(stage) + uint32_t(warp - kOrRoleWarps) * 4096u;
  const uint32_t tlane = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(wg * Cfg::kHalf);
  int b = 0;
  uint32_t aph = 0;
  uint32_t passed = 0;
  pdl_wait_prerequisites();
  for (int64_t t = owner; t < or_total(args); t += args.owners) {
    const OrTile o = or_tile<Cfg>(args, t);
    const int32_t row0 = o.tm * Cfg::kTileM + int32_t(rank) * 128 + q * 32;
    const int32_t col0 = o.tn * Cfg::kTileN + wg * Cfg::kHalf;
    const bool apply = o.kind == kApply;
    const int32_t rows = apply ? args.rows : args.n;
    const int32_t col_end = apply ? int32_t(args.ld_x) : int32_t(args.ld_a);
    const OrthoStep& co = args.step[o.step];
    const float alpha = apply ? co.apply_alpha : o.kind == kPoly ? co.poly_alpha : co.gram_alpha;
    const float beta = apply ? co.apply_beta : co.poly_beta, scale = co.scale;
    // What the tile adds to its sums is sent for while the MMAs still run: A's tile once
    // its piece of K may be loaded, the iterate's once any of B may be.  (A chunk ahead,
    // each chunk took 1.4 us, the loads' latency.)
    constexpr int kChunks = Cfg::kHalf / 32;
    OrOld old[kChunks];
    bool ok = true;
    if (o.kind != kGram) {
      const uint32_t need = passed + (apply ? 1 : o.tn / Cfg::kRatio + 1);
      ok = __all_sync(0xffffffffu, or_wait_ready(ready, need, wc));
      if (ok) {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          if (row0 >= rows || col0 + 32 * i >= col_end) break;
          const OrChunk k{row0, col0 + 32 * i, rows, col_end};
          if (apply) or_read_iterate(args, old[i], o.z, k, lane);
          else or_read_symmetric(args, old[i], o.z, k, lane);
        }
      }
    }
    passed += or_pieces<Cfg>(args, o.kind);
    ok = ok && wait_bounded(smem_u32(&acc_full[b]), aph, wc, kSiteEpilogue);
    if (!__all_sync(0xffffffffu, ok)) break;
    tc_fence_after();
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = 32 * i;
      if (row0 >= rows || col0 + c >= col_end) break;
      uint32_t r[32];
      float v[32];
      __syncwarp();
      tmem_ld32(tlane + uint32_t(b * Cfg::kTileN + c), r);
      tmem_wait_ld32(r);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
      const OrChunk k{row0, col0 + c, rows, col_end};
      if (apply) or_store_iterate(args, v, old[i], stage_w, o, alpha, beta, scale, k, lane);
      else or_store_symmetric(args, v, old[i], stage_w, o, alpha, beta, k, lane);
    }
    // the tile's counter: this warp's stores, for copies and loads of other SMs
    __syncwarp();
    if (lane == 0) red_release_gpu(or_counters(args, o.step, o.kind, o.z) +
                                   or_index<Cfg>(args, o.kind, o.tm, o.tn));
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if constexpr (Cfg::kPair) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[b]), 0));
      else mbar_arrive(smem_u32(&acc_empty[b]));
    }
    if (++b == 2) {
      b = 0;
      aph ^= 1;
    }
  }
}

template <class Cfg>
__global__ void __launch_bounds__(kOrThreads, 1)
    ortho_tc_kernel(const __grid_constant__ OrMaps maps, const __grid_constant__ OrTcArgs args) {
  constexpr uint32_t S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stage = ring + S * Cfg::kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stage + Cfg::kEpiBytes);
  uint64_t* full = bars;               // a stage's bytes have landed (the leader's)
  uint64_t* empty = full + S;          // its MMAs are done
  uint64_t* acc_full = empty + S;      // a tile's sum is in TMEM
  uint64_t* acc_empty = acc_full + 2;  // all epilogue warps have read it (the leader's)
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* peer_filled = tmem_slot + 2;  // leader: stages that the peer's producer filled
  volatile uint32_t* ready = tmem_slot + 3;

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = Cfg::kPair ? cluster_rank() : 0;
  const int32_t owner = Cfg::kPair ? int32_t(blockIdx.x >> 1) : int32_t(blockIdx.x);
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), kOrEpiWarps * (Cfg::kPair ? 2 : 1));
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *peer_filled = 0;
    *ready = 0;
    fence_barrier_init();
    tma_prefetch_map(&maps.x[0].ka);
    tma_prefetch_map(args.tall && Cfg::kBRows == 64 ? &maps.x[0].mn : &maps.x[0].kb);
  }
  if (warp == 1) {
    if constexpr (Cfg::kPair) {
      tmem_alloc_pair(smem_u32(tmem_slot), Cfg::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (Cfg::kPair) cluster_sync_all();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  const WaitCtl wc{args.wait_limit_ns, args.status, abort_flag};

  uint32_t filled = 0;
  bool issued = false;
  if (warp >= kOrRoleWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOrEpiRegs));
    or_epilogue<Cfg>(args, acc_full, acc_empty, ready, wc, tmem_base, stage, rank, owner);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOrRoleRegs));
    if (warp == 0 && lane == 0) {
      filled = or_producer<Cfg>(maps, args, smem_u32(ring), full, empty, ready, wc, rank, owner);
      if (Cfg::kPair && rank != 0) st_dsmem_u32(map_to_rank(smem_u32(peer_filled), 0), filled);
    } else if (warp == 2) {
      or_watch<Cfg>(args, ready, wc, owner);
    } else {
      pdl_wait_prerequisites();
      if (warp == 1 && lane == 0 && rank == 0) {
        issued = or_mma<Cfg>(args, smem_u32(ring), full, empty, acc_full, acc_empty, wc,
                              tmem_base, owner);
        // every MMA finishes before TMEM is freed, also when an epilogue gave up
        if (issued) {
          if constexpr (Cfg::kPair) tc_commit_pair_self(smem_u32(drain));
          else tc_commit(smem_u32(drain));
          wait_drain(smem_u32(drain), 0, wc);
        }
      }
    }
  }
  __syncthreads();
  tc_fence_before();
  if constexpr (Cfg::kPair) cluster_sync_all();
  // after an abort copies may still be in flight: each stage's last one (of a pair, see
  // tc2_drain_loads)
  if (rank == 0 && threadIdx.x == 0) {
    const uint32_t n0 = filled, n1 = Cfg::kPair ? *peer_filled : filled, n = n0 > n1 ? n0 : n1;
#pragma unroll 1
    for (uint32_t s = 0; s < S && s < n; ++s) {
      const uint32_t at = s + ((n - 1 - s) / S) * S;
      const uint32_t bar = smem_u32(&full[s]);
      if (at >= n0) mbar_arrive_expect_tx(bar, Cfg::kStageBytes);
      else if (at >= n1) mbar_complete_tx(bar, Cfg::kStageBytes);
      wait_drain(bar, (at / S) & 1, wc);
    }
  }
  if constexpr (Cfg::kPair) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (Cfg::kPair) tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

}  // namespace dg

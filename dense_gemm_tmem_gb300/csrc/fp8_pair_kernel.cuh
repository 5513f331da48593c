// fp8_pair_kernel.cuh: the block-scaled product on the tensor cores, two SMs a
// tile (tcgen05.mma.cta_group::2.kind::f8f6f4).
//
//   C[m, n] = sum over kb of sa[m, kb] sb[n, kb] P_kb[m, n],
//   P_kb[m, n] = sum over the 128 k of block kb of a[m, k] b[n, k]
//
// The scales change every 128 k, so no accumulator may run past a block: each
// k-block's P is its own short MMA chain (4 x K = 32) into a TMEM buffer, and
// the sum over k-blocks is kept in fp32 registers.  A k-block of 128 bytes is
// one 128-byte swizzle row, so the ring is that of the 16-bit kernel with twice
// the k per stage:
//   warp 0, one lane   TMA producer: this CTA's 128 rows of A and BN / 2 rows of
//                      B per k-block into an S-stage ring.
//   warp 1, one lane   (leader CTA) 4 MMAs of 256 x BN x 32 per k-block into the
//                      next of NB TMEM buffers; commits free the stage and hand
//                      the buffer to both CTAs' epilogues.
//   warps 4-11         epilogue, two warpgroups of BN / 2 columns: TMEM ->
//                      registers, acc += (sa sb) * P, and the buffer goes back.
//                      A 256 x 256 tile keeps 128 fp32 sums a thread.
// What bounds it: the tensor pipe (512 cycles a k-block of a 256 x 256 tile at
// the e4m3 rate) if the epilogue's TMEM reads (256 cycles) and FMAs (128 packed
// issue slots a scheduler) stay behind it; with only two buffers of 256 columns the
// hand-over latency between the roles shows.  For skinny problems
// (TRANS: operands swapped, C stored transposed) the stream of the weights.
// Small problems split the k-blocks of all tiles evenly over the pairs; the
// last pair to finish a tile adds the fp32 partials in ascending k order, so
// the sum does not depend on who is last and no CTA waits for another.
#pragma once

#include "fp8.cuh"
#include "tc2_kernel.cuh"

namespace dg {

constexpr int kF8EpiWarps = 8;
constexpr int kF8RoleWarps = 4;  // producer, MMA issuer, two idle: one warpgroup
constexpr int kF8Threads = 32 * (kF8RoleWarps + kF8EpiWarps);
// Registers a thread: 3 warpgroups launch with 168 each (504 in all); for a
// 256-wide tile, whose epilogue threads keep 128 sums, the role warpgroup gives
// up all but 40 and the epilogue's two take 232 each (40 + 2 * 232 = 504).
constexpr int kF8RoleRegs = 40, kF8EpiRegs = 232;

template <int BN>
struct Fp8PairConfig {
  static constexpr int kABytes = kBM * kFp8Block;         // 16 KiB: this CTA's 128 rows
  static constexpr int kBBytes = (BN / 2) * kFp8Block;    // this CTA's half of B
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : 8;
  static constexpr int kBuffers = BN == 256 ? 2 : 4;      // TMEM accumulators
  static constexpr int kTmemCols = BN * kBuffers;         // a power of two >= 32
  static constexpr int kHalf = BN / 2;                    // columns per warpgroup
  static constexpr int kChunk = kHalf < 32 ? kHalf : 32;  // columns per TMEM load
  static constexpr int kStoreCols = 16;                   // columns per staged store
  static constexpr int kStoreLd = kStoreCols + 4;
  static constexpr int kEpiBytes = kF8EpiWarps * 32 * kStoreLd * 4;
  static constexpr int kScaleBytes = 2 * 2 * kHalf * 4;   // [buffer][warpgroup][column]
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes =
      1024 + kStages * kStageBytes + kEpiBytes + kScaleBytes + kBarBytes;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static_assert((2 * kStages + 2 * kBuffers + 1) * 8 + 16 <= kBarBytes, "barrier area");
};

// One operand's scales in the MMA view: row (or column) r of k-block kb at
// p[(r >> shift) * stride + kb * kb_stride].
struct Fp8Scales {
  const float* p;
  int64_t stride, kb_stride;
  int32_t shift;
};

struct Fp8PairArgs {
  WorkSpec work;
  int32_t Mm, Nm;      // MMA-view extents
  Fp8Scales row, col;  // of the MMA-view A and B operands
  void* C;             // row-major in the problem's view
  int64_t ldc;
  const float* bias;   // NULL or one per column of C
  int32_t out_dtype;
  int32_t c_vec;       // 1: C's base is 16-byte aligned, its pitch a multiple of 16 bytes
  int32_t a_mn, b_mn;  // 1: the operand is MN-major (b_mn: BN = 256 only)
  float* workspace;
  int* tickets;
  int* status;
  uint64_t wait_limit_ns;
  uint32_t idesc;
};

__device__ __forceinline__ void tc_mma_f8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Barrier among the 128 threads of epilogue warpgroup wg, or all 256.
__device__ __forceinline__ void f8_wg_sync(int wg) {
  asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
}
__device__ __forceinline__ void f8_epi_sync() {
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ void fma2(float2& d, float2 a, float2 b) {
  uint64_t x, y, z;
  __builtin_memcpy(&x, &a, 8);
  __builtin_memcpy(&y, &b, 8);
  __builtin_memcpy(&z, &d, 8);
  asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(z) : "l"(x), "l"(y));
  __builtin_memcpy(&d, &z, 8);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t x, y, z;
  __builtin_memcpy(&x, &a, 8);
  __builtin_memcpy(&y, &b, 8);
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  float2 d;
  __builtin_memcpy(&d, &z, 8);
  return d;
}

template <int BN>
__device__ __forceinline__ uint32_t f8_producer(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                                const Fp8PairArgs& args, uint8_t* sA, uint8_t* sB,
                                                uint64_t* full, uint64_t* empty,
                                                const WaitCtl& wc, uint32_t rank,
                                                int32_t pair_id) {
  using Cfg = Fp8PairConfig<BN>;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init(W, pair_id);
  Unit u;
  int s = 0;
  uint32_t ph = 0, filled = 0;
  pdl_wait_prerequisites();
  while (it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    const int32_t a_row = tm * kPairBM + int32_t(rank) * kBM;
    const int32_t b_row = tn * BN + int32_t(rank) * (BN / 2);
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      if (!wait_bounded(smem_u32(&empty[s]), ph ^ 1, wc, kSiteProducer)) return filled;
      const uint32_t local = smem_u32(&full[s]);
      if (rank == 0) mbar_arrive_expect_tx(local, 2 * Cfg::kStageBytes);
      const uint32_t fb = map_to_rank(local, 0);
      const int32_t k0 = kb * kFp8Block;
      const uint32_t a_dst = smem_u32(sA + s * Cfg::kABytes);
      const uint32_t b_dst = smem_u32(sB + s * Cfg::kBBytes);
      if (args.a_mn) tma_load_2d_pair(a_dst, &tmA, fb, a_row, k0);
      else tma_load_2d_pair(a_dst, &tmA, fb, k0, a_row);
      if (args.b_mn) tma_load_2d_pair(b_dst, &tmB, fb, b_row, k0);
      else tma_load_2d_pair(b_dst, &tmB, fb, k0, b_row);
      ++filled;
      if (++s == Cfg::kStages) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  return filled;
}

// After both producers have stopped (leader's thread 0): waits until every
// load issued has landed.  n0 and n1 count the stages the leader and the peer
// filled; they differ only after an abort, by less than one ring, so only a
// stage's last filling can be one-sided: the peer's alone is armed for the
// peer's bytes here, the leader's alone has the peer's missing bytes counted
// as done.
template <int BN>
__device__ __forceinline__ void f8_drain_loads(uint64_t* full, uint32_t n0, uint32_t n1,
                                               const WaitCtl& wc) {
  using Cfg = Fp8PairConfig<BN>;
  constexpr uint32_t S = Cfg::kStages;
  const uint32_t n = n0 > n1 ? n0 : n1;
#pragma unroll 1
  for (uint32_t s = 0; s < S && s < n; ++s) {
    const uint32_t q = s + ((n - 1 - s) / S) * S;
    const uint32_t bar = smem_u32(&full[s]);
    if (q >= n0) mbar_arrive_expect_tx(bar, Cfg::kStageBytes);
    else if (q >= n1) mbar_complete_tx(bar, Cfg::kStageBytes);
    wait_drain(bar, (q / S) & 1, wc);
  }
}

template <int BN>
__device__ __forceinline__ void f8_mma(const Fp8PairArgs& args, uint8_t* sA, uint8_t* sB,
                                       uint64_t* full, uint64_t* empty, uint64_t* acc_full,
                                       uint64_t* acc_empty, uint64_t* drain, const WaitCtl& wc,
                                       uint32_t tmem_base, int32_t pair_id) {
  using Cfg = Fp8PairConfig<BN>;
  const WorkSpec& W = args.work;
  WorkIter it;
  it.init(W, pair_id);
  Unit u;
  int s = 0, b = 0;
  uint32_t ph = 0, aph = 0;
  bool ok = true, any = false;
  // K = 32 steps: 32 bytes along a K-major row, 32 rows of 128 bytes MN-major
  const uint32_t a_step = args.a_mn ? (4096u >> 4) : (32u >> 4);
  const uint32_t b_step = args.b_mn ? (4096u >> 4) : (32u >> 4);
  while (ok && it.next(W, u)) {
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      if (!wait_bounded(smem_u32(&acc_empty[b]), aph ^ 1, wc, kSiteMmaAccum) ||
          !wait_bounded(smem_u32(&full[s]), ph, wc, kSiteMmaFull)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint64_t adesc = make_sdesc_sw128(smem_u32(sA + s * Cfg::kABytes), 16, 1024);
      const uint64_t bdesc = make_sdesc_sw128(smem_u32(sB + s * Cfg::kBBytes), 16, 1024);
      const uint32_t d = tmem_base + uint32_t(b * BN);
#pragma unroll
      for (int kk = 0; kk < kFp8Block / 32; ++kk)
        tc_mma_f8_pair(d, adesc + uint64_t(kk * a_step), bdesc + uint64_t(kk * b_step),
                       args.idesc, kk > 0 ? 1u : 0u);
      any = true;
      tc_commit_pair_both(smem_u32(&empty[s]));
      tc_commit_pair_both(smem_u32(&acc_full[b]));
      if (++s == Cfg::kStages) {
        s = 0;
        ph ^= 1;
      }
      if (++b == Cfg::kBuffers) {
        b = 0;
        aph ^= 1;
      }
    }
  }
  if (!ok && any) {  // every MMA issued so far must finish before TMEM is freed
    tc_commit_pair_self(smem_u32(drain));
    wait_drain(smem_u32(drain), 0, wc);
  }
}

// Four neighbouring outputs along C's rows, the first `valid` of them.
__device__ __forceinline__ void f8_put4(const Fp8PairArgs& a, int64_t off, float4 v, int valid) {
  if (a.out_dtype == GEMM_F32) {
    float* p = static_cast<float*>(a.C) + off;
    if (valid == 4 && a.c_vec) {
      *reinterpret_cast<float4*>(p) = v;
      return;
    }
  } else if (valid == 4 && a.c_vec) {
    uint2 pk;
    if (a.out_dtype == GEMM_F16) {
      const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
      __builtin_memcpy(&pk.x, &x, 4);
      __builtin_memcpy(&pk.y, &y, 4);
    } else {
      const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
      __builtin_memcpy(&pk.x, &x, 4);
      __builtin_memcpy(&pk.y, &y, 4);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.C) + off) = pk;
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < valid) store_typed(a.C, off + j, f[j], a.out_dtype);
}

template <int BN, bool TRANS, bool COLVEC>
__device__ __forceinline__ void f8_epilogue(const Fp8PairArgs& args, uint64_t* acc_full,
                                            uint64_t* acc_empty, const WaitCtl& wc,
                                            uint32_t tmem_base, uint32_t rank, int32_t pair_id,
                                            float* stage, float* scales, volatile int* last_flag) {
  using Cfg = Fp8PairConfig<BN>;
  constexpr int HC = Cfg::kHalf, CW = Cfg::kChunk;
  const WorkSpec& W = args.work;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3;               // TMEM lane quarter this warp may access
  const int wg = (warp - kF8RoleWarps) >> 2;       // which half of the columns
  const int row = q * 32 + lane;
  const int wtid = ((warp - kF8RoleWarps) & 3) * 32 + lane;  // thread of the warpgroup
  float* stage_w = stage + (warp - kF8RoleWarps) * 32 * Cfg::kStoreLd;
  WorkIter it;
  it.init(W, pair_id);
  pdl_wait_prerequisites();
  Unit u;
  int b = 0;
  uint32_t aph = 0;
  bool ok = true;
  // After a wait gave up the loops run on without waiting or storing, so that
  // every warp still meets every barrier below.
  while (it.next(W, u)) {
    int32_t tm, tn;
    tile_coords(W, u.tile, tm, tn);
    const int32_t mrow0 = tm * kPairBM + int32_t(rank) * kBM;
    const int32_t mm = mrow0 + row;
    const int32_t nn0 = tn * BN + wg * HC;
    const int32_t mc = mm < args.Mm ? mm : args.Mm - 1;
    const float* rp = args.row.p + int64_t(mc >> args.row.shift) * args.row.stride;
    // the scale this thread fetches along the columns: its own column's, or
    // the one that all the warpgroup's columns share
    int32_t nc = nn0 + (COLVEC && wtid < HC ? wtid : 0);
    nc = nc < args.Nm ? nc : args.Nm - 1;
    const float* cp = args.col.p + int64_t(nc >> args.col.shift) * args.col.stride;
    auto ld_row = [&](int32_t kb) {
      return __ldg(rp + int64_t(kb < u.kb1 ? kb : u.kb1 - 1) * args.row.kb_stride);
    };
    auto ld_col = [&](int32_t kb) {
      return __ldg(cp + int64_t(kb < u.kb1 ? kb : u.kb1 - 1) * args.col.kb_stride);
    };
    float r0 = ld_row(u.kb0), r1 = ld_row(u.kb0 + 1);
    float c0 = ld_col(u.kb0), c1 = ld_col(u.kb0 + 1);
    float2 acc[HC / 2];
#pragma unroll
    for (int j = 0; j < HC / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    if (COLVEC && wtid < HC) scales[wg * HC + wtid] = c0;
    for (int32_t kb = u.kb0; kb < u.kb1; ++kb) {
      const float r2 = ld_row(kb + 2), c2 = ld_col(kb + 2);
      const int par = (kb - u.kb0) & 1;
      if (COLVEC) {
        f8_wg_sync(wg);  // this k-block's column scales are in; the other buffer is free
        if (wtid < HC) scales[((par ^ 1) * 2 + wg) * HC + wtid] = c1;
      }
      if (ok) ok = __all_sync(0xffffffffu, wait_bounded(smem_u32(&acc_full[b]), aph, wc,
                                                        kSiteEpilogue));
      if (ok) {
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + (uint32_t(q * 32) << 16) + uint32_t(b * BN + wg * HC);
        const float rs = COLVEC ? r0 : r0 * c0;
        const float2 rs2 = make_float2(rs, rs);
#pragma unroll
        for (int c = 0; c < HC / CW; ++c) {
          float v[CW];
          tmem_load_chunk<CW>(taddr + c * CW, v);
          if (c == HC / CW - 1) {  // the buffer's last read: back to the MMA issuer
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[b]), 0));
          }
#pragma unroll
          for (int j = 0; j < CW / 2; ++j) {
            const float2 p2 = make_float2(v[2 * j], v[2 * j + 1]);
            if constexpr (COLVEC) {
              const float2 cs = *reinterpret_cast<const float2*>(
                  scales + (par * 2 + wg) * HC + c * CW + 2 * j);
              fma2(acc[c * (CW / 2) + j], mul2(cs, rs2), p2);
            } else {
              fma2(acc[c * (CW / 2) + j], rs2, p2);
            }
          }
        }
      }
      r0 = r1; r1 = r2;
      c0 = c1; c1 = c2;
      if (++b == Cfg::kBuffers) {
        b = 0;
        aph ^= 1;
      }
    }
    if (COLVEC) f8_wg_sync(wg);  // the scales' buffers may be refilled for the next unit

    // Split tile: this CTA's fp32 half goes to the workspace (128 rows x BN, as
    // float4 j of row r at j * 128 + r); the last pair to arrive adds the halves.
    bool mine = true;
    int32_t first = pair_id, last = pair_id;
    const int32_t st = u.tile - W.dp_tiles;
    const bool partial = unit_is_partial(W, u);
    auto half_of = [&](int32_t p) {
      return reinterpret_cast<float4*>(args.workspace) +
             (size_t(split_slot(W, p, st)) * 2 + rank) * (size_t(kBM) * BN / 4) +
             size_t(wg) * (HC / 4) * kBM + row;
    };
    if (partial) {
      float4* dst = half_of(pair_id);
#pragma unroll
      for (int j = 0; j < HC / 4; ++j)
        __stcg(dst + j * kBM, make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x,
                                          acc[2 * j + 1].y));
      __threadfence();
      f8_epi_sync();
      split_contributors(W, st, first, last);
      int* ticket = args.tickets + 2 * st + int32_t(rank);
      if (threadIdx.x == 32 * kF8RoleWarps) {
        const int old = atomicAdd(ticket, 1);
        *last_flag = (old == last - first) ? 1 : 0;
        if (old == last - first) atomicExch(ticket, 0);  // ready for the next launch
      }
      f8_epi_sync();
      mine = *last_flag != 0;
      if (mine) __threadfence();
    }
    if (!mine || !ok) continue;
    const float* bias = args.bias;
#pragma unroll
    for (int c = 0; c < HC / 16; ++c) {  // 16 columns at a time
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[2 * j] = acc[c * 8 + j].x;
        v[2 * j + 1] = acc[c * 8 + j].y;
      }
      if (partial) {
        float tot[16];
#pragma unroll 1
        for (int32_t p = first; p <= last; ++p) {
          float4 x[4];
          const float4* src = half_of(p) + size_t(c) * 4 * kBM;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = __ldcg(src + j * kBM);
            const float w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[4 * j + i] = p == first ? w[i] : tot[4 * j + i] + w[i];
          }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = tot[j];
      }
      const int32_t nn = nn0 + c * 16;
      if (TRANS) {
        if (mm < args.Mm) {
          const float bv = bias ? __ldg(bias + mm) : 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (nn + j < args.Nm)
              store_typed(args.C, int64_t(nn + j) * args.ldc + mm, v[j] + bv, args.out_dtype);
        }
      } else {
        // through the warp's shared rows, so that neighbouring lanes store
        // neighbouring columns: 4 lanes a row, 8 rows an instruction
        __syncwarp();
        float4* own = reinterpret_cast<float4*>(stage_w + lane * Cfg::kStoreLd);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          own[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        __syncwarp();
        const int c4 = lane & 3, rs = lane >> 2;
        const int32_t n4 = nn + 4 * c4;
        const int valid = min(4, args.Nm - n4);
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const float4*>(stage_w + (i * 8 + rs) * Cfg::kStoreLd + 4 * c4);
        if (valid > 0) {
          float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);
          if (bias) {
            b4.x = __ldg(bias + n4);
            if (valid > 1) b4.y = __ldg(bias + n4 + 1);
            if (valid > 2) b4.z = __ldg(bias + n4 + 2);
            if (valid > 3) b4.w = __ldg(bias + n4 + 3);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t m = mrow0 + q * 32 + i * 8 + rs;
            if (m < args.Mm)
              f8_put4(args, int64_t(m) * args.ldc + n4,
                      make_float4(x[i].x + b4.x, x[i].y + b4.y, x[i].z + b4.z, x[i].w + b4.w),
                      valid);
          }
        }
      }
    }
  }
}

// args.work counts pair tiles (256 x BN) and pairs (grid / 2).
template <int BN, bool TRANS, bool COLVEC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kF8Threads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                    const __grid_constant__ CUtensorMap tmB, const Fp8PairArgs args) {
  using Cfg = Fp8PairConfig<BN>;
  constexpr int S = Cfg::kStages, NB = Cfg::kBuffers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + S * Cfg::kABytes;
  float* stage = reinterpret_cast<float*>(sB + S * Cfg::kBBytes);
  float* scales = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(stage) + Cfg::kEpiBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(scales) +
                                               Cfg::kScaleBytes);
  uint64_t* full = bars;              // leader's counts both CTAs' bytes
  uint64_t* empty = bars + S;         // one multicast commit per phase, in both CTAs
  uint64_t* acc_full = empty + S;     // the same, per k-block
  uint64_t* acc_empty = acc_full + NB;  // leader's: 8 epilogue warps x 2 CTAs
  uint64_t* drain = acc_empty + NB;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = reinterpret_cast<volatile int*>(tmem_slot + 2);
  uint32_t* peer_filled = tmem_slot + 3;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int32_t pair_id = int32_t(blockIdx.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), 2 * kF8EpiWarps);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *last_flag = 0;
    *peer_filled = 0;
    fence_barrier_init();
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();  // both CTAs' barriers initialised and TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  const WaitCtl wc{args.wait_limit_ns, args.status, abort_flag};

  uint32_t filled = 0;
  if (warp >= kF8RoleWarps) {
    if (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kF8EpiRegs));
    f8_epilogue<BN, TRANS, COLVEC>(args, acc_full, acc_empty, wc, tmem_base, rank, pair_id, stage,
                                   scales, last_flag);
  } else {
    if (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kF8RoleRegs));
    if (warp == 0 && lane == 0) {
      filled = f8_producer<BN>(tmA, tmB, args, sA, sB, full, empty, wc, rank, pair_id);
      if (rank != 0) st_dsmem_u32(map_to_rank(smem_u32(peer_filled), 0), filled);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      pdl_wait_prerequisites();
      f8_mma<BN>(args, sA, sB, full, empty, acc_full, acc_empty, drain, wc, tmem_base, pair_id);
    } else {
      pdl_wait_prerequisites();
    }
  }
  __syncthreads();
  tc_fence_before();
  // both CTAs' roles are done: no MMA or remote arrive is still aimed at
  // either CTA, no load will be issued, and the peer's fill count is in
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) f8_drain_loads<BN>(full, filled, *peer_filled, wc);
  cluster_sync_all();  // no copy still lands in either CTA's shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
  }
}

}  // namespace dg

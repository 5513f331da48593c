// ortho_tc_kernel.cuh: the products of the orthogonalising call on the tensor cores
// (tcgen05.mma.kind::f16, fp32 sums in TMEM), for all matrices of the batch in one
// launch:
//   kGram   A16 = half(alpha X·Xᵀ)               symmetric
//   kPoly   B16 = half(alpha A·Aᵀ + beta A)      symmetric
//   kApply  X   = alpha B·X + beta X             (or X·B), fp32, and its 16-bit copy
// Of a symmetric result only the tiles on and below the diagonal are computed; the
// epilogue stores each also mirrored, which takes the step from 4 to 3 m^2 n + m^3
// flops.  Operands are K-major or MN-major as they lie in memory (Xᵀ is never formed);
// rows are padded with zeros to 64 elements, so a k-block is always whole.
//   warp 0, one lane   TMA producer, two k-blocks per stage (an SM's TMA unit takes
//                      about as long for a copy of 32 KiB as for one of 16)
//   warp 1, one lane   MMAs into one of two accumulators
//   warps 4-11         epilogue, two warpgroups of half the columns each, beside the
//                      next tile's MMAs
// PAIR: two CTAs on two SMs own a 256 x 256 tile (cta_group::2), else one a 128 x 128
// tile, for matrices too small to fill the SMs with pairs' tiles.
#pragma once

#include "fp8_tc_kernel.cuh"
#include "ortho.cuh"
#include "tc2_kernel.cuh"

namespace dg {

constexpr int kOrRoleWarps = 4, kOrEpiWarps = 8;
constexpr int kOrThreads = 32 * (kOrRoleWarps + kOrEpiWarps);
// Registers a thread: 3 warpgroups launch with 168 each (504 in all); the roles keep 56,
// the epilogue's two take 224 each, for the chunk that is sent for ahead.
constexpr int kOrRoleRegs = 56, kOrEpiRegs = 224;
constexpr int kOrGroup = 2;   // k-blocks of 64 per stage
constexpr int kOrStages = 3;

template <bool PAIR>
struct OrConfig {
  static constexpr int kTile = PAIR ? 256 : 128;          // rows and columns
  static constexpr int kBlockBytes = 128 * 128;           // 128 rows (or columns) of a k-block
  static constexpr int kOperandBytes = kOrGroup * kBlockBytes;
  static constexpr int kStageBytes = 2 * kOperandBytes;
  static constexpr int kTmemCols = 2 * kTile;
  static constexpr int kHalf = kTile / 2;                 // columns per warpgroup
  static constexpr int kEpiBytes = kOrEpiWarps * 4096;    // 32 x 32 floats a warp
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes = 1024 + kOrStages * kStageBytes + kEpiBytes + kBarBytes;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

struct OrTcArgs {
  int32_t batch, tiles_m, tiles_n;  // tiles of one matrix
  int32_t per;                      // tiles of one matrix that are computed
  int32_t group_m, k_blocks, owners;
  int32_t a_mn, b_mn;
  int32_t rows, cols, n;
  int64_t ld_x, ld_a, stride_x, stride_a;
  OrthoProduct p;
  int32_t out_vec;                  // 8-byte stores of `out`
  uint32_t idesc;
  int* status;
  uint64_t wait_limit_ns;
};

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

// Tile t: matrix z and tile coordinates; of a symmetric result tn <= tm.
__device__ __forceinline__ void or_tile(const OrTcArgs& a, int32_t t, int32_t& z, int32_t& tm,
                                        int32_t& tn) {
  z = t / a.per;
  const int32_t x = t - z * a.per;
  if (a.p.kind != kApply) {
    int32_t i = int32_t((sqrtf(8.f * float(x) + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > x) --i;
    while ((i + 1) * (i + 2) / 2 <= x) ++i;
    tm = i;
    tn = x - i * (i + 1) / 2;
  } else {
    const int32_t per_group = a.group_m * a.tiles_n, g = x / per_group, first = g * a.group_m;
    const int32_t gm = min(a.group_m, a.tiles_m - first), r = x - g * per_group;
    tm = first + r % gm;
    tn = r / gm;
  }
}

// TMA producer (one thread).  Returns how many stages it filled.
template <bool PAIR>
__device__ __forceinline__ uint32_t or_producer(const CUtensorMap& mA, const CUtensorMap& mB,
                                                const OrTcArgs& args, uint32_t ring,
                                                uint64_t* full, uint64_t* empty,
                                                const WaitCtl& wc, uint32_t rank, int32_t owner) {
  using Cfg = OrConfig<PAIR>;
  int s = 0;
  uint32_t ph = 0, filled = 0;
  pdl_wait_prerequisites();
  for (int32_t t = owner; t < args.per * args.batch; t += args.owners) {
    int32_t z, tm, tn;
    or_tile(args, t, z, tm, tn);
    const int32_t a_row = tm * Cfg::kTile + int32_t(rank) * 128;
    const int32_t b_row = tn * Cfg::kTile + int32_t(rank) * 128;
    for (int32_t kb = 0; kb < args.k_blocks; kb += kOrGroup) {
      if (!wait_bounded(smem_u32(&empty[s]), ph ^ 1, wc, kSiteProducer)) return filled;
      const uint32_t own = smem_u32(&full[s]);
      if (rank == 0) mbar_arrive_expect_tx(own, (PAIR ? 2 : 1) * Cfg::kStageBytes);
      // K-major: 128 rows of two k-blocks; MN-major: two 64-wide halves of 128 k
      auto load = [&](uint32_t dst, const CUtensorMap* map, int mn, int32_t row) {
        if constexpr (PAIR) {
          const uint32_t bar = map_to_rank(own, 0);
          if (!mn) {
            tma_load_4d_pair(dst, map, bar, 0, row, kb, z);
          } else {
            tma_load_3d_pair(dst, map, bar, row, kb * kBK, z);
            tma_load_3d_pair(dst + kOrGroup * 8192, map, bar, row + 64, kb * kBK, z);
          }
        } else {
          if (!mn) {
            tma_load_4d(dst, map, own, 0, row, kb, z);
          } else {
            tma_load_3d(dst, map, own, row, kb * kBK, z);
            tma_load_3d(dst + kOrGroup * 8192, map, own, row + 64, kb * kBK, z);
          }
        }
      };
      const uint32_t dst = ring + uint32_t(s) * Cfg::kStageBytes;
      load(dst, &mA, args.a_mn, a_row);
      load(dst + Cfg::kOperandBytes, &mB, args.b_mn, b_row);
      ++filled;
      if (++s == kOrStages) {
        s = 0;
        ph ^= 1;
      }
    }
  }
  return filled;
}

// MMA issuer (one thread).  Whether it issued anything.
template <bool PAIR>
__device__ __forceinline__ bool or_mma(const OrTcArgs& args, uint32_t ring, uint64_t* full,
                                       uint64_t* empty, uint64_t* acc_full, uint64_t* acc_empty,
                                       const WaitCtl& wc, uint32_t tmem_base, int32_t owner) {
  using Cfg = OrConfig<PAIR>;
  int s = 0, b = 0;
  uint32_t ph = 0, aph = 1;
  bool any = false;
  auto commit = [&](uint64_t* bar) {
    if constexpr (PAIR) tc_commit_pair_both(smem_u32(bar));
    else tc_commit(smem_u32(bar));
  };
  const uint32_t a_lbo = args.a_mn ? uint32_t(kOrGroup) * 8192u : 16u;
  const uint32_t b_lbo = args.b_mn ? uint32_t(kOrGroup) * 8192u : 16u;
  const uint32_t a_step = args.a_mn ? (2048u >> 4) : (32u >> 4);
  const uint32_t b_step = args.b_mn ? (2048u >> 4) : (32u >> 4);
  const uint32_t a_blk = args.a_mn ? 8192u : uint32_t(Cfg::kBlockBytes);
  const uint32_t b_blk = args.b_mn ? 8192u : uint32_t(Cfg::kBlockBytes);
  for (int32_t t = owner; t < args.per * args.batch; t += args.owners) {
    if (!wait_bounded(smem_u32(&acc_empty[b]), aph, wc, kSiteMmaAccum)) return any;
    tc_fence_after();
    const uint32_t d = tmem_base + uint32_t(b * Cfg::kTile);
    for (int32_t kb = 0; kb < args.k_blocks; kb += kOrGroup) {
      if (!wait_bounded(smem_u32(&full[s]), ph, wc, kSiteMmaFull)) return any;
      tc_fence_after();
      const uint32_t a0 = ring + uint32_t(s) * Cfg::kStageBytes, b0 = a0 + Cfg::kOperandBytes;
#pragma unroll
      for (int j = 0; j < kOrGroup; ++j) {
        if (kb + j >= args.k_blocks) break;
        const uint64_t adesc = make_sdesc_sw128(a0 + uint32_t(j) * a_blk, a_lbo, 1024);
        const uint64_t bdesc = make_sdesc_sw128(b0 + uint32_t(j) * b_blk, b_lbo, 1024);
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
          const uint32_t acc = kb > 0 || j > 0 || kk > 0 ? 1u : 0u;
          if constexpr (PAIR)
            tc_mma_f16_pair(d, adesc + uint64_t(kk * a_step), bdesc + uint64_t(kk * b_step),
                            args.idesc, acc);
          else
            tc_mma_f16(d, adesc + uint64_t(kk * a_step), bdesc + uint64_t(kk * b_step),
                       args.idesc, acc);
        }
      }
      any = true;
      commit(&empty[s]);
      if (++s == kOrStages) {
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

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// A warp's 32 x 32 floats (lane i holds row i) turned, through shared memory, so that 8
// lanes hold a row: x[i] is floats 4 (lane % 8) ... + 3 of row 4 i + lane / 8.  16-byte
// pieces are swapped about by row, so that neither side meets a bank twice.  (Shared
// addresses, not pointers: through generic ones a chunk took 1.3 us even alone, as no
// load passed a store.)
__device__ __forceinline__ void or_turn(uint32_t at, const float (&v)[32], float4 (&x)[8],
                                        int lane) {
  __syncwarp();  // the last chunk has been read
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st_shared_v4(at + lane * 128 + ((c ^ (lane & 7)) << 4), __float_as_uint(v[4 * c]),
                 __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                 __float_as_uint(v[4 * c + 3]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    x[i] = lds4(at + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
  }
}

// What a chunk adds: 8 x 4 neighbours of the iterate, or of A as halves in x and y.
struct OrOld {
  float4 v[8];
};

// One chunk of a symmetric result: 32 rows from row0, 32 columns from col0.  `old`: what
// or_read_symmetric brought of A.  The mirrored chunk goes through shared memory too, as
// halves in rows of 72 bytes (8-byte pieces read back; the 2-byte stores meet a bank at
// most twice): 64 bytes a row are stored at a time.  (Stored from registers, 2 bytes a
// lane, it took 1.7 of a chunk's 2.2 us.)
constexpr int kMirrorLd = 36;  // halves
__device__ __forceinline__ void or_read_symmetric(const OrTcArgs& a, OrOld& old, int32_t z,
                                                  int32_t row0, int32_t col0, int lane) {
  const int32_t c = col0 + (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int32_t r = row0 + 4 * i + (lane >> 3);
    const uint2 x = r < a.n && c < a.ld_a ? *reinterpret_cast<const uint2*>(
                                                a.p.a + z * a.stride_a + int64_t(r) * a.ld_a + c)
                                          : make_uint2(0, 0);
    old.v[i].x = __uint_as_float(x.x);
    old.v[i].y = __uint_as_float(x.y);
  }
}
__device__ __forceinline__ void or_store_symmetric(const OrTcArgs& a, const float (&v)[32],
                                                   const OrOld& old, uint32_t stage,
                                                   int32_t z, int32_t row0, int32_t col0,
                                                   bool mirror, int lane) {
  const OrthoProduct& p = a.p;
  float4 turned[8];
  or_turn(stage, v, turned, lane);
  __half* const to = p.c + z * a.stride_a;
  const int32_t c = col0 + (lane & 7) * 4;
  uint2 h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3);
    float4 x = turned[i];
    x.x *= p.alpha;
    x.y *= p.alpha;
    x.z *= p.alpha;
    x.w *= p.alpha;
    if (p.kind == kPoly) {
      __half2 lo, hi;
      __builtin_memcpy(&lo, &old.v[i].x, 4);
      __builtin_memcpy(&hi, &old.v[i].y, 4);
      const float2 l = __half22float2(lo), u = __half22float2(hi);
      x.x = fmaf(p.beta, l.x, x.x);
      x.y = fmaf(p.beta, l.y, x.y);
      x.z = fmaf(p.beta, u.x, x.z);
      x.w = fmaf(p.beta, u.y, x.w);
    }
    h[i] = make_uint2(pack_half2(x.x, x.y), pack_half2(x.z, x.w));
    if (row0 + r < a.n && c < a.ld_a)
      *reinterpret_cast<uint2*>(to + int64_t(row0 + r) * a.ld_a + c) = h[i];
  }
  if (!mirror) return;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t at = stage + ((lane & 7) * 4 * kMirrorLd + 4 * i + (lane >> 3)) * 2;
    st_shared_u16(at, uint16_t(h[i].x));
    st_shared_u16(at + 2 * kMirrorLd, uint16_t(h[i].x >> 16));
    st_shared_u16(at + 4 * kMirrorLd, uint16_t(h[i].y));
    st_shared_u16(at + 6 * kMirrorLd, uint16_t(h[i].y >> 16));
  }
  __syncwarp();
  uint2 m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    m[i] = ld_shared_v2(stage + ((4 * i + (lane >> 3)) * kMirrorLd + (lane & 7) * 4) * 2);
  const int32_t r = row0 + (lane & 7) * 4;  // a column of the mirrored rows
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int cc = 4 * i + (lane >> 3);
    if (col0 + cc < a.n && r < a.ld_a)
      *reinterpret_cast<uint2*>(to + int64_t(col0 + cc) * a.ld_a + r) = m[i];
  }
}

// One chunk of the new iterate; `old`: what or_read_iterate brought.
__device__ __forceinline__ void or_read_iterate(const OrTcArgs& a, OrOld& old, int32_t z,
                                                int32_t row0, int32_t col0, int lane) {
  const int32_t c = col0 + (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int32_t r = row0 + 4 * i + (lane >> 3);
    old.v[i] = r < a.rows && c < a.ld_x
                   ? *reinterpret_cast<const float4*>(a.p.x32 + z * a.stride_x +
                                                      int64_t(r) * a.ld_x + c)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
__device__ __forceinline__ void or_store_iterate(const OrTcArgs& a, const float (&v)[32],
                                                 const OrOld& old, uint32_t stage,
                                                 int32_t z, int32_t row0, int32_t col0,
                                                 int lane) {
  const OrthoProduct& p = a.p;
  float4 turned[8];
  or_turn(stage, v, turned, lane);
  const int32_t c = col0 + (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rr = 4 * i + (lane >> 3);
    const int32_t r = row0 + rr;
    float4 x = turned[i];
    if (r >= a.rows) continue;
    x.x = fmaf(p.alpha, x.x, p.beta * old.v[i].x);
    x.y = fmaf(p.alpha, x.y, p.beta * old.v[i].y);
    x.z = fmaf(p.alpha, x.z, p.beta * old.v[i].z);
    x.w = fmaf(p.alpha, x.w, p.beta * old.v[i].w);
    if (p.out) {
      __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + z * p.stride_out +
                          int64_t(r) * p.ld_out + c;
      if (a.out_vec && c + 4 <= a.cols) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(x.z, x.w);
        uint2 w;
        __builtin_memcpy(&w.x, &lo, 4);
        __builtin_memcpy(&w.y, &hi, 4);
        *reinterpret_cast<uint2*>(to) = w;
      } else {
        const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (c + k < a.cols) to[k] = __float2bfloat16_rn(e[k]);
      }
    } else if (c < a.ld_x) {
      const int64_t at = z * a.stride_x + int64_t(r) * a.ld_x + c;
      *reinterpret_cast<float4*>(p.x32 + at) = x;
      *reinterpret_cast<uint2*>(p.c + at) = make_uint2(pack_half2(x.x * p.scale, x.y * p.scale),
                                                       pack_half2(x.z * p.scale, x.w * p.scale));
    }
  }
}

template <bool PAIR>
__device__ __forceinline__ void or_epilogue(const OrTcArgs& args, uint64_t* acc_full,
                                            uint64_t* acc_empty, const WaitCtl& wc,
                                            uint32_t tmem_base, uint8_t* stage, uint32_t rank,
                                            int32_t owner) {
  using Cfg = OrConfig<PAIR>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, wg = (warp - kOrRoleWarps) >> 2;
  const uint32_t stage_w = smem_u32(stage) + uint32_t(warp - kOrRoleWarps) * 4096u;
  const uint32_t tlane = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(wg * Cfg::kHalf);
  int b = 0;
  uint32_t aph = 0;
  pdl_wait_prerequisites();
  for (int32_t t = owner; t < args.per * args.batch; t += args.owners) {
    int32_t z, tm, tn;
    or_tile(args, t, z, tm, tn);
    const int32_t row0 = tm * Cfg::kTile + int32_t(rank) * 128 + q * 32;
    const int32_t col0 = tn * Cfg::kTile + wg * Cfg::kHalf;
    const bool apply = args.p.kind == kApply;
    const int32_t rows = apply ? args.rows : args.n;
    // a mirrored tile's rows past the matrix fill the padding of the mirrored rows
    const int32_t row_end = apply || tm == tn ? rows : int32_t(args.ld_a);
    const int32_t col_end = apply ? int32_t(args.ld_x) : int32_t(args.ld_a);
    // what a chunk adds to its sums is sent for a chunk ahead, the first one's while the
    // MMAs still run: two chunks a turn, so that registers have fixed names
    OrOld old[2];
    auto inside = [&](int c) { return row0 < row_end && col0 + c < col_end; };
    auto fetch = [&](OrOld& o, int c) {
      if (c >= Cfg::kHalf || !inside(c)) return;
      if (apply) or_read_iterate(args, o, z, row0, col0 + c, lane);
      else if (args.p.kind == kPoly) or_read_symmetric(args, o, z, row0, col0 + c, lane);
    };
    auto chunk = [&](const OrOld& o, int c) {
      if (!inside(c)) return;
      uint32_t r[32];
      float v[32];
      __syncwarp();
      tmem_ld32(tlane + uint32_t(b * Cfg::kTile + c), r);
      tmem_wait_ld32(r);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
      if (apply) or_store_iterate(args, v, o, stage_w, z, row0, col0 + c, lane);
      else or_store_symmetric(args, v, o, stage_w, z, row0, col0 + c, tm != tn, lane);
    };
    fetch(old[0], 0);
    if (!__all_sync(0xffffffffu, wait_bounded(smem_u32(&acc_full[b]), aph, wc, kSiteEpilogue)))
      break;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < Cfg::kHalf; c += 64) {
      fetch(old[1], c + 32);
      chunk(old[0], c);
      fetch(old[0], c + 64);
      chunk(old[1], c + 32);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if constexpr (PAIR) mbar_arrive_cluster(map_to_rank(smem_u32(&acc_empty[b]), 0));
      else mbar_arrive(smem_u32(&acc_empty[b]));
    }
    if (++b == 2) {
      b = 0;
      aph ^= 1;
    }
  }
}

template <bool PAIR>
__global__ void __launch_bounds__(kOrThreads, 1)
    ortho_tc_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB,
                    const OrTcArgs args) {
  using Cfg = OrConfig<PAIR>;
  constexpr uint32_t S = kOrStages;
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

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const int32_t owner = PAIR ? int32_t(blockIdx.x >> 1) : int32_t(blockIdx.x);
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), kOrEpiWarps * (PAIR ? 2 : 1));
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    *peer_filled = 0;
    fence_barrier_init();
    tma_prefetch_map(&mA);
    tma_prefetch_map(&mB);
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
  if (warp >= kOrRoleWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kOrEpiRegs));
    or_epilogue<PAIR>(args, acc_full, acc_empty, wc, tmem_base, stage, rank, owner);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOrRoleRegs));
    if (warp == 0 && lane == 0) {
      filled = or_producer<PAIR>(mA, mB, args, smem_u32(ring), full, empty, wc, rank, owner);
      if (PAIR && rank != 0) st_dsmem_u32(map_to_rank(smem_u32(peer_filled), 0), filled);
    } else {
      pdl_wait_prerequisites();
      if (warp == 1 && lane == 0 && rank == 0) {
        issued = or_mma<PAIR>(args, smem_u32(ring), full, empty, acc_full, acc_empty, wc,
                              tmem_base, owner);
        // every MMA finishes before TMEM is freed, also when an epilogue gave up
        if (issued) {
          if constexpr (PAIR) tc_commit_pair_self(smem_u32(drain));
          else tc_commit(smem_u32(drain));
          wait_drain(smem_u32(drain), 0, wc);
        }
      }
    }
  }
  __syncthreads();
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all();
  // after an abort copies may still be in flight: each stage's last one (of a pair, see
  // tc2_drain_loads)
  if (rank == 0 && threadIdx.x == 0) {
    const uint32_t n0 = filled, n1 = PAIR ? *peer_filled : filled, n = n0 > n1 ? n0 : n1;
#pragma unroll 1
    for (uint32_t s = 0; s < S && s < n; ++s) {
      const uint32_t at = s + ((n - 1 - s) / S) * S;
      const uint32_t bar = smem_u32(&full[s]);
      if (at >= n0) mbar_arrive_expect_tx(bar, Cfg::kStageBytes);
      else if (at >= n1) mbar_complete_tx(bar, Cfg::kStageBytes);
      wait_drain(bar, (at / S) & 1, wc);
    }
  }
  if constexpr (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
    else tmem_dealloc(tmem_base, Cfg::kTmemCols);
  }
}

}  // namespace dg

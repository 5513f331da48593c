// fp8_moe.cu: a whole mixture-of-experts layer for a few tokens in one launch.
//
//   l = x·routerᵀ, top-k and gates;  h = silu(gate_e x̂) * (up_e x̂);
//   out[t] = sum over the chosen e of gate[t, e] (down_e ĥ)
//
// With few tokens the layer is the stream of the chosen experts' weights, each
// byte used once per token that chose the expert, so the kernel is built around
// that stream: one persistent CTA per SM (a cooperative launch), and the k-blocks
// (128 rows x 128 k of one expert's matrix) of all chosen experts are shared out
// over the CTAs, first for gate and up, then for down: laid end to end and cut
// into equal ranges when they are few, handed out in fixed pieces at run time when
// they are many.  The weights are the MMA's 128-row side, the expert's tokens (x̂
// or ĥ, 16 to 64 rows) its columns; tensor cores because a weight then costs the
// same for one token or sixteen, and the TMA ring keeps 128 KiB a CTA in flight.
//
//   phase A  all workers: router logits, x̂                  -> barrier 1
//   phase B  every CTA for itself: top-k, token lists
//   phase C  gate and up: fp32 partial sums of each part     -> barrier 2
//            ĥ from those, each row once                     -> barrier 3
//   phase D  down: as C                                      -> barrier 4
//   phase E  out from phase D's partials and the gates
//
// Roles in C and D: warp 0 streams weights by TMA (it runs ahead into D: weights
// need no barrier), warp 1 issues MMAs, warp 2 copies the weights' scales, warps
// 4-7 read each k-block's product from TMEM and add it, scaled, into fp32
// registers, warps 8-11 copy the token operand into shared memory (swizzled as
// the MMA reads it), one buffer ahead.  The producer draws the work up and hands
// it to the other roles through a small ring.  A tile cut between CTAs leaves one
// partial per part; whoever reads it adds them in their order along K, so results
// do not depend on timing.  Every wait is bounded.
//
// Measured, weights from HBM: 32 tokens, 8 of 128 experts of 4096 x 1024: 231 to
// 235 us, 6.0 TB/s, 88 % of a copy's rate, so HBM bounds it; one token, 8 of 64 of 2048 x
// 1024: 29.1 us, of which 50 MB take 7.5: the rest is four grid barriers, code
// fetched cold and each phase's first loads.  ĥ formed by every CTA for its own
// tiles instead of once spares a barrier (28.5 us for the one token) but takes
// 173 instead of 92 us for 64 tokens, 2 of 16 experts of 4096 x 2048.
#include <algorithm>

#include "context.h"
#include "fp8_tc_kernel.cuh"
#include "moe_order.h"

namespace dg {
namespace {

constexpr int kMoeThreads = 384;
constexpr int kMoeStages = 4;                      // of two k-blocks
constexpr int kMoeStageBytes = 2 * kBM * kFp8Block;
constexpr int kMoeOperandBytes = 32768;            // one token operand buffer: 256 rows of 128 B
constexpr int kMoeRows = kMoeOperandBytes / kFp8Block;
constexpr int kMoeBuffers = 4;                     // TMEM accumulators, two of 64 columns each
constexpr int kMoeScaleGroup = 8, kMoeScaleRing = 4;
// A phase's k-blocks are cut into equal ranges of at least kMoeMinUnits (2 to 8
// time alike, 16 cost 8 us at 512 k-blocks), unless there are kMoeDynamicPieces
// pieces a CTA to hand out at run time: SMs get unequal shares of HBM, and whole
// tiles leave one partial each.  Measured, pieces against ranges: 238 and 246 us
// (32 tokens, 114 of 128 experts of 4096 x 1024), 86 and 92 (32 tokens, 63 of 64
// of 2048 x 1024); with 2 or 3 pieces a CTA 63 and 58 (8 tokens, 10 of 16 of 4096
// x 2048), 80 and 78 (4 tokens, 29 of 128 of 4096 x 1024).
constexpr int kMoeMinUnits = 4;
constexpr int kMoeDynamicPieces = 4;
// A piece is a part of one tile or several tiles, of about as many k-blocks as
// this (gate and up; down), and several only while kMoeRunPieces a CTA remain.
// Parts of 16 instead of 32: 4 us of 250 more; pieces of 64 and 32 for down alike.
constexpr int kMoePieceC = 32, kMoePieceD = 64;
constexpr int kMoeRunC = 16, kMoeRunD = 32;
constexpr int kMoeRunPieces = 6;

// Rows of B (tokens) of an MMA, a power of two, and k-blocks of them that an
// operand buffer holds.  Rows past the expert's tokens hold anything: they only
// reach columns that nobody reads.
__host__ __device__ constexpr int moe_shift(int n) { return n <= 16 ? 4 : n <= 32 ? 5 : 6; }
__host__ __device__ constexpr int moe_cap(int cols) { return kMoeRows / cols; }

struct MoeMaps {
  CUtensorMap group, one;  // {128, rows, k-block, expert}, {K, rows, expert}
};

// How a phase's tiles are cut when they are handed out at run time: `chunks`
// pieces of `chunk` k-blocks a tile, or up to `run` tiles of one expert a piece.
struct MoePieces {
  int32_t run, chunks, chunk;
};

struct MoeArgs {
  gemm_moe_fp8_t L;
  int32_t tiles_i, tiles_h, kb_h, kb_i;
  uint8_t* xq;      // tokens x kb_h * 128
  float* xs;        // tokens x kb_h
  float* logits;    // tokens x experts
  uint8_t* hq;      // picks x kb_i * 128
  float* hs;        // picks x kb_i
  float* part1;     // [segment][gate, up][pick][tiles_i * 128]
  float* part2;     // [segment][pick][tiles_h * 128]
  int* counters;    // barriers 1-4, exits, C's and D's pieces; 0 at launch and after
  int* status;
  uint64_t wait_limit_ns;
  int32_t vec;      // x and router rows are 16-byte aligned
  MoePieces pieces[2];
  int32_t dynamic;  // 1: pieces are handed out at run time whatever their number
};

// What phase B leaves in shared memory.
struct MoeRoute {
  uint64_t mask[GEMM_MOE_MAX_EXPERTS];   // tokens that chose the expert
  uint16_t off[GEMM_MOE_MAX_EXPERTS];    // first of its picks in `pick`
  uint16_t index[GEMM_MOE_MAX_EXPERTS];  // its place among the chosen experts
  uint16_t act[GEMM_MOE_MAX_EXPERTS];    // the chosen experts, ascending
  uint16_t ids[GEMM_MOE_MAX_TOKENS * GEMM_MOE_MAX_TOP_K];
  uint16_t pick[GEMM_MOE_MAX_TOKENS * GEMM_MOE_MAX_TOP_K];  // token * top_k + choice
  uint8_t token[GEMM_MOE_MAX_TOKENS * GEMM_MOE_MAX_TOP_K];  // and its token
  int32_t active;
};

// A quotient of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (((uint64_t(n) | uint64_t(d)) >> 32) == 0) return uint32_t(n) / uint32_t(d);
  return n / d;
}

// One phase's work: k-blocks laid end to end in `ctas` equal ranges, or (dynamic)
// pieces handed out by a counter.
struct MoeWork {
  int64_t blocks;   // k-blocks
  int64_t total;    // pieces
  int32_t per, kb;  // tiles of an expert, k-blocks of a tile
  int32_t ctas;
  const MoePieces& p;
  bool dynamic;
  int32_t run;      // tiles a piece
  int32_t pieces;   // of an expert
  __device__ __forceinline__ MoeWork(const MoeArgs& a, const MoeRoute& r, int32_t ph)
      : p(a.pieces[ph]) {
    kb = ph == 0 ? a.kb_h : a.kb_i;
    per = ph == 0 ? 2 * a.tiles_i : a.tiles_h;
    blocks = int64_t(r.active) * per * kb;
    const int64_t most = blocks / kMoeMinUnits;
    ctas = int32_t(most < 1 ? 1 : most < int64_t(gridDim.x) ? most : int64_t(gridDim.x));
    const int64_t tiles = int64_t(r.active) * per;
    dynamic = a.dynamic || tiles * p.chunks >= kMoeDynamicPieces * int64_t(gridDim.x);
    run = 1;
    if (p.run > 1)
      run = int32_t(max(int64_t(1), min(int64_t(p.run),
                                        quotient(tiles, kMoeRunPieces * gridDim.x))));
    pieces = p.chunks > 1 ? per * p.chunks : (per + run - 1) / run;
    total = int64_t(r.active) * pieces;
  }
  __device__ __forceinline__ int64_t begin(int32_t c) const {
    return c >= ctas ? blocks : quotient(blocks * c, ctas);
  }
  __device__ __forceinline__ int32_t owner(int64_t x) const {
    return int32_t(quotient((x + 1) * ctas - 1, blocks));
  }
  // Partials that a tile leaves.
  __device__ __forceinline__ int32_t segments(int64_t tile) const {
    if (dynamic) return p.chunks;
    return owner((tile + 1) * kb - 1) - owner(tile * kb) + 1;
  }
};

// A CTA's part of one tile.
struct MoeSeg {
  int32_t phase;     // 0 gate and up, 1 down
  int32_t expert, n; // and its tokens; n == 0: the phase is over
  int32_t which;     // 0 gate, 1 up, 2 down
  int32_t tile;      // 128-row tile of the matrix
  int32_t kb0, kb1, kb;
  int32_t seg;       // which of the tile's partials
};

// A CTA's segments of a phase, one after the other (the producer's; the other
// roles read them from its ring).
struct MoeSource {
  const MoeArgs& a;
  const MoeRoute& r;
  const MoeWork w;
  const int32_t phase;
  int64_t left = 0;           // static: k-blocks left of this CTA's range; dynamic: tiles
                              // left of the piece
  int32_t expert = 0, rest = 0, kb0 = 0, kb1 = 0, seg = 0;
  int32_t ahead = 0;          // dynamic: the piece after this one
  __device__ __forceinline__ MoeSource(const MoeArgs& a_, const MoeRoute& r_, int32_t ph)
      : a(a_), r(r_), w(a_, r_, ph), phase(ph) {
    if (w.dynamic) {
      ahead = int32_t(blockIdx.x);  // the counter hands out the rest
      return;
    }
    const int64_t x = w.begin(blockIdx.x);
    left = w.begin(blockIdx.x + 1) - x;
    if (left == 0) return;
    const int64_t tile = quotient(x, w.kb);
    expert = int32_t(quotient(tile, w.per));
    rest = int32_t(tile - int64_t(expert) * w.per);
    kb0 = int32_t(x - tile * w.kb);
    // only a range's first tile can have begun in another CTA's range
    if (kb0 > 0) seg = int32_t(blockIdx.x) - w.owner(tile * w.kb);
  }
  __device__ __forceinline__ bool next(MoeSeg& s) {
    if (w.dynamic && left == 0) {
      const int64_t piece = ahead;
      if (piece >= w.total) return false;
      // asked for one piece early: the answer takes about a microsecond
      ahead = int32_t(gridDim.x) + atomicAdd(a.counters + 5 + phase, 1);
      expert = int32_t(quotient(piece, w.pieces));
      const int32_t i = int32_t(piece - int64_t(expert) * w.pieces);
      if (w.p.chunks > 1) {
        rest = i / w.p.chunks;
        seg = i - rest * w.p.chunks;
        kb0 = seg * w.p.chunk;
        kb1 = min(kb0 + w.p.chunk, w.kb);
        left = 1;
      } else {
        rest = i * w.run;
        seg = kb0 = 0;
        kb1 = w.kb;
        left = min(w.run, w.per - rest);
      }
    }
    if (left == 0) return false;
    if (!w.dynamic) kb1 = left < w.kb - kb0 ? int32_t(kb0 + left) : w.kb;
    s.phase = phase;
    s.kb = w.kb;
    s.kb0 = kb0;
    s.kb1 = kb1;
    s.seg = seg;
    s.expert = r.act[expert];
    s.n = __popcll(r.mask[s.expert]);
    const int32_t second = phase == 0 && rest >= a.tiles_i;
    s.which = phase == 1 ? 2 : second;
    s.tile = second ? rest - a.tiles_i : rest;
    left -= w.dynamic ? 1 : kb1 - kb0;
    if (!w.dynamic) kb0 = seg = 0;
    if (++rest == w.per && !w.dynamic) {
      rest = 0;
      ++expert;
    }
    return true;
  }
};

// The ring of segments, from the producer to the warps of the other roles.
constexpr int kMoeSegs = 4;
constexpr int kMoeSegReaders = 1 + 1 + 4 + 4;  // warps: MMA, scales, accumulators, builders
struct MoeRing {
  const MoeSeg* slot;
  uint32_t full, empty;
  uint32_t d = 0, ph = 0;
  // The next segment; false at the end of a phase, or (ok cleared) when the wait
  // gave up.
  __device__ __forceinline__ bool next(MoeSeg& s, const WaitCtl& wc, bool& ok) {
    ok = __all_sync(0xffffffffu, ok && wait_bounded(full + 8 * d, ph, wc, kSiteEpilogue));
    if (!ok) return false;
    s = slot[d];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * d);
    if (++d == kMoeSegs) {
      d = 0;
      ph ^= 1;
    }
    return s.n > 0;
  }
};

// The token operand's buffers as every role sees them: content is one expert's
// rows for a range of k-blocks; a whole-K content serves every segment of the
// same phase and expert that follows.
struct MoeContent {
  int32_t phase = -1, expert = -1;
  bool whole = false;
  uint32_t count = 0;  // contents so far; buffer (count - 1) & 1
  // True if the chunk needs a new content.
  __device__ __forceinline__ bool advance(const MoeSeg& s, bool whole_) {
    if (whole_ && whole && phase == s.phase && expert == s.expert) return false;
    phase = s.phase;
    expert = s.expert;
    whole = whole_;
    ++count;
    return true;
  }
  __device__ __forceinline__ uint32_t buf() const { return (count - 1) & 1; }
  __device__ __forceinline__ uint32_t parity() const { return ((count - 1) >> 1) & 1; }
};

// Floats in a total order as integers: NaN above +inf, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float f) {
  if (f != f) return 0xffffffffu;
  const uint32_t u = __float_as_uint(f + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float from16(uint16_t h, int dtype) {
  if (dtype == GEMM_F16) {
    __half v;
    __builtin_memcpy(&v, &h, 2);
    return __half2float(v);
  }
  return __uint_as_float(uint32_t(h) << 16);
}

__device__ __forceinline__ void widen8(const uint4& w, int dtype, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = from16(uint16_t(u[j / 2] >> (16 * (j & 1))), dtype);
}

// One block of 128 values, 4 per lane, quantised by a warp: this lane's 4 bytes;
// every lane gets the scale.
__device__ __forceinline__ uint32_t quant_block(const float (&v)[4], float& scale) {
  float m = 0.f, w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = fabsf(v[j]) == INFINITY ? NAN : v[j];
    m = fmaxf(m, fabsf(w[j]));
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float inv = fp8_inverse(m);
  scale = fp8_scale(m);
  return pack_e4m3x4(__fmul_rn(w[0], inv), __fmul_rn(w[1], inv), __fmul_rn(w[2], inv),
                     __fmul_rn(w[3], inv));
}

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// One thread arrives on a barrier's counter for its CTA, after a barrier among
// the threads whose writes the arrival is to publish: the fence covers theirs too.
__device__ __forceinline__ void grid_arrive(int* counter) {
  __threadfence();
  atomicAdd(counter, 1);
}

// Waits (bounded) until all CTAs have arrived on a barrier's counter.  A barrier
// among the CTA's threads then hands what was acquired on to them.
__device__ __forceinline__ bool grid_wait(const int* counter, const WaitCtl& wc) {
  const uint64_t t0 = globaltimer_ns();
  while (ld_acquire(counter) < int(gridDim.x)) {
    if (*wc.abort) return false;
    if (globaltimer_ns() - t0 > wc.limit_ns) {
      *wc.abort = 1;
      atomicCAS(wc.status, 0, 1 + kSiteEpilogue);
      return false;
    }
  }
  return true;
}

// Weights are read once: they leave L2 first, and the partials, x and the code stay.
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void load_weights_4d(uint32_t dst, const CUtensorMap* map,
                                                uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                                                int32_t c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}
__device__ __forceinline__ void load_weights_3d(uint32_t dst, const CUtensorMap* map,
                                                uint32_t bar, int32_t c0, int32_t c1, int32_t c2,
                                                uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ------------------------------------------------------------------- phase A --
// Router logits: a CTA takes (expert, 8 tokens) tasks, its 8 worker warps an
// eighth of the hidden axis each.  x̂: a warp per (token, k-block).
__device__ __forceinline__ void moe_phase_a(const MoeArgs& a, float* red0, int tid) {
  const gemm_moe_fp8_t& L = a.L;
  const int warp = tid >> 5, lane = tid & 31;
  const int64_t H = L.hidden;
  const uint16_t* x = static_cast<const uint16_t*>(L.x);
  const uint16_t* router = static_cast<const uint16_t*>(L.router);
  const int32_t T = int32_t(L.tokens), E = int32_t(L.experts);
  const int32_t groups = (T + 7) / 8;
  float* red = red0;
  int turn = 0;
  for (int32_t task = blockIdx.x; task < E * groups; task += gridDim.x) {
    const int32_t e = task / groups, t0 = (task - e * groups) * 8;
    float s[8] = {};
    for (int64_t c = (warp * 32 + lane) * 8; c < H; c += 8 * 256) {
      if (a.vec && c + 8 <= H) {  // every load in flight before the first is used
        uint4 raw[9];
        raw[8] = __ldg(reinterpret_cast<const uint4*>(router + e * L.ld_router + c));
#pragma unroll
        for (int i = 0; i < 8; ++i)  // tokens past the last repeat it
          if (i == 0 || T > 1)
            raw[i] = __ldg(reinterpret_cast<const uint4*>(x + min(t0 + i, T - 1) * L.ld_x + c));
        float w[8];
        widen8(raw[8], L.dtype, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i > 0 && T == 1) break;
          float v[8];
          widen8(raw[i], L.dtype, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) s[i] = fmaf(v[j], w[j], s[i]);
        }
      } else {
        for (int j = 0; j < 8 && c + j < H; ++j) {
          const float w = from16(router[e * L.ld_router + c + j], L.dtype);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            s[i] = fmaf(from16(x[min(t0 + i, T - 1) * L.ld_x + c + j], L.dtype), w, s[i]);
        }
      }
    }
    // 8 sums over 32 lanes: halve the sums a lane holds three times, then add
    // over the 4 lanes left; token i's sum ends in lanes 4 i ... 4 i + 3
#pragma unroll
    for (int h = 4; h > 0; h >>= 1) {
      const bool high = (lane & (h * 4)) != 0;
#pragma unroll
      for (int i = 0; i < h; ++i) {
        const float give = high ? s[i] : s[i + h], keep = high ? s[i + h] : s[i];
        s[i] = keep + __shfl_xor_sync(0xffffffffu, give, h * 4);
      }
    }
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 1);
    s[0] += __shfl_xor_sync(0xffffffffu, s[0], 2);
    red = red0 + (turn ^= 64);  // the other half: the task before last has been read
    if ((lane & 3) == 0) red[warp * 8 + (lane >> 2)] = s[0];
    bar_sync(1, 256);
    if (tid < 8 && t0 + tid < T) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) v += red[w * 8 + tid];
      a.logits[(t0 + tid) * E + e] = v;
    }
  }
  // from the last CTA backwards, as the logits' tasks go from the first on
  const int64_t tasks = int64_t(T) * a.kb_h;
  for (int64_t i = int64_t(gridDim.x - 1 - blockIdx.x) * 8 + warp; i < tasks;
       i += int64_t(gridDim.x) * 8) {
    const int64_t t = i / a.kb_h, kb = i - t * a.kb_h;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = kb * kFp8Block + lane * 4 + j;
      v[j] = c < H ? from16(x[t * L.ld_x + c], L.dtype) : 0.f;
    }
    float scale;
    const uint32_t q = quant_block(v, scale);
    reinterpret_cast<uint32_t*>(a.xq + (t * a.kb_h + kb) * kFp8Block)[lane] = q;
    if (lane == 0) a.xs[t * a.kb_h + kb] = scale;
  }
}

// ------------------------------------------------------------------- phase B --
// The experts of a token, by one warp: one largest key after the other, of equal
// ones the lowest index.  PER keys a lane.
template <int PER>
__device__ __forceinline__ void moe_choose(const MoeArgs& a, MoeRoute& r, int32_t t, int lane) {
  const int32_t E = int32_t(a.L.experts), k = a.L.top_k;
  uint32_t key[PER], mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int32_t e = i * 32 + lane;
    key[i] = e < E ? order_key(__ldcg(a.logits + int64_t(t) * E + e)) : 0;  // 0: below all
  }
#pragma unroll 1
  for (int32_t j = 0; j < k; ++j) {
    uint32_t most = key[0];
#pragma unroll
    for (int i = 1; i < PER; ++i) most = max(most, key[i]);
    most = __reduce_max_sync(0xffffffffu, most);
    uint32_t e = 0xffffu;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) e = key[i] == most ? uint32_t(i * 32 + lane) : e;
    e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = e == uint32_t(i * 32 + lane) ? 0 : key[i];
    mine = lane == j ? e : mine;
  }
  if (lane < k) {
    r.ids[t * k + lane] = uint16_t(mine);
    atomicOr(reinterpret_cast<unsigned long long*>(&r.mask[mine]), 1ull << t);
  }
}

// Every warp of the CTA: the experts of its tokens; then, by one, who was chosen and
// where each expert's picks begin.
__device__ __forceinline__ void moe_phase_b(const MoeArgs& a, MoeRoute& r) {
  const gemm_moe_fp8_t& L = a.L;
  const int32_t T = int32_t(L.tokens), E = int32_t(L.experts);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int32_t t = warp; t < T; t += kMoeThreads / 32) {
    if (E <= 64) moe_choose<2>(a, r, t, lane);
    else if (E <= 128) moe_choose<4>(a, r, t, lane);
    else moe_choose<GEMM_MOE_MAX_EXPERTS / 32>(a, r, t, lane);
  }
  __syncthreads();
  if (tid < 32) {  // prefix sums over the experts
    int32_t picks = 0, active = 0;
    for (int32_t e0 = 0; e0 < E; e0 += 32) {
      const int32_t e = e0 + tid;
      const int32_t n = e < E ? __popcll(r.mask[e]) : 0;
      int32_t sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, sum, d);
        if (tid >= d) sum += o;
      }
      const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
      const int32_t place = active + __popc(some & ((1u << tid) - 1));
      if (e < E) {
        r.off[e] = uint16_t(picks + sum - n);
        r.index[e] = uint16_t(place);
        if (n > 0) r.act[place] = uint16_t(e);
      }
      picks += __shfl_sync(0xffffffffu, sum, 31);
      active += __popc(some);
    }
    if (tid == 0) r.active = active;
  }
  __syncthreads();
}

// Who of an expert's tokens picked it as what: its readers' own (warps 4-11).
__device__ __forceinline__ void moe_picks(const MoeArgs& a, MoeRoute& r) {
  const int32_t T = int32_t(a.L.tokens), k = a.L.top_k;
  for (int32_t p = int32_t(threadIdx.x) - 128; p < T * k; p += 256) {
    const int32_t t = p / k, e = r.ids[p];
    const int32_t at = r.off[e] + __popcll(r.mask[e] & ((1ull << t) - 1));
    r.pick[at] = uint16_t(p);
    r.token[at] = uint8_t(t);
  }
  bar_sync(1, 256);
}

// Token t's gates, choice j's in lane j (one warp): the exponentials of the chosen
// logits over the sum of theirs, or of all.
__device__ __forceinline__ float moe_gate(const MoeArgs& a, const MoeRoute& r, int32_t t,
                                          int lane) {
  const int32_t E = int32_t(a.L.experts), k = a.L.top_k;
  const float* l = a.logits + int64_t(t) * E;
  const float top = __ldcg(l + r.ids[t * k]);
  const float mine = lane < k ? expf(__ldcg(l + r.ids[t * k + lane]) - top) : 0.f;
  float sum = mine;
  if (!a.L.renormalize) {
    sum = 0.f;
    for (int32_t e = lane; e < E; e += 32) sum += expf(__ldcg(l + e) - top);
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return mine / sum;
}

// Gates and ids, as the layer returns them: one warp per token, spread over the
// CTAs (warp 3, beside the streaming).
__device__ __forceinline__ void moe_gates(const MoeArgs& a, const MoeRoute& r, int lane) {
  const int32_t k = a.L.top_k;
  for (int32_t t = int32_t(blockIdx.x); t < int32_t(a.L.tokens); t += int32_t(gridDim.x)) {
    const float gate = moe_gate(a, r, t, lane);
    if (lane < k) {
      a.L.ids[t * k + lane] = r.ids[t * k + lane];
      a.L.gates[t * k + lane] = gate;
    }
  }
}

// --------------------------------------------------------------- phases C, D --
__device__ __forceinline__ uint32_t moe_producer(const MoeArgs& a, const MoeRoute& r,
                                                 const MoeMaps& gate, const MoeMaps& up,
                                                 const MoeMaps& down, MoeSeg* segs,
                                                 uint32_t seg_full, uint32_t seg_empty,
                                                 uint32_t ring, uint32_t full,
                                                 uint32_t empty, const WaitCtl& wc) {
  uint32_t s = 0, ph = 0, filled = 0;
  const uint64_t policy = policy_evict_first();
  uint32_t d = 0, dph = 0;
  auto publish = [&](const MoeSeg& g) {
    if (!wait_bounded(seg_empty + 8 * d, dph ^ 1, wc, kSiteProducer)) return false;
    segs[d] = g;
    mbar_arrive(seg_full + 8 * d);
    if (++d == kMoeSegs) {
      d = 0;
      dph ^= 1;
    }
    return true;
  };
  for (int phase = 0; phase < 2; ++phase) {
    MoeSource source(a, r, phase);
    const int32_t k_full = int32_t((phase == 0 ? a.L.hidden : a.L.inner) / kFp8Block);
    MoeSeg g;
    while (source.next(g)) {
      if (!publish(g)) return filled;
      const MoeMaps* m = g.which == 0 ? &gate : g.which == 1 ? &up : &down;
      for (int32_t kb = g.kb0; kb < g.kb1; kb += 2) {
        if (!wait_bounded(empty + 8 * s, ph ^ 1, wc, kSiteProducer)) return filled;
        const uint32_t bar = full + 8 * s, dst = ring + s * kMoeStageBytes;
        mbar_arrive_expect_tx(bar, kMoeStageBytes);
        if (kb + 2 <= k_full) {
          load_weights_4d(dst, &m->group, bar, 0, g.tile * kBM, kb, g.expert, policy);
        } else {
          for (int j = 0; j < 2; ++j)
            load_weights_3d(dst + j * kBM * kFp8Block, &m->one, bar, (kb + j) * kFp8Block,
                            g.tile * kBM, g.expert, policy);
        }
        ++filled;
        if (++s == kMoeStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    g.n = 0;
    if (!publish(g)) return filled;
  }
  return filled;
}

// The weights' scales (one per k-block of a tile): 8 at a time, one per lane.
__device__ __forceinline__ void moe_scales(const MoeArgs& a, MoeRing segs, uint32_t ring,
                                           uint32_t sc_full, uint32_t sc_empty, int lane,
                                           const WaitCtl& wc) {
  uint32_t slot = 0, ph = 0;
  bool ok = true;
  for (int phase = 0; phase < 2 && ok; ++phase) {
    MoeSeg g;
    while (segs.next(g, wc, ok)) {
      const gemm_fp8_experts_t& w = g.which == 0 ? a.L.gate : g.which == 1 ? a.L.up : a.L.down;
      const float* p = w.scale + g.expert * w.scale_stride_e + g.tile * w.scale_stride_r;
      for (int32_t kb = g.kb0; kb < g.kb1; kb += kMoeScaleGroup) {
        ok = __all_sync(0xffffffffu, wait_bounded(sc_empty + 8 * slot, ph ^ 1, wc, kSiteProducer));
        if (!ok) break;
        if (lane < kMoeScaleGroup && kb + lane < g.kb1)
          cp_async4(ring + (slot * kMoeScaleGroup + lane) * 4, p + (kb + lane) * w.scale_stride_c);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sc_full +
                                                                                 8 * slot)
                     : "memory");
        if (++slot == kMoeScaleRing) {
          slot = 0;
          ph ^= 1;
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Whether it issued anything.
__device__ __forceinline__ bool moe_mma(MoeRing segs, uint32_t ring, uint32_t operand,
                                        uint32_t full, uint32_t empty, uint32_t acc_full,
                                        uint32_t acc_empty, uint32_t b_full, uint32_t b_empty,
                                        uint32_t tmem_base, const WaitCtl& wc) {
  uint32_t s = 0, ph = 0, b = 0, phases = (1u << kMoeBuffers) - 1;
  bool ok = true, any = false;
  const bool leader = f8_elect();
  const uint64_t adesc0 = make_sdesc_sw128(ring, 16, 1024);
  const uint64_t bdesc0 = make_sdesc_sw128(operand, 16, 1024);
  MoeContent content;
  auto wait = [&](uint32_t bar, uint32_t parity, int site) {
    if (ok && !mbar_test(bar, parity)) ok = wait_bounded(bar, parity, wc, site);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  for (int phase = 0; phase < 2 && ok; ++phase) {
    MoeSeg g;
    while (segs.next(g, wc, ok)) {
      const int cols = 1 << moe_shift(g.n), cap = moe_cap(cols);
      const bool whole = g.kb <= cap;
      const uint32_t idesc = make_idesc_f16(kBM, cols, 0, 0);
      for (int32_t c0 = g.kb0; ok && c0 < g.kb1; c0 += cap) {
        const int32_t c1 = whole ? g.kb1 : min(c0 + cap, g.kb1);
        const int32_t base = whole ? 0 : c0;  // the content's first k-block
        const uint32_t old = content.buf();
        const bool had = content.count > 0;
        if (content.advance(g, whole)) {
          if (had && leader) tc_commit(b_empty + 8 * old);
          if (!wait(b_full + 8 * content.buf(), content.parity(), kSiteMmaFull)) break;
          tc_fence_after();
        }
        const uint64_t bd = bdesc0 + ((content.buf() * kMoeOperandBytes) >> 4);
        for (int32_t kb = c0; ok && kb < c1; kb += 2) {
          if (!wait(full + 8 * s, ph, kSiteMmaFull)) break;
          if (!wait(acc_empty + 8 * b, (phases >> b) & 1, kSiteMmaAccum)) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (kb + j >= c1) break;
              const uint64_t ad = adesc0 + ((s * kMoeStageBytes + j * kBM * kFp8Block) >> 4);
              const uint64_t bj = bd + uint64_t(((kb + j - base) * cols * kFp8Block) >> 4);
#pragma unroll
              for (int kk = 0; kk < kFp8Block / 32; ++kk)
                tc_mma_f8(tmem_base + b * 128 + j * 64, ad + 2 * kk, bj + 2 * kk, idesc,
                          kk > 0 ? 1u : 0u);
            }
            tc_commit(empty + 8 * s);
            tc_commit(acc_full + 8 * b);
          }
          __syncwarp();
          any = true;
          phases ^= 1u << b;
          b = (b + 1) & (kMoeBuffers - 1);
          if (++s == kMoeStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (whole) break;
      }
    }
  }
  return any;
}

// Warps 4-7: thread `row` owns one weight row; sums of up to 64 tokens.  A block's sum
// meets the weight's scale, then the token's, whose product might not fit fp32.
__device__ __forceinline__ void moe_accumulate(const MoeArgs& a, const MoeRoute& r, MoeRing segs,
                                               const float* scale_ring, const float* b_scale,
                                               uint32_t acc_full, uint32_t acc_empty,
                                               uint32_t b_full, uint32_t b_empty, uint32_t sc_full,
                                               uint32_t sc_empty, uint32_t tmem_base,
                                               const WaitCtl& wc) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int row = warp * 32 + lane;
  const uint32_t tlane = tmem_base + (uint32_t(warp * 32) << 16);
  uint32_t b = 0, phases = 0, slot = 0, sph = 0;
  bool ok = true;
  const int32_t picks = int32_t(a.L.tokens) * a.L.top_k;
  MoeContent content;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok && !mbar_test(bar, parity)) ok = wait_bounded(bar, parity, wc, kSiteEpilogue);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  for (int phase = 0; phase < 2; ++phase) {
    MoeSeg g;
    while (segs.next(g, wc, ok)) {
      const int cols = 1 << moe_shift(g.n), cap = moe_cap(cols);
      const bool whole = g.kb <= cap;
      float acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0.f;
      for (int32_t c0 = g.kb0; ok && c0 < g.kb1; c0 += cap) {
        const int32_t c1 = whole ? g.kb1 : min(c0 + cap, g.kb1);
        const int32_t base = whole ? 0 : c0;
        const uint32_t old = content.buf();
        const bool had = content.count > 0;
        if (content.advance(g, whole)) {
          __syncwarp();
          if (had && lane == 0) mbar_arrive(b_empty + 8 * old);
          if (!wait(b_full + 8 * content.buf(), content.parity())) break;
        }
        const float* bs = b_scale + content.buf() * kMoeRows;
        for (int32_t kb = c0; ok && kb < c1; kb += 2) {
          const int32_t i = (kb - g.kb0) % kMoeScaleGroup;
          if (i == 0 && !wait(sc_full + 8 * slot, sph)) break;
          const bool two = kb + 1 < c1;
          const float w0 = scale_ring[slot * kMoeScaleGroup + i];
          const float w1 = two ? scale_ring[slot * kMoeScaleGroup + i + 1] : 0.f;
          if (!wait(acc_full + 8 * b, (phases >> b) & 1)) break;
          tc_fence_after();
          const float* bk = bs + (kb - base) * cols;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c * 16 >= cols) break;
            uint32_t v0[16], v1[16];
            tmem_issue<16>(tlane + b * 128 + c * 16, v0);
            if (two) tmem_issue<16>(tlane + b * 128 + 64 + c * 16, v1);
            tmem_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) fma_tmem2(acc[c * 16 + j], w0, bk[c * 16 + j], v0[j]);
            if (two) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                fma_tmem2(acc[c * 16 + j], w1, bk[cols + c * 16 + j], v1[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(acc_empty + 8 * b);
          phases ^= 1u << b;
          b = (b + 1) & (kMoeBuffers - 1);
          if (i + 2 >= kMoeScaleGroup || kb + 2 >= g.kb1) {
            if (lane == 0) mbar_arrive(sc_empty + 8 * slot);
            if (++slot == kMoeScaleRing) {
              slot = 0;
              sph ^= 1;
            }
          }
        }
        if (whole) break;
      }
      if (!ok) break;
      const int64_t ld = int64_t(phase == 0 ? a.tiles_i : a.tiles_h) * kBM;
      float* out = phase == 0 ? a.part1 + (int64_t(g.seg) * 2 + g.which) * picks * ld
                              : a.part2 + int64_t(g.seg) * picks * ld;
      out += g.tile * kBM + row;
      const uint16_t* pick = r.pick + r.off[g.expert];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c * 16 >= g.n) break;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c * 16 + i < g.n) __stcg(out + int64_t(pick[c * 16 + i]) * ld, acc[c * 16 + i]);
      }
    }
    // this CTA's partials of the phase are written
    bar_sync(2, 128);
    if (threadIdx.x == 128) grid_arrive(a.counters + 1 + 2 * phase);
  }
}

// The sum of `n` partials, the first four's loads in flight together.
__device__ __forceinline__ float4 sum_segments(const float* p, int64_t step, int32_t n) {
  constexpr int kAhead = 4;
  float4 v[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) v[i] = __ldcg(reinterpret_cast<const float4*>(p + i * step));
  }
  float4 s = v[0];
#pragma unroll
  for (int i = 1; i < kAhead; ++i) {
    s.x += v[i].x; s.y += v[i].y; s.z += v[i].z; s.w += v[i].w;
  }
  for (int32_t i = kAhead; i < n; ++i) {
    const float4 w = __ldcg(reinterpret_cast<const float4*>(p + i * step));
    s.x += w.x; s.y += w.y; s.z += w.z; s.w += w.w;
  }
  return s;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// ĥ from phase C's partials, quantised, shared out over all CTAs: a warp takes a
// row of 128 values (a pick's k-block), two at a time (warps 8-11).
__device__ __forceinline__ void moe_rows(const MoeArgs& a, const MoeRoute& r, int warp, int lane) {
  constexpr int kRows = 2;
  const MoeWork w(a, r, 0);
  const int64_t picks = a.L.tokens * a.L.top_k, rows = picks * a.kb_i;
  const int64_t ld = int64_t(a.tiles_i) * kBM, to_up = picks * ld;
  const int64_t step = 4 * int64_t(gridDim.x);
  for (int64_t i0 = blockIdx.x + int64_t(warp) * gridDim.x; i0 < rows; i0 += step * kRows) {
    float4 gt[kRows], up[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t i = i0 + step * j;
      if (i >= rows) break;
      const int32_t pick = int32_t(quotient(i, a.kb_i)), kb = int32_t(i - int64_t(pick) * a.kb_i);
      const float* p = a.part1 + pick * ld + kb * kFp8Block + lane * 4;
      const int64_t tile = int64_t(r.index[r.ids[pick]]) * 2 * a.tiles_i + kb;
      const int32_t n = w.segments(tile + (lane & 1) * a.tiles_i);
      gt[j] = sum_segments(p, 2 * to_up, __shfl_sync(0xffffffffu, n, 0));
      up[j] = sum_segments(p + to_up, 2 * to_up, __shfl_sync(0xffffffffu, n, 1));
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t i = i0 + step * j;
      if (i >= rows) break;
      const float h[4] = {gt[j].x / (1.f + expf(-gt[j].x)) * up[j].x,
                          gt[j].y / (1.f + expf(-gt[j].y)) * up[j].y,
                          gt[j].z / (1.f + expf(-gt[j].z)) * up[j].z,
                          gt[j].w / (1.f + expf(-gt[j].w)) * up[j].w};
      float scale;
      const uint32_t q = quant_block(h, scale);
      __stcg(reinterpret_cast<uint32_t*>(a.hq + i * kFp8Block) + lane, q);
      if (lane == 0) __stcg(a.hs + i, scale);
    }
  }
}

// Warps 8-11: ĥ between the phases, and the token operand.  The order is
// builder_run's.
struct MoeBuilder {
  const MoeArgs& a;
  const MoeRoute& r;
  MoeRing segs;
  uint8_t* operand;
  float* b_scale;
  uint32_t b_full, b_empty;
  volatile int* flag;     // whether the grid's barrier came
  volatile int* gave_up;  // 1: a warp's wait in phase C ran out
  const WaitCtl& wc;
  MoeContent content;

  // Every CTA's partials of phase C, also in a CTA without work in phase D.  (A
  // barrier that votes, bar.red, cost the one-token layer 0.35 of 29 us.)
  __device__ __forceinline__ bool partials(bool ok) {
    if (!ok) *gave_up = 1;
    if (threadIdx.x == 256) *flag = ok && grid_wait(a.counters + 1, wc);
    bar_sync(3, 128);
    return *flag != 0 && *gave_up == 0;
  }
  __device__ __forceinline__ void rows() {
    moe_rows(a, r, int(threadIdx.x - 256) >> 5, threadIdx.x & 31);
  }
  __device__ __forceinline__ bool rows_done() {
    bar_sync(3, 128);
    if (threadIdx.x == 256) {
      grid_arrive(a.counters + 2);
      *flag = grid_wait(a.counters + 2, wc);
    }
    bar_sync(3, 128);
    return *flag != 0;
  }
  __device__ __forceinline__ bool contents(int phase) {
    const int tid = threadIdx.x - 256;
    bool ok = true;
    const uint8_t* rows_q = phase == 0 ? a.xq : a.hq;
    const float* rows_s = phase == 0 ? a.xs : a.hs;
    MoeSeg g;
    while (segs.next(g, wc, ok)) {
      const int cols = 1 << moe_shift(g.n), cap = moe_cap(cols);
      const bool whole = g.kb <= cap;
      for (int32_t c0 = g.kb0; ok && c0 < g.kb1; c0 += cap) {
        const int32_t base = whole ? 0 : c0;
        const int32_t blocks = whole ? g.kb : min(cap, g.kb1 - c0);
        if (content.advance(g, whole)) {
          const uint32_t buf = content.buf();
          ok = __all_sync(0xffffffffu, wait_bounded(b_empty + 8 * buf, content.parity() ^ 1, wc,
                                                    kSiteProducer));
          if (!ok) break;
          uint8_t* dst = operand + buf * kMoeOperandBytes;
          float* bs = b_scale + buf * kMoeRows;
          const uint16_t* pick = r.pick + r.off[g.expert];
          const uint8_t* token = r.token + r.off[g.expert];
          const int32_t rows = blocks * g.n;
          auto at = [&](int32_t i, int32_t& row) {  // row i of the content: its block in memory
            const int32_t kb = i / g.n, n = i - kb * g.n;
            row = kb * cols + n;
            return int64_t(phase == 0 ? token[n] : pick[n]) * g.kb + base + kb;
          };
          // the real rows' 16-byte pieces, all in flight together
          const int c = tid & 7;
          int32_t row;
          for (int32_t i = tid >> 3; i < rows; i += 16) {
            const uint8_t* src = rows_q + at(i, row) * kFp8Block + c * 16;
            cp_async16(smem_u32(dst + row * kFp8Block + ((c ^ (row & 7)) << 4)), src);
          }
          for (int32_t i = tid; i < rows; i += 128) {
            const float s = __ldcg(rows_s + at(i, row));
            bs[row] = s;
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          fence_proxy_async_smem();  // the MMA reads the operand through the async proxy
          mbar_arrive(b_full + 8 * buf);
        }
        if (whole) break;
      }
    }
    return ok;
  }
};

// ------------------------------------------------------------------- phase E --
// `arrived` is called once, before the first partial is read.
template <class F>
__device__ __forceinline__ void moe_phase_e(const MoeArgs& a, const MoeRoute& r, F&& arrived) {
  const gemm_moe_fp8_t& L = a.L;
  const int32_t k = L.top_k, picks = int32_t(L.tokens) * k;
  const int64_t H = L.hidden, ld = int64_t(a.tiles_h) * kBM, step = int64_t(picks) * ld;
  const MoeWork w(a, r, 1);
  // A warp takes (token, 128 columns): lane j works out choice j's gate and how
  // many partials its tile has (the first item's before the barrier), then all
  // lanes add 4 columns each.
  const int lane = threadIdx.x & 31;
  const int64_t items = L.tokens * a.tiles_h;
  int64_t i = int64_t(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  bool waiting = true;
  do {
    const int32_t t = int32_t(quotient(i, a.tiles_h)), tile = int32_t(i - int64_t(t) * a.tiles_h);
    int32_t my_n = 0;
    if (lane < k && i < items)
      my_n = w.segments(int64_t(r.index[r.ids[t * k + lane]]) * a.tiles_h + tile);
    const float my_gate = i < items ? moe_gate(a, r, t, lane) : 0.f;
    if (waiting && !arrived()) return;
    waiting = false;
    if (i >= items) return;
    const int64_t h = int64_t(tile) * kBM + lane * 4;
    const float* src = a.part2 + int64_t(t) * k * ld + h;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int32_t j = 0; j < k; ++j) {
      const float gate = __shfl_sync(0xffffffffu, my_gate, j);
      const int32_t n = __shfl_sync(0xffffffffu, my_n, j);
      const float4 y = sum_segments(src + j * ld, step, n);
      o.x = fmaf(gate, y.x, o.x);
      o.y = fmaf(gate, y.y, o.y);
      o.z = fmaf(gate, y.z, o.z);
      o.w = fmaf(gate, y.w, o.w);
    }
    const float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (h + j < H) store_typed(L.out, t * L.ld_out + h + j, v[j], L.dtype);
    i += int64_t(gridDim.x) * (kMoeThreads / 32);
  } while (i < items);
}

// Shared memory: weight ring, two operand buffers, routing, scales, barriers.
struct MoeSmem {
  static constexpr int ring = 0;
  static constexpr int operand = ring + kMoeStages * kMoeStageBytes;
  static constexpr int route = operand + 2 * kMoeOperandBytes;
  static constexpr int b_scale = route + int((sizeof(MoeRoute) + 15) / 16 * 16);
  static constexpr int scale_ring = b_scale + 2 * kMoeRows * 4;
  static constexpr int red = scale_ring + kMoeScaleRing * kMoeScaleGroup * 4;
  static constexpr int segs = red + 2 * 64 * 4;
  static constexpr int bars = segs + int(sizeof(MoeSeg)) * kMoeSegs;
  static constexpr int kBars = 2 * kMoeStages + 2 * kMoeBuffers + 2 * 2 + 2 * kMoeScaleRing + 1 +
                               2 * kMoeSegs;
  static constexpr int words = bars + kBars * 8;
  // TMEM, abort, barrier, abort in phase E, builders (2)
  static constexpr int bytes = 1024 + words + 32;
};
static_assert(MoeSmem::bytes <= 227 * 1024, "shared memory per CTA");

__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_kernel(const __grid_constant__ MoeMaps gate, const __grid_constant__ MoeMaps up,
               const __grid_constant__ MoeMaps down, const __grid_constant__ MoeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  MoeRoute& r = *reinterpret_cast<MoeRoute*>(smem + MoeSmem::route);
  float* b_scale = reinterpret_cast<float*>(smem + MoeSmem::b_scale);
  float* scale_ring = reinterpret_cast<float*>(smem + MoeSmem::scale_ring);
  const uint32_t full = smem_u32(smem + MoeSmem::bars);
  const uint32_t empty = full + 8 * kMoeStages;
  const uint32_t acc_full = empty + 8 * kMoeStages;
  const uint32_t acc_empty = acc_full + 8 * kMoeBuffers;
  const uint32_t b_full = acc_empty + 8 * kMoeBuffers;
  const uint32_t b_empty = b_full + 16;
  const uint32_t sc_full = b_empty + 16;
  const uint32_t sc_empty = sc_full + 8 * kMoeScaleRing;
  const uint32_t seg_full = sc_empty + 8 * kMoeScaleRing;
  const uint32_t seg_empty = seg_full + 8 * kMoeSegs;
  const uint32_t drain = seg_empty + 8 * kMoeSegs;
  MoeSeg* seg_slot = reinterpret_cast<MoeSeg*>(smem + MoeSmem::segs);
  const MoeRing segs{seg_slot, seg_full, seg_empty};
  int* words = reinterpret_cast<int*>(smem + MoeSmem::words);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
  volatile int* abort_flag = words + 1;
  const WaitCtl wc{a.wait_limit_ns, a.status, abort_flag};

  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < int(a.L.experts); e += kMoeThreads) r.mask[e] = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMoeStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kMoeBuffers; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_full + 8 * i, 128);
      mbar_init(b_empty + 8 * i, 1 + 4);  // the MMA issuer's commit, four reading warps
    }
    for (int i = 0; i < kMoeScaleRing; ++i) {
      mbar_init(sc_full + 8 * i, 32);
      mbar_init(sc_empty + 8 * i, 4);
    }
    for (int i = 0; i < kMoeSegs; ++i) {
      mbar_init(seg_full + 8 * i, 1);
      mbar_init(seg_empty + 8 * i, kMoeSegReaders);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    words[3] = words[5] = 0;
    fence_barrier_init();
    tma_prefetch_map(&gate.group);
    tma_prefetch_map(&up.group);
    tma_prefetch_map(&down.group);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp >= 4) {
    moe_phase_a(a, reinterpret_cast<float*>(smem + MoeSmem::red), threadIdx.x - 128);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (threadIdx.x == 0) {
    grid_arrive(a.counters);
    words[2] = grid_wait(a.counters, wc) ? 1 : 0;
  }
  __syncthreads();
  const bool routed = words[2] != 0;
  uint32_t filled = 0;
  bool issued = false;
  if (routed) {
    moe_phase_b(a, r);
    const uint32_t ring = smem_u32(smem + MoeSmem::ring);
    if (warp >= 4) moe_picks(a, r);
    if (warp >= 8) {
      MoeBuilder builder{a,       r,         segs,      smem + MoeSmem::operand, b_scale, b_full,
                         b_empty, words + 4, words + 5, wc,                      {}};
      builder_run(builder);
    } else if (warp >= 4) {
      moe_accumulate(a, r, segs, scale_ring, b_scale, acc_full, acc_empty, b_full, b_empty, sc_full,
                     sc_empty, tmem_base, wc);
    } else if (warp == 3) {
      moe_gates(a, r, lane);
    } else if (warp == 2) {
      moe_scales(a, segs, smem_u32(scale_ring), sc_full, sc_empty, lane, wc);
    } else if (warp == 1) {
      issued = moe_mma(segs, ring, smem_u32(smem + MoeSmem::operand), full, empty, acc_full,
                       acc_empty, b_full, b_empty, tmem_base, wc);
    } else if (warp == 0 && lane == 0) {
      filled = moe_producer(a, r, gate, up, down, seg_slot, seg_full, seg_empty, ring, full, empty,
                            wc);
    }
  }
  // after an abort, copies may still be in flight: each stage's last one
  if (threadIdx.x == 0)
    for (uint32_t s = 0; s < uint32_t(kMoeStages) && s < filled; ++s)
      wait_drain(full + 8 * s, ((filled - 1 - s) / kMoeStages) & 1, wc);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (issued) f8_drain(drain, wc);
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
  // All warps or none: a wait of phase E that runs out has a flag of its own, as a
  // slower warp may have this one still to read.
  if (!routed || *abort_flag) return;  // gemm_status clears the counters
  const WaitCtl last{a.wait_limit_ns, a.status, words + 3};
  moe_phase_e(a, r, [&]() {
    if (threadIdx.x == 0) words[2] = grid_wait(a.counters + 3, last) ? 1 : 0;
    __syncthreads();
    return words[2] != 0;
  });
  if (words[2] == 0) return;
  // the last CTA through the last barrier leaves the counters at 0
  if (threadIdx.x == 0 && atomicAdd(a.counters + 4, 1) == int(gridDim.x) - 1) {
#pragma unroll
    for (int i = 0; i < 7; ++i) atomicExch(a.counters + i, 0);
  }
}

int64_t up256(int64_t b) { return (b + 255) & ~int64_t(255); }
int64_t ceil128(int64_t n) { return (n + 127) / 128; }

// Most partials that one tile of `kb` k-blocks can leave: in equal ranges, when at
// least `tiles` tiles are shared out over at most `ctas` CTAs, or in pieces.
int64_t most_segments(int64_t tiles, int64_t kb, int64_t ctas, int64_t piece) {
  const int64_t least = std::max<int64_t>(kMoeMinUnits, tiles * kb / ctas);
  const int64_t pieces = (kb + piece - 1) / piece;
  return std::max(pieces, std::min(kb, kb / least + 2));
}

MoePieces pieces_of(int64_t kb, int64_t budget, int64_t run) {
  MoePieces p{};
  p.run = int32_t(kb < run ? run / kb : 1);
  const int64_t chunks = (kb + budget - 1) / budget;
  p.chunk = int32_t(((kb + chunks - 1) / chunks + 1) & ~int64_t(1));  // weights come in pairs
  p.chunks = int32_t((kb + p.chunk - 1) / p.chunk);
  return p;
}

struct MoeSpace {
  int64_t xq, xs, logits, hq, hs, part1, part2;
  MoeSpace(const gemm_moe_fp8_t& L, int64_t ctas) {
    const int64_t T = L.tokens, P = T * L.top_k, kb_h = ceil128(L.hidden), kb_i = ceil128(L.inner);
    // a token's choices are different experts, so at least top_k are chosen
    const int64_t s1 = most_segments(2 * L.top_k * kb_i, kb_h, ctas, kMoePieceC);
    const int64_t s2 = most_segments(L.top_k * kb_h, kb_i, ctas, kMoePieceD);
    xq = up256(T * kb_h * kFp8Block);
    xs = up256(T * kb_h * 4);
    logits = up256(T * L.experts * 4);
    hq = up256(P * kb_i * kFp8Block);
    hs = up256(P * kb_i * 4);
    part1 = up256(s1 * 2 * P * kb_i * kBM * 4);
    part2 = up256(s2 * P * kb_h * kBM * 4);
  }
  int64_t bytes() const { return xq + xs + logits + hq + hs + part1 + part2; }
};

bool encode_experts(MoeMaps* m, const gemm_fp8_experts_t& w, int64_t rows, int64_t K,
                    int64_t experts) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t pitch = cuuint64_t(w.ld);
  const cuuint64_t next = cuuint64_t(experts > 1 ? w.expert_stride : rows * w.ld);
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  auto encode = [&](CUtensorMap* map, cuuint32_t rank, const cuuint64_t* dims,
                    const cuuint64_t* strides, const cuuint32_t* box) {
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(w.data), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t dims3[3] = {cuuint64_t(K), cuuint64_t(rows), cuuint64_t(experts)};
  const cuuint64_t strides3[2] = {pitch, next};
  const cuuint32_t box3[3] = {kFp8Block, kBM, 1};
  if (!encode(&m->one, 3, dims3, strides3, box3)) return false;
  m->group = m->one;
  if (K < 2 * kFp8Block) return true;  // no whole group: never used
  const cuuint64_t dims4[4] = {kFp8Block, cuuint64_t(rows), cuuint64_t(K / kFp8Block),
                               cuuint64_t(experts)};
  const cuuint64_t strides4[3] = {pitch, kFp8Block, next};
  const cuuint32_t box4[4] = {kFp8Block, kBM, 2, 1};
  return encode(&m->group, 4, dims4, strides4, box4);
}

}  // namespace

int64_t moe_workspace_bytes(const gemm_ctx* h, const gemm_moe_fp8_t& L) {
  return MoeSpace(L, h->num_sms).bytes();
}

cudaError_t launch_moe(gemm_ctx* h, const gemm_moe_fp8_t& L, void* workspace,
                       cudaStream_t stream) {
  const MoeSpace space(L, h->num_sms);
  MoeArgs a{};
  a.L = L;
  a.kb_h = int32_t(ceil128(L.hidden));
  a.kb_i = int32_t(ceil128(L.inner));
  a.tiles_h = a.kb_h;
  a.tiles_i = a.kb_i;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.xq = w;
  a.xs = reinterpret_cast<float*>(w += space.xq);
  a.logits = reinterpret_cast<float*>(w += space.xs);
  a.hq = w += space.logits;
  a.hs = reinterpret_cast<float*>(w += space.hq);
  a.part1 = reinterpret_cast<float*>(w += space.hs);
  a.part2 = reinterpret_cast<float*>(w += space.part1);
  a.counters = h->tickets + kMoeCounters;
  a.status = h->status;
  a.wait_limit_ns = h->opt.wait_limit_ns;
  a.vec = ((reinterpret_cast<uintptr_t>(L.x) | reinterpret_cast<uintptr_t>(L.router)) & 15) == 0 &&
          L.ld_x % 8 == 0 && L.ld_router % 8 == 0;
  a.pieces[0] = pieces_of(a.kb_h, kMoePieceC, kMoeRunC);
  a.pieces[1] = pieces_of(a.kb_i, kMoePieceD, kMoeRunD);
  a.dynamic = h->opt.dyn_sched > 0;
  MoeMaps gate, up, down;
  if (!encode_experts(&gate, L.gate, L.inner, L.hidden, L.experts) ||
      !encode_experts(&up, L.up, L.inner, L.hidden, L.experts) ||
      !encode_experts(&down, L.down, L.hidden, L.inner, L.experts))
    return cudaErrorInvalidValue;
  static SharedMemoryOnce once;
  cudaError_t e = once.allow(moe_kernel, MoeSmem::bytes, h->device);
  if (e != cudaSuccess) return e;
  // the CTAs wait for one another: a cooperative launch, all resident at once
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3(unsigned(h->num_sms), 1, 1);
  cfg.blockDim = dim3(kMoeThreads, 1, 1);
  cfg.dynamicSmemBytes = MoeSmem::bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_kernel, gate, up, down, a);
}

}  // namespace dg

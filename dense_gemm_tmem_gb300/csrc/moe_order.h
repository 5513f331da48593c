// moe_order.h: the order in which each of the expert layer's four builder warps
// works and meets the others.  Plain C++, so that it also runs on the host.
#pragma once

#ifdef __CUDACC__
#define DG_ORDER __device__ __forceinline__
#else
#define DG_ORDER inline
#endif

namespace dg {

// Warp: contents(phase) lays out a phase's token operands, false when one of this
// warp's waits gave up.  partials(ok) and rows_done() are barriers of the four
// warps, which all of them answer alike: whether every warp is ok and the grid's
// barrier came.
//
// A wait that gives up does so for one warp at a time: another that polls the same
// barrier a moment later may find it complete.  So a warp that gave up in phase C
// still comes to partials(); only what the four decide there together ends them.
template <class Warp>
DG_ORDER void builder_run(Warp& w) {
#ifdef __CUDACC__
#pragma unroll 1  // contents() stands in the code once: code is fetched cold, 1 us of 29
#endif
  for (int phase = 0;; ++phase) {
    const bool ok = w.contents(phase);
    if (phase == 1 || !w.partials(ok)) return;
    w.rows();
    if (!w.rows_done()) return;
  }
}

}  // namespace dg

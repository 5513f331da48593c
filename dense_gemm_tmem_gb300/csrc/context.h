// context.h: the handle behind gemm_handle_t and what the API files share.
#pragma once

#include <atomic>
#include <mutex>

#include "internal.h"

namespace dg {

constexpr int kMaxTileN = 256;
constexpr int kTicketCap = 16384;     // split tiles one launch may have
// after the tickets: the two-SM kernel's tile counter and finished-pair count
// and the expert layer's four barriers, its exits and its two piece counters
constexpr int kMoeCounters = kTicketCap + 2;
constexpr int kCounterInts = kMoeCounters + 7;
constexpr int kTmapCacheSize = 32;
constexpr int64_t kMaxCoord = (int64_t(1) << 31) - 1024;  // TMA coordinates are int32

struct TmapKey {
  const void* ptr;
  int64_t rows, k;
  int mn_major, box_rows;
  int kind;  // 0 fp16 operand, 1 fp32 output, 2 fp16 output
  int kgroup;  // k-blocks per box (operands)
  bool operator==(const TmapKey& o) const {
    return ptr == o.ptr && rows == o.rows && k == o.k && mn_major == o.mn_major &&
           box_rows == o.box_rows && kind == o.kind && kgroup == o.kgroup;
  }
};

struct TmapEntry {
  TmapKey key;
  CUtensorMap map;
  bool valid = false;
};

// A kernel's dynamic shared memory limit, raised once per device (on every launch it
// cost 0.5 us of a product's 4.4 of host time).
struct SharedMemoryOnce {
  std::atomic<uint64_t> devices{0};  // those that have it; past 63, none is noted
  template <class Kernel>
  cudaError_t allow(Kernel kern, int bytes, int device) {
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) devices.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// Runs `f` with the handle's device current, restoring the caller's.
template <class F>
int on_device(int device, F&& f) {
  int prev = -1;
  if (cudaGetDevice(&prev) != cudaSuccess) return GEMM_ERR_CUDA;
  if (prev != device && cudaSetDevice(device) != cudaSuccess) return GEMM_ERR_CUDA;
  const int rc = f();
  if (prev != device) cudaSetDevice(prev);
  return rc;
}

}  // namespace dg

struct gemm_ctx {
  int device = 0;
  int num_sms = 0;
  float* workspace = nullptr;
  size_t workspace_bytes = 0;
  int* tickets = nullptr;
  int* status = nullptr;
  int last_detail = 0;
  uint64_t* trace = nullptr;  // caller's device buffer for phase stamps, or NULL
  int64_t trace_ctas = 0;     // CTA rows it holds (kTraceSlots stamps each)
  dg::Options opt;
  void* host_stage = nullptr;   // gemm_run_host: device copies of A, B, bias and C
  size_t host_stage_bytes = 0;  // grow-only
  std::mutex host_mu;           // serialises gemm_run_host's enqueueing
  cudaEvent_t host_done = nullptr;  // recorded after each gemm_run_host call's work
  bool host_done_recorded = false;
  std::mutex mu;  // guards the tensor-map cache
  dg::TmapEntry cache[dg::kTmapCacheSize];
  int cache_next = 0;
};

// Bounded waits on mbarriers, shared by the persistent tensor-core kernels.
#pragma once
#include <cstdint>
#include "common.cuh"
#include "ptx_sm100.cuh"

namespace cutbce {

struct WaitCtx {
  volatile int* abort_flag;
  WsHeader* hdr;
  long long limit;
};

// Where a wait happens, recorded if it gives up: role (1 producer, 2 MMA,
// 4 epilogue), barrier id, and the role's tile or item counter.
__device__ __forceinline__ int wait_tag(int role, int barrier, uint32_t counter) {
  return (role << 28) | (barrier << 20) | static_cast<int>(counter & 0xFFFFFu);
}

// Bounded wait for phase `parity` of `bar`.  Returns false if the CTA aborted
// or the limit ran out (then it records the timeout, where it happened, and
// raises the abort flag).
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const WaitCtx& w, int tag = 0) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    if (*w.abort_flag) {
      // record where each role stood when the CTA gave up (first record per role wins)
      const int role = (tag >> 28) & 7;
      if (tag != 0 && role >= 1) atomicCAS(&w.hdr->role_wait_tag[role - 1], 0, tag);
      return false;
    }
    if (static_cast<long long>(global_timer_ns() - t0) > w.limit) {
      *w.abort_flag = 1;
      if (atomicCAS(&w.hdr->status, 0, kErrTimeout) == 0) {
        w.hdr->wait_tag = tag;
        w.hdr->wait_block = static_cast<int>(blockIdx.x);
      }
      return false;
    }
  }
}
// Bounded wait that ignores the abort flag (used to drain in-flight copies/MMAs).
__device__ __forceinline__ bool wait_bar_drain(uint64_t* bar, uint32_t parity, long long limit) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (static_cast<long long>(global_timer_ns() - t0) > limit) return false;
  }
  return true;
}
// Whole-warp wait.  Fast path: every lane tests the phase itself (one
// shared-memory instruction for the warp, each lane acquiring the phase) and a
// vote, not a shuffle, gathers the answers.  Otherwise lane 0 waits (bounded)
// and the warp then synchronises with it, which orders the other lanes after
// lane 0's acquire of the phase.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, const WaitCtx& w, int tag = 0) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, w, tag);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

}  // namespace cutbce

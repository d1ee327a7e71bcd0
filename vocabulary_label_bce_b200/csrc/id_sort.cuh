// Stable radix sort of (item id, entry index) pairs and the sum of rows grouped
// by id: the table's gradient from its sparse side (lookup gradient, and the
// target part of the softmax losses).
//
// Sort: LSD over at most 11 bits a pass, so V up to 2047 takes one pass and V up
// to 4 M two.  Up to 16,384 entries it is one kernel (k_sort_cluster); beyond, a block
// owns a tile of consecutive entries; each warp ranks a contiguous part of it with
// match_any and 16-bit counters in shared memory, so equal ids keep entry order.
// Every scatter block forms its own offsets from the
// tile histograms (they sit in L2), and the scatter of one pass counts the
// histogram of the next with integer atomics, whose order changes nothing.
// An entry without a row (an empty id, or one out of range, which also sets the status)
// has the key V and sorts to the end.
//
// Sums: a block takes a chunk of consecutive sorted entries, cut into sub-chunks;
// the lanes of a row add the rows of their sub-chunk in order, four in flight.  A
// segment (equal ids) inside a sub-chunk is written at once; one that crosses
// sub-chunks is joined in shared memory, in order; one that crosses blocks leaves
// one partial per block, and k_segment_join adds those (eight interleaved running
// sums, then a fixed order).  Hot ids neither serialise nor need atomics.
//
// Measured, ids drawn from Zipf laws: N = 12,800, V = 876,000, D = 64 bf16: sort 22 us
// beside the 112 MB of zeros (17 us at the measured copy rate), sums 8.6, join 2.8.
// N = 200,003, V = 100,000, D = 200 fp32: keys 6 us, two passes beside 80 MB of zeros
// 24, sums 48 (160 MB read, 3.5 TB/s: several waves of blocks whose rows are 800 random
// bytes each), join 8.  The sorts are bound by latency: a few dozen blocks, each a
// chain of loads, counts and scattered stores.
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
  if (s.bits < 2) s.bits = 2;                 // a thread of the scatter holds four digits
  // Tiles of 1024, 2048 or 4096 entries; past 128 tiles their histograms are scanned.
  // Lookup gradients over 40,000 ids, D = 8, for 4 / 8 / 16 entries a thread: 100,000
  // entries 45 / 48 / - us, 200,003 53 / 51 / 54, 1,000,000 111 / 107 / 104, 10,000,000
  // 739 / 639 / 628 (and half the histograms' memory).
  s.ipt = N <= 131072 ? 4 : N <= 4194304 ? 8 : 16;
  s.nblk = static_cast<int>(ceil_div(N, int64_t(kSortThreads) * s.ipt));
  s.scan = s.nblk > 128;
  s.hist_bytes = sizeof(int) * static_cast<size_t>(s.passes) * s.nblk * (size_t(1) << s.bits);
}

// Memory to set (zeros for a dense gradient's rows, -1 for an index), written by
// blocks of their own beside a sort kernel that leaves most SMs idle: `n` pieces of 16
// bytes, every 32-bit word `value`.
struct FillJob {
  uint4* dst;
  int64_t n;                // 0: nothing to fill
  uint32_t value;
};
__device__ __forceinline__ void fill_words(const FillJob& f, int64_t block, int64_t blocks) {
  const uint4 v = make_uint4(f.value, f.value, f.value, f.value);
  const int64_t step = blocks * blockDim.x;
  int64_t i = block * blockDim.x + threadIdx.x;
  for (; i + 3 * step < f.n; i += 4 * step) {
#pragma unroll
    for (int u = 0; u < 4; ++u) f.dst[i + u * step] = v;
  }
  for (; i < f.n; i += step) f.dst[i] = v;
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
#pragma unroll 16
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
// A block has 32 digits; its warps take consecutive shares of the tiles.
constexpr int kScanWarps = 16;
__global__ void __launch_bounds__(32 * kScanWarps) k_sort_scan(int* __restrict__ hist, int* __restrict__ total, int bins,
                                                               int nblk) {
  __shared__ int s_sum[kScanWarps][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane;
  const int per = (nblk + kScanWarps - 1) / kScanWarps;
  const int b0 = min(nblk, w * per), b1 = d < bins ? min(nblk, b0 + per) : b0;
  // the counts of this share's tiles, eight in flight
  auto walk = [&](auto each) {
    for (int b = b0; b < b1; b += 8) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = b + u < b1 ? hist[static_cast<int64_t>(b + u) * bins + d] : 0;
#pragma unroll
      for (int u = 0; u < 8; ++u) each(b + u, v[u]);
    }
  };
  int own = 0;
  walk([&](int, int v) { own += v; });
  s_sum[w][lane] = own;
  __syncthreads();
  int run = 0;
#pragma unroll
  for (int k = 0; k < kScanWarps; ++k) run += k < w ? s_sum[k][lane] : 0;
  if (w == kScanWarps - 1 && d < bins) total[d] = run + own;
  walk([&](int b, int v) {
    if (b < b1) hist[static_cast<int64_t>(b) * bins + d] = run;
    run += v;
  });
}

// One pass over (id, entry index) pairs.  ids (first pass, else null): the plain ids,
// empty and out-of-range ones counting as V, the index being the entry's own.
// hist_next (null in the last pass): the next pass's histogram, cleared before the
// call.  Blocks from nblk on fill.  With `stop` (or null) the pass is left out where it
// holds an error.
// The bound of two blocks an SM leaves registers for the histogram loads in flight:
// without it the compiler holds fewer (two passes over 51,200 entries 20.7 us, with
// it 13.7; over 200,003 29.0 and 24.5).
template <int IPT>
__global__ void __launch_bounds__(kSortThreads, 2) k_sort_scatter(const int* __restrict__ ids,
                                                               const int2* __restrict__ in, int64_t N, int V,
                                                               int shift, int bits, int nblk,
                                                               const int* __restrict__ hist,
                                                               const int* __restrict__ digit_total,
                                                               int2* __restrict__ out, int* __restrict__ hist_next,
                                                               const int* __restrict__ stop, FillJob fill) {
  __shared__ __align__(16) uint16_t cnt[kSortWarps][kSortMaxBins];
  __shared__ int off[kSortMaxBins];
  __shared__ int wsum[kSortWarps];
  if (static_cast<int>(blockIdx.x) >= nblk) {
    fill_words(fill, static_cast<int>(blockIdx.x) - nblk, static_cast<int>(gridDim.x) - nblk);
    return;
  }
  const int failed = stop != nullptr ? *stop : 0;   // looked at before anything is written
  const int bins = 1 << bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // offset of (digit, this tile): all smaller digits, then this digit in earlier
  // tiles.  A thread holds four consecutive digits (of each 1024), sixteen tiles'
  // histograms in flight; with fewer than 1024 digits, groups of threads share the tiles.
  const int quads = min(bins / 4, kSortThreads), groups = kSortThreads / quads;
  int* s_total = reinterpret_cast<int*>(&cnt[0][0]);
  int carry = 0;
  for (int h0 = 0; h0 < bins; h0 += 4 * kSortThreads) {
    const int d0 = h0 + 4 * tid;
    int before[4] = {0, 0, 0, 0}, total[4] = {0, 0, 0, 0};
    auto add_tiles = [&](int d, int first, int stride) {
      const int4* src = reinterpret_cast<const int4*>(hist + d);
      const int step = bins / 4;
      constexpr int kTiles = 16;                        // tiles in flight; the last group is guarded, not looped
      for (int b0 = first * kTiles; b0 < nblk; b0 += stride * kTiles) {
        int4 v[kTiles];
#pragma unroll
        for (int u = 0; u < kTiles; ++u)
          v[u] = b0 + u < nblk ? __ldg(src + static_cast<int64_t>(b0 + u) * step) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          const int keep = b0 + u < static_cast<int>(blockIdx.x) ? -1 : 0;
          total[0] += v[u].x, total[1] += v[u].y, total[2] += v[u].z, total[3] += v[u].w;
          before[0] += v[u].x & keep, before[1] += v[u].y & keep, before[2] += v[u].z & keep, before[3] += v[u].w & keep;
        }
      }
    };
    if (digit_total != nullptr) {
      if (d0 < bins) {
        const int4 v = *reinterpret_cast<const int4*>(hist + static_cast<int64_t>(blockIdx.x) * bins + d0);
        const int4 t = *reinterpret_cast<const int4*>(digit_total + d0);
        before[0] = v.x, before[1] = v.y, before[2] = v.z, before[3] = v.w;
        total[0] = t.x, total[1] = t.y, total[2] = t.z, total[3] = t.w;
      }
    } else if (groups == 1) {
      if (d0 < bins) add_tiles(d0, 0, 1);
    } else {
      for (int d = tid; d < bins; d += kSortThreads) off[d] = s_total[d] = 0;
      __syncthreads();
      const int d = 4 * (tid & (quads - 1));
      add_tiles(d, tid / quads, groups);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        atomicAdd(off + d + k, before[k]);
        atomicAdd(s_total + d + k, total[k]);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        before[k] = d0 < bins ? off[d0 + k] : 0;
        total[k] = d0 < bins ? s_total[d0 + k] : 0;
      }
    }
    const int sum = total[0] + total[1] + total[2] + total[3];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int run = carry + inc - sum;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) run += wsum[w];
      carry += wsum[w];
    }
    if (d0 < bins) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        off[d0 + k] = run + before[k];
        run += total[k];
      }
    }
    __syncthreads();
  }
  for (int d = lane; d < bins; d += 32) cnt[warp][d] = 0;
  __syncwarp();
  // ranks: warp w owns entries [w * 32 * IPT, (w + 1) * 32 * IPT) of the tile, 32 at a time
  const int64_t wbase = static_cast<int64_t>(blockIdx.x) * kSortThreads * IPT + static_cast<int64_t>(warp) * 32 * IPT;
  const unsigned lt = (1u << lane) - 1u;
  int2 key[IPT];
  int rank[IPT];
  auto load_pair = [&](int64_t i) {
    if (ids == nullptr) return in[i];
    const int k = ids[i];
    return make_int2((k < 0 || k > V) ? V : k, static_cast<int>(i));
  };
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    const int64_t i = wbase + r * 32 + lane;
    key[r] = i < N ? load_pair(i) : make_int2(0, 0);
  }
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    const bool live = wbase + r * 32 + lane < N;
    const int d = live ? (key[r].x >> shift) & (bins - 1) : bins;
    const unsigned peers = __match_any_sync(0xffffffffu, d);
    const int old = live ? cnt[warp][d] : 0;
    rank[r] = old + __popc(peers & lt);
    __syncwarp();
    if (live && (peers & lt) == 0) cnt[warp][d] = static_cast<uint16_t>(old + __popc(peers));
    __syncwarp();
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
  if (failed != 0) return;
#pragma unroll
  for (int r = 0; r < IPT; ++r) {
    const bool live = wbase + r * 32 + lane < N;
    const int d = (key[r].x >> shift) & (bins - 1);
    const int pos = live ? off[d] + cnt[warp][d] + rank[r] : 0;
    if (live) out[pos] = key[r];
    if (hist_next != nullptr) {
      // one atomic per distinct counter of the warp: entries of a hot id share theirs
      const int bin = live ? (pos / (kSortThreads * IPT)) * bins + ((key[r].x >> (shift + bits)) & (bins - 1)) : -1;
      const unsigned peers = __match_any_sync(0xffffffffu, bin);
      if (live && (peers & lt) == 0) atomicAdd(hist_next + bin, __popc(peers));
    }
  }
}

// The whole sort in one kernel, for up to 16,384 entries: a cluster of
// eight CTAs, whose warps own consecutive entries (held in registers over a pass).
// The CTAs read each other's digit totals from shared memory; the pairs of a pass go
// through L2.  No launch, histogram or clearing between the passes: 12,800 entries
// of 20-bit ids take 18 us with one launch, the kernels above 19 us with four; at
// 51,200 entries it is 35 against 23.  ids as there;
// `clear_status`: the status starts here, and bad ids set it.  Clusters past the
// first fill.
constexpr int kClusterCtas = 8;
constexpr int kClusterThreads = 1024;
constexpr int kClusterRounds = 2;                       // entries per thread: 16,384 in all
constexpr int64_t kClusterEntries = 16384;

__device__ __forceinline__ int ld_cluster_shared(const int* local, uint32_t rank) {
  uint32_t addr;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads)
    k_sort_cluster(const int* __restrict__ ids, int N, int V, int bits, int passes, int2* buf0, int2* buf1, int* status,
                   int clear_status, FillJob fill) {
  if (blockIdx.x >= kClusterCtas) {                         // clusters past the first
    fill_words(fill, static_cast<int>(blockIdx.x) - kClusterCtas, static_cast<int>(gridDim.x) - kClusterCtas);
    return;
  }
  extern __shared__ __align__(16) uint16_t s_cnt[];                       // [32 warps][bins]
  __shared__ int tot[kSortMaxBins], off[kSortMaxBins];
  __shared__ int wsum[32];
  const int bins = 1 << bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  uint16_t* cnt = s_cnt + warp * bins;
  const unsigned lt = (1u << lane) - 1u;
  const int per = (N + kClusterCtas * 1024 - 1) / (kClusterCtas * 1024);   // rounds of 32 entries a warp
  const int base = (static_cast<int>(rank) * 32 + warp) * per * 32;
  if (clear_status) {
    if (rank == 0 && tid == 0) *status = 0;
    cluster_sync_all();
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits;
    const int2* in = (p & 1) ? buf0 : buf1;                 // pass p writes buf0 for even p
    int2* out = (p & 1) ? buf1 : buf0;
    int2 key[kClusterRounds];
    int rk[kClusterRounds];
    for (int i = tid; i < 4 * bins; i += kClusterThreads) reinterpret_cast<uint4*>(s_cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int r = 0; r < kClusterRounds; ++r) {
      const int i = base + r * 32 + lane;
      key[r] = make_int2(V, 0);
      if (r < per && i < N) {
        if (p == 0) {
          const int id = __ldg(ids + i);
          const bool real = id >= 0 && id < V;
          if (!real && id != -1) atomicCAS(status, 0, kErrTargetRange);
          key[r] = make_int2(real ? id : V, i);
        } else {
          key[r] = __ldcg(in + i);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kClusterRounds; ++r) {
      if (r >= per) break;
      const bool live = base + r * 32 + lane < N;
      const int d = live ? (key[r].x >> shift) & (bins - 1) : bins;
      const unsigned peers = __match_any_sync(0xffffffffu, d);
      const int old = live ? cnt[d] : 0;
      rk[r] = old + __popc(peers & lt);
      __syncwarp();
      if (live && (peers & lt) == 0) cnt[d] = static_cast<uint16_t>(old + __popc(peers));
      __syncwarp();
    }
    __syncthreads();
    // this CTA's totals, and each warp's start within them
    for (int d = tid; d < bins; d += kClusterThreads) {
      int run = 0;
#pragma unroll
      for (int w = 0; w < 32; ++w) {
        const int c = s_cnt[w * bins + d];
        s_cnt[w * bins + d] = static_cast<uint16_t>(run);
        run += c;
      }
      tot[d] = run;
    }
    cluster_sync_all();
    // offsets: smaller digits in the whole cluster, then this digit in earlier CTAs
    int carry = 0;
    for (int d0 = 0; d0 < bins; d0 += kClusterThreads) {
      const int d = d0 + tid;
      int before = 0, total = 0;
      if (d < bins) {
#pragma unroll
        for (uint32_t c = 0; c < kClusterCtas; ++c) {
          const int v = ld_cluster_shared(tot + d, c);
          total += v;
          if (c < rank) before += v;
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
      if (warp == 0) {
        int s = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, s, o);
          if (lane >= o) s += v;
        }
        wsum[lane] = s;
      }
      __syncthreads();
      if (d < bins) off[d] = carry + (warp > 0 ? wsum[warp - 1] : 0) + inc - total + before;
      carry += wsum[31];
      __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < kClusterRounds; ++r) {
      if (r >= per || base + r * 32 + lane >= N) break;
      const int d = (key[r].x >> shift) & (bins - 1);
      out[off[d] + cnt[d] + rk[r]] = key[r];
    }
    // the pairs are visible to the cluster, and no CTA still reads another's totals
    cluster_sync_all();
  }
}

// ------------------------------------------------------------------ segment sums
struct SegmentParams {
  const int2* pairs;          // sorted (id, entry index): id V has no row; indices ascend within an id
  int64_t N;
  int V, D;
  const void* src;            // [rows, src_stride] rows to add; entry p reads row p / K
  int64_t src_stride;
  int K;
  const float* share;         // [N] factor of entry p, or null
  const float* row_coef;      // [rows] factor of its row, or null
  float scale;                // factor of the whole sum
  float* part;                // [2 * chunks, D]: the chunk's first (continued) and last (continuing) segment
  void* out;                  // by item: [V, D] fp32 or bf16; by segment (first != null): fp32 row at the segment's first index
  int* first;                 // [V] first sorted index of each id's segment (cleared to -1), or null
  uint32_t* columns;          // [N] row of each sorted entry, 2^31 added to the first of an id, or null
  int out_bf16, accumulate;
  const int* stop;            // nothing is added up where it holds an error, or null
};

template <int VEC>
__device__ __forceinline__ void store_floats(float* o, const float (&v)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) *reinterpret_cast<float4*>(o + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
  } else {
    o[0] = v[0];
  }
}

// VEC > 1: rows of the output start on 16-byte boundaries.
template <int VEC, typename TOut>
__device__ __forceinline__ void write_sum(const SegmentParams& p, int id, int64_t start, int col, const float (&acc)[VEC]) {
  float v[VEC];
  if (p.first != nullptr) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[k] = acc[k] * p.scale;
    store_floats<VEC>(static_cast<float*>(p.out) + start * p.D + col, v);
    return;
  }
  TOut* o = static_cast<TOut*>(p.out) + static_cast<int64_t>(id) * p.D + col;
#pragma unroll
  for (int k = 0; k < VEC; ++k) {
    v[k] = __fmul_rn(acc[k], p.scale);
    if (p.accumulate) v[k] = __fadd_rn(v[k], static_cast<float>(o[k]));
  }
  if constexpr (sizeof(TOut) == 4) {
    store_floats<VEC>(reinterpret_cast<float*>(o), v);
  } else if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4)
      *reinterpret_cast<uint2*>(o + k) = make_uint2(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]));
  } else {
    o[0] = TOut(v[0]);
  }
}

// A piece of a row as loaded (16 bytes, or one element), and its values.
template <int VEC, typename T>
struct RowPiece {
  uint4 raw;
  __device__ __forceinline__ void load(const T* src) { raw = __ldg(reinterpret_cast<const uint4*>(src)); }
  __device__ __forceinline__ void values(float (&x)[VEC]) const {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        x[k] = __uint_as_float(u[k]);
      } else {
        x[2 * k] = __uint_as_float(u[k] << 16);
        x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
      }
    }
  }
};
template <typename T>
struct RowPiece<1, T> {
  T raw;
  __device__ __forceinline__ void load(const T* src) { raw = *src; }
  __device__ __forceinline__ void values(float (&x)[1]) const { x[0] = static_cast<float>(raw); }
};

// Geometry for rows of D elements in pieces of VEC: `lanes` threads a row (wide
// rows in `slices`), `subs` rows side by side in a block, each sub-chunk summing
// kSumBatch * rounds consecutive entries.
constexpr int kSumBatch = 4;                // rows in flight per thread
constexpr int kMinChunk = 4 * kSumBatch;    // fewest entries of a block
struct SumGeometry {
  int lanes, slices, subs, rounds;
  int64_t chunk, chunks;                    // entries per block, blocks (per slice)
};
inline SumGeometry sum_geometry(int64_t N, int64_t D, int vec) {
  SumGeometry g;
  const int pieces = static_cast<int>(ceil_div(D, vec));
  g.slices = static_cast<int>(ceil_div(pieces, 64));
  g.lanes = static_cast<int>(ceil_div(pieces, g.slices));
  g.subs = 256 / g.lanes;
  if (g.subs > 64) g.subs = 64;
  // rounds so that about eight blocks an SM remain: fewer leave SMs idle at the end (626
  // blocks in waves of 592: a third lost), more leave more partials to join
  int64_t r = N / (static_cast<int64_t>(g.subs) * kSumBatch * 1184);
  g.rounds = static_cast<int>(r < 1 ? 1 : r > 16 ? 16 : r);
  g.chunk = static_cast<int64_t>(g.subs) * kSumBatch * g.rounds;
  g.chunks = ceil_div(N, g.chunk);
  return g;
}

// One block per (chunk, slice).  A sub-chunk writes the segments that lie inside it
// and leaves its first (continued) and last (continuing) ones in shared memory; the
// lanes of sub-chunk 0 then walk the sub-chunks in order.
template <int VEC, typename TIn, typename TOut>
__global__ void __launch_bounds__(256, VEC == 8 ? 3 : 4) k_segment_sum(const SegmentParams p, int lanes, int subs, int rounds) {
  __shared__ float s_first[256 * VEC], s_last[256 * VEC];
  __shared__ int s_kind[64], s_key[64], s_start[64];     // 1: first closes, 2: first goes through, 4: last is open
  if (p.stop != nullptr && *p.stop != 0) return;
  const int sub = static_cast<int>(threadIdx.x) / lanes, lane = static_cast<int>(threadIdx.x) % lanes;
  const int col = (static_cast<int>(blockIdx.y) * lanes + lane) * VEC;
  const int per = kSumBatch * rounds;
  const int64_t chunk = blockIdx.x;
  const int64_t i0 = (chunk * subs + sub) * per;
  const int64_t i1 = min(p.N, i0 + per);
  const bool live = col < p.D;
  const TIn* src = static_cast<const TIn*>(p.src) + col;
  if (sub < subs) {
    int kind = 0;
    int cur = i0 < i1 ? __ldg(&p.pairs[i0].x) : p.V;
    bool open_left = i0 > 0 && i0 < i1 && __ldg(&p.pairs[i0 - 1].x) == cur;
    const int after = i1 < p.N && i0 < i1 ? __ldg(&p.pairs[i1].x) : -1;
    int start = static_cast<int>(i0);
    float acc[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
    // ends the running segment; `goes_on`: the next sub-chunk continues it
    auto flush = [&](bool goes_on) {
      if (cur >= p.V) return;
      if (p.first != nullptr && !open_left && col == 0) p.first[cur] = start;
      if (!open_left && !goes_on) {
        if (live) write_sum<VEC, TOut>(p, cur, start, col, acc);
        return;
      }
      float* o = (open_left ? s_first : s_last) + threadIdx.x * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = acc[k];
      kind |= open_left ? (goes_on ? 2 : 1) : 4;
    };
    // Every load is unconditional, so that a batch's are in flight together: indices
    // are held below N, and an entry without a row (key V) reads its row all the same
    // and adds it to a segment that is never written.  The next batch's keys and
    // indices are loaded before this one's rows are added.
    int id[kSumBatch], e[kSumBatch];
    auto load_entries = [&](int64_t i) {
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) {
        const int64_t at = min(i + u, p.N - 1);
        const int2 pair = __ldg(p.pairs + at);
        id[u] = pair.x;
        e[u] = pair.y;
      }
    };
    if (i0 < i1) load_entries(i0);
    for (int64_t i = i0; i < i1; i += kSumBatch) {
      RowPiece<VEC, TIn> x[kSumBatch];
      float w[kSumBatch];
      int now[kSumBatch], from[kSumBatch];
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) {
        const int64_t row = p.K == 1 ? e[u] : e[u] / p.K;
        w[u] = p.share != nullptr ? __ldg(p.share + e[u]) : 1.f;
        if (p.row_coef != nullptr) w[u] *= __ldg(p.row_coef + row);
        x[u].load(src + (live ? row * p.src_stride : -col));       // lanes past the row's end read its first element
        now[u] = id[u];
        from[u] = static_cast<int>(row);
      }
      if (i + kSumBatch < i1) load_entries(i + kSumBatch);
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) {
        if (i + u >= i1) break;
        if (now[u] != cur) {
          flush(false);
          cur = now[u];
          open_left = false;
          start = static_cast<int>(i + u);
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
        }
        if (p.columns != nullptr && col == 0)
          p.columns[i + u] = static_cast<uint32_t>(from[u]) | (i + u == start && !open_left ? 0x80000000u : 0u);
        float v[VEC];
        x[u].values(v);
#pragma unroll
        for (int k = 0; k < VEC; ++k) acc[k] = fmaf(w[u], v[k], acc[k]);
      }
    }
    if (i0 < i1) flush(after == cur);
    if (lane == 0) {
      s_kind[sub] = kind;
      s_key[sub] = cur;
      s_start[sub] = start;
    }
  }
  __syncthreads();
  if (sub != 0 || !live) return;
  // the running segment across sub-chunks; it may have begun in an earlier block
  float run[VEC];
  bool open = (s_kind[0] & 3) != 0, here = false;
  int key = 0, start = 0;
#pragma unroll
  for (int k = 0; k < VEC; ++k) run[k] = 0.f;
  auto leave = [&](int slot) {
    store_floats<VEC>(p.part + (2 * chunk + slot) * p.D + col, run);
  };
  for (int s = 0; s < subs; ++s) {
    const int kind = s_kind[s];
    if (kind == 0) continue;
    if (kind & 3) {
      const float* f = s_first + (s * lanes + lane) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) run[k] += f[k];
      if (kind & 1) {
        if (here) write_sum<VEC, TOut>(p, key, start, col, run);
        else leave(0);
        open = false;
      }
    }
    if (kind & 4) {
      const float* f = s_last + (s * lanes + lane) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) run[k] = f[k];
      key = s_key[s];
      start = s_start[s];
      open = here = true;
    }
  }
  if (open) leave(here ? 1 : 0);
}

// One block per chunk whose last segment continues: adds that segment's partials.
constexpr int kJoinBatch = 8;               // partials in flight per thread
template <int VEC, typename TOut>
__global__ void __launch_bounds__(256, 4) k_segment_join(const SegmentParams p, int64_t chunk_entries) {
  __shared__ float red[8][32 * VEC];
  if (p.stop != nullptr && *p.stop != 0) return;
  const int64_t c0 = blockIdx.x, b0 = c0 * chunk_entries, end = b0 + chunk_entries;
  if (end >= p.N) return;
  const int id = __ldg(&p.pairs[end - 1].x);
  const bool goes_on = __ldg(&p.pairs[end].x) == id;
  const bool middle = b0 > 0 && __ldg(&p.pairs[b0].x) == id && __ldg(&p.pairs[b0 - 1].x) == id;
  if (id >= p.V || !goes_on || middle) return;          // nothing continues, or this chunk is not the segment's first
  // the last chunk it reaches: chunks whose first entry has the id, 256 at a time
  int64_t c1 = c0;
  while (true) {
    const int64_t at = (c1 + 1 + threadIdx.x) * chunk_entries;
    const int hit = __syncthreads_count(at < p.N && __ldg(&p.pairs[min(at, p.N - 1)].x) == id);
    c1 += hit;
    if (hit < 256) break;
  }
  // its first entry (needed where sums are filed by it)
  int64_t start = b0;
  if (p.first != nullptr) {
    int below = 0;
    for (int64_t i = b0 + threadIdx.x; i < end; i += 256) below += __ldg(&p.pairs[i].x) < id;
    __shared__ int s_below;
    if (threadIdx.x == 0) s_below = 0;
    __syncthreads();
    below = __reduce_add_sync(0xffffffffu, below);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s_below, below);
    __syncthreads();
    start = b0 + s_below;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int col = (static_cast<int>(blockIdx.y) * 32 + lane) * VEC;
  float acc[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc[k] = 0.f;
  if (col < p.D) {
    for (int64_t cb = c0 + w; cb <= c1; cb += 8 * kJoinBatch) {
      RowPiece<VEC, float> q[kJoinBatch];
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        const int64_t c = min(cb + 8 * u, c1);
        q[u].load(p.part + (2 * c + (c == c0 ? 1 : 0)) * p.D + col);
      }
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        float v[VEC];
        q[u].values(v);
        if (cb + 8 * u <= c1) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) acc[k] += v[k];
        }
      }
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
}

}  // namespace cutbce

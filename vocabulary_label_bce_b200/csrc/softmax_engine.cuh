// Tensor-core passes of the softmax losses over the whole item table: one
// persistent, warp-specialised sm_100a kernel template that forms logit tiles on
// tcgen05 (accumulators in tensor memory) and takes exponentials of them in
// registers.  No logit and no probability ever reaches device memory.
//
//   kLse   a CTA owns 128 positions and streams the items of one vocabulary
//          split; each thread keeps a running maximum and sum of one row's slab.
//   kRows  the same tiles with the exponent's offset known: P = 2^(c z - l_t) is
//          rounded to bf16, written back over the logits in tensor memory and
//          contracted with the item tile: dH partial += P E.
//   kItems a CTA owns 128 items and streams the positions: P = 2^(c z + b_t),
//          b_t = log2 |w_t| - l_t, and dE += +-P H.  Here a logit's row offset
//          runs along the columns of the tile; b_t / c, split into three bf16
//          values (24 bits), enters as one more K step of the logit MMA against
//          ones, so the epilogue loads nothing (2.89 to 2.44 ms at D = 64).  Above
//          D = 128 the pass is bound by the MMAs, and the epilogue loads b_t.  Rows are compacted by the sign
//          of w_t (the negative ones from a tile boundary on), so the sign is
//          the negate-A bit of the contraction's instruction descriptor.
//
// A row's targets are left out of all three passes (their exponentials are 0 in the
// sums and in P): p - q of a target is a small difference where the loss is small,
// and bf16(p) would swamp it.  softmax_head.cuh carries them in fp32.  Each epilogue
// thread owns a stationary row and walks its targets (kLse, kRows: the row's ids; kItems:
// the item's positions, from the sorted pairs) with a forward cursor; a tile without one
// pays a comparison and a vote.
//
// c = log2(e) / tau.  Warp roles, tensor-memory layout and hand-over of the tiles
// follow the BCE engine (warp 0 loads by TMA, 16 epilogue warps in two groups take
// alternate tiles), with one difference: the logit MMAs and the contractions are
// issued by two warps with blocking waits instead of one that polls for both.  With
// no element math at all the dH pass then takes 1.39 ms instead of 2.5 at 9.0e9 logits
// and D = 64.  Every wait is bounded.
//
// What bounds it, at T = 12,800 positions (10,240 count), V = 876,000, D = 64:
//   kLse   2.15 ms (2.02 with nothing left out).  One exponential per logit: 1.37 ms of SFU time with 5 of 16 on
//          the FMA pipe, which the maximum and the polynomial then share with the
//          sums.  256-item tiles: the hand-over alone takes 0.65 ms, with 128-item
//          tiles 1.08.
//   kRows  2.24 ms and kItems 2.10 ms in a few steps, 2.5 and 2.3 in a loop of them,
//          where the card holds its power limit (sw_power_cap); without the walk over the
//          targets 1% to 3% less.  The MMAs take 1.4 and
//          1.6 ms (the D = 64 contraction runs at two thirds of the tensor rate), the
//          exponentials 1.4 of SFU time; three logit buffers are all that fits beside
//          the accumulator.  Tried and no better: 64-item tiles with six buffers (2.27 /
//          2.28 ms), one or three epilogue groups, one arrival per warp.
//   D = 256, T = 8,192 (7,376 count), V = 1,000,000: kRows 5.7 ms, 1,330 TFLOP/s of its
//          two products, against 1,404 that a library bf16 product sustains on this
//          card.  Bound by the tensor cores under the power limit.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <type_traits>
#include "common.cuh"
#include "elementwise.cuh"
#include "ptx_sm100.cuh"
#include "softmax_head.cuh"
#include "wait.cuh"

namespace cutbce {

enum : int { kPassLse = 0, kPassRows = 1, kPassItems = 2 };

template <int DP, int kPass>
struct SoftmaxCfg {
  static constexpr bool kGrad = kPass != kPassLse;
  static constexpr bool kItems = kPass == kPassItems;
  static constexpr int GROUPS = 2;                          // epilogue groups taking tiles in turn
  // the dE pass's exponent offsets as one more K step of the logit MMA (see the top)
  static constexpr bool OFF_MMA = kItems && DP <= 128;
  static constexpr int GROUP_WARPS = 8;
  static constexpr int G_WARP = 2 + GROUPS * GROUP_WARPS;   // issuer of the contractions
  static constexpr int THREADS = 32 * (kGrad ? G_WARP + 1 : G_WARP);
  static constexpr int SLABS = GROUP_WARPS / 4;
  static constexpr int BN = DP == 64 && !kGrad ? 256 : DP <= 128 ? 128 : 64;   // streamed rows per tile
  static constexpr int NKB = DP / 64;
  static constexpr int NX = DP == 64 ? (kItems ? 9 : BN == 256 ? 6 : 12) : DP == 128 ? 5 : DP == 192 ? 7 : 4;
  static constexpr int NZ = kGrad ? 3 : BN == 256 ? 2 : 4;  // logit buffers in tensor memory
  static constexpr uint32_t S_BYTES = kTileM * DP * 2;
  static constexpr uint32_t X_BYTES = BN * DP * 2;
  static constexpr uint32_t O_BYTES = OFF_MMA ? BN * 32 : 0;         // exponent offsets of a streamed tile (16 bf16 a row)
  static constexpr uint32_t ONES_BYTES = OFF_MMA ? kTileM * 32 : 0;  // their other operand
  static constexpr int ZC = BN / SLABS;                     // logit columns per epilogue warp (64 or 32)
  static constexpr int ACC_COL = kGrad ? 3 * BN : 0;
  static constexpr int S_COL = ACC_COL + DP;
  static constexpr bool S_IN_TMEM = kGrad && S_COL + DP / 2 <= 512;
  static constexpr int ONES_COL = S_COL + DP / 2;
  static constexpr bool ONES_IN_TMEM = OFF_MMA && S_IN_TMEM && ONES_COL + 8 <= 512;
  static constexpr int NUM_BARS = 2 + 2 * NX + 3 * NZ + 3 + GROUPS;
  static constexpr uint32_t SMEM_BYTES = 1024 + S_BYTES + NX * (X_BYTES + O_BYTES) + ONES_BYTES + NUM_BARS * 8 + 16 + 64;
  static_assert((!kGrad || ACC_COL + DP <= 512) && NZ * BN <= 512, "TMEM budget");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(GROUPS * SLABS == 4, "partials per split");
  static_assert(SMEM_BYTES > 232448 / 2, "one CTA per SM keeps the TMEM allocation uncontended");
};

struct SoftmaxParams {
  int V, D;
  int64_t Tc;                  // rows of the compacted buffers
  HeadHeader* hdr;
  float c2;                    // log2(e) / tau
  const float* off2;           // kRows: [Tc] l_t; kItems without OFF_MMA: [Tc] b_t (log2 domain)
  float2* part;                // kLse, and kRows where it takes the sums: [splits * groups * slabs, Tc] (reference, sum)
  const float2* wide_part;     // kRows: partials of the log-sum-exp pass, the reference where hdr->wide is set
  int wide_slots;              // their number per row
  int only_wide;               // kLse: run only where hdr->wide is set
  float* dh_part;              // kRows: [splits, Tc, DP]
  const int* targets;          // kLse, kRows: [Tc, K] ids of each row's targets, ascending, then -1
  int K;
  const uint32_t* columns;     // kItems: [n_pairs] compacted positions of the sorted pairs, 2^31 added to an item's first
  int n_pairs;
  const int* first;            // kItems: [V] first pair of each item, and its row of `sparse`; -1 none
  const float* sparse;         // kItems: [.., D] sum of (q - p) h over the item's pairs
  void* dE;                    // kItems: [V, D]
  int de_bf16, de_acc;
  int nsplit, tiles_per_split, n_item_tiles_bn;
  long long timeout_ns;
};

// Pairs of every 16 whose exponential runs on the FMA pipe instead of the SFU.
// Measured at 9.0e9 logits, D = 64, nothing left out, for 2 / 4 / 5 / 6 / 7 pairs: dH pass 2.20 / 2.17 /
// 2.15 / 2.15 / 2.26 ms, dE pass 2.23 / 2.09 / 2.11 / 2.10 / 2.16 ms; log-sum-exp
// pass for 4 / 5 / 6 / 7: 2.09 / 2.01 / 2.05 / 2.14 ms.
constexpr int kPolyLse = 5, kPolyRows = 5, kPolyItems = 5;

// The larger (largest) of two (three): NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^x of a pair on the FMA pipe, x clamped below at -125: as exp2_poly3_pair, with
// the degree chosen by what the value feeds.  kDegree 3 (relative error 7.5e-5) for
// values that are rounded to bf16 next, 4 (2.7e-6) for the sums of a log-sum-exp.
// NaN gives the largest float (its bits 0x7FFFFFFF and, shifted, 0xFF800000 add up to
// 0x7F7FFFFF): a row's sum then passes 2^64, which no finite row's does, and the join of the
// sums takes it for NaN.
template <int kDegree>
__device__ __forceinline__ float2 exp2_fma_pair(float2 x) {
  constexpr float kShift = 12582912.0f;   // 1.5 * 2^23
  x = f2(max_nan(x.x, -125.f), max_nan(x.y, -125.f));
  const float2 j = __fadd2_rn(x, f2(kShift, kShift));
  const float2 jr = __fadd2_rn(j, f2(-kShift, -kShift));
  const float2 f = __ffma2_rn(jr, f2(-1.f, -1.f), x);
  float2 p;
  if (kDegree == 3) {
    p = __ffma2_rn(f2(0.0551716685f, 0.0551716685f), f, f2(0.2426111251f, 0.2426111251f));
    p = __ffma2_rn(p, f, f2(0.6932609677f, 0.6932609677f));
    p = __ffma2_rn(p, f, f2(0.9999280572f, 0.9999280572f));
  } else {
    p = __ffma2_rn(f2(0.0095701022f, 0.0095701022f), f, f2(0.0559178591f, 0.0559178591f));
    p = __ffma2_rn(p, f, f2(0.2402474433f, 0.2402474433f));
    p = __ffma2_rn(p, f, f2(0.6931217909f, 0.6931217909f));
    p = __ffma2_rn(p, f, f2(0.9999992847f, 0.9999992847f));
  }
  uint32_t rx, ry;
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(rx) : "r"(__float_as_uint(j.x)), "r"(1u << 23), "r"(__float_as_uint(p.x)));
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(ry) : "r"(__float_as_uint(j.y)), "r"(1u << 23), "r"(__float_as_uint(p.y)));
  return f2(__uint_as_float(rx), __uint_as_float(ry));
}
// Pair e / 2 of a chunk of 16: `kPoly` of them, evenly spread, run on the FMA pipe.
template <int kPoly, int kDegree>
__device__ __forceinline__ float2 exp2_pair(int pair, float2 x) {
  if ((pair * kPoly) % 16 < kPoly) return exp2_fma_pair<kDegree>(x);
  return f2(ex2_approx(x.x), ex2_approx(x.y));
}

// Forward-only cursor over the columns that a stationary row leaves out: `next` is the
// first not yet passed, `ahead` the one behind it (2^31 and above: none is left).  Passing
// one loads another, which is not looked at before the one after it is passed, so that the
// load's latency is hidden (waiting for it made the log-sum-exp pass 2.33 ms instead of 2.15
// at T = 12,800, V = 876,000, K = 16).
// The list is the row's of `targets`, or the item's run of `columns`.
constexpr uint32_t kNoTarget = 0xFFFFFFFFu;
struct TargetCursor {
  int at;                       // index of `next`: slot of the row's list, or entry of `columns`
  uint32_t next, ahead;
};

template <bool kItems>
__device__ __forceinline__ uint32_t load_target(const SoftmaxParams& p, int s_row, int at) {
  if (kItems) return at < p.n_pairs ? __ldg(p.columns + at) : kNoTarget;
  return at < p.K ? static_cast<uint32_t>(__ldg(p.targets + static_cast<int64_t>(s_row) * p.K + at)) : kNoTarget;
}

// kLse, kRows: starts at the first id of the row's list that is not below col0.  Halved down
// to eight slots, which are loaded together: one round trip for K <= 8, two for 16.
__device__ __forceinline__ TargetCursor row_cursor(const SoftmaxParams& p, int s_row, uint32_t col0) {
  int lo = 0, n = p.K;
  while (n > 8) {
    const int half = n >> 1;
    if (load_target<false>(p, s_row, lo + half) < col0) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  // the answer is one of slots lo .. lo + n
  uint32_t v[9];
#pragma unroll
  for (int i = 0; i < 9; ++i) v[i] = i <= n ? load_target<false>(p, s_row, lo + i) : kNoTarget;
  TargetCursor cur{lo, kNoTarget, kNoTarget};
#pragma unroll
  for (int i = 0; i < 9; ++i) {
    cur.at += v[i] < col0;
    if (v[i] >= col0) cur.next = min(cur.next, v[i]);
  }
  cur.ahead = load_target<false>(p, s_row, cur.at + 1);
  return cur;
}

// The targets in columns [lo, lo + 32 N), lo a multiple of 32, as bits of mask[N]; passes all
// below the end (those below lo are in another warp's columns).  A list may name a column
// twice.  Where a row has more than one, up to kBatch others are loaded together; rows of an
// item that has still more in this tile (an item of many positions) are then taken one by
// one by the whole warp, 32 entries at a time.  With ids of a Zipf law (4,834 positions, half
// of them in one tile of items) the dE pass takes 0.154 ms, 0.26 entry by entry, 0.14
// if nothing were left out.
template <bool kItems, int N>
__device__ __forceinline__ void take_targets(TargetCursor& cur, const SoftmaxParams& p, int s_row, uint32_t lo, uint32_t (&mask)[N]) {
  constexpr int kBatch = 8;
  const uint32_t hi = lo + 32u * N;
  const int lane = threadIdx.x & 31;
  auto set = [&](uint32_t (&m)[N], uint32_t col) {
#pragma unroll
    for (int w = 0; w < N; ++w)
      if (col - (lo + 32u * w) < 32u) m[w] |= 1u << (col & 31u);
  };
  bool more = false;
  if (cur.next < hi) {
    set(mask, cur.next);
    cur.next = cur.ahead;
    ++cur.at;
    more = cur.next < hi;
    if (!more) cur.ahead = load_target<kItems>(p, s_row, cur.at + 1);
  }
  if (!__any_sync(0xffffffffu, more)) return;
  if (!kItems) {
    while (cur.next < hi) {
      set(mask, cur.next);
      cur.next = load_target<false>(p, s_row, ++cur.at);
    }
    if (more) cur.ahead = load_target<false>(p, s_row, cur.at + 1);
    return;
  }
  const bool again = more;
  if (more) {
    set(mask, cur.next);
    uint32_t col[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) col[u] = load_target<kItems>(p, s_row, cur.at + 1 + u);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!more) continue;
      ++cur.at;
      cur.next = col[u];
      more = col[u] < hi;
      if (more) set(mask, col[u]);
    }
  }
  // rows with `more`: the entry cur.at is taken, those behind it are not
  for (unsigned todo = __ballot_sync(0xffffffffu, more); todo != 0u; todo &= todo - 1u) {
    const int from = __ffs(todo) - 1;
    int at = __shfl_sync(0xffffffffu, cur.at, from) + 1;
    uint32_t bits[N], next;
#pragma unroll
    for (int w = 0; w < N; ++w) bits[w] = 0u;
    while (true) {
      const uint32_t col = load_target<kItems>(p, s_row, at + lane);
      // columns ascend up to the next item's first, whose top bit is set; what follows is not this item's
      const unsigned past = __ballot_sync(0xffffffffu, col >= hi);
      const int below = past != 0u ? __ffs(past) - 1 : 32;
      if (lane < below) set(bits, col);
      at += below;
      next = __shfl_sync(0xffffffffu, col, below & 31);
      if (below < 32) break;
    }
#pragma unroll
    for (int w = 0; w < N; ++w) {
      bits[w] = __reduce_or_sync(0xffffffffu, bits[w]);
      if (lane == from) mask[w] |= bits[w];
    }
    if (lane == from) {
      cur.at = at;
      cur.next = next;
    }
  }
  if (again) cur.ahead = load_target<kItems>(p, s_row, cur.at + 1);
}

template <int DP, int kPass>
__global__ void __launch_bounds__(SoftmaxCfg<DP, kPass>::THREADS, 1)
    k_softmax(const __grid_constant__ CUtensorMap tmS, const __grid_constant__ CUtensorMap tmX,
              const __grid_constant__ CUtensorMap tmO, SoftmaxParams p) {
  constexpr bool kGrad = kPass != kPassLse;
  constexpr bool kItems = kPass == kPassItems;
  using Cfg = SoftmaxCfg<DP, kPass>;
  constexpr int BN = Cfg::BN, NKB = Cfg::NKB, NX = Cfg::NX, NZ = Cfg::NZ, ZC = Cfg::ZC;
  constexpr uint32_t S_BYTES = Cfg::S_BYTES, X_BYTES = Cfg::X_BYTES;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sS = smem;
  uint8_t* sX = sS + S_BYTES;
  uint8_t* sO = sX + NX * X_BYTES;                // kItems: [NX] offsets, 32-byte rows, 32-byte swizzle
  uint8_t* sOne = sO + NX * Cfg::O_BYTES;         // kItems: 128 rows of (1, 1, 1, 0, ..)
  uint64_t* bars = reinterpret_cast<uint64_t*>(sOne + Cfg::ONES_BYTES);
  uint64_t* bar_sfull = bars + 0;                 // stationary tile landed (TMA)
  uint64_t* bar_sempty = bars + 1;                // stationary tile no longer read (commit)
  uint64_t* bar_xfull = bars + 2;                 // [NX] streamed tile landed
  uint64_t* bar_xempty = bar_xfull + NX;          // [NX] streamed tile free (commit)
  uint64_t* bar_zfull = bar_xempty + NX;          // [NZ] logit tile ready (commit)
  uint64_t* bar_zfree = bar_zfull + NZ;           // [NZ] buffer free: P contracted (commit), or logits loaded (epilogue)
  uint64_t* bar_pready = bar_zfree + NZ;          // [NZ] P written over the logits (epilogue)
  uint64_t* bar_accfull = bar_pready + NZ;        // [groups] accumulator complete, for the group that reads it (commit)
  uint64_t* bar_accempty = bar_accfull + Cfg::GROUPS;  // accumulator read out (epilogue)
  uint64_t* bar_drain = bar_accempty + 1;         // every logit MMA done
  uint64_t* bar_gdrain = bar_drain + 1;           // every contraction done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + Cfg::NUM_BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  WsHeader* hdr = &p.hdr->w;
  __shared__ int s_status, s_rows, s_neg0, s_wide;
  if (threadIdx.x == 0) {
    s_status = *reinterpret_cast<volatile int*>(&hdr->status);
    s_rows = p.hdr->n_rows;
    s_neg0 = p.hdr->neg0;
    s_wide = p.hdr->wide;
  }
  __syncthreads();
  if (s_status != 0 || (kPass == kPassLse && p.only_wide && !s_wide)) return;
  const int n_rows = s_rows;                      // compacted rows, a multiple of 128
  const int neg_tile = s_neg0 / BN;               // kItems: first streamed tile of negative rows
  const int n_row_tiles = n_rows / kTileM;
  const int n_items = kItems ? static_cast<int>(ceil_div(p.V, kTileM)) : p.nsplit * n_row_tiles;
  if (kItems && n_rows == 0) {
    // no position counts: dE is zero
    if (p.de_acc) return;
    const int64_t n = static_cast<int64_t>(p.V) * p.D;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * Cfg::THREADS + threadIdx.x; k < n;
         k += static_cast<int64_t>(gridDim.x) * Cfg::THREADS) {
      if (p.de_bf16) static_cast<__nv_bfloat16*>(p.dE)[k] = __float2bfloat16_rn(0.f);
      else static_cast<float*>(p.dE)[k] = 0.f;
    }
    return;
  }
  if (static_cast<int>(blockIdx.x) >= n_items) return;

  if (threadIdx.x == 0) {
    mbar_init(bar_sfull, 1);
    mbar_init(bar_sempty, 1);
    for (int s = 0; s < NX; ++s) {
      mbar_init(bar_xfull + s, 1);
      mbar_init(bar_xempty + s, 1);
    }
    for (int b = 0; b < NZ; ++b) {
      mbar_init(bar_zfull + b, 1);
      mbar_init(bar_zfree + b, kGrad ? 1 : Cfg::GROUP_WARPS * 32);
      mbar_init(bar_pready + b, Cfg::GROUP_WARPS * 32);
    }
    for (int g = 0; g < Cfg::GROUPS; ++g) mbar_init(bar_accfull + g, 1);
    mbar_init(bar_accempty, Cfg::GROUP_WARPS);
    mbar_init(bar_drain, 1);
    mbar_init(bar_gdrain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmS);
    tma_prefetch_desc(&tmX);
    if (Cfg::OFF_MMA) tma_prefetch_desc(&tmO);
  }
  if (Cfg::OFF_MMA) {
    // the two 16-byte halves of a row trade places in rows 4..7 of each 8 (32-byte swizzle)
    if (threadIdx.x < kTileM) {
      const int r = threadIdx.x, sw = (r >> 2) & 1;
      uint4* dst = reinterpret_cast<uint4*>(sOne + 32 * r);
      dst[sw] = make_uint4(0x3F803F80u, 0x00003F80u, 0u, 0u);
      dst[sw ^ 1] = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtx wc{abort_flag, hdr, p.timeout_ns};

  // work item i: a tile of items (kItems), or (vocabulary split, tile of positions), split-major
  auto item = [&](int i, int& s_row0, int& x0, int& nx, int& split) {
    if (kItems) {
      // The first round goes from the last CTA to the first: where ids are ranks, the tile
      // with the most pairs goes to a CTA that has no tile of the last round (0.175 to 0.154 ms
      // for the dE pass of 4,834 positions of a Zipf law, V = 100,000; 0.166 either way of 51,200
      // evenly spread pairs).
      s_row0 = (i < static_cast<int>(gridDim.x) ? static_cast<int>(gridDim.x) - 1 - i : i) * kTileM;
      x0 = 0;
      nx = n_rows / BN;
      split = 0;
    } else {
      split = i / n_row_tiles;
      s_row0 = (i - split * n_row_tiles) * kTileM;
      x0 = split * p.tiles_per_split;
      nx = min(p.tiles_per_split, p.n_item_tiles_bn - x0);
    }
  };

  if (warp == 0) {
    // ============================================================ TMA producer
    if (lane == 0) {
      uint32_t ic = 0, xc = 0;
      for (int i = blockIdx.x; i < n_items; i += gridDim.x, ++ic) {
        int s_row0, x0, nx, split;
        item(i, s_row0, x0, nx, split);
        if (!wait_bar(bar_sempty, (ic & 1) ^ 1, wc, wait_tag(1, 1, ic))) break;
        mbar_arrive_expect_tx(bar_sfull, S_BYTES);
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) tma_load_2d(sS + kb * (kTileM * 128), &tmS, kb * 64, s_row0, bar_sfull);
        bool ok = true;
        for (int j = 0; j < nx; ++j, ++xc) {
          const uint32_t st = xc % NX;
          if (!wait_bar(bar_xempty + st, ((xc / NX) & 1) ^ 1, wc, wait_tag(1, 3, xc))) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(bar_xfull + st, X_BYTES + Cfg::O_BYTES);
          if (Cfg::OFF_MMA) tma_load_2d(sO + st * Cfg::O_BYTES, &tmO, 0, (x0 + j) * BN, bar_xfull + st);
#pragma unroll
          for (int kb = 0; kb < NKB; ++kb)
            tma_load_2d(sX + st * X_BYTES + kb * (BN * 128), &tmX, kb * 64, (x0 + j) * BN, bar_xfull + st);
        }
        if (!ok) {
          ++ic;
          break;
        }
      }
      // wait (bounded) for every copy this thread issued to land
      if (ic > 0) wait_bar_drain(bar_sfull, (ic - 1) & 1, p.timeout_ns);
      for (uint32_t st = 0; st < NX; ++st) {
        const uint32_t issued = xc > st ? (xc - st + NX - 1) / NX : 0;
        if (issued > 0) wait_bar_drain(bar_xfull + st, (issued - 1) & 1, p.timeout_ns);
      }
    }
  } else if (warp == 1) {
    // ============================================================ MMA issuer
    // The logit tiles, in order, by blocking waits.  The contractions have a warp of
    // their own: one warp polling for both took 1250 cycles a tile even with no element
    // math at all, this form 820.
    constexpr uint32_t idesc_z = idesc_bf16_f32(kTileM, BN, false, false);
    constexpr uint32_t kXStep = X_BYTES >> 4;
    const uint64_t dS = smem_desc_sw128(smem_u32(sS), 16, 1024);
    const uint64_t dXk = smem_desc_sw128(smem_u32(sX), 16, 1024);
    const uint64_t dO = smem_desc_sw32(smem_u32(sO)), dOne = smem_desc_sw32(smem_u32(sOne));
    const uint32_t tS = tmem_base + Cfg::S_COL;
    uint32_t ic = 0, c = 0, st = 0, ph = 0, zb = 0, zph = 0;
    bool ok = true;
    if (Cfg::ONES_IN_TMEM) {
      if (elect_one()) tmem_cp_128x256b(tmem_base + Cfg::ONES_COL, dOne);
      __syncwarp();
    }
    for (int i = blockIdx.x; i < n_items && ok; i += gridDim.x, ++ic) {
      int row0, x0, nx, split;
      item(i, row0, x0, nx, split);
      if (!wait_bar_warp(bar_sfull, ic & 1, wc, wait_tag(2, 0, ic))) break;
      tc_fence_after();
      if (Cfg::S_IN_TMEM) {
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks)
            tmem_cp_128x256b(tS + 8 * ks, dS + static_cast<uint32_t>((ks >> 2) * (kTileM * 8) + (ks & 3) * 2));
          umma_commit(bar_sempty);
        }
        __syncwarp();
      }
      for (int j = 0; j < nx; ++j, ++c) {
        if (!wait_bar_warp(bar_xfull + st, ph, wc, wait_tag(2, 1, c)) ||
            !wait_bar_warp(bar_zfree + zb, zph ^ 1, wc, wait_tag(2, 2, c))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dB = dXk + st * kXStep;
        const uint32_t tD = tmem_base + zb * BN;
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            const uint64_t bd = dB + static_cast<uint32_t>((ks >> 2) * (BN * 8) + (ks & 3) * 2);
            if (Cfg::S_IN_TMEM) umma_bf16_tmem_a(tD, tS + 8 * ks, bd, idesc_z, ks > 0 ? 1u : 0u);
            else umma_bf16(tD, dS + static_cast<uint32_t>((ks >> 2) * (kTileM * 8) + (ks & 3) * 2), bd, idesc_z,
                           ks > 0 ? 1u : 0u);
          }
          if (Cfg::ONES_IN_TMEM) umma_bf16_tmem_a(tD, tmem_base + Cfg::ONES_COL, dO + st * (Cfg::O_BYTES >> 4), idesc_z, 1u);
          else if (Cfg::OFF_MMA) umma_bf16(tD, dOne, dO + st * (Cfg::O_BYTES >> 4), idesc_z, 1u);
          umma_commit(bar_zfull + zb);
          if (!kGrad) umma_commit(bar_xempty + st);
          if (!Cfg::S_IN_TMEM && j + 1 == nx) umma_commit(bar_sempty);
        }
        __syncwarp();
        if (++st == static_cast<uint32_t>(NX)) {
          st = 0;
          ph ^= 1;
        }
        if (++zb == static_cast<uint32_t>(NZ)) {
          zb = 0;
          zph ^= 1;
        }
      }
    }
    // every MMA this warp issued has completed once the drain barrier flips
    if (elect_one()) umma_commit(bar_drain);
    __syncwarp();
    if (lane == 0) wait_bar_drain(bar_drain, 0, p.timeout_ns);
    __syncwarp();
  } else if (kGrad && warp == Cfg::G_WARP) {
    // ============================================================ contraction issuer
    constexpr uint32_t idesc_acc = idesc_bf16_f32(kTileM, DP, false, true);
    constexpr uint32_t kNegateA = 1u << 13;
    constexpr uint32_t kXStep = X_BYTES >> 4;
    constexpr int kKsPerSlab = ZC / 16;
    const uint64_t dXmn = smem_desc_sw128(smem_u32(sX), BN * 128, 1024);
    const uint32_t tAcc = tmem_base + Cfg::ACC_COL;
    uint32_t ic = 0, c = 0, st = 0, gb = 0, gph = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < n_items && ok; i += gridDim.x, ++ic) {
      int row0, x0, nx, split;
      item(i, row0, x0, nx, split);
      if (!wait_bar_warp(bar_accempty, (ic & 1) ^ 1, wc, wait_tag(2, 4, ic))) break;
      for (int j = 0; j < nx; ++j, ++c) {
        if (!wait_bar_warp(bar_pready + gb, gph, wc, wait_tag(2, 3, c))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t dB = dXmn + st * kXStep;
        const uint32_t tA = tmem_base + gb * BN;
        const bool last = j + 1 == nx;
        const uint32_t idesc = kItems && j >= neg_tile ? idesc_acc | kNegateA : idesc_acc;
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < BN / 16; ++ks) {
            const uint32_t a_col = (ks / kKsPerSlab) * ZC + 8 * (ks % kKsPerSlab);
            umma_bf16_tmem_a(tAcc, tA + a_col, dB + static_cast<uint32_t>(ks * 128), idesc, (j > 0 || ks > 0) ? 1u : 0u);
          }
          umma_commit(bar_zfree + gb);
          umma_commit(bar_xempty + st);
          if (last) umma_commit(bar_accfull + c % Cfg::GROUPS);
        }
        __syncwarp();
        if (++st == static_cast<uint32_t>(NX)) st = 0;
        if (++gb == static_cast<uint32_t>(NZ)) {
          gb = 0;
          gph ^= 1;
        }
      }
    }
    if (elect_one()) umma_commit(bar_gdrain);
    __syncwarp();
    if (lane == 0) wait_bar_drain(bar_gdrain, 0, p.timeout_ns);
    __syncwarp();
  } else {
    // ============================================================ epilogue
    constexpr int NCH = ZC / 32;                  // chunks of 32 columns per warp and tile
    constexpr int AC = DP / Cfg::SLABS;           // accumulator columns per warp
    const int ew = warp - kEpiWarp0;
    const uint32_t grp = static_cast<uint32_t>(ew / Cfg::GROUP_WARPS);
    const int q = warp & 3;
    const int slab = (ew >> 2) % Cfg::SLABS;
    const int row = q * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    const float2 c2 = f2(p.c2, p.c2);
    uint32_t cnt = 0, ic = 0, acc_reads = 0;
    bool ok = true;
    // kItems: the item's first pair, read ahead (the next item's beside this one's tiles)
    auto first_of = [&](int v) { return v < p.V ? __ldg(p.first + v) : -1; };
    int first = -1;
    TargetCursor cur{-1, kNoTarget, kNoTarget};
    auto item_cursor = [&] {                      // at the item's first pair, whose top bit goes
      cur = TargetCursor{first, kNoTarget, kNoTarget};
      if (first < 0) return;
      cur.next = load_target<true>(p, 0, first) & 0x7FFFFFFFu;
      cur.ahead = load_target<true>(p, 0, first + 1);
    };
    if (kItems) {
      int s_row0, x0, nx, split;
      item(static_cast<int>(blockIdx.x), s_row0, x0, nx, split);
      first = first_of(s_row0 + row);
      item_cursor();
    }
    for (int i = blockIdx.x; i < n_items && ok; i += gridDim.x, ++ic) {
      int s_row0, x0, n, split;
      item(i, s_row0, x0, n, split);
      float m = -1e30f, sum = 0.f;                // reference (log2 domain) and sum of 2^(x - m)
      float off = 0.f;                            // kRows: -m
      if (kPass == kPassRows) {
        m = __ldg(p.off2 + s_row0 + row);
        if (p.wide_part != nullptr && s_wide) {
          // the row's log-sum-exp from the partials of the pass before
          const int slots = p.wide_slots;
          float mx = -3.0e38f, s = 0.f;
          for (int k = 0; k < slots; ++k) mx = fmaxf(mx, p.wide_part[k * p.Tc + s_row0 + row].x);
          for (int k = 0; k < slots; ++k) {
            const float2 v = p.wide_part[k * p.Tc + s_row0 + row];
            s += v.y * exp2f(v.x - mx);
          }
          m = mx + log2f(s);
        }
        off = -m;
      }
      const int s_row = s_row0 + row;
      int first_next = -1;
      if (!kItems) cur = row_cursor(p, s_row, static_cast<uint32_t>(x0) * BN);
      else if (i + static_cast<int>(gridDim.x) < n_items) first_next = first_of((i + static_cast<int>(gridDim.x)) * kTileM + row);
      const int j0 = static_cast<int>((grp + Cfg::GROUPS - cnt % Cfg::GROUPS) % Cfg::GROUPS);
      for (int j = j0; j < n; j += Cfg::GROUPS) {
        const uint32_t c = cnt + j, bz = c % NZ;
        const int tile_col0 = (x0 + j) * BN + slab * ZC;      // item (or compacted position) of the slab's first column
        // columns that count as -infinity: the row's targets, and those past the table's end
        uint32_t drop[NCH];
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) drop[ch] = 0u;
        unsigned hit = 0u;                        // chunks that have such a column in some row of the warp
        if (__any_sync(0xffffffffu, cur.next < static_cast<uint32_t>(tile_col0) + ZC)) {
          take_targets<kItems>(cur, p, s_row, static_cast<uint32_t>(tile_col0), drop);
#pragma unroll
          for (int ch = 0; ch < NCH; ++ch) hit |= __any_sync(0xffffffffu, drop[ch] != 0u) ? 1u << ch : 0u;
        }
        if (!kItems && (x0 + j + 1) * static_cast<int64_t>(BN) > p.V) {
          hit = (1u << NCH) - 1u;
#pragma unroll
          for (int ch = 0; ch < NCH; ++ch) {
            const int valid = p.V - (tile_col0 + ch * 32);
            if (valid < 32) drop[ch] |= valid <= 0 ? 0xFFFFFFFFu : 0xFFFFFFFFu << valid;
          }
        }
        if (!wait_bar_warp(bar_zfull + bz, (c / NZ) & 1, wc, wait_tag(4, 4, c))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int ch = 0; ch < NCH; ++ch) {
          uint32_t r[32];
          tmem_ld32(tmem_base + lane_base + bz * BN + slab * ZC + ch * 32, r);
          tmem_ld_wait();
          if (!kGrad && ch == NCH - 1) {
            tc_fence_before();
            mbar_arrive(bar_zfree + bz);
          }
          const int col = tile_col0 + ch * 32;
          if (hit >> ch & 1u) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (drop[ch] >> e & 1u) r[e] = 0xFF800000u;
          }
          if constexpr (kPass == kPassLse) {
            float mx4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mx4[k] = max_nan(__uint_as_float(r[8 * k]), __uint_as_float(r[8 * k + 1]));
#pragma unroll
              for (int e = 2; e < 8; e += 2)
                mx4[k] = max_nan(mx4[k], __uint_as_float(r[8 * k + e]), __uint_as_float(r[8 * k + e + 1]));
            }
            const float mx = max_nan(max_nan(mx4[0], mx4[1], mx4[2]), mx4[3]) * p.c2;
            // the reference moves only when the maximum has grown by 2^8: sums stay far from
            // overflow; a NaN moves it, and the sum is NaN from there on
            const float mn = !(mx <= m + 8.f) ? mx : m;
            sum *= ex2_approx(m - mn);
            m = mn;
            const float2 nm = f2(-m, -m);
            float2 s4[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 x = __ffma2_rn(f2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), c2, nm);
              s4[(e >> 1) & 3] = __fadd2_rn(s4[(e >> 1) & 3], exp2_pair<kPolyLse, 4>(e >> 1, x));
            }
            const float2 s2 = __fadd2_rn(__fadd2_rn(s4[0], s4[1]), __fadd2_rn(s4[2], s4[3]));
            sum += s2.x + s2.y;
          } else {
            uint32_t pk[16];
            float2 s2 = f2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 z = f2(__uint_as_float(r[e]), __uint_as_float(r[e + 1]));
              float2 x;
              if (Cfg::OFF_MMA) x = __fmul2_rn(z, c2);
              else if (kItems) x = __ffma2_rn(z, c2, __ldg(reinterpret_cast<const float2*>(p.off2 + col + e)));
              else x = __ffma2_rn(z, c2, f2(off, off));
              const float2 y = kItems ? exp2_pair<kPolyItems, 3>(e >> 1, x) : exp2_pair<kPolyRows, 4>(e >> 1, x);
              if (!kItems) s2 = __fadd2_rn(s2, y);
              pk[e >> 1] = pack_bf16x2(y.x, y.y);
            }
            tmem_st16(tmem_base + lane_base + bz * BN + slab * ZC + ch * 16, pk);
            if (!kItems) sum += s2.x + s2.y;
          }
        }
        if constexpr (kGrad) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar_pready + bz);
        }
      }
      if (!ok) break;
      const int64_t sp = first;                   // kItems: the item's row of `sparse`
      if (kItems) {
        first = first_next;
        item_cursor();
      }
      if (kPass == kPassLse || (kPass == kPassRows && p.part != nullptr)) {
        const int slot = (split * Cfg::GROUPS + static_cast<int>(grp)) * Cfg::SLABS + slab;
        p.part[static_cast<int64_t>(slot) * p.Tc + s_row0 + row] = make_float2(m, sum);
      }
      if (kGrad && (cnt + n - 1) % Cfg::GROUPS == grp) {
        // the group that took the last tile reads the accumulator out; each group's
        // barrier counts its own read-outs (with one tile an item, a shared barrier could
        // be tested a whole phase early)
        if (!wait_bar_warp(bar_accfull + grp, acc_reads & 1, wc, wait_tag(4, 9, ic))) break;
        ++acc_reads;
        tc_fence_after();
        const int v = s_row0 + row;
        // a row whose probabilities are NaN makes every row of dE NaN
        const float gs = !kItems ? 0.f : p.hdr->nan_rows != 0 ? __int_as_float(0x7FFFFFFF) : hdr->grad_scale;
#pragma unroll 1
        for (int ch = 0; ch < AC / 16; ++ch) {
          uint32_t r[16];
          const int col0 = slab * AC + ch * 16;
          tmem_ld<16>(tmem_base + lane_base + Cfg::ACC_COL + col0, r);
          tmem_ld_wait();
          if (!kItems) {
            float* dst = p.dh_part + (static_cast<int64_t>(split) * p.Tc + s_row0 + row) * DP + col0;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(dst + e) = make_float4(__uint_as_float(r[e]), __uint_as_float(r[e + 1]),
                                                                __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
          } else if (v < p.V) {
            // eight columns at a time (D is a multiple of 8): 16-byte stores in either dtype
            const int64_t o = static_cast<int64_t>(v) * p.D + col0;
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              if (col0 + e >= p.D) continue;
              float g[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) g[k] = __uint_as_float(r[e + k]);
              if (sp >= 0) {
                const float4* s4 = reinterpret_cast<const float4*>(p.sparse + sp * p.D + col0 + e);
                const float4 lo = __ldg(s4), hi = __ldg(s4 + 1);
                g[0] -= lo.x, g[1] -= lo.y, g[2] -= lo.z, g[3] -= lo.w;
                g[4] -= hi.x, g[5] -= hi.y, g[6] -= hi.z, g[7] -= hi.w;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) g[k] = __fmul_rn(g[k], gs);
              if (p.de_bf16) {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dE) + o + e);
                if (p.de_acc) {
                  float old[8];
                  unpack8(*dst, old);
#pragma unroll
                  for (int k = 0; k < 8; ++k) g[k] = __fadd_rn(g[k], old[k]);
                }
                *dst = make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]),
                                  pack_bf16x2(g[6], g[7]));
              } else {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.dE) + o + e);
                if (p.de_acc) {
                  const float4 lo = dst[0], hi = dst[1];
                  g[0] = __fadd_rn(g[0], lo.x), g[1] = __fadd_rn(g[1], lo.y);
                  g[2] = __fadd_rn(g[2], lo.z), g[3] = __fadd_rn(g[3], lo.w);
                  g[4] = __fadd_rn(g[4], hi.x), g[5] = __fadd_rn(g[5], hi.y);
                  g[6] = __fadd_rn(g[6], hi.z), g[7] = __fadd_rn(g[7], hi.w);
                }
                dst[0] = make_float4(g[0], g[1], g[2], g[3]);
                dst[1] = make_float4(g[4], g[5], g[6], g[7]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_accempty);
      }
      cnt += n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace cutbce

// CUDA-core kernels around the softmax tile engine (softmax_engine.cuh): the
// losses with a softmax over the whole item table.
//
//   rows    which positions count, their class (sign of their gradient's factor),
//           the checks of ids and offsets, and the normalisation;
//   gather  compacts the rows of H (positive class first, the negative class from
//           the next multiple of 128 rows), sorts each row's targets, takes their
//           logits and their part of dH in fp32;
//   lse     joins the sums of a row's exponentials, forms p - q of its targets, and
//           the distillation loss;
//   pairs   the preference loss, from the sums over each sequence;
//   dh      adds the split partials of dH and the targets' part, scales.
//
// With p = softmax(z / tau) and q the sparse target weights of a position, the
// gradient of every such loss is  dz = w (p - q).  Where the losses are small, p is
// close to q, and p rounded to bf16 would leave only the rounding of that difference
// (with p = 0.996 it was off by half in the norm).  So an item that is a target of a
// row (q != 0) is left out of that row in the tile engine: its exponential counts as
// 0 in the sums and in the contractions, which carry w p of the other items alone, each
// rounded to bf16 relative to itself.  The targets are the sparse side's, in fp32.  With
// t_k = 2^(x_k - x_max) over the row's targets, T = sum t_k, and R the sum of the
// other items' exponentials on the same reference,
//   p_k = t_k / (T + R),  p_k - q_k = (t_k / T - q_k) - omp t_k / T,  omp = R / (T + R):
// omp = 1 - sum_k p_k comes from a sum, not from a difference, so one dominating
// target keeps all the bits of 1 - p.  (Where omp is the larger part, that difference
// would lose a small q, and p_k - q_k is formed as (1 - omp) t_k / T - q_k, with
// 1 - omp = T / (T + R).)  For dH the gather forms sum_k (q_k - t_k / T) e_k and
// sum_k t_k / T e_k, which the dh kernel joins by omp; for dE the factors q_k - p_k
// weigh the rows of H in the sums over sorted ids.
//
// All of them are short next to the tile passes and bound by memory latency; at
// T = 12,800, K = 16, V = 876,000, D = 64: rows 7 us, or 32 with the norms of the
// 112 MB table, gather 17 us (164,000 rows of E; 23 with gradients, which read them twice),
// lse 12 us (15 with q - p of the pairs), pairs 9 to 11 us, dh 20 us (79 MB of partials, mostly
// from L2).
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "common.cuh"
#include "id_sort.cuh"
#include "ptx_sm100.cuh"

namespace cutbce {

enum : int { kHeadDistill = 0, kHeadPreference = 1 };

// First 256 bytes of a softmax head's workspace.
struct HeadHeader {
  WsHeader w;               // status first; n_valid, grad_scale, waits
  int n_pos;                // rows of the positive class: compacted rows [0, n_pos)
  int n_neg;                // rows of the negative class: [neg0, neg0 + n_neg)
  int neg0;                 // first row of the negative class (a multiple of 128)
  int n_rows;               // compacted rows with padding (a multiple of 128)
  int rows_ticket;          // blocks done, per kernel that has a last block
  int lse_ticket;
  int pairs_ticket;
  unsigned emax2;           // bits of max |e_v|^2 (with a dH pass that takes the row sums too)
  int wide;                 // 1: some row's logits may lie too far below its bound (see the gather)
  int nan_rows;             // 1: some row's factor or probabilities are NaN
};
static_assert(sizeof(HeadHeader) <= 256, "the workspace header is 256 bytes");

struct HeadParams {
  int kind;
  int T, V, D, DP, K;
  int P;                         // preference pairs
  const __nv_bfloat16* H;
  const __nv_bfloat16* E;
  const int32_t* ids;            // [T, K]
  const float* logits;           // [T, K] teacher logits (distillation)
  const int32_t* offsets;        // [2P + 1] (preference)
  const float* ref;              // [2P] reference log-probabilities, or null
  const uint8_t* mask;
  const float* weights;          // [T], or null (distillation)
  float inv_tau, tau, beta;
  int reduction;
  const float* grad_loss;
  HeadHeader* hdr;
  uint8_t* cls;                  // [T] 0 none, 1 positive, 2 negative
  int* blk;                      // [2 * ceil(T / 256)] rows per class and block, then their prefix
  int n_blk;
  int* cidx;                     // [T] compacted row or -1
  int* orig;                     // [Tc] position of a compacted row, -1 padding
  __nv_bfloat16* Hc;             // [Tc, DP]
  double* rowterm;               // [Tc] distillation: sum_k q (ln q - (x_k - x_max) ln 2); preference: log p of the target
  float* sparse;                 // [Tc, 2, DP] sum_k (q_k - t_k / T) e_k, sum_k t_k / T e_k, or null
  float* tref;                   // [Tc] x_max: the largest x = c2 z of the row's targets
  float* tsum;                   // [Tc] T
  float* omp;                    // [Tc] 1 - the targets' probabilities
  int* targets;                  // [Tc, K] ids of the row's targets, ascending, then -1
  int* keys;                     // [Tc * K] ids of the pairs (-1 none; an id's first slot has all its weight), or null
  float* share;                  // [Tc * K] q of the pairs, then q - p, or null
  float* zt;                     // [Tc * K] x of the pairs, or null
  float* coef;                   // [Tc] signed factor of the row's gradient
  float* b2;                     // [Tc] log2 |factor| - lse (log2 domain; with dE, wide D), or null
  __nv_bfloat16* off16;          // [Tc, 16] (log2 |factor| - lse) tau in three bf16 pieces, then zeros (with dE), or null
  float* lse2;                   // [Tc] lse in the log2 domain
  const float* lse_in;           // [T] lse of an earlier forward, or null
  float* m2;                     // [Tc] reference of the exponentials in a dH pass that takes the row sums, or null
  float c2;                      // log2(e) / tau
  float* rescale;                // [Tc] 2^(reference - lse): factor of the dense part of dH
  const float2* part;            // [slots, Tc] (reference, sum) of the items that are not targets, log2 domain, or null
  int slots;
  int64_t Tc;                    // rows of the compacted buffers
  double* loss_part;             // per-block (distillation) or per-pair (preference) partials
  double* loss;                  // output or null
  float* lse_out;                // [T] output or null
  float* logp_out;               // [2P] output or null
};

// The exponent offset b of a row of the item-owned pass (log2 domain): as it is, or
// u = b / c2 as three bf16 values whose sum is u to 24 bits; clamped to +-1e30 (2^b is
// 0 there, as for padding).  NaN is noted in the header: the tile pass would lose it where
// it clamps.
__device__ __forceinline__ void write_offset(const HeadParams& p, int64_t c, float b2) {
  if (b2 != b2) p.hdr->nan_rows = 1;
  if (p.b2 != nullptr) p.b2[c] = b2;
  if (p.off16 == nullptr) return;
  float u = b2 / p.c2;
  u = fminf(fmaxf(u, -1e30f), 1e30f);
  const float a = __bfloat162float(__float2bfloat16_rn(u));
  const float b = __bfloat162float(__float2bfloat16_rn(u - a));
  const float d = (u - a) - b;
  uint4* o = reinterpret_cast<uint4*>(p.off16 + c * 16);
  o[0] = make_uint4(pack_bf16x2(a, b), pack_bf16x2(d, 0.f), 0u, 0u);
  o[1] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ rows
// The class of position t (0: it does not count); `bad` if its ids are out of range.
__device__ __forceinline__ int row_class(const HeadParams& p, int t, bool& bad) {
  int cls = 0;
  if (t < p.T && (p.mask == nullptr || p.mask[t] != 0)) {
    if (p.kind == kHeadDistill) {
      const float w = p.weights != nullptr ? p.weights[t] : 1.f;
      if (w != 0.f) {
        const int64_t r = static_cast<int64_t>(t) * p.K;
        bool any = false;
#pragma unroll 4
        for (int k = 0; k < p.K; ++k) {
          const int id = __ldg(p.ids + r + k);
          const float l = __ldg(p.logits + r + k);
          if (id == -1) continue;
          if (id < 0 || id >= p.V) bad = true;
          any |= !(l == -INFINITY);
        }
        if (any) cls = w < 0.f ? 2 : 1;
      }
    } else {
      const int id = p.ids[t];
      const int o0 = p.offsets[0], o1 = p.offsets[2 * p.P];
      if (id != -1 && t >= o0 && t < o1) {
        if (id < 0 || id >= p.V) bad = true;
        int lo = 0, hi = 2 * p.P;                     // the last sequence that starts at or before t
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.offsets + mid) <= t) lo = mid;
          else hi = mid;
        }
        cls = 1 + (lo & 1);
      }
    }
  }
  return cls;
}

// The header from the rows of each class.
__device__ __forceinline__ void write_counts(const HeadParams& p, int np, int nn) {
  HeadHeader* hdr = p.hdr;
  const int neg0 = (np + kTileM - 1) / kTileM * kTileM;
  hdr->n_pos = np;
  hdr->n_neg = nn;
  hdr->neg0 = neg0;
  hdr->n_rows = neg0 + (nn + kTileM - 1) / kTileM * kTileM;
  hdr->w.n_valid = np + nn;
  double s = 1.0;
  if (p.reduction == kMeanValidPositions) {
    const int n = p.kind == kHeadDistill ? np + nn : p.P;
    s = n > 0 ? 1.0 / n : 0.0;
  }
  const double g = p.grad_loss != nullptr ? static_cast<double>(*p.grad_loss) : 1.0;
  hdr->w.loss_scale = s;
  hdr->w.grad_scale = static_cast<float>(g * s * (p.kind == kHeadDistill ? p.tau : p.beta));
}


// Preference offsets ascend within [0, T]; thread i of n looks at every n-th from i on.
__device__ __forceinline__ bool bad_offsets(const HeadParams& p, int i0, int n) {
  bool bad = false;
  if (p.kind != kHeadPreference) return bad;
  for (int64_t i = i0; i <= 2 * static_cast<int64_t>(p.P); i += n) {
    const int o = p.offsets[i];
    if (o < 0 || o > p.T || (i > 0 && p.offsets[i - 1] > o)) bad = true;
  }
  return bad;
}

// Largest |e_v|^2 over the table: eight lanes a row, 16 bytes a lane, four rows in
// flight.  The maximum is over float bits (all >= 0), so the order of the atomics
// changes nothing; a NaN stays the maximum.
__device__ __forceinline__ void table_norm(const __nv_bfloat16* __restrict__ E, int64_t V, int D, HeadHeader* hdr,
                                           int block, int blocks) {
  constexpr int U = 4;
  const int sub = threadIdx.x & 7;
  const int64_t step = static_cast<int64_t>(blocks) * 32;
  unsigned best = 0u;
  // every lane of a warp runs the same trips, so that the sums below are whole
  for (int64_t v0 = static_cast<int64_t>(block) * 32; v0 < V; v0 += U * step) {
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = 0.f;
    for (int i = sub; i < D / 8; i += 8) {
      uint4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t v = min(v0 + u * step + (threadIdx.x >> 3), V - 1);     // a row read twice changes nothing
        x[u] = __ldg(reinterpret_cast<const uint4*>(E + v * D) + i);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xFFFF0000u);
          s[u] = fmaf(a, a, fmaf(b, b, s[u]));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
      best = max(best, __float_as_uint(s[u]) & 0x7FFFFFFFu);
    }
  }
  best = __reduce_max_sync(0xffffffffu, best);
  if ((threadIdx.x & 31) == 0 && best > *reinterpret_cast<volatile unsigned*>(&hdr->emax2)) atomicMax(&hdr->emax2, best);
}

// Blocks from n_blk on read the table's norms (with m2).
__global__ void __launch_bounds__(256) k_head_rows(const HeadParams p) {
  if (static_cast<int>(blockIdx.x) >= p.n_blk) {
    table_norm(p.E, p.V, p.D, p.hdr, static_cast<int>(blockIdx.x) - p.n_blk, static_cast<int>(gridDim.x) - p.n_blk);
    return;
  }
  __shared__ int cnt[2];
  __shared__ int last;
  __shared__ int tot[2][256];
  HeadHeader* hdr = p.hdr;
  const int tid = threadIdx.x;
  const int t = blockIdx.x * 256 + tid;
  if (tid < 2) cnt[tid] = 0;
  __syncthreads();
  bool bad = bad_offsets(p, t, p.n_blk * 256);
  const int cls = row_class(p, t, bad);
  if (bad) atomicCAS(&hdr->w.status, 0, kErrTargetRange);
  if (t < p.T) p.cls[t] = static_cast<uint8_t>(cls);
  const unsigned b1 = __ballot_sync(0xffffffffu, cls == 1), b2 = __ballot_sync(0xffffffffu, cls == 2);
  if ((tid & 31) == 0) {
    atomicAdd(&cnt[0], __popc(b1));
    atomicAdd(&cnt[1], __popc(b2));
  }
  __syncthreads();
  if (tid == 0) {
    p.blk[2 * blockIdx.x] = cnt[0];
    p.blk[2 * blockIdx.x + 1] = cnt[1];
    __threadfence();
    last = atomicAdd(&hdr->rows_ticket, 1) == p.n_blk - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  // the last block: exclusive prefix of the block counts, then the header
  const int per = (p.n_blk + 255) / 256;
  const int a = min(p.n_blk, tid * per), e = min(p.n_blk, a + per);
  int s0 = 0, s1 = 0;
  for (int i = a; i < e; ++i) {
    s0 += __ldcg(p.blk + 2 * i);
    s1 += __ldcg(p.blk + 2 * i + 1);
  }
  tot[0][tid] = s0;
  tot[1][tid] = s1;
  __syncthreads();
  for (int off = 1; off < 256; off <<= 1) {
    const int x0 = tid >= off ? tot[0][tid - off] : 0, x1 = tid >= off ? tot[1][tid - off] : 0;
    __syncthreads();
    tot[0][tid] += x0;
    tot[1][tid] += x1;
    __syncthreads();
  }
  int r0 = tot[0][tid] - s0, r1 = tot[1][tid] - s1;
  for (int i = a; i < e; ++i) {
    const int c0 = __ldcg(p.blk + 2 * i), c1 = __ldcg(p.blk + 2 * i + 1);
    p.blk[2 * i] = r0;
    p.blk[2 * i + 1] = r1;
    r0 += c0;
    r1 += c1;
  }
  if (tid == 0) write_counts(p, tot[0][255], tot[1][255]);
}

// ------------------------------------------------------------------ gather
// One warp per position; a warp whose position does not count, or that has none,
// takes an unused compacted row instead (padding: zeros, no targets).
// `L` lanes hold a row in 16-byte pieces (8, 16 or 32 for DP = 64, 128 and above),
// so a warp reads the rows of 32 / L targets at once, kGatherU of those in flight.
//
// With m2 it also sets the reference of the row's exponentials in a dH pass that
// takes the row's sum on the way: the lse of an earlier forward, or m = |h| max|e| c, a
// bound of every logit (Cauchy-Schwarz), so 2^(x - m) never overflows.  It must not lie
// too far above the row's largest logit either: terms below 2^-126 are lost, and with a
// gap of at most 70 (log2) the V < 2^31 lost terms are below 2^-25 of the sum.  The gap
// is bounded by a logit that the row is known to have, its largest sparse target.
// Rows beyond it set `wide`, and then the log-sum-exp pass runs first and its
// result is the reference.
//
// kSmall (up to kSmallRows positions and kSmallSlots slots in all): every block works out
// the classes of all positions itself, and block 0 writes the header, so a short call has
// neither the row kernel nor a memset before this one (one launch of 4 us less for the
// host).  The blocks' repeated reads grow with T^2 K.  Distillation losses, V = 2,048, D = 64,
// this way / with the row kernel, us on the device: T = 64, K = 16 18 / 25; T = 1,024, K = 16
// 27 / 28; T = 256, K = 64 49 / 57; T = 512, K = 64 67 / 57; T = 1,024, K = 64 100 / 57.
constexpr int kGatherU = 4;
constexpr float kMaxRefGap = 70.f;
constexpr int kSmallRows = 1024;
constexpr int kSmallSlots = 16384;

__device__ __forceinline__ void unpack8(uint4 r, float (&x)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(u[k] << 16);
    x[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
  }
}

// J: groups of 32 slots (1, 2 or 4).
template <int L, int J, bool kSmall>
__global__ void __launch_bounds__(256) k_head_gather(const HeadParams p) {
  constexpr int G = 32 / L;                     // targets side by side
  const HeadHeader* hdr = p.hdr;
  __shared__ uint8_t s_cls[kSmall ? kSmallRows : 1];
  __shared__ int s_cnt[kSmallRows / 256][2];    // rows per class of each 256 positions
  __shared__ int s_bad;
  int n_pos, n_neg, neg0;
  if (kSmall) {
    const int tid = threadIdx.x;
    if (tid < kSmallRows / 128) (&s_cnt[0][0])[tid] = 0;
    if (tid == 0) s_bad = 0;
    if (blockIdx.x == 0 && tid < static_cast<int>(sizeof(HeadHeader) / 4)) reinterpret_cast<int*>(p.hdr)[tid] = 0;
    __syncthreads();
    bool bad = bad_offsets(p, tid, 256);
#pragma unroll 1
    for (int g = 0; g * 256 < p.T; ++g) {
      const int cl = row_class(p, g * 256 + tid, bad);
      s_cls[g * 256 + tid] = static_cast<uint8_t>(cl);
      const unsigned pos = __ballot_sync(0xffffffffu, cl == 1), neg = __ballot_sync(0xffffffffu, cl == 2);
      if ((tid & 31) == 0) {
        atomicAdd(&s_cnt[g][0], __popc(pos));
        atomicAdd(&s_cnt[g][1], __popc(neg));
      }
    }
    if (bad) s_bad = 1;
    __syncthreads();
    n_pos = n_neg = 0;
#pragma unroll
    for (int g = 0; g < kSmallRows / 256; ++g) {
      n_pos += s_cnt[g][0];
      n_neg += s_cnt[g][1];
    }
    neg0 = (n_pos + kTileM - 1) / kTileM * kTileM;
    if (blockIdx.x == 0 && tid == 0) {
      write_counts(p, n_pos, n_neg);
      if (s_bad != 0) p.hdr->w.status = kErrTargetRange;
    }
    if (s_bad != 0) return;
  } else {
    if (hdr->w.status != 0) return;
    n_pos = hdr->n_pos;
    n_neg = hdr->n_neg;
    neg0 = hdr->neg0;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane % L, grp = lane / L;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + warp;
  const bool piece = 8 * sub < p.DP, real = 8 * sub < p.D;       // this lane's piece of a padded row, and of a row
  if (t >= p.Tc) return;
  // the rows of each class before t: the prefix of its 256 and those before it in them
  int cls = 0;
  int64_t n1 = n_pos, n2 = n_neg;
  if (t < p.T) {
    cls = kSmall ? s_cls[t] : p.cls[t];
    const int b = static_cast<int>(t >> 8), n = static_cast<int>(t & 255);
    int before = 0;                                              // the second class in the upper half
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = lane + 32 * i;
      const int o = k < n ? (kSmall ? s_cls[(b << 8) + k] : p.cls[(static_cast<int64_t>(b) << 8) + k]) : 0;
      before += (o == 1) + ((o == 2) << 16);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    n1 = before & 0xffff;
    n2 = before >> 16;
    if (kSmall) {
      for (int g = 0; g < b; ++g) n1 += s_cnt[g][0], n2 += s_cnt[g][1];
    } else {
      n1 += p.blk[2 * b];
      n2 += p.blk[2 * b + 1];
    }
  }
  if (cls == 0) {
    // the unused rows in order: those between the classes, then those behind both
    const int64_t r = t - n1 - n2, gap = neg0 - n_pos;
    const int64_t c = r < gap ? n_pos + r : neg0 + n_neg + (r - gap);
    if (grp == 0 && piece) reinterpret_cast<uint4*>(p.Hc + c * p.DP)[sub] = make_uint4(0u, 0u, 0u, 0u);
    for (int k = lane; k < p.K; k += 32) {
      p.targets[c * p.K + k] = -1;
      if (p.keys != nullptr) p.keys[c * p.K + k] = -1;
    }
    if (lane == 0) {
      p.orig[c] = -1;
      write_offset(p, c, -1e30f);
      p.lse2[c] = 0.f;
      if (p.m2 != nullptr) p.m2[c] = 0.f;
      if (t < p.T) {
        p.cidx[t] = -1;
        if (p.lse_out != nullptr) p.lse_out[t] = 0.f;
      }
    }
    return;
  }
  const int64_t c = cls == 2 ? neg0 + n2 : n1;
  const int64_t r = t * p.K, rc = c * p.K;
  // the row, and the ids and logits of its slots (slot k = lane + 32 j), all in flight
  const uint4 hraw = real ? __ldg(reinterpret_cast<const uint4*>(p.H + t * p.D) + sub) : make_uint4(0u, 0u, 0u, 0u);
  float q[J], lq[J];
  int id[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int k = lane + 32 * j;
    id[j] = k < p.K ? __ldg(p.ids + r + k) : -1;
    lq[j] = p.kind == kHeadDistill && k < p.K ? __ldg(p.logits + r + k) : 0.f;
  }
  if (grp == 0 && piece) reinterpret_cast<uint4*>(p.Hc + c * p.DP)[sub] = hraw;
  float h[8];
  unpack8(hraw, h);
  // the targets' weights; the largest logit is subtracted before the division by tau, so that
  // finite ones of any size stay finite and only their differences are rounded
  if (p.kind == kHeadDistill) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (id[j] < 0) lq[j] = -INFINITY;
      m = fmaxf(m, lq[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      lq[j] = (lq[j] - m) * p.inv_tau;
      q[j] = expf(lq[j]);                        // an empty slot: e^-inf = 0
      s += q[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float ls = logf(s);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      q[j] /= s;
      lq[j] -= ls;
    }
  } else {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      q[j] = j == 0 && lane == 0 ? 1.f : 0.f;
      lq[j] = 0.f;
    }
  }
  // The row's targets, the slots with q != 0, in ascending order of id; an id's weights
  // are added up in its first slot.  A slot's rank: the live ones that sort before it.
  bool own[J];                                   // a live slot, the first of its id
  {
    float all[J];
    int rank[J], live_n = 0;
    bool again[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      all[j] = 0.f;
      rank[j] = 0;
      again[j] = false;
    }
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const unsigned live = __ballot_sync(0xffffffffu, id[i] >= 0 && q[i] != 0.f);
      live_n += __popc(live);
#pragma unroll 1
      for (unsigned todo = live; todo != 0u; todo &= todo - 1u) {
        const int from = __ffs(todo) - 1;
        const int v = __shfl_sync(0xffffffffu, id[i], from);
        const float w = __shfl_sync(0xffffffffu, q[i], from);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const bool earlier = 32 * i + from < lane + 32 * j;
          if (v == id[j]) {
            all[j] += w;
            again[j] |= earlier;
          }
          rank[j] += v < id[j] || (v == id[j] && earlier);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int k = lane + 32 * j;
      const bool live = id[j] >= 0 && q[j] != 0.f;
      own[j] = live && !again[j];
      if (live) p.targets[rc + rank[j]] = id[j];
      if (k >= live_n && k < p.K) p.targets[rc + k] = -1;
      if (p.keys != nullptr && k < p.K) {
        p.keys[rc + k] = own[j] ? id[j] : -1;
        p.share[rc + k] = own[j] ? all[j] : 0.f;
      }
    }
  }
  // calls what(slots k + u G + grp, their pieces of E) for the slots of group j, kGatherU
  // rows a lane in flight; rows of weight 0 are zeros
  auto walk = [&](int j, int n, auto what) {
    for (int k = 0; k < n; k += G * kGatherU) {
      uint4 e[kGatherU];
#pragma unroll
      for (int u = 0; u < kGatherU; ++u) {
        const int slot = k + u * G + grp, from = min(slot, 31);
        const int v = __shfl_sync(0xffffffffu, id[j], from);
        const float w = __shfl_sync(0xffffffffu, q[j], from);
        const bool load = slot < n && v >= 0 && v < p.V && w != 0.f && real;
        e[u] = load ? __ldg(reinterpret_cast<const uint4*>(p.E + static_cast<int64_t>(v) * p.D) + sub)
                    : make_uint4(0u, 0u, 0u, 0u);
      }
      what(k, e);
    }
  };
  // the logits: lane k keeps x of its slot
  float x[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    x[j] = 0.f;
    const int n = min(32, p.K - 32 * j);
    if (n <= 0) break;
    walk(j, n, [&](int k, const uint4 (&e)[kGatherU]) {
      float z[kGatherU];
#pragma unroll
      for (int u = 0; u < kGatherU; ++u) {
        float row[8];
        unpack8(e[u], row);
        z[u] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) z[u] = fmaf(h[i], row[i], z[u]);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < kGatherU; ++u) z[u] += __shfl_xor_sync(0xffffffffu, z[u], o);
      const int mine = lane - k;                 // its place in this batch
#pragma unroll
      for (int u = 0; u < kGatherU; ++u) {
        const float y = __shfl_sync(0xffffffffu, z[u], (mine & (G - 1)) * L);
        if (mine >= u * G && mine < (u + 1) * G) x[j] = y * p.c2;
      }
    });
  }
  // their maximum, and the sum of 2^(x - maximum) over the ids
  float zref = -3.0e38f, tsum = 0.f;
#pragma unroll
  for (int j = 0; j < J; ++j)
    if (own[j]) zref = fmaxf(zref, x[j]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) zref = fmaxf(zref, __shfl_xor_sync(0xffffffffu, zref, o));
  float y[J];
  double term = 0.0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    y[j] = own[j] ? exp2f(x[j] - zref) : 0.f;
    tsum += y[j];
    if (p.kind == kHeadDistill && id[j] >= 0 && q[j] != 0.f)
      term += static_cast<double>(q[j]) * (static_cast<double>(lq[j]) - (static_cast<double>(x[j]) - zref) * 0.6931471805599453);
    if (p.zt != nullptr && lane + 32 * j < p.K) p.zt[rc + 32 * j + lane] = own[j] ? x[j] : -INFINITY;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tsum += __shfl_xor_sync(0xffffffffu, tsum, o);
    if (p.kind == kHeadDistill) term += __shfl_xor_sync(0xffffffffu, term, o);
  }
  if (p.sparse != nullptr) {
    // sum (q - y / T) e and sum y / T e; the rows come from the caches this time
    float sp[8], sb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sp[i] = sb[i] = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = min(32, p.K - 32 * j);
      if (n <= 0) break;
      y[j] = __fdiv_rn(y[j], tsum);
      const float d = q[j] - y[j];
      walk(j, n, [&](int k, const uint4 (&e)[kGatherU]) {
#pragma unroll
        for (int u = 0; u < kGatherU; ++u) {
          const int from = min(k + u * G + grp, 31);
          const float a = __shfl_sync(0xffffffffu, d, from), b = __shfl_sync(0xffffffffu, y[j], from);
          float row[8];
          unpack8(e[u], row);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sp[i] = fmaf(a, row[i], sp[i]);
            sb[i] = fmaf(b, row[i], sb[i]);
          }
        }
      });
    }
    // the groups' parts, in a fixed order
#pragma unroll
    for (int o = L; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sp[i] += __shfl_xor_sync(0xffffffffu, sp[i], o);
        sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], o);
      }
    }
    if (grp == 0 && piece) {
      store_floats<8>(p.sparse + 2 * c * p.DP + 8 * sub, sp);
      store_floats<8>(p.sparse + (2 * c + 1) * p.DP + 8 * sub, sb);
    }
  }
  if (p.m2 != nullptr && p.lse_in == nullptr) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(h[i], h[i], s);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      const float bound = sqrtf(s) * sqrtf(__uint_as_float(hdr->emax2)) * p.c2;
      const float m = bound * 1.0001f + 0.01f;               // above the rounding of the norms
      p.m2[c] = m;
      if (!(m - zref <= kMaxRefGap)) p.hdr->wide = 1;        // NaN counts as wide
    }
  }
  if (lane == 0) {
    if (p.m2 != nullptr && p.lse_in != nullptr) p.m2[c] = p.lse_in[t] * 1.4426950408889634f;
    p.cidx[t] = static_cast<int>(c);
    p.orig[c] = static_cast<int>(t);
    p.tref[c] = zref;
    p.tsum[c] = tsum;
    if (p.kind == kHeadDistill) {
      p.rowterm[c] = term;
      p.coef[c] = p.weights != nullptr ? p.weights[t] : 1.f;
    }
  }
}

// Sum over the block in a fixed order (contiguous values per thread, then a tree).
__device__ __forceinline__ double head_block_sum(double v, double* red) {
  red[threadIdx.x] = v;
  __syncthreads();
  for (int s = blockDim.x / 2; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  const double r = red[0];
  __syncthreads();
  return r;
}

// A call with a data error has no loss: NaN, so that it does not pass unnoticed where
// the status is not read.
__device__ __forceinline__ void failed_loss(const HeadParams& p) {
  if (p.loss != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.loss = NAN;
}

// ------------------------------------------------------------------ lse
// Several threads per compacted row join the (reference, sum) partials of the row's
// splits and slabs with the sum over its targets (or take the lse of an earlier
// forward), write lse, the exponent offset of the item-owned pass, q - p of the row's
// pairs and its share of the distillation loss, which the last block adds up in
// block order.
//
// kLseLanes threads share a row: 4, or 32 where a row has more than 128 partials (few
// positions, many splits: 14 us with 592 partials and 4 threads).
constexpr int kLseThreads = 128;
constexpr int kLseManySlots = 128;
constexpr float kMaxRowSum = 18446744073709551616.f;   // 2^64: V terms of at most 2^8 stay below 2^39

template <int kLseLanes>
__global__ void __launch_bounds__(kLseThreads) k_head_lse(const HeadParams p) {
  constexpr int kLseRows = kLseThreads / kLseLanes;
  __shared__ double red[kLseThreads];
  __shared__ int last;
  HeadHeader* hdr = p.hdr;
  if (hdr->w.status != 0) {
    failed_loss(p);
    return;
  }
  // consecutive threads take consecutive rows, so that a slot's partials are read together
  const int part_of = static_cast<int>(threadIdx.x) / kLseRows;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kLseRows + threadIdx.x % kLseRows;
  __shared__ float sm[kLseLanes][kLseRows], ss[kLseLanes][kLseRows];
  const int t = c < hdr->n_rows ? p.orig[c] : -1;
  if (p.part != nullptr) {
    // running (reference, sum) over every kLseLanes-th slot, eight loads in flight
    float m = -3.0e38f, sum = 0.f;
    bool bad = false;
    if (t >= 0) {
      for (int s0 = part_of; s0 < p.slots; s0 += 8 * kLseLanes) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int s = s0 + u * kLseLanes;
          v[u] = s < p.slots ? __ldg(p.part + s * p.Tc + c) : make_float2(-3.0e38f, 0.f);
        }
        float mx = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          mx = fmaxf(mx, v[u].x);
          bad |= v[u].x != v[u].x;
        }
        sum *= exp2f(m - mx);
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += v[u].y * exp2f(v[u].x - mx);
        m = mx;
      }
    }
    sm[part_of][threadIdx.x % kLseRows] = bad ? NAN : m;
    ss[part_of][threadIdx.x % kLseRows] = sum;
    __syncthreads();
  }
  __shared__ float s_omp[kLseRows], s_mass[kLseRows], s_ref[kLseRows], s_sum[kLseRows];
  double row_loss = 0.0;
  if (t >= 0 && part_of == 0) {
    const float zref = p.tref[c], tsum = p.tsum[c];
    double l2;
    float omp, mass, ref = 0.f;                  // the probability of the other items, and of the targets
    if (p.part == nullptr) {
      // 1 - p from the lse alone: to half a step of it
      l2 = static_cast<double>(p.lse_in[t]) * 1.4426950408889634;
      mass = static_cast<float>(tsum * exp2(zref - l2));
      omp = static_cast<float>(1.0 - tsum * exp2(zref - l2));
      if (omp < 0.f) omp = 0.f;
    } else {
      float m = sm[0][threadIdx.x], sum = 0.f;
#pragma unroll
      for (int q = 1; q < kLseLanes; ++q) m = fmaxf(m, sm[q][threadIdx.x]);
      bool bad = false;
#pragma unroll
      for (int q = 0; q < kLseLanes; ++q) {
        const float mq = sm[q][threadIdx.x];
        bad |= mq != mq;
        sum += ss[q][threadIdx.x] * exp2f(mq - m);
      }
      bad |= !(sum < kMaxRowSum);                    // a NaN logit (see the tile passes)
      const float top = fmaxf(m, zref);
      const double rest = static_cast<double>(sum * exp2f(m - top)), own = static_cast<double>(tsum * exp2f(zref - top));
      const double all = rest + own;
      l2 = bad ? NAN : static_cast<double>(top) + log2(all);
      omp = bad ? NAN : static_cast<float>(rest / all);
      mass = bad ? NAN : static_cast<float>(own / all);
      ref = m;
    }
    const float l2f = static_cast<float>(l2);
    p.rescale[c] = p.m2 != nullptr ? static_cast<float>(exp2(static_cast<double>(ref) - l2)) : 1.f;
    p.lse2[c] = l2f;
    p.omp[c] = omp;
    s_omp[threadIdx.x] = omp;
    s_mass[threadIdx.x] = mass;
    s_ref[threadIdx.x] = zref;
    s_sum[threadIdx.x] = tsum;
    if (p.lse_out != nullptr) p.lse_out[t] = static_cast<float>(l2 * 0.6931471805599453);
    const double above = (l2 - static_cast<double>(zref)) * 0.6931471805599453;      // lse - the largest target's logit
    if (p.kind == kHeadDistill) {
      const float w = p.weights != nullptr ? p.weights[t] : 1.f;
      write_offset(p, c, (p.weights != nullptr ? log2f(fabsf(w)) : 0.f) - l2f);
      row_loss = static_cast<double>(w) * p.tau * p.tau * (p.rowterm[c] + above);
    } else {
      p.rowterm[c] = -above;
    }
  }
  if (p.share != nullptr) {
    __syncthreads();
    if (t >= 0) {
      const int i = static_cast<int>(threadIdx.x) % kLseRows;
      const float omp = s_omp[i], mass = s_mass[i], ref = s_ref[i], sum = s_sum[i];
#pragma unroll 4
      for (int k = part_of; k < p.K; k += kLseLanes) {
        const int64_t e = c * p.K + k;
        const float y = __fdiv_rn(exp2f(p.zt[e] - ref), sum);
        p.share[e] = omp < mass ? fmaf(omp, y, p.share[e] - y) : fmaf(-mass, y, p.share[e]);
      }
    }
  }
  if (p.kind != kHeadDistill || p.loss == nullptr) return;
  const double b = head_block_sum(row_loss, red);
  if (threadIdx.x == 0) {
    p.loss_part[blockIdx.x] = b;
    __threadfence();
    last = atomicAdd(&hdr->lse_ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double a = 0.0;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kLseThreads) a += __ldcg(p.loss_part + i);
  const double all = head_block_sum(a, red);
  if (threadIdx.x == 0) *p.loss = hdr->w.loss_scale * all;
}

// ------------------------------------------------------------------ pairs
// One block per preference pair: the log-probability of both sequences (fixed
// order), x = beta ((Lc - Lr) - (Rc - Rr)), the loss softplus(-x), and the factor
// sigmoid(-x) of the pair's rows (positive for the chosen sequence).
constexpr int kPairThreads = 128;

__global__ void __launch_bounds__(kPairThreads) k_head_pairs(const HeadParams p) {
  __shared__ double red[kPairThreads];
  __shared__ int last;
  HeadHeader* hdr = p.hdr;
  if (hdr->w.status != 0) {
    failed_loss(p);
    return;
  }
  const int pr = blockIdx.x;
  double L[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int a = p.offsets[2 * pr + q], b = p.offsets[2 * pr + q + 1];
    double s = 0.0;
    for (int t = a + static_cast<int>(threadIdx.x); t < b; t += kPairThreads) {
      const int c = p.cidx[t];
      if (c >= 0) s += p.rowterm[c];
    }
    L[q] = head_block_sum(s, red);
  }
  double x = L[0] - L[1];
  if (p.ref != nullptr) x -= static_cast<double>(p.ref[2 * pr]) - static_cast<double>(p.ref[2 * pr + 1]);
  x *= p.beta;
  const double ex = exp(-fabs(x));
  const double sig = (x >= 0.0 ? ex : 1.0) / (1.0 + ex);           // sigmoid(-x)
  const float f = static_cast<float>(sig);
  const float lf = log2f(f);
  for (int q = 0; q < 2; ++q) {
    const int a = p.offsets[2 * pr + q], b = p.offsets[2 * pr + q + 1];
    for (int t = a + static_cast<int>(threadIdx.x); t < b; t += kPairThreads) {
      const int c = p.cidx[t];
      if (c < 0) continue;
      p.coef[c] = q == 0 ? f : -f;
      write_offset(p, c, lf - p.lse2[c]);
    }
  }
  if (threadIdx.x == 0) {
    if (p.logp_out != nullptr) {
      p.logp_out[2 * pr] = static_cast<float>(L[0]);
      p.logp_out[2 * pr + 1] = static_cast<float>(L[1]);
    }
    p.loss_part[pr] = fmax(-x, 0.0) + log1p(ex) + (x != x ? x : 0.0);
    __threadfence();
    last = atomicAdd(&hdr->pairs_ticket, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!last || p.loss == nullptr) return;
  __threadfence();
  double a = 0.0;
  for (int i = threadIdx.x; i < p.P; i += kPairThreads) a += __ldcg(p.loss_part + i);
  const double all = head_block_sum(a, red);
  if (threadIdx.x == 0) *p.loss = hdr->w.loss_scale * all;
}

// ------------------------------------------------------------------ dh
// dH[t] = g s w_t (sum over splits of the dense part - sum_k (q_k - p_k) e_k), four
// columns per thread; rows that do not count are zero.
struct HeadDhParams {
  int T, D, DP, S;
  int64_t Tc;
  const int* cidx;
  const float* coef;      // [Tc]
  const float* part;      // [S, Tc, DP]
  const float* sparse;    // [Tc, 2, DP]
  const float* omp;       // [Tc] factor of the second sparse row
  const float* rescale;   // [Tc] factor of the dense part
  void* dH;
  int bf16, accumulate;
  const HeadHeader* hdr;
};

// kLanes threads share four columns and add every kLanes-th split, their sums are
// then added in order: 1, or 8 where the positions alone leave SMs idle (131 splits of
// 9 rows took 30 us with one thread each).
template <int kLanes>
__global__ void __launch_bounds__(256, 4) k_head_dh(const HeadDhParams p) {
  if (p.hdr->w.status != 0) return;
  constexpr int kCols = 256 / kLanes;             // groups of four columns per block
  __shared__ float4 s_part[kLanes > 1 ? kLanes : 1][kLanes > 1 ? kCols : 1];
  const int part_of = kLanes > 1 ? static_cast<int>(threadIdx.x) / kCols : 0;
  const int per_row = p.D / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x % kCols;
  const int64_t t = i / per_row;
  const int col = static_cast<int>(i - t * per_row) * 4;
  const int c = t < p.T ? p.cidx[t] : -1;
  float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c >= 0) {
    const float* src = p.part + static_cast<int64_t>(c) * p.DP + col;
    const int64_t stride = p.Tc * p.DP;
    for (int s0 = part_of; s0 < p.S; s0 += 8 * kLanes) {      // eight loads in flight, added in split order
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = s0 + u * kLanes;
        v[u] = s < p.S ? __ldg(reinterpret_cast<const float4*>(src + s * stride)) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        a.x += v[u].x;
        a.y += v[u].y;
        a.z += v[u].z;
        a.w += v[u].w;
      }
    }
  }
  if (kLanes > 1) {
    s_part[part_of][threadIdx.x % kCols] = a;
    __syncthreads();
    if (part_of != 0) return;
#pragma unroll
    for (int q = 1; q < kLanes; ++q) {
      const float4 v = s_part[q][threadIdx.x % kCols];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
  }
  if (t >= p.T) return;
  if (c >= 0) {
    const float* sp = p.sparse + static_cast<int64_t>(c) * 2 * p.DP + col;
    float4 q = __ldg(reinterpret_cast<const float4*>(sp));
    const float4 b = __ldg(reinterpret_cast<const float4*>(sp + p.DP));
    const float o = p.omp[c];
    q = make_float4(fmaf(o, b.x, q.x), fmaf(o, b.y, q.y), fmaf(o, b.z, q.z), fmaf(o, b.w, q.w));
    const float f = p.hdr->w.grad_scale * p.coef[c];
    const float r = p.rescale[c];
    g = make_float4(__fmul_rn(fmaf(a.x, r, -q.x), f), __fmul_rn(fmaf(a.y, r, -q.y), f),
                    __fmul_rn(fmaf(a.z, r, -q.z), f), __fmul_rn(fmaf(a.w, r, -q.w), f));
  }
  const int64_t o = t * p.D + col;
  if (p.bf16) {
    uint2* dst = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.dH) + o);
    if (p.accumulate) {
      const uint2 old = *dst;
      g.x = __fadd_rn(g.x, __uint_as_float(old.x << 16));
      g.y = __fadd_rn(g.y, __uint_as_float(old.x & 0xFFFF0000u));
      g.z = __fadd_rn(g.z, __uint_as_float(old.y << 16));
      g.w = __fadd_rn(g.w, __uint_as_float(old.y & 0xFFFF0000u));
    }
    *dst = make_uint2(pack_bf16x2(g.x, g.y), pack_bf16x2(g.z, g.w));
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.dH) + o);
    if (p.accumulate) {
      const float4 old = *dst;
      g.x = __fadd_rn(g.x, old.x);
      g.y = __fadd_rn(g.y, old.y);
      g.z = __fadd_rn(g.z, old.z);
      g.w = __fadd_rn(g.w, old.w);
    }
    *dst = g;
  }
}

}  // namespace cutbce

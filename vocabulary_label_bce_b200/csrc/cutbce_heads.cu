// Host side of the item-table operators: row lookup and its gradient, and the
// softmax losses over the whole table (distillation, preference).  Argument
// checks, workspace layouts and launch sequences; no device memory is allocated.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "cutbce.h"
#include "common.cuh"
#include "host_util.cuh"
#include "id_sort.cuh"
#include "embed.cuh"
#include "softmax_head.cuh"
#include "softmax_engine.cuh"

namespace {
using namespace cutbce;

#define CUTBCE_CK(x)                                \
  do {                                              \
    if ((x) != cudaSuccess) return CUTBCE_ERR_CUDA; \
  } while (0)

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Offsets of a workspace, 256-byte aligned pieces in order.
struct Layout {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total = align256(total + bytes);
    return at;
  }
};

cutbce_status check_device() {
  DeviceFacts dev;
  const cutbce_status s = device_facts(dev);
  if (s != CUTBCE_OK) return s;
  return dev.major == 10 && dev.minor == 0 ? CUTBCE_OK : CUTBCE_ERR_UNSUPPORTED;
}

// Sets a kernel's dynamic shared memory limit once per device (the attribute belongs
// to the current device).
template <int kTag, typename Kernel>
cudaError_t set_smem_once(Kernel kern, size_t bytes) {
  static std::atomic<uint64_t> configured{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const uint64_t bit = uint64_t(1) << dev;
  if ((configured.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) configured.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

// ---------------------------------------------------------------- sort and segment sums
constexpr int64_t kMaxSortEntries = int64_t(1) << 28;

// Buffers of the sort and of the sums over N entries.
struct SortBuffers {
  SortPlan sp;
  bool cluster;
  size_t o_hist, o_total, o_pairs[2], o_part;
};

void plan_sort(int64_t N, int64_t V, int64_t D, SortBuffers& b, Layout& l) {
  make_sort_plan(N, V, b.sp);
  b.cluster = N <= kClusterEntries;
  if (b.cluster) b.sp.hist_bytes = 0;
  b.o_hist = l.take(b.sp.hist_bytes);                 // right after the header: one memset clears both
  b.o_total = l.take(b.cluster ? 0 : sizeof(int) * (size_t(1) << b.sp.bits));
  for (int i = 0; i < 2; ++i) b.o_pairs[i] = l.take(8 * static_cast<size_t>(N));
  b.o_part = l.take(4 * 2 * static_cast<size_t>(ceil_div(N, kMinChunk)) * D);   // the most blocks of any geometry
}

// Sorts the entries by id into *pairs.  stop: see k_sort_scatter.
template <int IPT>
cutbce_status run_sort_ipt(const SortBuffers& b, const int32_t* ids, int V, void* ws, int* status, const int* stop,
                           FillJob fill, cudaStream_t st, const int2** pairs) {
  const SortPlan& sp = b.sp;
  const size_t pass_hist = static_cast<size_t>(sp.nblk) << sp.bits;
  int* hist = at<int>(ws, b.o_hist);
  int* total = at<int>(ws, b.o_total);
  // the passes take equal shares of the fill: they last longer than the counting of the keys
  const int64_t share = ceil_div(fill.n, sp.passes);
  k_sort_keys<IPT><<<sp.nblk, kSortThreads, 0, st>>>(ids, sp.N, V, sp.bits, hist, status);
  const int2* in = nullptr;
  for (int p = 0; p < sp.passes; ++p) {
    int* h = hist + p * pass_hist;
    int* next = p + 1 < sp.passes ? h + pass_hist : nullptr;
    if (sp.scan) k_sort_scan<<<static_cast<unsigned>(ceil_div(1 << sp.bits, 32)), 32 * kScanWarps, 0, st>>>(h, total, 1 << sp.bits, sp.nblk);
    int2* out = at<int2>(ws, b.o_pairs[p & 1]);
    const FillJob part{fill.dst + p * share, std::max<int64_t>(0, std::min(share, fill.n - p * share)), fill.value};
    const int fill_blocks = static_cast<int>(std::min<int64_t>(ceil_div(part.n, 4 * kSortThreads), 8 * 148));
    k_sort_scatter<IPT><<<sp.nblk + fill_blocks, kSortThreads, 0, st>>>(p == 0 ? ids : nullptr, in, sp.N, V, p * sp.bits, sp.bits, sp.nblk,
                                                          h, sp.scan ? total : nullptr, out, next, stop, part);
    in = out;
  }
  *pairs = in;
  return cudaGetLastError() == cudaSuccess ? CUTBCE_OK : CUTBCE_ERR_CUDA;
}

// clear_status: the status word is not yet cleared (one-kernel sort only: the others
// follow a memset of the header and the histograms).
cutbce_status run_sort(const SortBuffers& b, const int32_t* ids, int V, void* ws, int* status, const int* stop,
                       bool clear_status, FillJob fill, cudaStream_t st, const int2** pairs) {
  LaunchScope ls(CUTBCE_KERNEL_ID_SORT, st);
  if (b.cluster) {
    const size_t smem = size_t(64) << b.sp.bits;           // a 16-bit counter per warp and digit
    const cudaError_t e = set_smem_once<0>(k_sort_cluster, size_t(64) << kSortMaxBits);
    if (e != cudaSuccess) return CUTBCE_ERR_CUDA;
    const int fill_clusters = static_cast<int>(std::min<int64_t>(ceil_div(fill.n, 2 * kClusterCtas * kClusterThreads), 36));
    k_sort_cluster<<<kClusterCtas * (1 + fill_clusters), kClusterThreads, smem, st>>>(ids, static_cast<int>(b.sp.N), V, b.sp.bits, b.sp.passes,
                                                                at<int2>(ws, b.o_pairs[0]), at<int2>(ws, b.o_pairs[1]),
                                                                status, clear_status ? 1 : 0, fill);
    *pairs = at<int2>(ws, b.o_pairs[(b.sp.passes - 1) & 1]);
    return cudaGetLastError() == cudaSuccess ? CUTBCE_OK : CUTBCE_ERR_CUDA;
  }
  if (b.sp.ipt == 4) return run_sort_ipt<4>(b, ids, V, ws, status, stop, fill, st, pairs);
  if (b.sp.ipt == 8) return run_sort_ipt<8>(b, ids, V, ws, status, stop, fill, st, pairs);
  return run_sort_ipt<16>(b, ids, V, ws, status, stop, fill, st, pairs);
}

template <int VEC, typename TIn, typename TOut>
cutbce_status run_sums_t(const SegmentParams& p, cudaStream_t st) {
  const SumGeometry g = sum_geometry(p.N, p.D, VEC);
  LaunchScope ls(CUTBCE_KERNEL_SEGMENT_SUM, st);
  k_segment_sum<VEC, TIn, TOut><<<dim3(static_cast<unsigned>(g.chunks), static_cast<unsigned>(g.slices)),
                                  g.lanes * g.subs, 0, st>>>(p, g.lanes, g.subs, g.rounds);
  constexpr int kJoinVec = VEC == 8 ? 4 : VEC;
  if (g.chunks > 1)
    k_segment_join<kJoinVec, TOut><<<dim3(static_cast<unsigned>(g.chunks - 1), static_cast<unsigned>(ceil_div(p.D, 32 * kJoinVec))),
                                     256, 0, st>>>(p, g.chunk);
  return cudaGetLastError() == cudaSuccess ? CUTBCE_OK : CUTBCE_ERR_CUDA;
}

template <typename TIn, typename TOut>
cutbce_status run_sums_vec(const SegmentParams& p, cudaStream_t st) {
  constexpr int VEC = 16 / sizeof(TIn);
  if (p.D % VEC == 0 && aligned(p.src, 16) && aligned(p.out, 16)) return run_sums_t<VEC, TIn, TOut>(p, st);
  return run_sums_t<1, TIn, TOut>(p, st);
}

cutbce_status run_sums(const SegmentParams& p, bool in_bf16, cudaStream_t st) {
  if (p.first != nullptr) return run_sums_vec<__nv_bfloat16, float>(p, st);
  if (in_bf16) {
    return p.out_bf16 ? run_sums_vec<__nv_bfloat16, __nv_bfloat16>(p, st)
                      : run_sums_vec<__nv_bfloat16, float>(p, st);
  }
  return p.out_bf16 ? run_sums_vec<float, __nv_bfloat16>(p, st) : run_sums_vec<float, float>(p, st);
}

// ---------------------------------------------------------------- row lookup
cutbce_status check_embed(int64_t N, int64_t V, int64_t D, int32_t dtype) {
  if (N <= 0 || V <= 0 || D <= 0) return CUTBCE_ERR_INVALID_ARG;
  if (dtype != CUTBCE_BF16 && dtype != CUTBCE_F32) return CUTBCE_ERR_UNSUPPORTED;
  if (V >= (int64_t(1) << 31) - 1 || D > kMaxEmbedDim || N >= kMaxSortEntries) return CUTBCE_ERR_UNSUPPORTED;
  return CUTBCE_OK;
}

struct EmbedPlan {
  size_t o_hdr;
  SortBuffers sort;
  size_t total;
};

void plan_embed(int64_t N, int64_t V, int64_t D, EmbedPlan& pl) {
  Layout l;
  pl.o_hdr = l.take(256);
  plan_sort(N, V, D, pl.sort, l);
  pl.total = l.total;
}

template <int VEC, typename T>
cutbce_status launch_embed(const void* E, int64_t V, const int32_t* ids, int64_t N, int64_t D, float scale, void* X,
                           int32_t* status, cudaStream_t st) {
  const int64_t blocks = ceil_div(N * (D / VEC), 256);
  if (blocks >= (int64_t(1) << 31)) return CUTBCE_ERR_UNSUPPORTED;
  LaunchScope ls(CUTBCE_KERNEL_EMBED, st);
  k_embed<VEC, T><<<static_cast<unsigned>(blocks), 256, 0, st>>>(static_cast<const T*>(E), V, ids, N,
                                                                 static_cast<int>(D), scale, static_cast<T*>(X), status);
  return cudaGetLastError() == cudaSuccess ? CUTBCE_OK : CUTBCE_ERR_CUDA;
}

// ---------------------------------------------------------------- softmax heads
struct HeadProblem {
  int kind;
  int64_t T, V, D, K, P;
  int32_t dtype, reduction;
  const void *H, *E;
  const int32_t* ids;
  const float* logits;
  const int32_t* offsets;
  const float* ref;
  const uint8_t* mask;
  const float* weights;
  float tau, beta;
};

HeadProblem head_problem(const cutbce_distill_problem* p) {
  return HeadProblem{kHeadDistill, p->T, p->V, p->D, p->K, 0, p->dtype, p->reduction, p->H, p->E, p->ids, p->logits,
                     nullptr, nullptr, p->mask, p->weights, p->temperature, 1.f};
}
HeadProblem head_problem(const cutbce_preference_problem* p) {
  return HeadProblem{kHeadPreference, p->T, p->V, p->D, 1, p->P, p->dtype, p->reduction, p->H, p->E, p->ids, nullptr,
                     p->offsets, p->ref_logp, p->mask, nullptr, 1.f, p->beta};
}

cutbce_status check_head(const HeadProblem& p, bool need_data) {
  if (p.T <= 0 || p.V <= 0 || p.D <= 0 || p.K <= 0) return CUTBCE_ERR_INVALID_ARG;
  if (p.dtype != CUTBCE_BF16) return CUTBCE_ERR_UNSUPPORTED;
  if (p.reduction != CUTBCE_MEAN_VALID_POSITIONS && p.reduction != CUTBCE_SUM) return CUTBCE_ERR_INVALID_ARG;
  if (p.K > kMaxK || p.D > kMaxDim || p.D % 8 != 0) return CUTBCE_ERR_UNSUPPORTED;
  if (p.V >= (int64_t(1) << 31) - 1 || p.T >= (int64_t(1) << 24) - 255 || p.T * p.K >= kMaxSortEntries)
    return CUTBCE_ERR_UNSUPPORTED;
  if (p.kind == kHeadDistill) {
    const float c = kLog2eF / p.tau;
    if (!(p.tau > 0.f) || !std::isfinite(c) || !std::isfinite(p.tau * p.tau)) return CUTBCE_ERR_INVALID_ARG;
  } else {
    if (p.P <= 0 || !std::isfinite(p.beta)) return CUTBCE_ERR_INVALID_ARG;
    if (p.P >= (int64_t(1) << 30)) return CUTBCE_ERR_UNSUPPORTED;
  }
  if (need_data) {
    if (p.H == nullptr || p.E == nullptr || p.ids == nullptr) return CUTBCE_ERR_INVALID_ARG;
    if (p.kind == kHeadDistill ? p.logits == nullptr : p.offsets == nullptr) return CUTBCE_ERR_INVALID_ARG;
    if (!aligned(p.H, 16) || !aligned(p.E, 16) || !aligned(p.ids, 4) || !aligned(p.logits, 4) ||
        !aligned(p.offsets, 4) || !aligned(p.ref, 4) || !aligned(p.weights, 4))
      return CUTBCE_ERR_INVALID_ARG;
  }
  return CUTBCE_OK;
}

constexpr int kMaxHeadSplits = 148;
constexpr int kHeadSlots = 4;                  // partials per split: column slabs x epilogue groups

struct HeadPlan {
  int DP, BN, S, tps, n_vtiles, n_blk;
  int BN_lse, n_vtiles_lse, S_lse, tps_lse;   // the log-sum-exp pass's tiles and splits
  bool fused;                    // the dH pass takes the row sums: no log-sum-exp pass of its own
  bool rows_first;               // the dH pass runs ahead of the join of the row sums (fused, or given the lse)
  int64_t Tc;
  size_t o_hdr, o_blk, o_cls, o_cidx, o_orig, o_coef, o_off16, o_b2, o_lse2, o_term, o_hc, o_lpart, o_part, o_wide, o_m2, o_rescale, o_sparse, o_dhpart,
      o_targets, o_tref, o_tsum, o_omp, o_keys, o_share, o_zt, o_usum, o_first, o_columns, total;
  SortBuffers sort;
  size_t clear_bytes;            // header and histograms
};

// A call that needs both the log-sum-exps and dH can take the row sums in the dH
// pass, with a bound as the exponentials' reference (see the gather): it saves the
// log-sum-exp pass and costs a read of E's norms.
// Measured for the whole gradient call, V = 20,000, D = 64, K = 8, with / without: 60.0 / 60.3
// us at T V = 2.6e6 logits, 72.2 / 69.9 at 1.0e7, 85.4 / 87.9 at 2.0e7, 130 / 152 at 6.4e7.
constexpr int64_t kFusedLogits = 8000000;

// Vocabulary splits of a pass that owns position tiles (nT of them) and streams
// `tiles` item tiles: the count with the least estimated time, in units of a streamed
// tile.  A work item costs its tiles and about kItemColumns streamed rows more (stationary
// tile, accumulator, pipeline fill); the persistent grid runs ceil(items / 148) of them one
// after the other; a split of dH costs `split_cost` to add up.  Masked positions leave
// fewer position tiles than the host knows, so the estimate is taken at three counts.
// The splits depend on sizes alone (148 is a constant, not the device's SM count).
// At T = 4,900, V = 100,000: 15 splits, 4 rounds of 56, where "16 items an SM" took 61
// splits, 17 rounds of 16.
constexpr double kItemColumns = 3.0 * 128;

int choose_splits(int64_t nT, int64_t tiles, int BN, double split_cost) {
  const double item_tiles = kItemColumns / BN;
  int best = 1;
  double best_cost = 1e300;
  for (int64_t want = 1; want <= std::min<int64_t>(kMaxHeadSplits, tiles); ++want) {
    const int64_t tps = ceil_div(tiles, want), S = ceil_div(tiles, tps);
    if (S != want) continue;                       // the same cut as a smaller count
    double cost = split_cost * static_cast<double>(S);
    for (const int64_t n : {nT, nT, ceil_div(9 * nT, 10), ceil_div(8 * nT, 10)})
      cost += 0.25 * static_cast<double>(ceil_div(S * n, 148)) * (static_cast<double>(tps) + item_tiles);
    if (cost < best_cost) {
      best_cost = cost;
      best = static_cast<int>(S);
    }
  }
  return best;
}

void plan_head(const HeadProblem& p, bool dH, bool dE, bool lse_pass, HeadPlan& pl) {
  pl.DP = static_cast<int>(round_up(p.D, 64));
  pl.BN = pl.DP > 128 ? 64 : 128;
  pl.BN_lse = pl.DP == 64 ? SoftmaxCfg<64, kPassLse>::BN : pl.BN;
  pl.n_vtiles = static_cast<int>(ceil_div(p.V, pl.BN));
  pl.n_blk = static_cast<int>(ceil_div(p.T, 256));
  pl.fused = lse_pass && dH && p.T * p.V >= kFusedLogits;
  pl.rows_first = dH && (pl.fused || !lse_pass);
  pl.Tc = round_up(p.T, kTileM) + kTileM;
  const int64_t nT = ceil_div(p.T, kTileM);
  // dH partials are read at about 5 MB a microsecond, a streamed tile takes about 0.6
  const double split_cost = 4.0 * static_cast<double>(pl.Tc) * pl.DP / 5e6 / 0.6;
  pl.S = choose_splits(nT, pl.n_vtiles, pl.BN, split_cost);
  pl.tps = static_cast<int>(ceil_div(pl.n_vtiles, pl.S));
  pl.n_vtiles_lse = static_cast<int>(ceil_div(p.V, pl.BN_lse));
  pl.S_lse = choose_splits(nT, pl.n_vtiles_lse, pl.BN_lse, 0.1);
  pl.tps_lse = static_cast<int>(ceil_div(pl.n_vtiles_lse, pl.S_lse));
  const size_t T = static_cast<size_t>(p.T), Tc = static_cast<size_t>(pl.Tc), TK = Tc * p.K;
  Layout l;
  pl.o_hdr = l.take(256);
  pl.sort = SortBuffers{};
  if (dE) plan_sort(pl.Tc * p.K, p.V, p.D, pl.sort, l);
  pl.clear_bytes = dE ? pl.sort.o_hist + pl.sort.sp.hist_bytes : 256;
  pl.o_blk = l.take(8 * static_cast<size_t>(pl.n_blk));
  pl.o_cls = l.take(T);
  pl.o_cidx = l.take(4 * T);
  pl.o_orig = l.take(4 * Tc);
  pl.o_coef = l.take(4 * Tc);
  pl.o_off16 = dE && pl.DP <= 128 ? l.take(32 * Tc) : 0;
  pl.o_b2 = dE && pl.DP > 128 ? l.take(4 * Tc) : 0;
  pl.o_lse2 = l.take(4 * Tc);
  pl.o_term = l.take(8 * Tc);
  pl.o_hc = l.take(2 * Tc * pl.DP);
  pl.o_lpart = l.take(8 * std::max<size_t>(static_cast<size_t>(p.P), Tc * 32 / kLseThreads));
  pl.o_part = lse_pass || dH ? l.take(8 * static_cast<size_t>(pl.rows_first ? pl.S : pl.S_lse) * kHeadSlots * Tc) : 0;
  pl.o_wide = pl.fused ? l.take(8 * static_cast<size_t>(pl.S_lse) * kHeadSlots * Tc) : 0;
  pl.o_m2 = pl.rows_first ? l.take(4 * Tc) : 0;
  pl.o_rescale = l.take(4 * Tc);
  pl.o_targets = l.take(4 * TK);
  pl.o_tref = l.take(4 * Tc);
  pl.o_tsum = l.take(4 * Tc);
  pl.o_omp = l.take(4 * Tc);
  pl.o_sparse = dH ? l.take(2 * 4 * Tc * pl.DP) : 0;
  pl.o_dhpart = dH ? l.take(4 * static_cast<size_t>(pl.S) * Tc * pl.DP) : 0;
  pl.o_keys = dE ? l.take(4 * TK) : 0;
  pl.o_share = dE ? l.take(4 * TK) : 0;
  pl.o_zt = dE ? l.take(4 * TK) : 0;
  pl.o_columns = dE ? l.take(4 * TK) : 0;
  pl.o_usum = dE ? l.take(4 * TK * p.D) : 0;
  pl.o_first = dE ? l.take(16 * static_cast<size_t>(ceil_div(p.V, 4))) : 0;
  pl.total = l.total;
}

template <int DP, int kPass>
cudaError_t launch_softmax(int grid, const CUtensorMap& s, const CUtensorMap& x, const CUtensorMap& o,
                           const SoftmaxParams& sp, cudaStream_t st) {
  auto kern = k_softmax<DP, kPass>;
  constexpr uint32_t smem = SoftmaxCfg<DP, kPass>::SMEM_BYTES;
  const cudaError_t e = set_smem_once<DP + kPass>(kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, SoftmaxCfg<DP, kPass>::THREADS, smem, st>>>(s, x, o, sp);
  return cudaGetLastError();
}

template <int kPass>
cudaError_t launch_softmax_dp(int DP, int grid, const CUtensorMap& s, const CUtensorMap& x, const CUtensorMap& o,
                              const SoftmaxParams& sp, cudaStream_t st) {
  switch (DP) {
    case 64: return launch_softmax<64, kPass>(grid, s, x, o, sp, st);
    case 128: return launch_softmax<128, kPass>(grid, s, x, o, sp, st);
    case 192: return launch_softmax<192, kPass>(grid, s, x, o, sp, st);
    case 256: return launch_softmax<256, kPass>(grid, s, x, o, sp, st);
    default: return cudaErrorInvalidValue;
  }
}

template <int L, bool kSmall>
void launch_gather_width(unsigned grid, const HeadParams& hp, cudaStream_t st) {
  if (hp.K <= 32) k_head_gather<L, 1, kSmall><<<grid, 256, 0, st>>>(hp);
  else if (hp.K <= 64) k_head_gather<L, 2, kSmall><<<grid, 256, 0, st>>>(hp);
  else k_head_gather<L, 4, kSmall><<<grid, 256, 0, st>>>(hp);
}

template <bool kSmall>
void launch_gather(int DP, unsigned grid, const HeadParams& hp, cudaStream_t st) {
  if (DP == 64) launch_gather_width<8, kSmall>(grid, hp, st);
  else if (DP == 128) launch_gather_width<16, kSmall>(grid, hp, st);
  else launch_gather_width<32, kSmall>(grid, hp, st);
}

struct HeadOutputs {
  double* loss = nullptr;
  float* lse = nullptr;
  float* logp = nullptr;
  void* dH = nullptr;
  void* dE = nullptr;
  int grad_dtype = CUTBCE_GRAD_F32, accumulate = 0;
};

cutbce_status check_grad_options(const cutbce_grad_options* o, HeadOutputs& out) {
  if (o == nullptr) return CUTBCE_OK;
  if (o->grad_dtype != CUTBCE_GRAD_F32 && o->grad_dtype != CUTBCE_GRAD_BF16) return CUTBCE_ERR_UNSUPPORTED;
  if (o->accumulate < 0 || o->accumulate > (CUTBCE_ACCUMULATE_DH | CUTBCE_ACCUMULATE_DE)) return CUTBCE_ERR_INVALID_ARG;
  out.grad_dtype = o->grad_dtype;
  out.accumulate = o->accumulate;
  return CUTBCE_OK;
}

// lse_in: the log-sum-exps of an earlier forward on the same inputs, or null (then
// they are computed first).
cutbce_status run_head(const HeadProblem& p, const float* lse_in, const float* grad_loss, const HeadOutputs& out,
                       void* ws, size_t ws_bytes, cudaStream_t st) {
  cutbce_status s = check_head(p, true);
  if (s != CUTBCE_OK) return s;
  const bool dH = out.dH != nullptr, dE = out.dE != nullptr;
  if (ws == nullptr || !aligned(ws, 256) || !aligned(out.dH, 16) || !aligned(out.dE, 16) || !aligned(out.loss, 8) ||
      !aligned(out.lse, 4) || !aligned(out.logp, 4) || !aligned(lse_in, 4) || !aligned(grad_loss, 4))
    return CUTBCE_ERR_INVALID_ARG;
  HeadPlan pl;
  plan_head(p, dH, dE, lse_in == nullptr, pl);
  if (ws_bytes < pl.total) return CUTBCE_ERR_WORKSPACE;
  DeviceFacts dev;
  if ((s = device_facts(dev)) != CUTBCE_OK) return s;
  if (!(dev.major == 10 && dev.minor == 0)) return CUTBCE_ERR_UNSUPPORTED;

  HeadParams hp{};
  hp.kind = p.kind;
  hp.T = static_cast<int>(p.T);
  hp.V = static_cast<int>(p.V);
  hp.D = static_cast<int>(p.D);
  hp.DP = pl.DP;
  hp.K = static_cast<int>(p.K);
  hp.P = static_cast<int>(p.P);
  hp.H = static_cast<const __nv_bfloat16*>(p.H);
  hp.E = static_cast<const __nv_bfloat16*>(p.E);
  hp.ids = p.ids;
  hp.logits = p.logits;
  hp.offsets = p.offsets;
  hp.ref = p.ref;
  hp.mask = p.mask;
  hp.weights = p.weights;
  hp.tau = p.tau;
  hp.inv_tau = 1.f / p.tau;
  hp.beta = p.beta;
  hp.reduction = p.reduction;
  hp.grad_loss = grad_loss;
  hp.hdr = at<HeadHeader>(ws, pl.o_hdr);
  hp.cls = at<uint8_t>(ws, pl.o_cls);
  hp.blk = at<int>(ws, pl.o_blk);
  hp.n_blk = pl.n_blk;
  hp.cidx = at<int>(ws, pl.o_cidx);
  hp.orig = at<int>(ws, pl.o_orig);
  hp.Hc = at<__nv_bfloat16>(ws, pl.o_hc);
  hp.rowterm = at<double>(ws, pl.o_term);
  hp.sparse = dH ? at<float>(ws, pl.o_sparse) : nullptr;
  hp.keys = dE ? at<int>(ws, pl.o_keys) : nullptr;
  hp.share = dE ? at<float>(ws, pl.o_share) : nullptr;
  hp.zt = dE ? at<float>(ws, pl.o_zt) : nullptr;
  hp.targets = at<int>(ws, pl.o_targets);
  hp.tref = at<float>(ws, pl.o_tref);
  hp.tsum = at<float>(ws, pl.o_tsum);
  hp.omp = at<float>(ws, pl.o_omp);
  hp.coef = at<float>(ws, pl.o_coef);
  hp.off16 = dE && pl.DP <= 128 ? at<__nv_bfloat16>(ws, pl.o_off16) : nullptr;
  hp.b2 = dE && pl.DP > 128 ? at<float>(ws, pl.o_b2) : nullptr;
  hp.lse2 = at<float>(ws, pl.o_lse2);
  hp.lse_in = lse_in;
  hp.c2 = kLog2eF / p.tau;
  hp.m2 = pl.rows_first ? at<float>(ws, pl.o_m2) : nullptr;
  hp.rescale = at<float>(ws, pl.o_rescale);
  hp.part = lse_in == nullptr || dH ? at<float2>(ws, pl.o_part) : nullptr;
  hp.slots = kHeadSlots * (pl.rows_first ? pl.S : pl.S_lse);
  hp.Tc = pl.Tc;
  hp.loss_part = at<double>(ws, pl.o_lpart);
  hp.loss = out.loss;
  hp.lse_out = out.lse;
  hp.logp_out = out.logp;
  int* status = &hp.hdr->w.status;

  const bool small = p.T <= kSmallRows && p.T * p.K <= kSmallSlots && p.P <= kSmallRows && pl.clear_bytes <= 256 && !pl.fused;
  if (!small) CUTBCE_CK(cudaMemsetAsync(hp.hdr, 0, pl.clear_bytes, st));
  {
    LaunchScope ls(CUTBCE_KERNEL_HEAD_PREP, st);
    const unsigned grid = static_cast<unsigned>(pl.Tc / 8);
    if (!small) {
      const int64_t norm_blocks = pl.fused ? std::min<int64_t>(ceil_div(p.V, 128), 8 * 148) : 0;
      k_head_rows<<<static_cast<unsigned>(pl.n_blk + norm_blocks), 256, 0, st>>>(hp);
    }
    if (small) launch_gather<true>(pl.DP, grid, hp, st);
    else launch_gather<false>(pl.DP, grid, hp, st);
    CUTBCE_CK(cudaGetLastError());
  }
  SoftmaxParams sp{};
  sp.V = hp.V;
  sp.D = hp.D;
  sp.Tc = pl.Tc;
  sp.hdr = hp.hdr;
  sp.c2 = kLog2eF / p.tau;
  sp.nsplit = pl.S;
  sp.tiles_per_split = pl.tps;
  sp.n_item_tiles_bn = pl.n_vtiles;
  sp.timeout_ns = kDefaultTimeoutNs;
  sp.targets = hp.targets;
  sp.K = hp.K;
  CUtensorMap m_rows_s;                                      // the positions as stationary operand
  if (!make_map(&m_rows_s, hp.Hc, pl.DP, pl.Tc, pl.DP, kTileM)) return CUTBCE_ERR_CUDA;
  auto row_grid = [&](int splits) {                          // persistent: at most one CTA per SM
    const int64_t items = static_cast<int64_t>(splits) * (pl.Tc / kTileM);
    return static_cast<int>(std::min<int64_t>({static_cast<int64_t>(dev.sms), items, static_cast<int64_t>(kMaxCtas)}));
  };
  auto row_pass = [&]() -> cudaError_t {
    LaunchScope ls(CUTBCE_KERNEL_HEAD_ROW_PASS, st);
    sp.dh_part = at<float>(ws, pl.o_dhpart);
    CUtensorMap m_items_x;
    if (!make_map(&m_items_x, p.E, p.D, p.V, p.D, pl.BN)) return cudaErrorInvalidValue;
    return launch_softmax_dp<kPassRows>(pl.DP, row_grid(pl.S), m_rows_s, m_items_x, m_items_x, sp, st);
  };
  if (lse_in == nullptr) {
    {
      LaunchScope ls(CUTBCE_KERNEL_HEAD_LSE_PASS, st);
      sp.part = at<float2>(ws, pl.fused ? pl.o_wide : pl.o_part);
      sp.only_wide = pl.fused ? 1 : 0;
      CUtensorMap m_lse_x;
      if (!make_map(&m_lse_x, p.E, p.D, p.V, p.D, pl.BN_lse)) return CUTBCE_ERR_CUDA;
      SoftmaxParams lp = sp;
      lp.n_item_tiles_bn = pl.n_vtiles_lse;
      lp.tiles_per_split = pl.tps_lse;
      lp.nsplit = pl.S_lse;
      CUTBCE_CK(launch_softmax_dp<kPassLse>(pl.DP, row_grid(pl.S_lse), m_rows_s, m_lse_x, m_lse_x, lp, st));
    }
    if (pl.fused) {
      sp.wide_part = at<float2>(ws, pl.o_wide);
      sp.wide_slots = kHeadSlots * pl.S_lse;
    }
  }
  if (pl.rows_first) {
    sp.off2 = hp.m2;
    sp.part = at<float2>(ws, pl.o_part);
    CUTBCE_CK(row_pass());
  }
  sp.part = nullptr;
  sp.wide_part = nullptr;
  {
    LaunchScope ls(CUTBCE_KERNEL_HEAD_FINISH, st);
    if (hp.part != nullptr && hp.slots > kLseManySlots) k_head_lse<32><<<static_cast<unsigned>(pl.Tc * 32 / kLseThreads), kLseThreads, 0, st>>>(hp);
    else k_head_lse<4><<<static_cast<unsigned>(pl.Tc * 4 / kLseThreads), kLseThreads, 0, st>>>(hp);
    if (p.kind == kHeadPreference) k_head_pairs<<<static_cast<unsigned>(p.P), kPairThreads, 0, st>>>(hp);
    CUTBCE_CK(cudaGetLastError());
  }
  if (dH) {
    if (!pl.rows_first) {
      sp.off2 = hp.lse2;
      CUTBCE_CK(row_pass());
    }
    HeadDhParams dp{};
    dp.T = hp.T;
    dp.D = hp.D;
    dp.DP = pl.DP;
    dp.S = pl.S;
    dp.Tc = pl.Tc;
    dp.cidx = hp.cidx;
    dp.coef = hp.coef;
    dp.part = at<float>(ws, pl.o_dhpart);
    dp.sparse = hp.sparse;
    dp.omp = hp.omp;
    dp.rescale = hp.rescale;
    dp.dH = out.dH;
    dp.bf16 = out.grad_dtype == CUTBCE_GRAD_BF16;
    dp.accumulate = (out.accumulate & CUTBCE_ACCUMULATE_DH) != 0;
    dp.hdr = hp.hdr;
    LaunchScope ls(CUTBCE_KERNEL_HEAD_FINISH, st);
    const int64_t groups = p.T * (p.D / 4);
    if (groups < 148 * 512) k_head_dh<8><<<static_cast<unsigned>(ceil_div(groups, 32)), 256, 0, st>>>(dp);
    else k_head_dh<1><<<static_cast<unsigned>(ceil_div(groups, 256)), 256, 0, st>>>(dp);
    CUTBCE_CK(cudaGetLastError());
  }
  if (dE) {
    // the targets' part of dE: sum of coef (q - p) h over the pairs of each item, in fp32
    SegmentParams gp{};
    const FillJob none{at<uint4>(ws, pl.o_first), ceil_div(p.V, 4), 0xFFFFFFFFu};
    if ((s = run_sort(pl.sort, hp.keys, hp.V, ws, status, status, false, none, st, &gp.pairs)) != CUTBCE_OK) return s;
    gp.N = pl.Tc * p.K;
    gp.V = hp.V;
    gp.D = hp.D;
    gp.src = hp.Hc;
    gp.src_stride = pl.DP;
    gp.K = hp.K;
    gp.share = hp.share;
    gp.row_coef = hp.coef;
    gp.scale = 1.f;
    gp.part = at<float>(ws, pl.sort.o_part);
    gp.out = at<float>(ws, pl.o_usum);
    gp.first = at<int>(ws, pl.o_first);
    gp.columns = at<uint32_t>(ws, pl.o_columns);
    gp.stop = status;
    if ((s = run_sums(gp, true, st)) != CUTBCE_OK) return s;
    sp.first = gp.first;
    sp.columns = gp.columns;
    sp.n_pairs = static_cast<int>(gp.N);
    sp.sparse = at<float>(ws, pl.o_usum);
    sp.dE = out.dE;
    sp.de_bf16 = out.grad_dtype == CUTBCE_GRAD_BF16;
    sp.de_acc = (out.accumulate & CUTBCE_ACCUMULATE_DE) != 0;
    sp.off2 = hp.b2;
    CUtensorMap m_items_s, m_rows_x;
    if (!make_map(&m_items_s, p.E, p.D, p.V, p.D, kTileM) || !make_map(&m_rows_x, hp.Hc, pl.DP, pl.Tc, pl.DP, pl.BN))
      return CUTBCE_ERR_CUDA;
    CUtensorMap m_off = m_rows_x;
    if (hp.off16 != nullptr && !make_map_sw32(&m_off, hp.off16, pl.Tc, pl.BN)) return CUTBCE_ERR_CUDA;
    const int grid = static_cast<int>(std::min<int64_t>({static_cast<int64_t>(dev.sms), ceil_div(p.V, kTileM), static_cast<int64_t>(kMaxCtas)}));
    LaunchScope ls(CUTBCE_KERNEL_HEAD_ITEM_PASS, st);
    CUTBCE_CK(launch_softmax_dp<kPassItems>(pl.DP, grid, m_items_s, m_rows_x, m_off, sp, st));
  }
  return CUTBCE_OK;
}

cutbce_status head_workspace(const HeadProblem& p, int outputs, size_t* bytes) {
  if (bytes == nullptr || outputs <= 0 || outputs > (CUTBCE_OUT_LOSS | CUTBCE_OUT_DH | CUTBCE_OUT_DE))
    return CUTBCE_ERR_INVALID_ARG;
  const cutbce_status s = check_head(p, false);
  if (s != CUTBCE_OK) return s;
  HeadPlan with, without;                          // a pass for the log-sum-exps, or those of a forward
  plan_head(p, (outputs & CUTBCE_OUT_DH) != 0, (outputs & CUTBCE_OUT_DE) != 0, true, with);
  plan_head(p, (outputs & CUTBCE_OUT_DH) != 0, (outputs & CUTBCE_OUT_DE) != 0, false, without);
  *bytes = std::max(with.total, without.total);
  return CUTBCE_OK;
}

}  // namespace

extern "C" {

cutbce_status cutbce_embed_forward(const void* E, int64_t V, int64_t D, int32_t dtype, const int32_t* ids, int64_t N,
                                   float scale, void* X, int32_t* status, cutbce_stream_t stream) {
  cutbce_status s = check_embed(N, V, D, dtype);
  if (s != CUTBCE_OK) return s;
  const size_t e = dtype == CUTBCE_BF16 ? 2 : 4;
  if (E == nullptr || ids == nullptr || X == nullptr || !aligned(E, e) || !aligned(X, e) || !aligned(ids, 4) ||
      !aligned(status, 4))
    return CUTBCE_ERR_INVALID_ARG;
  if ((s = check_device()) != CUTBCE_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = aligned(E, 16) && aligned(X, 16);
  if (dtype == CUTBCE_BF16) {
    return wide && D % 8 == 0 ? launch_embed<8, __nv_bfloat16>(E, V, ids, N, D, scale, X, status, st)
                              : launch_embed<1, __nv_bfloat16>(E, V, ids, N, D, scale, X, status, st);
  }
  return wide && D % 4 == 0 ? launch_embed<4, float>(E, V, ids, N, D, scale, X, status, st)
                            : launch_embed<1, float>(E, V, ids, N, D, scale, X, status, st);
}

cutbce_status cutbce_embed_workspace_size(int64_t N, int64_t V, int64_t D, size_t* bytes) {
  if (bytes == nullptr) return CUTBCE_ERR_INVALID_ARG;
  const cutbce_status s = check_embed(N, V, D, CUTBCE_BF16);
  if (s != CUTBCE_OK) return s;
  EmbedPlan pl;
  plan_embed(N, V, D, pl);
  *bytes = pl.total;
  return CUTBCE_OK;
}

cutbce_status cutbce_embed_backward(const void* dX, int32_t dtype, const int32_t* ids, int64_t N, int64_t V, int64_t D,
                                    float scale, void* dE, int32_t grad_dtype, int32_t accumulate, void* ws,
                                    size_t ws_bytes, cutbce_stream_t stream) {
  cutbce_status s = check_embed(N, V, D, dtype);
  if (s != CUTBCE_OK) return s;
  if (grad_dtype != CUTBCE_GRAD_F32 && grad_dtype != CUTBCE_GRAD_BF16) return CUTBCE_ERR_UNSUPPORTED;
  const size_t ei = dtype == CUTBCE_BF16 ? 2 : 4, eo = grad_dtype == CUTBCE_GRAD_BF16 ? 2 : 4;
  if (dX == nullptr || ids == nullptr || dE == nullptr || ws == nullptr || !aligned(ws, 256) || !aligned(dX, ei) ||
      !aligned(dE, eo) || !aligned(ids, 4) || (accumulate != 0 && accumulate != 1))
    return CUTBCE_ERR_INVALID_ARG;
  EmbedPlan pl;
  plan_embed(N, V, D, pl);
  if (ws_bytes < pl.total) return CUTBCE_ERR_WORKSPACE;
  if ((s = check_device()) != CUTBCE_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int* status = at<int>(ws, pl.o_hdr);
  if (!pl.sort.cluster) CUTBCE_CK(cudaMemsetAsync(status, 0, pl.sort.o_hist + pl.sort.sp.hist_bytes, st));
  // dE starts at zero: by blocks beside the sort, or ahead of it where its ends are not 16-byte aligned
  const size_t de_bytes = eo * static_cast<size_t>(V) * D;
  FillJob fill{};
  if (!accumulate && aligned(dE, 16) && de_bytes % 16 == 0) fill = FillJob{static_cast<uint4*>(dE), static_cast<int64_t>(de_bytes / 16), 0u};
  else if (!accumulate) CUTBCE_CK(cudaMemsetAsync(dE, 0, de_bytes, st));
  SegmentParams p{};
  // an id out of range sets the status and counts as empty: dE is the gradient of what the lookup gave
  s = run_sort(pl.sort, ids, static_cast<int>(V), ws, status, nullptr, true, fill, st, &p.pairs);
  if (s != CUTBCE_OK) return s;
  p.N = N;
  p.V = static_cast<int>(V);
  p.D = static_cast<int>(D);
  p.src = dX;
  p.src_stride = D;
  p.K = 1;
  p.scale = scale;
  p.part = at<float>(ws, pl.sort.o_part);
  p.out = dE;
  p.out_bf16 = grad_dtype == CUTBCE_GRAD_BF16;
  p.accumulate = accumulate;
  return run_sums(p, dtype == CUTBCE_BF16, st);
}

cutbce_status cutbce_distill_workspace_size(const cutbce_distill_problem* prob, int outputs, size_t* bytes) {
  if (prob == nullptr) return CUTBCE_ERR_INVALID_ARG;
  return head_workspace(head_problem(prob), outputs, bytes);
}

cutbce_status cutbce_distill_forward(const cutbce_distill_problem* prob, double* loss, float* lse, void* ws,
                                     size_t ws_bytes, cutbce_stream_t stream) {
  if (prob == nullptr || (loss == nullptr && lse == nullptr)) return CUTBCE_ERR_INVALID_ARG;
  HeadOutputs o;
  o.loss = loss;
  o.lse = lse;
  return run_head(head_problem(prob), nullptr, nullptr, o, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

cutbce_status cutbce_distill_backward(const cutbce_distill_problem* prob, const cutbce_grad_options* opts,
                                      const float* lse, const float* grad_loss, void* dH, void* dE, void* ws,
                                      size_t ws_bytes, cutbce_stream_t stream) {
  if (prob == nullptr || lse == nullptr || (dH == nullptr && dE == nullptr)) return CUTBCE_ERR_INVALID_ARG;
  HeadOutputs o;
  const cutbce_status s = check_grad_options(opts, o);
  if (s != CUTBCE_OK) return s;
  o.dH = dH;
  o.dE = dE;
  return run_head(head_problem(prob), lse, grad_loss, o, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

cutbce_status cutbce_distill_forward_backward(const cutbce_distill_problem* prob, const cutbce_grad_options* opts,
                                              const float* grad_loss, double* loss, float* lse, void* dH, void* dE,
                                              void* ws, size_t ws_bytes, cutbce_stream_t stream) {
  if (prob == nullptr || (loss == nullptr && lse == nullptr && dH == nullptr && dE == nullptr))
    return CUTBCE_ERR_INVALID_ARG;
  HeadOutputs o;
  const cutbce_status s = check_grad_options(opts, o);
  if (s != CUTBCE_OK) return s;
  o.loss = loss;
  o.lse = lse;
  o.dH = dH;
  o.dE = dE;
  return run_head(head_problem(prob), nullptr, grad_loss, o, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

cutbce_status cutbce_preference_workspace_size(const cutbce_preference_problem* prob, int outputs, size_t* bytes) {
  if (prob == nullptr) return CUTBCE_ERR_INVALID_ARG;
  return head_workspace(head_problem(prob), outputs, bytes);
}

cutbce_status cutbce_preference_forward(const cutbce_preference_problem* prob, double* loss, float* logp, float* lse,
                                        void* ws, size_t ws_bytes, cutbce_stream_t stream) {
  if (prob == nullptr || (loss == nullptr && logp == nullptr && lse == nullptr)) return CUTBCE_ERR_INVALID_ARG;
  HeadOutputs o;
  o.loss = loss;
  o.logp = logp;
  o.lse = lse;
  return run_head(head_problem(prob), nullptr, nullptr, o, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

cutbce_status cutbce_preference_backward(const cutbce_preference_problem* prob, const cutbce_grad_options* opts,
                                         const float* lse, const float* grad_loss, void* dH, void* dE, void* ws,
                                         size_t ws_bytes, cutbce_stream_t stream) {
  if (prob == nullptr || lse == nullptr || (dH == nullptr && dE == nullptr)) return CUTBCE_ERR_INVALID_ARG;
  HeadOutputs o;
  const cutbce_status s = check_grad_options(opts, o);
  if (s != CUTBCE_OK) return s;
  o.dH = dH;
  o.dE = dE;
  return run_head(head_problem(prob), lse, grad_loss, o, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

cutbce_status cutbce_preference_forward_backward(const cutbce_preference_problem* prob,
                                                 const cutbce_grad_options* opts, const float* grad_loss, double* loss,
                                                 float* logp, float* lse, void* dH, void* dE, void* ws,
                                                 size_t ws_bytes, cutbce_stream_t stream) {
  if (prob == nullptr || (loss == nullptr && logp == nullptr && lse == nullptr && dH == nullptr && dE == nullptr))
    return CUTBCE_ERR_INVALID_ARG;
  HeadOutputs o;
  const cutbce_status s = check_grad_options(opts, o);
  if (s != CUTBCE_OK) return s;
  o.loss = loss;
  o.logp = logp;
  o.lse = lse;
  o.dH = dH;
  o.dE = dE;
  return run_head(head_problem(prob), nullptr, grad_loss, o, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

// Tokens to their experts and back.  P = T k (token, choice) pairs, pair p = t k + j:
//   sort     rows of the sorted buffer by expert, pairs of one expert in their order (stable):
//            offsets [E + 1], row_of [P] (the row of a pair), order [P] (the pair of a row).  Pairs
//            without an expert (choice outside [0, E)) follow the last group; their row r is
//            held as ~r, below zero
//   gather   rows[row_of[t, j]] = x[t]; rows of pairs without an expert are zero
//   combine  out[t] = add[t] + sum_j gate[t, j] y[row_of[t, j]] over the pairs that have an expert
//   and combine's gradient  dy[row_of[t, j]] = gate[t, j] dout[t],  dgate[t, j] = dout[t] . y[row_of[t, j]]
// The gradient of gather is combine without gates.
//
// Bound: gather, combine and its gradient move rows and are bound by HBM: the threads of a token
// go over its k rows together, so a token's own row is read or written once, and each sum is
// taken by one thread in the order of j (no atomics).  The sort moves 12 bytes a pair and is
// latency: a counting sort without atomics.  A warp counts its own run of pairs in its own
// counters (lanes with one expert find each other by a match), counters are summed over the
// warps, and each warp walks its run again with its running positions; up to 2^18 pairs in one
// launch of a cluster.
// All begin while the grid before them ends (8 tokens of 8 rows of 4096 through sort, gather and combine in a graph 9.5 us,
// 10.8 without; sort and gather of 16384 pairs 28.8, 29.7).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "api_internal.h"
#include "row_ops.cuh"

namespace dp {
namespace {

constexpr int64_t kMaxExpertCount = 1024;
constexpr int64_t kMaxPairs = 0x7FFFFFFF - 256;
constexpr int64_t kMaxColumns = 0x7FFFFFFF / 2048 * 2048;  // a thread's next column, up to 2048 further on, fits in 32 bits
constexpr uint32_t kAll = 0xffffffffu;

// ------------------------------------------------------------------------ sort

struct SortArgs {
  const void* choice;
  int wide;  // int64 choices
  int32_t P, E;
  int32_t per_block, per_warp;  // pairs, multiples of 32
  int32_t bits;                 // of the keys 0 .. E
  int32_t* counts;              // [blocks][E + 1], of two launches
  int32_t* offsets;
  int32_t* row_of;
  int32_t* order;
};

__device__ __forceinline__ int key_of(const SortArgs& a, int i) {
  const int64_t e = a.wide ? static_cast<const int64_t*>(a.choice)[i] : static_cast<const int32_t*>(a.choice)[i];
  return e >= 0 && e < a.E ? static_cast<int>(e) : a.E;
}

// The lanes whose keys (below 2^bits; -1: none) are this lane's.  A vote for each bit: the hardware's match takes longer the
// more keys differ.
__device__ __forceinline__ uint32_t same_keys(int key, int bits) {
  uint32_t same = __ballot_sync(kAll, key >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool set = (key >> b) & 1;
    const uint32_t m = __ballot_sync(kAll, set);
    same &= set ? m : ~m;
  }
  return same;
}

// The warp's own counts of the pairs in its run, in shared memory (zero before).
__device__ __forceinline__ void count_run(const SortArgs& a, int begin, int end, int32_t* mine) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  for (int i = begin + lane; i - lane < end; i += 32) {
    const int key = i < end ? key_of(a, i) : -1;
    const uint32_t same = same_keys(key, a.bits);
    if (key >= 0 && lane == __ffs(static_cast<int>(same)) - 1) mine[key] += __popc(same);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(1024) sort_count_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t warp_counts[];  // [warps][E + 1]
  const int n = a.E + 1, warp = static_cast<int>(threadIdx.x) >> 5, warps = static_cast<int>(blockDim.x) >> 5;
  for (int i = static_cast<int>(threadIdx.x); i < warps * n; i += static_cast<int>(blockDim.x)) warp_counts[i] = 0;
  pdl_begin();
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.per_block;
  const int begin = static_cast<int>(min(static_cast<int64_t>(a.P), first + warp * a.per_warp));
  const int end = static_cast<int>(min(static_cast<int64_t>(a.P), min(first + a.per_block, first + (warp + 1) * a.per_warp)));
  count_run(a, begin, end, warp_counts + warp * n);
  __syncthreads();
  for (int e = static_cast<int>(threadIdx.x); e < n; e += static_cast<int>(blockDim.x)) {
    int32_t s = 0;
    for (int w = 0; w < warps; ++w) s += warp_counts[w * n + e];
    a.counts[static_cast<int64_t>(blockIdx.x) * n + e] = s;
  }
}

__global__ void __launch_bounds__(1024) sort_place_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t warp_counts[];  // [warps][E + 1], then base [E + 1]
  __shared__ int32_t scan[33];
  const int n = a.E + 1, tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  int32_t* base = warp_counts + warps * n;
  for (int i = tid; i < warps * n; i += threads) warp_counts[i] = 0;
  pdl_begin();
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * a.per_block;
  const int begin = static_cast<int>(min(static_cast<int64_t>(a.P), first + warp * a.per_warp));
  const int end = static_cast<int>(min(static_cast<int64_t>(a.P), min(first + a.per_block, first + (warp + 1) * a.per_warp)));
  count_run(a, begin, end, warp_counts + warp * n);
  __syncthreads();
  // positions of the warps within their block, the pairs of each expert in all blocks and before this one
  int32_t carry = 0;
  for (int e0 = 0; e0 < n; e0 += threads) {
    const int e = e0 + tid;
    int32_t own = 0, total = 0, before = 0;
    if (e < n) {
      for (int w = 0; w < warps; ++w) {
        const int32_t c = warp_counts[w * n + e];
        warp_counts[w * n + e] = own;
        own += c;
      }
      for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
        if (b == static_cast<int>(blockIdx.x)) before = total;
        total += a.counts[static_cast<int64_t>(b) * n + e];
      }
    }
    int32_t incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kAll, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int32_t lower = carry;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) lower += scan[w];
      carry += scan[w];
    }
    if (e < n) {
      const int32_t start = lower + incl - total;
      base[e] = start + before;
      if (blockIdx.x == 0) a.offsets[e] = start;
    }
    __syncthreads();
  }
  int32_t* mine = warp_counts + warp * n;
  for (int i = begin + lane; i - lane < end; i += 32) {
    const int key = i < end ? key_of(a, i) : -1;
    const uint32_t same = same_keys(key, a.bits);
    const int32_t at = key >= 0 ? base[key] + mine[key] + __popc(same & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (key >= 0) {
      if (lane == __ffs(static_cast<int>(same)) - 1) mine[key] += __popc(same);
      a.row_of[i] = key < a.E ? at : ~at;
      a.order[at] = i;
    }
    __syncwarp();
  }
}

// The same in one launch, for pairs that one cluster can go through: the blocks read each other's
// counts from their shared memory.  Latency: 16384 pairs over 64 experts 6.1 us (14.1 in two launches; 11 with keys that
// meet by the hardware's match, in an earlier form of 8 us), 64 pairs 3 us.
__global__ void __launch_bounds__(1024) sort_cluster_kernel(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t warp_counts[];  // [warps][E + 1], then the block's totals [E + 1] and base [E + 1]
  __shared__ int32_t scan[32];
  constexpr int HELD = 4;  // runs of 32 pairs whose keys stay in registers
  const int n = a.E + 1, tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int threads = static_cast<int>(blockDim.x), warps = threads >> 5;
  const int rank = static_cast<int>(blockIdx.x), ranks = static_cast<int>(gridDim.x);
  const int stride = n | 1;  // (counters of one expert lie in different banks)
  int32_t* const totals = warp_counts + warps * stride;
  int32_t* const base = totals + n;
  const int begin = static_cast<int>(min(static_cast<int64_t>(a.P), static_cast<int64_t>(rank) * a.per_block + warp * a.per_warp));
  const int end = static_cast<int>(min(static_cast<int64_t>(a.P), static_cast<int64_t>(begin) + a.per_warp));
  pdl_begin();
  int held[HELD];
#pragma unroll
  for (int r = 0; r < HELD; ++r) held[r] = begin + r * 32 + lane < end ? key_of(a, begin + r * 32 + lane) : -1;
  for (int i = tid; i < warps * stride; i += threads) warp_counts[i] = 0;
  uint32_t held_same[HELD];
#pragma unroll
  for (int r = 0; r < HELD; ++r)
    if (begin + r * 32 < end) held_same[r] = same_keys(held[r], a.bits);
  __syncthreads();
  int32_t* const mine = warp_counts + warp * stride;
  auto walk = [&](auto step) {  // the warp's runs in order: first pair of the run, this lane's key (-1: none) and the lanes that share it
#pragma unroll
    for (int r = 0; r < HELD; ++r)
      if (begin + r * 32 < end) step(begin + r * 32, held[r], held_same[r]);
    for (int i = begin + HELD * 32; i < end; i += 32) {
      const int key = i + lane < end ? key_of(a, i + lane) : -1;
      step(i, key, same_keys(key, a.bits));
    }
  };
  walk([&](int, int key, uint32_t same) {
    if (key >= 0 && lane == __ffs(static_cast<int>(same)) - 1) mine[key] += __popc(same);
    __syncwarp();
  });
  __syncthreads();
  for (int e = warp; e < n; e += warps) {  // positions of the warps within their block: lane w has warp w's count
    const int32_t own = lane < warps ? warp_counts[lane * stride + e] : 0;
    int32_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kAll, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane < warps) warp_counts[lane * stride + e] = incl - own;
    if (lane == 31) totals[e] = incl;
  }
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  int32_t carry = 0;
  for (int e0 = 0; e0 < n; e0 += threads) {
    const int e = e0 + tid;
    int32_t total = 0, before = 0;
    if (e < n) {
      const uint32_t at = smem_addr(totals + e);
      for (int r = 0; r < ranks; ++r) {
        int32_t c = totals[e];
        if (r != rank) asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(map_shared_rank(at, r)) : "memory");
        if (r < rank) before += c;
        total += c;
      }
    }
    int32_t incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kAll, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int32_t sums = lane < warps ? scan[lane] : 0;  // of the warps up to this lane's
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kAll, sums, d);
      if (lane >= d) sums += o;
    }
    const int32_t up_to = __shfl_sync(kAll, sums, warp > 0 ? warp - 1 : 0);
    const int32_t lower = carry + (warp > 0 ? up_to : 0);
    carry += __shfl_sync(kAll, sums, 31);
    if (e < n) {
      const int32_t start = lower + incl - total;
      base[e] = start + before;
      if (rank == 0) a.offsets[e] = start;
    }
    __syncthreads();
  }
  walk([&](int first, int key, uint32_t same) {
    const int32_t at = key >= 0 ? base[key] + mine[key] + __popc(same & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (key >= 0) {
      if (lane == __ffs(static_cast<int>(same)) - 1) mine[key] += __popc(same);
      a.row_of[first + lane] = key < a.E ? at : ~at;
      a.order[at] = first + lane;
    }
    __syncwarp();
  });
  if (ranks > 1) cluster_sync();  // (no block ends while others read its totals)
}

struct SortShape {
  int ranks;  // of the cluster that sorts alone (0: two launches)
  int warps, blocks;  // (of the two)
  int32_t per_warp, per_block;
  size_t smem;
};

constexpr int kSortBlocks = 128;
// Up to 2^18 pairs (32 runs a warp) a cluster, which needs no workspace.  One launch of a cluster / two launches, us:
//   8 experts     32768 pairs 5.9 / 11.8, 65536 11.1 / 12.5, 131072 21.2 / 14.0, 262144 41.0 / 17.2
//   64 experts    32768 8.1 / 14.2, 65536 15.3 / 15.0, 131072 28.1 / 16.1, 262144 52.3 / 18.5
//   1024 experts  32768 16.0 / 24.2, 65536 24.6 / 34.6, 131072 39.8 / 53.4, 262144 69.8 / 67.9
// so that between 2^16 and 2^18 pairs of few experts two launches would be faster, for callers who bring their workspace.
constexpr int64_t kClusterPairs = 1 << 18;

SortShape sort_shape(int64_t P, int64_t E) {
  SortShape s = {};
  const int want = tuning_override("DP_FORCE_SORT_CLUSTER", -1);
  if (want < 0 ? P <= kClusterPairs : want != 0) {
    const int64_t all = (P + 31) / 32;
    s.ranks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, (all + 63) / 64)));
    s.warps = all <= 16 ? 8 : 32;
    s.per_warp = static_cast<int32_t>((all + s.ranks * s.warps - 1) / (s.ranks * s.warps) * 32);
    s.per_block = s.per_warp * s.warps;
    s.smem = (static_cast<size_t>(s.warps) * ((E + 1) | 1) + 2 * (E + 1)) * 4;
    return s;
  }
  // (counters and positions: at most 46 KB)
  s.warps = static_cast<int>(std::min<int64_t>(32, (46 << 8) / (E + 1) - 1));
  const int64_t runs = (P + 31) / 32;  // 32 pairs each
  s.blocks = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kSortBlocks, runs / (s.warps * 4))));
  const int64_t per = (runs + static_cast<int64_t>(s.blocks) * s.warps - 1) / (static_cast<int64_t>(s.blocks) * s.warps);
  s.per_warp = static_cast<int32_t>(per * 32);
  s.per_block = s.per_warp * s.warps;
  s.smem = static_cast<size_t>(s.warps + 1) * (E + 1) * 4;
  return s;
}

// ------------------------------------------------------------- gather, combine

struct RowArgs {
  const void* x;  // gather: x; combine: y; gradient: dout
  int64_t ldx;
  const void* y;  // gradient: y
  int64_t ld_y;
  const int32_t* row_of;
  const float* gates;  // null: 1
  const void* add;     // null: 0
  int64_t ld_add;
  void* out;  // gather: rows; combine: out; gradient: dy
  int64_t ldo;
  float* dgates;
  int64_t T;
  int32_t k, C, tpr, P;
  uint32_t* fault;
};

// The row that a pair's entry names and whether the pair has an expert.  An entry that names no
// row of the buffer is reported, and its pair left out.
struct Place {
  int32_t row;  // -1: none
  bool live;
};

__device__ __forceinline__ Place place_of(const RowArgs& a, int64_t pair) {
  const int32_t r = a.row_of[pair], row = r < 0 ? ~r : r;
  if (row < a.P) return {row, r >= 0};
  atomicOr(a.fault, kFaultOffsets);
  return {-1, false};
}

// 2048 tokens to 8 rows each of 4096 in BF16: 22 us, 6.8 TB/s.
template <bool F32>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ RowArgs a) {
  const int sub = static_cast<int>(threadIdx.x) / a.tpr, lane = static_cast<int>(threadIdx.x) % a.tpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / a.tpr) + sub;
  pdl_begin();
  if (t >= a.T) return;
  for (int col = lane * 8; col < a.C; col += a.tpr * 8) {
    const Raw8<F32> v = load_raw8<F32, true>(a.x, t * a.ldx + col);
    for (int j = 0; j < a.k; ++j) {
      const Place at = place_of(a, t * a.k + j);
      if (at.row >= 0) store_raw8<F32>(a.out, at.row * a.ldo + col, at.live ? v : zero_raw8<F32>());
    }
  }
}

constexpr int kBatch = 4;  // rows of a token whose loads are in flight together (combine: 2 where there are no more)

// (With loads for no more rows than there are: 8192 tokens of 2 rows of 4096 in BF16 36.5 us, 38.8 with room for four;
// 16384 of one row of 1024 16.4, 19.2.  BF16 rows, five blocks an SM: 2048 tokens of 8 rows of 4096 26.3 us, 4096 of 3 rows
// 26.3; with six 27.6 and 25.4; with the four that 50 registers leave 28.4 and 26.  At five, 48 registers, the form for four BF16
// rows spills two words, and it is the faster one all the same.  FP32 rows need their registers: 27 us, 40 with 40.)
template <bool YF32, bool OF32, int BATCH>
__global__ void __launch_bounds__(256, YF32 ? 4 : 5) combine_kernel(const __grid_constant__ RowArgs a) {
  const int sub = static_cast<int>(threadIdx.x) / a.tpr, lane = static_cast<int>(threadIdx.x) % a.tpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / a.tpr) + sub;
  pdl_begin();
  if (t >= a.T) return;
  for (int col = lane * 8; col < a.C; col += a.tpr * 8) {
    float s[8];
    if (a.add != nullptr) {
      load8<OF32, true>(a.add, t * a.ld_add + col, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    }
    for (int j0 = 0; j0 < a.k; j0 += BATCH) {
      Raw8<YF32> v[BATCH];
      float g[BATCH];
      bool live[BATCH];
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const Place at = j0 + j < a.k ? place_of(a, t * a.k + j0 + j) : Place{-1, false};
        live[j] = at.live, g[j] = 1.0f;
        v[j] = at.live ? load_raw8<YF32, true>(a.x, at.row * a.ldx + col) : zero_raw8<YF32>();
        if (at.live && a.gates != nullptr) g[j] = a.gates[t * a.k + j0 + j];
      }
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        if (!live[j]) continue;
        float x[8];
        unpack8<YF32>(v[j], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(g[j], x[i], s[i]);
      }
    }
    store8<OF32>(a.out, t * a.ldo + col, s);
  }
}

// dy goes out as y comes in, kBatch rows at a time, and the rows' dots meet together: 2048 tokens of 8 rows of 4096 in
// BF16 45 us, 6.3 TB/s (62 with a row at a time; with combine before it batches of 2, 4, 8 rows took 84, 80, 88).
template <bool DF32, bool YF32, bool OF32>
__global__ void __launch_bounds__(256) combine_bwd_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float part[2][32][kBatch];
  const int sub = static_cast<int>(threadIdx.x) / a.tpr, lane = static_cast<int>(threadIdx.x) % a.tpr;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / a.tpr) + sub;
  pdl_begin();
  GroupSum<kBatch> sum(part, a.tpr);
  for (int j0 = 0; j0 < a.k; j0 += kBatch) {  // (every thread of the block: the sums meet in barriers)
    Place at[kBatch];
    float g[kBatch], dot[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      at[j] = t < a.T && j0 + j < a.k ? place_of(a, t * a.k + j0 + j) : Place{-1, false};
      g[j] = at[j].live ? a.gates[t * a.k + j0 + j] : 0.0f;
      dot[j] = 0.0f;
    }
    for (int col = lane * 8; t < a.T && col < a.C; col += a.tpr * 8) {
      Raw8<YF32> v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        v[j] = at[j].live ? load_raw8<YF32, true>(a.y, at[j].row * a.ld_y + col) : zero_raw8<YF32>();
      float d[8];
      load8<DF32, true>(a.x, t * a.ldx + col, d);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (at[j].row < 0) continue;
        float x[8];
        unpack8<YF32>(v[j], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (at[j].live) dot[j] = fmaf(d[i], x[i], dot[j]);
          x[i] = at[j].live ? d[i] * g[j] : 0.0f;
        }
        store8<OF32>(a.out, at[j].row * a.ldo + col, x);
      }
    }
    sum(dot);
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (t < a.T && lane == 0 && j0 + j < a.k) a.dgates[t * a.k + j0 + j] = dot[j];
  }
}

int threads_per_token(int64_t C) {
  int tpr = 8;
  while (tpr < 256 && tpr * 8 < C) tpr *= 2;
  return tpr;
}

bool flag(int v) { return v == 0 || v == 1; }

template <typename F>
void by_bool(bool v, F f) {
  v ? f(std::true_type()) : f(std::false_type());
}

dp_status check_pairs(const int32_t* row_of, int64_t T, int64_t k, int64_t C) {
  if (T < 0 || k < 1 || C < 1) return DP_ERR_INVALID_ARG;
  if (C % 8 != 0 || C > kMaxColumns || T > kMaxPairs || k > kMaxPairs || T * k > kMaxPairs) return DP_ERR_UNSUPPORTED;
  if (T > 0 && row_of == nullptr) return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(row_of) & 3) != 0) return DP_ERR_ALIGNMENT;
  return DP_OK;
}

RowArgs row_args(const int32_t* row_of, const float* gates, int64_t T, int64_t k, int64_t C, const DeviceContext& ctx) {
  RowArgs a = {};
  a.row_of = row_of, a.gates = gates, a.T = T, a.k = static_cast<int32_t>(k), a.C = static_cast<int32_t>(C);
  a.tpr = threads_per_token(C), a.P = static_cast<int32_t>(T * k), a.fault = ctx.fault;
  return a;
}

unsigned token_blocks(const RowArgs& a) { return static_cast<unsigned>((a.T + 256 / a.tpr - 1) / (256 / a.tpr)); }

}  // namespace

cudaError_t set_attributes_experts() {
  return cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>((32 + 2) * (kMaxExpertCount + 2) * 4));
}

}  // namespace dp

extern "C" dp_status dp_expert_sort_workspace_size(int64_t pairs, int64_t E, size_t* bytes) {
  using namespace dp;
  if (bytes == nullptr || pairs < 0 || E < 1) return DP_ERR_INVALID_ARG;
  if (E > kMaxExpertCount || pairs > kMaxPairs) return DP_ERR_UNSUPPORTED;
  const SortShape s = sort_shape(pairs, E);
  *bytes = static_cast<size_t>(s.blocks) * (E + 1) * 4;  // (0 for a cluster)
  return DP_OK;
}

extern "C" dp_status dp_expert_sort(const void* choice, int choice_bits, int64_t pairs, int64_t E, int32_t* offsets,
                                    int32_t* row_of, int32_t* order, void* workspace, size_t workspace_bytes,
                                    dp_stream stream) {
  using namespace dp;
  if ((choice_bits != 32 && choice_bits != 64) || pairs < 0 || E < 1 || offsets == nullptr) return DP_ERR_INVALID_ARG;
  if (E > kMaxExpertCount || pairs > kMaxPairs) return DP_ERR_UNSUPPORTED;
  if (pairs > 0 && (choice == nullptr || row_of == nullptr || order == nullptr)) return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(choice) & (choice_bits / 8 - 1)) != 0 ||
      ((reinterpret_cast<uintptr_t>(offsets) | reinterpret_cast<uintptr_t>(row_of) | reinterpret_cast<uintptr_t>(order) |
        reinterpret_cast<uintptr_t>(workspace)) & 3) != 0)
    return DP_ERR_ALIGNMENT;
  const SortShape s = sort_shape(pairs, E);
  if (s.ranks == 0 && (workspace == nullptr || workspace_bytes < static_cast<size_t>(s.blocks) * (E + 1) * 4))
    return DP_ERR_WORKSPACE;
  DeviceContext ctx;
  const dp_status st = device_context(&ctx);
  if (st != DP_OK) return st;
  SortArgs a = {};
  a.choice = choice, a.wide = choice_bits == 64, a.P = static_cast<int32_t>(pairs), a.E = static_cast<int32_t>(E);
  while ((1 << a.bits) <= a.E) ++a.bits;
  a.per_block = s.per_block, a.per_warp = s.per_warp, a.counts = static_cast<int32_t*>(workspace);
  a.offsets = offsets, a.row_of = row_of, a.order = order;
  if (s.ranks > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(s.ranks));
    cfg.blockDim = dim3(static_cast<unsigned>(s.warps * 32));
    cfg.dynamicSmemBytes = s.smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.ranks), attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.ranks > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, sort_cluster_kernel, a) == cudaSuccess) return DP_OK;
    cudaGetLastError();
    return DP_ERR_LAUNCH;
  }
  const dp_status counted = launch_dependent(sort_count_kernel, s.blocks, s.warps * 32, s.smem, stream, a);
  if (counted != DP_OK) return counted;
  return launch_dependent(sort_place_kernel, s.blocks, s.warps * 32, s.smem, stream, a);
}

extern "C" dp_status dp_expert_gather(const void* x, int64_t ldx, int x_f32, const int32_t* row_of, void* rows, int64_t ldr,
                                      int64_t T, int64_t k, int64_t C, dp_stream stream) {
  using namespace dp;
  if (!flag(x_f32)) return DP_ERR_INVALID_ARG;
  dp_status st = check_pairs(row_of, T, k, C);
  if (st == DP_OK) st = check_operand(x, T, C, &ldx, x_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(rows, T, C, &ldr, x_f32 ? 4 : 2);
  if (st != DP_OK) return st;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  RowArgs a = row_args(row_of, nullptr, T, k, C, ctx);
  a.x = x, a.ldx = ldx, a.out = rows, a.ldo = ldr;
  by_bool(x_f32, [&](auto f) { st = launch_dependent(gather_kernel<decltype(f)::value>, token_blocks(a), 256, 0, stream, a); });
  return st;
}

extern "C" dp_status dp_expert_combine(const void* y, int64_t ldy, int y_f32, const int32_t* row_of, const float* gates,
                                       const void* add, int64_t ld_add, void* out, int64_t ldo, dp_out_dtype out_dtype,
                                       int64_t T, int64_t k, int64_t C, dp_stream stream) {
  using namespace dp;
  const int code = static_cast<int>(out_dtype);
  if (!flag(y_f32) || !flag(code)) return DP_ERR_INVALID_ARG;
  dp_status st = check_pairs(row_of, T, k, C);
  if (st == DP_OK) st = check_operand(y, T, C, &ldy, y_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(out, T, C, &ldo, code ? 4 : 2);
  if (st == DP_OK && add != nullptr) st = check_operand(add, T, C, &ld_add, code ? 4 : 2);
  if (st != DP_OK) return st;
  if ((reinterpret_cast<uintptr_t>(gates) & 3) != 0) return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  RowArgs a = row_args(row_of, gates, T, k, C, ctx);
  a.x = y, a.ldx = ldy, a.add = add, a.ld_add = ld_add, a.out = out, a.ldo = ldo;
  by_bool(y_f32, [&](auto yf) {
    by_bool(code, [&](auto of) {
      constexpr bool Y = decltype(yf)::value, O = decltype(of)::value;
      st = launch_dependent(k <= 2 ? combine_kernel<Y, O, 2> : combine_kernel<Y, O, kBatch>, token_blocks(a), 256, 0, stream, a);
    });
  });
  return st;
}

extern "C" dp_status dp_expert_combine_bwd(const void* dout, int64_t ldd, int dout_f32, const void* y, int64_t ldy, int y_f32,
                                           const int32_t* row_of, const float* gates, void* dy, int64_t ld_dy,
                                           dp_out_dtype dy_dtype, float* dgates, int64_t T, int64_t k, int64_t C,
                                           dp_stream stream) {
  using namespace dp;
  const int code = static_cast<int>(dy_dtype);
  if (!flag(dout_f32) || !flag(y_f32) || !flag(code)) return DP_ERR_INVALID_ARG;
  dp_status st = check_pairs(row_of, T, k, C);
  if (st == DP_OK) st = check_operand(dout, T, C, &ldd, dout_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(y, T, C, &ldy, y_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(dy, T, C, &ld_dy, code ? 4 : 2);
  if (st != DP_OK) return st;
  if (T > 0 && (gates == nullptr || dgates == nullptr)) return DP_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(gates) | reinterpret_cast<uintptr_t>(dgates)) & 3) != 0) return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  RowArgs a = row_args(row_of, gates, T, k, C, ctx);
  a.x = dout, a.ldx = ldd, a.y = y, a.ld_y = ldy, a.out = dy, a.ldo = ld_dy, a.dgates = dgates;
  by_bool(dout_f32, [&](auto df) {
    by_bool(y_f32, [&](auto yf) {
      by_bool(code, [&](auto of) {
        st = launch_dependent(combine_bwd_kernel<decltype(df)::value, decltype(yf)::value, decltype(of)::value>, token_blocks(a), 256, 0,
                              stream, a);
      });
    });
  });
  return st;
}

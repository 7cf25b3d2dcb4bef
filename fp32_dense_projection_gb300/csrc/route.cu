// The router's choice: the k largest of each token's E logits (FP32) and their gates, and the
// gradient of the gates with respect to the logits.
//   chosen by value, the lowest index first among equals; a logit of -infinity is a closed expert:
//   it is never chosen (choice -1, gate 0, where fewer than k are open)
//   gate_j = exp(l_j - m) / sum exp(l - m), the sum over the chosen or over all experts
// Gradient, with s = sum_j dg_j gate_j over the chosen:
//   over the chosen:  dl_e = gate_e (dg_e - s), 0 for the others
//   over all:         dl_e = p_e ([e chosen] dg_e - s)
//
// Exponentials are expf's, within 2 ulp at any distance from the largest (__expf's grows with it: 3.8e-6 of a gate 60 to 80
// below, 2.9e-7 now).
//
// Bound: instructions (16384 tokens of 256 experts, k = 8, over all: 10.1 us and 6.4 the gradient, 2.5 of them the
// logits' bytes); a few rows are latency.  One warp a token holds its logits in registers, so they are read
// once.  Keys order floats as integers: -0 as +0, NaN above all.
// 3 to 16 choices: the k-th of the lanes' largest keys is a lower bound of the k-th of all; what is above it goes
// to shared memory in the order of indexes, and if a warp's lanes can hold it, each counts how many come before its own.
// Otherwise a choice is a warp-wide maximum and the votes for it, register by register, up to the first that has it.
// By the bound / by the search, 16384 tokens, us (more choices leave more above the bound than lanes):
//   64 experts    k = 1 4.1 / 3.7, 3 4.9 / 4.7, 8 6.8 / 7.0, 16 10.0 / 10.9, 20 12.2 / 12.8, 24 17.0 / 14.8
//   256 experts   k = 1 7.3 / 6.1, 3 8.1 / 8.2, 8 10.1 / 13.5, 16 13.9 / 21.8, 20 22.5 / 26.0, 24 35.1 / 30.1
//   1024 experts  k = 1 21.3 / 17.7, 3 22.4 / 26.5, 8 24.6 / 46.8, 16 38.0 / 77.7, 20 110 / 93
// (Whether the gradient's choices differ, each lane sees from who holds its expert: 7.2 us, 8.8 by matching lanes, both before
// closed experts lost their selections.)
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "api_internal.h"
#include "ptx.cuh"

namespace dp {
namespace {

constexpr int kMaxRouted = 1024, kMaxChosen = 32;
constexpr int kWarps = 8;  // tokens a block has at a time
constexpr int kBoundFrom = 3, kBoundTo = 16;  // choices that are looked for above a lower bound of the last
constexpr uint32_t kAll = 0xffffffffu;

struct RouteArgs {
  const float* logits;
  int64_t ld;
  int64_t T;
  int32_t E, k, renormalize;
  float* gates;
  int32_t* choice;
  const float* dgates;
  float* dlogits;
  int64_t ldd;
};

// An integer that orders as the float does; above 0 for every float.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 becomes +0)
  const uint32_t key = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return x != x ? 0xFFFFFFFFu : key;
}

__device__ __forceinline__ float key_value(uint32_t key) {
  if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

constexpr uint32_t kClosed = 0x007FFFFFu;  // order_key(-infinity)

template <int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ uint2 found[kWarps][32];  // candidates: key, index
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  pdl_begin();
  if (t >= a.T) return;
  const float* p = a.logits + t * a.ld;
  float x[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] = lane + 32 * i < a.E ? p[lane + 32 * i] : -INFINITY;
  uint32_t key[VPL], most = 0;  // this lane's largest
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = order_key(x[i]);
    most = max(most, key[i]);
  }
  // the k-th of the lanes' largest is a lower bound of the k-th of all (lanes that share a value count as one)
  const bool bounded = a.k >= kBoundFrom && a.k <= kBoundTo;
  uint32_t first = __reduce_max_sync(kAll, most), least = max(first, kClosed + 1), rest = most == first ? 0 : most;
  for (int j = 1; j < a.k && bounded; ++j) {
    const uint32_t best = __reduce_max_sync(kAll, rest);
    least = max(best, kClosed + 1);
    if (best <= kClosed) break;
    if (rest == best) rest = 0;
  }
  int count = bounded ? 0 : 33;
#pragma unroll
  for (int i = 0; i < VPL && bounded; ++i) {  // in the order of their indexes
    const bool in = key[i] >= least;
    const uint32_t have = __ballot_sync(kAll, in);
    if (in) found[warp][(count + __popc(have & ((1u << lane) - 1))) & 31] = make_uint2(key[i], lane + 32 * i);
    count += __popc(have);
  }
  const float m = key_value(first);
  float total = 0.0f;
  if (!a.renormalize && first != kClosed) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) total += expf(x[i] - m);  // (0 for what is closed: m is above)
    total = warp_sum(total);
  }
  uint32_t mine = 0;  // a choice's key, index and place
  int at = -1, place = lane;
  if (count <= 32) {
    __syncwarp();
    if (lane < count) mine = found[warp][lane].x, at = static_cast<int>(found[warp][lane].y), place = 0;
    for (int s = 0; s < count; ++s) {  // how many come before it
      const uint32_t other = __shfl_sync(kAll, mine, s);
      if (lane < count && (s < lane ? other >= mine : other > mine)) ++place;
    }
  } else {
    for (int j = 0; j < a.k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(kAll, best);
      if (best <= kClosed) break;
      // the lowest index that has it, which is taken out: indexes go up by lanes, then by registers
      int index = -1;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (index >= 0) continue;
        const uint32_t have = __ballot_sync(kAll, key[i] == best);
        if (have == 0) continue;
        const int owner = __ffs(static_cast<int>(have)) - 1;
        index = owner + 32 * i;
        if (lane == owner) key[i] = 0;
      }
      if (lane == j) mine = best, at = index;
    }
  }
  if (place >= a.k) at = -1;
  const float e = at >= 0 ? expf(key_value(mine) - m) : 0.0f;
  if (a.renormalize) total = warp_sum(e);
  if (place < a.k) {
    a.gates[t * a.k + place] = at >= 0 ? e / total : 0.0f;
    a.choice[t * a.k + place] = at;
  }
}

template <int VPL>
__global__ void __launch_bounds__(kWarps * 32) route_bwd_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ uint8_t holder[kWarps][VPL * 32];  // of an expert: a lane that has it
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  pdl_begin();
  if (t >= a.T) return;
  int at = -1;
  float g = 0.0f, dg = 0.0f;
  if (lane < a.k) {
    at = a.choice[t * a.k + lane];
    if (at < 0 || at >= a.E) at = -1;
    if (at >= 0) g = a.gates[t * a.k + lane], dg = a.dgates[t * a.k + lane];
  }
  const float s = warp_sum(at >= 0 ? g * dg : 0.0f);
  float d[VPL];
  if (a.renormalize) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
  } else {
    const float* p = a.logits + t * a.ld;
    float l[VPL], m = -INFINITY, total = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < a.E ? p[e] : -INFINITY;
      nan = nan || l[i] != l[i];
      m = fmaxf(m, l[i]);
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, w));
    if (__any_sync(kAll, nan)) {  // what is open is NaN
#pragma unroll
      for (int i = 0; i < VPL; ++i) l[i] = l[i] == -INFINITY ? l[i] : __uint_as_float(0x7FC00000u);
    }
    if (m == -INFINITY) m = 0.0f;  // (a closed expert's difference stays -infinity, its exponential 0)
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = expf(l[i] - m);
      total += l[i];
    }
    const float minus = -(s / warp_sum(total));
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = l[i] == 0.0f ? 0.0f : l[i] * minus;
  }
  float* out = a.dlogits + t * a.ldd;
  const float own = a.renormalize ? g * (dg - s) : g * dg;
  // choices that differ, as route_kernel makes them, are put into the row by the lanes that have them;
  // others are added up in their order
  if (at >= 0) holder[warp][at] = static_cast<uint8_t>(lane);
  __syncwarp();
  const bool repeated = __any_sync(kAll, at >= 0 && holder[warp][at] != lane);
  if (repeated) {
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl_sync(kAll, at, j);
      const float v = __shfl_sync(kAll, own, j);
      if (e < 0) continue;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (e == lane + 32 * i) d[i] += v;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    if (e < a.E) out[e] = d[i];
  }
  __syncwarp();
  // (gate_e is p_e: what stands there is -p_e s)
  if (!repeated && at >= 0) out[at] = g * (dg - s);
}

template <typename F>
void by_width(int64_t E, F f) {
  if (E <= 64)
    f(std::integral_constant<int, 2>());
  else if (E <= 128)
    f(std::integral_constant<int, 4>());
  else if (E <= 256)
    f(std::integral_constant<int, 8>());
  else if (E <= 512)
    f(std::integral_constant<int, 16>());
  else
    f(std::integral_constant<int, 32>());
}

dp_status check_route(const float* logits, int64_t* ld, int64_t T, int64_t E, int64_t k, int renormalize) {
  if (T < 0 || E < 1 || k < 1 || k > E || (renormalize != 0 && renormalize != 1)) return DP_ERR_INVALID_ARG;
  if (E > kMaxRouted || k > kMaxChosen || T > 0x7FFFFFFF) return DP_ERR_UNSUPPORTED;
  if (*ld == 0) *ld = E;
  if (*ld < E || (T > 0 && logits == nullptr)) return DP_ERR_INVALID_ARG;
  if (*ld > (int64_t{1} << 36)) return DP_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(logits) & 3) != 0) return DP_ERR_ALIGNMENT;
  return DP_OK;
}

}  // namespace
}  // namespace dp

extern "C" dp_status dp_route_topk(const float* logits, int64_t ld, float* gates, int32_t* choice, int64_t T, int64_t E,
                                   int64_t k, int renormalize, dp_stream stream) {
  using namespace dp;
  dp_status st = check_route(logits, &ld, T, E, k, renormalize);
  if (st != DP_OK) return st;
  if (T > 0 && (gates == nullptr || choice == nullptr)) return DP_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(gates) | reinterpret_cast<uintptr_t>(choice)) & 3) != 0) return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  RouteArgs a = {};
  a.logits = logits, a.ld = ld, a.T = T, a.E = static_cast<int32_t>(E), a.k = static_cast<int32_t>(k);
  a.renormalize = renormalize, a.gates = gates, a.choice = choice;
  const unsigned grid = static_cast<unsigned>((T + kWarps - 1) / kWarps);
  by_width(E, [&](auto v) {
    st = launch_dependent(route_kernel<decltype(v)::value>, grid, kWarps * 32, 0, stream, a);
  });
  return st;
}

extern "C" dp_status dp_route_topk_bwd(const float* dgates, const float* logits, int64_t ld, const float* gates,
                                       const int32_t* choice, float* dlogits, int64_t ldd, int64_t T, int64_t E, int64_t k,
                                       int renormalize, dp_stream stream) {
  using namespace dp;
  // (over the chosen, the gates say all: the logits are not read and may be null)
  dp_status st = check_route(renormalize ? dlogits : logits, &ld, T, E, k, renormalize);
  if (st == DP_OK) st = check_route(dlogits, &ldd, T, E, k, renormalize);
  if (st != DP_OK) return st;
  if (T > 0 && (gates == nullptr || choice == nullptr || dgates == nullptr)) return DP_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(gates) | reinterpret_cast<uintptr_t>(choice) | reinterpret_cast<uintptr_t>(dgates)) & 3) != 0)
    return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  RouteArgs a = {};
  a.logits = logits, a.ld = ld, a.T = T, a.E = static_cast<int32_t>(E), a.k = static_cast<int32_t>(k);
  a.renormalize = renormalize, a.gates = const_cast<float*>(gates), a.choice = const_cast<int32_t*>(choice);
  a.dgates = dgates, a.dlogits = dlogits, a.ldd = ldd;
  const unsigned grid = static_cast<unsigned>((T + kWarps - 1) / kWarps);
  by_width(E, [&](auto v) {
    st = launch_dependent(route_bwd_kernel<decltype(v)::value>, grid, kWarps * 32, 0, stream, a);
  });
  return st;
}

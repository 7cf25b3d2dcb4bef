// AdamW over many tensors in one launch, first and second moments in 32 or 8 bits.
//
//   g' = g * grad_scale
//   m  = beta1 m + (1 - beta1) g',      v = beta2 v + (1 - beta2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// in FP32 whatever the storage types.  The moments' operations are rounded one by one (no
// fused multiply-add, and for 8-bit moments the IEEE square root and reciprocal): a code on the
// edge between two values would else depend on how its FP32 value was computed, and a run
// would not be reproducible elsewhere.  The parameter's quotient, which no state depends on, takes
// the approximate instructions: root (2^-23) and reciprocal (2^-23), the constants' and three other
// roundings make up to 5.4e-7 of the update.  The parameter is rounded once to its type, and its
// optional BF16 copy (the working weight of the GEMMs) from the rounded parameter.
//
// 8-bit moments: 128 consecutive elements of a tensor share a scale.  m is held as E4M3
// codes of m / s with s = max|m| / 448.  sqrt(v), not v, is held the same way: the root
// halves the exponents' range, so E4M3's 2^17.8 covers v over 2^35; a v above zero never
// becomes zero (the smallest code is kept), since a lost v would blow up m / sqrt(v).
// A code's rounding is up to 1/16 of the value.  Rounding to nearest therefore drops every change
// of less than half a code against the block's maximum, and a step at rate 1 - beta changes m by
// that share of itself and sqrt(v) by half of it.  Where the rate is small the codes are rounded
// stochastically instead: up with the probability of the distance from the code below, so that
// the expected state follows the recurrence.  The 16 random bits an element are a hash of its index
// in the tensor and of the step (the splitmix64 sequence of Steele, Lea and Flood), so that a
// run repeats bit for bit, also after a resume.  Mean and standard deviation of sqrt(v) over its 32-bit
// value, normal gradients, stationary and six time constants after a tenfold fall of half of them
// (restated in numpy):
//     beta2        0.9           0.95          0.98          0.99          0.999
//     nearest      1.01 +- 0.07  1.06 +- 0.09  1.43 +- 0.25  1.31 +- 0.18  1.09 +- 0.22
//                  1.02 +- 0.08  1.34 +- 0.42  6.2 +- 5.1    6.1 +- 4.9    4.6 +- 3.9
//     stochastic   1.00 +- 0.09  1.00 +- 0.12  1.01 +- 0.15  1.01 +- 0.16  1.01 +- 0.16
//                  1.01 +- 0.11  1.01 +- 0.14  1.02 +- 0.17  1.02 +- 0.18  1.02 +- 0.19
// so it is used above beta2 = 0.95; below, nearest codes carry less noise.  Nearest codes of m
// keep its mean within 3% up to beta1 = 0.98 (0.9: 0.6%; 0.99: 5%; 0.999: off by its own size).
//
// Bound: HBM bytes (14 to 34 per element).  A CTA takes one chunk of 2048 elements, a
// thread 8 consecutive ones: every load of the chunk is in flight before the first use,
// and a block's maximum is a shuffle reduction over 16 lanes.  One CTA per chunk and not a
// persistent grid: 1216 CTAs of which 912 are resident left a third of the second round idle
// (153M elements, BF16 gradients and copies: 700 against 611 us with 32-bit, 495 against 415 us
// with 8-bit moments).  With 8-bit moments a warp computes half its time, too long for its
// loads alone to keep HBM busy, so each CTA also asks L2 for the chunk two per SM further:
// 427 -> 372 us or 6.6 TB/s (one per SM 422, three 375, four 379, six 382; with stochastic codes
// of sqrt(v) 432, of m too 502: bound by instructions).  32-bit moments, at 609
// us or 7.0 TB/s without, lose by it (643 at six per SM).  The tensors' table travels as a kernel
// parameter: no copy to the device, no state between calls.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "api_internal.h"
#include "ptx.cuh"

namespace dp {
namespace {

constexpr int kBlockElems = 128;   // 8-bit moments: elements per scale
constexpr int kChunkElems = 2048;  // elements per CTA step (256 threads x 8)
constexpr float kTop = 448.0f, kTinyMax = 1e-30f, kSmallest = 0.001953125f;  // E4M3: largest, smallest > 0
constexpr float kNormal = 0.015625f;                                            // E4M3: smallest normal
constexpr double kNearestBeta1 = 0.98, kNearestBeta2 = 0.95;  // 8 bits: stochastic codes above
constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;            // step of the splitmix64 sequence

struct Entry {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  int64_t n;
  int32_t flags;  // bit 0: p BF16, bit 1: g BF16, bit 2: every pointer 16-byte aligned
};

template <int MAX>
struct Table {
  Entry e[MAX];
  int64_t chunk0[MAX + 1];  // first chunk of each tensor
  int32_t count;
  int32_t ahead;  // 8-bit moments: chunks from one to the one it prefetches
  float beta1, one_beta1, beta2, one_beta2, eps, keep, root_scale, lr;
  float grad_scale;
  const float* grad_scale_ptr;
  uint64_t seed;             // of this step's random bits
  int32_t dither_m, dither_v;  // 8-bit moments: stochastic codes of m, of v's root
};

__device__ __forceinline__ float bf16_at(uint32_t w, int half) {
  return __uint_as_float(half ? (w & 0xFFFF0000u) : (w << 16));
}

// Eight values of a thread, from aligned storage or one by one (n of them exist).
__device__ __forceinline__ void load8(const void* base, int64_t at, bool bf16, bool fast, int n, float (&x)[8]) {
  if (fast) {
    if (bf16) {
      const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = bf16_at(u[j >> 1], j & 1);
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
      const float4 a = f[0], b = f[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = 0.0f;
    if (j < n)
      x[j] = bf16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at + j]) << 16)
                  : static_cast<const float*>(base)[at + j];
  }
}

__device__ __forceinline__ void store8(void* base, int64_t at, bool bf16, bool fast, int n, const float (&x)[8]) {
  if (fast) {
    if (bf16) {
      __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at),
             make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
    } else {
      float4* f = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
      __stcs(f, make_float4(x[0], x[1], x[2], x[3]));
      __stcs(f + 1, make_float4(x[4], x[5], x[6], x[7]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) {
      if (bf16)
        static_cast<uint16_t*>(base)[at + j] = static_cast<uint16_t>(pack_bf16x2(x[j], 0.0f) & 0xFFFFu);
      else
        static_cast<float*>(base)[at + j] = x[j];
    }
}

__device__ __forceinline__ uint2 load_codes(const void* base, int64_t at, bool fast, int n) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  if (fast) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(void* base, int64_t at, bool fast, int n, uint2 w) {
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if (fast) {
    __stcs(reinterpret_cast<uint2*>(p), w);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) p[j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
}

// Two FP32 operations in one instruction, each rounded to nearest.
struct Pair {
  uint64_t v;
  __device__ __forceinline__ float lo() const { return __uint_as_float(static_cast<uint32_t>(v)); }
  __device__ __forceinline__ float hi() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};
__device__ __forceinline__ Pair pair(float a, float b) {
  return {(static_cast<uint64_t>(__float_as_uint(b)) << 32) | __float_as_uint(a)};
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a.v), "l"(b.v));
  return {d};
}
// (two instructions: a paired sum of a paired product may be fused with it, into one rounding)
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  return pair(__fadd_rn(a.lo(), b.lo()), __fadd_rn(a.hi(), b.hi()));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a.v), "l"(b.v), "l"(c.v));
  return {d};
}

// Four E4M3 codes times their scale (squared: the second moment from its root).
__device__ __forceinline__ void decode4(uint32_t w, float s, bool square, float* x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t f16x2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f16x2) : "h"(static_cast<uint16_t>(w >> (16 * h))));
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(f16x2));
    Pair y = pair(lo, hi) * pair(s, s);
    if (square) y = y * y;
    x[2 * h] = y.lo();
    x[2 * h + 1] = y.hi();
  }
}

__device__ __forceinline__ uint32_t encode4(const float* x) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// The output function of splitmix64.
__host__ __device__ __forceinline__ uint64_t mix64(uint64_t z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// |x| up to 448 rounded to E4M3's values by 16 random bits: the 20 bits below the third of the mantissa get
// a uniform addend and are cut.  Values below the normal range have the spacing of the first
// normal binade and are rounded there.
__device__ __forceinline__ float stochastic(float x, uint32_t bits) {
  const float shift = fabsf(x) < kNormal ? kNormal : 0.0f;
  const uint32_t a = __float_as_uint(__fadd_rn(fabsf(x), shift));
  return copysignf(__uint_as_float((a + (bits << 4) + 8u) & 0xFFF00000u) - shift, x);
}
__device__ __forceinline__ void stochastic8(float (&x)[8], uint64_t counter) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t r = mix64(counter + h * kGamma);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[4 * h + j] = stochastic(x[4 * h + j], static_cast<uint32_t>(r >> (16 * j)) & 0xFFFFu);
  }
}

// max(|a|, |b|, |c|); a NaN wins.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// max |x| over the 16 lanes of a block, at least kTinyMax; a NaN wins.
__device__ __forceinline__ float block_max(const float (&x)[8]) {
  float m = max3_abs(x[0], x[1], kTinyMax);
#pragma unroll
  for (int j = 2; j < 8; j += 2) m = max3_abs(m, x[j], x[j + 1]);
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, m, d);
    m = max3_abs(m, o, o);
  }
  return m;
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Bring `bytes` (a multiple of 16, as is the address) into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// (8-bit moments: six CTAs an SM leave 40 registers a thread, and two words of it are spilled.)
template <int MAX, bool EIGHT, bool DITHER>
__global__ void __launch_bounds__(256, EIGHT ? 6 : 5) adamw_kernel(const __grid_constant__ Table<MAX> t) {
  const float gs = t.grad_scale_ptr ? t.grad_scale * __ldg(t.grad_scale_ptr) : t.grad_scale;
  const int64_t chunks = t.chunk0[t.count];
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    int lo = 0, hi = t.count - 1;  // the last tensor whose first chunk is <= c
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.chunk0[mid] <= c)
        lo = mid;
      else
        hi = mid - 1;
    }
    const Entry& e = t.e[lo];
    const int64_t at = (c - t.chunk0[lo]) * kChunkElems + static_cast<int64_t>(threadIdx.x) * 8;
    const int64_t left = e.n - at;
    const int n = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
    const bool fast = (e.flags & 4) != 0 && n == 8;
    const bool p16 = (e.flags & 1) != 0, g16 = (e.flags & 2) != 0;
    if (EIGHT && threadIdx.x < 4 && (e.flags & 4) != 0 && c + t.ahead + 1 < t.chunk0[lo + 1]) {
      // (a whole chunk of this tensor, of p, g, m or v)
      const int w = static_cast<int>(threadIdx.x);
      const int size = w == 0 ? (p16 ? 2 : 4) : w == 1 ? (g16 ? 2 : 4) : 1;
      prefetch_l2(static_cast<const char*>(w == 0 ? e.p : w == 1 ? e.g : w == 2 ? e.m : e.v) +
                      (c - t.chunk0[lo] + t.ahead) * kChunkElems * size,
                  size * kChunkElems);
    }
    float p[8], g[8], m[8], v[8];
    load8(e.p, at, p16, fast, n, p);
    load8(e.g, at, g16, fast, n, g);
    const int64_t blk = at / kBlockElems;
    if (EIGHT) {
      const uint2 mq = load_codes(e.m, at, fast, n), vq = load_codes(e.v, at, fast, n);
      const float ms = n > 0 ? e.ms[blk] : 0.0f, vs = n > 0 ? e.vs[blk] : 0.0f;
      decode4(mq.x, ms, false, m);
      decode4(mq.y, ms, false, m + 4);
      decode4(vq.x, vs, true, v);
      decode4(vq.y, vs, true, v + 4);
    } else {
      load8(e.m, at, false, fast, n, m);
      load8(e.v, at, false, fast, n, v);
    }
    float root[8];
    auto twice = [](float x) { return pair(x, x); };
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const Pair x = pair(g[j], g[j + 1]) * twice(gs);
      const Pair mm = pair(m[j], m[j + 1]) * twice(t.beta1) + x * twice(t.one_beta1);
      const Pair vv = pair(v[j], v[j + 1]) * twice(t.beta2) + (x * x) * twice(t.one_beta2);
      m[j] = mm.lo(), m[j + 1] = mm.hi();
      v[j] = vv.lo(), v[j + 1] = vv.hi();
      root[j] = EIGHT ? __fsqrt_rn(v[j]) : sqrt_approx(v[j]);
      root[j + 1] = EIGHT ? __fsqrt_rn(v[j + 1]) : sqrt_approx(v[j + 1]);
      const Pair den = fma2(pair(root[j], root[j + 1]), twice(t.root_scale), twice(t.eps));
      const Pair u = mm * pair(rcp_approx(den.lo()), rcp_approx(den.hi()));
      const Pair pp = fma2(u, twice(-t.lr), pair(p[j], p[j + 1]) * twice(t.keep));
      p[j] = pp.lo(), p[j + 1] = pp.hi();
    }
    store8(e.p, at, p16, fast, n, p);
    if (e.copy) store8(e.copy, at, true, fast, n, p);
    if (EIGHT) {
      if (n < 8) {  // elements past the end are no part of the block's maximum
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= n) m[j] = root[j] = 0.0f;
      }
      const float ma = block_max(m), va = block_max(root);
      const float mf = __fmul_rn(__frcp_rn(ma), kTop), vf = __fmul_rn(__frcp_rn(va), kTop);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const Pair mm = pair(m[j], m[j + 1]) * twice(mf), r = pair(root[j], root[j + 1]), vv = r * twice(vf);
        m[j] = mm.lo(), m[j + 1] = mm.hi();
        // (a root above zero is at least 1e-23: its floor is kSmallest, and zero's stays zero)
        const Pair floor = r * twice(1e30f);
        root[j] = fmaxf(vv.lo(), fminf(floor.lo(), kSmallest));
        root[j + 1] = fmaxf(vv.hi(), fminf(floor.hi(), kSmallest));
      }
      if (DITHER) {  // (a floor is a value of the grid's, which stays)
        const uint64_t counter = t.seed + static_cast<uint64_t>(at >> 3) * (4 * kGamma);
        if (t.dither_v) stochastic8(root, counter);
        if (t.dither_m) stochastic8(m, counter + 2 * kGamma);
      }
      store_codes(e.m, at, fast, n, make_uint2(encode4(m), encode4(m + 4)));
      store_codes(e.v, at, fast, n, make_uint2(encode4(root), encode4(root + 4)));
      if ((threadIdx.x & 15) == 0 && n > 0) {
        e.ms[blk] = __fmul_rn(ma, 1.0f / kTop);
        e.vs[blk] = __fmul_rn(va, 1.0f / kTop);
      }
    } else {
      store8(e.m, at, false, fast, n, m);
      store8(e.v, at, false, fast, n, v);
    }
  }
}

template <int MAX, bool EIGHT, bool DITHER = false>
cudaError_t launch_adamw(const dp_adamw_tensor* t, int64_t count, const dp_adamw_hyper& h, int sm_count,
                         cudaStream_t stream) {
  static_assert(sizeof(Table<MAX>) <= 32764, "kernel parameters");
  for (int64_t first = 0; first < count; first += MAX) {
    Table<MAX> tab;
    const int n = static_cast<int>(std::min<int64_t>(MAX, count - first));
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) {
      const dp_adamw_tensor& x = t[first + i];
      Entry& e = tab.e[i];
      e.p = x.param;
      e.g = x.grad;
      e.m = x.exp_avg;
      e.v = x.exp_avg_sq;
      e.ms = x.exp_avg_scale;
      e.vs = x.exp_avg_sq_scale;
      e.copy = static_cast<uint16_t*>(x.copy);
      e.n = x.grad == nullptr ? 0 : x.numel;
      const bool aligned = is_aligned16(x.param) && is_aligned16(x.grad) && is_aligned16(x.exp_avg) &&
                           is_aligned16(x.exp_avg_sq) && is_aligned16(x.copy);
      e.flags = (x.param_bf16 ? 1 : 0) | (x.grad_bf16 ? 2 : 0) | (aligned ? 4 : 0);
      tab.chunk0[i] = chunks;
      chunks += (e.n + kChunkElems - 1) / kChunkElems;
    }
    tab.chunk0[n] = chunks;
    if (chunks == 0) continue;
    tab.count = n;
    tab.ahead = 2 * sm_count;
    tab.beta1 = static_cast<float>(h.beta1);
    tab.one_beta1 = static_cast<float>(1.0 - h.beta1);
    tab.beta2 = static_cast<float>(h.beta2);
    tab.one_beta2 = static_cast<float>(1.0 - h.beta2);
    tab.eps = static_cast<float>(h.eps);
    tab.keep = static_cast<float>(1.0 - h.lr * h.weight_decay);
    tab.root_scale = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h.beta2, static_cast<double>(h.step))));
    tab.lr = static_cast<float>(h.lr / (1.0 - std::pow(h.beta1, static_cast<double>(h.step))));
    tab.grad_scale = static_cast<float>(h.grad_scale);
    tab.grad_scale_ptr = h.grad_scale_ptr;
    tab.seed = mix64(static_cast<uint64_t>(h.step) * kGamma);
    tab.dither_m = h.beta1 > kNearestBeta1;
    tab.dither_v = h.beta2 > kNearestBeta2;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(chunks, 0x7FFFFFFF));
    adamw_kernel<MAX, EIGHT, DITHER><<<grid, 256, 0, stream>>>(tab);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace dp

extern "C" dp_status dp_adamw_step(const dp_adamw_tensor* tensors, int64_t count, int state_bits,
                                   const dp_adamw_hyper* hyper, dp_stream stream) {
  using namespace dp;
  if (count < 0 || (count > 0 && tensors == nullptr) || hyper == nullptr) return DP_ERR_INVALID_ARG;
  if (state_bits != 8 && state_bits != 32) return DP_ERR_INVALID_ARG;
  const dp_adamw_hyper& h = *hyper;
  // (negated comparisons: a NaN is refused too)
  if (!(h.lr >= 0.0) || !(h.beta1 >= 0.0 && h.beta1 < 1.0) || !(h.beta2 >= 0.0 && h.beta2 < 1.0) || !(h.eps >= 0.0) ||
      !(h.weight_decay >= 0.0) || h.step < 1)
    return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(h.grad_scale_ptr) & 3) != 0) return DP_ERR_ALIGNMENT;
  for (int64_t i = 0; i < count; ++i) {
    const dp_adamw_tensor& t = tensors[i];
    if (t.numel < 0) return DP_ERR_INVALID_ARG;
    if (t.numel == 0 || t.grad == nullptr) continue;
    if (!t.param || !t.exp_avg || !t.exp_avg_sq) return DP_ERR_INVALID_ARG;
    if (state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return DP_ERR_INVALID_ARG;
    const uintptr_t p = t.param_bf16 ? 1 : 3, g = t.grad_bf16 ? 1 : 3, s = state_bits == 8 ? 0 : 3;
    if ((reinterpret_cast<uintptr_t>(t.param) & p) || (reinterpret_cast<uintptr_t>(t.grad) & g) ||
        (reinterpret_cast<uintptr_t>(t.exp_avg) & s) || (reinterpret_cast<uintptr_t>(t.exp_avg_sq) & s) ||
        (reinterpret_cast<uintptr_t>(t.exp_avg_scale) & 3) || (reinterpret_cast<uintptr_t>(t.exp_avg_sq_scale) & 3) ||
        (reinterpret_cast<uintptr_t>(t.copy) & 1))
      return DP_ERR_ALIGNMENT;
  }
  DeviceContext ctx;
  const dp_status st = device_context(&ctx);
  if (st != DP_OK) return st;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  // (a small table for few tensors: its launch carries 2 KB of parameters instead of 20)
  auto launch = [&](auto eight, auto dither) {
    return count <= 24 ? launch_adamw<24, decltype(eight)::value, decltype(dither)::value>(tensors, count, h, ctx.sm_count, str)
                       : launch_adamw<256, decltype(eight)::value, decltype(dither)::value>(tensors, count, h, ctx.sm_count, str);
  };
  cudaError_t e;
  if (state_bits == 32)
    e = launch(std::false_type(), std::false_type());
  else if (h.beta1 > kNearestBeta1 || h.beta2 > kNearestBeta2)
    e = launch(std::true_type(), std::true_type());
  else
    e = launch(std::true_type(), std::false_type());
  return e == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

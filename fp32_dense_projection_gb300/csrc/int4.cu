// Weights in 4 bits with a scale per group of G = 32, 64 or 128 values along the contraction:
//   w[n][k] = (q - z) s,   q in 0..15, two to a byte (the even k in the low half)
// z is 8, or a zero point of the group's own.
//
// Products of few rows, plain or grouped by expert:  Y[t][n] = sum over groups of s sum x[t][k] (q - z)
//
// Bound: the codes' bytes from HBM.  A CTA takes R rows of weights (16, 32 or 64) and a slab of the
// contraction, and asks for all of its codes at once with one bulk copy a row; several such CTAs
// share an SM, so there is nothing to pipeline by hand.  The CTAs of the slabs of one tile are a
// cluster and add their sums in rank order through shared memory.  A warp multiplies 16 rows of
// weights (the MMA's 16 rows) with 8 tokens (its 8 columns):
// - codes become BF16 by one OR (0x4300 | q is 128 + q) and one exact subtraction of 128 + z;
// - the MMA's sums run over one group and meet the group's scale in FP32, so the product is as
//   exact as with weights expanded in FP32.
// The order of the contraction within a group is free as long as both operands agree: a thread takes
// neighbouring codes, the words w of 8 codes, and reads pairs (i, i + 4) of a word with one mask;
// x is laid out in shared memory in that order, so that a thread's operands of two MMAs are 16
// neighbouring bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "api_internal.h"
#include "row_ops.cuh"

namespace dp {
namespace {

constexpr int kMaxInt4Experts = 1024;
constexpr int64_t kMaxInt4K = 32768;
constexpr int kThreads = 256, kWarpCount = kThreads / 32;
constexpr int kMaxSlabs = 8;  // CTAs of a cluster
constexpr uint32_t kAll = 0xffffffffu;

struct ProductArgs {
  const void* x;
  int64_t ldx;
  const uint8_t* q;  // [E][N][K / 2]
  const void* s;     // [E][N][K / G]
  const uint8_t* z;  // the same shape, or null
  int s_f32;
  const void* offsets;  // null: one group of all T rows
  int offsets64;
  int32_t E, T, N, K;
  int32_t R, slab, slabs, x_rows;  // rows of weights, contraction elements and CTAs a tile; rows of x in shared memory
  void* out;
  int64_t ldo;
  int out_f32;
  uint32_t* fault;
  uint64_t wait_ns;
};

// Shared memory of a CTA.
struct Layout {
  int32_t code_stride, x_stride, groups;
  int32_t x, scale, zero, red, red_stride, bytes;  // (codes at 0)
};

__host__ __device__ inline Layout layout_of(int G, int R, int slab, int x_rows, int tokens) {
  Layout l;
  // bytes of a row, padded so that the rows that a warp reads at a time lie in different banks: a
  // thread reads G / 8 bytes, the four threads of a row G / 2
  l.code_stride = (slab / 2 + 127) / 128 * 128 + G / 2;
  l.x_stride = slab * 2 + 64;
  l.groups = slab / G;
  l.red_stride = R + 4;
  l.x = R * l.code_stride;
  l.scale = l.x + x_rows * l.x_stride;
  l.zero = l.scale + R * l.groups * 4;
  l.red = (l.zero + R * l.groups * 2 + 15) / 16 * 16;
  l.bytes = l.red + kWarpCount / (R / 16) * tokens * l.red_stride * 4;
  return l;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes i and i + 4 of a word of 8, less their zero point (`zero`: twice 128 + z in BF16; exact).
__device__ __forceinline__ uint32_t code_pair(uint32_t word, int i, uint32_t zero) {
  const uint32_t v = ((word >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&zero));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Where the 8 elements of chunk c (0..15) of a block of 128 lie in shared memory: the chunk that
// thread t of a row's four needs for its word j is at 4 j + t.
template <int G>
__device__ __forceinline__ int chunk_place(int c) {
  if (G == 128) return (c & 3) * 4 + (c >> 2);
  if (G == 64) return ((c >> 3) * 2 + (c & 1)) * 4 + ((c >> 1) & 3);
  return c;
}

__device__ __forceinline__ float ld_float_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// The group's rows [lo, hi): offsets clamped to [0, T] and to the running maximum; all threads
// call it.  What had to be clamped is reported by the CTAs of the first tile.
__device__ __forceinline__ void group_rows(const ProductArgs& a, int e, int32_t& lo, int32_t& hi, int32_t& first, int32_t& last) {
  __shared__ int32_t most[3][kWarpCount];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  auto at = [&](int i) {
    return a.offsets64 ? static_cast<const int64_t*>(a.offsets)[i] : static_cast<int64_t>(static_cast<const int32_t*>(a.offsets)[i]);
  };
  int32_t m[3] = {0, 0, 0};  // maxima over offsets up to e, up to e + 1, all
  bool bad = false;
  int64_t before = 0;
  for (int i = tid; i <= a.E; i += kThreads) {
    const int64_t raw = at(i);
    if (i > 0) before = at(i - 1);
    bad = bad || raw < 0 || raw > a.T || (i > 0 && raw < before);
    const int32_t v = static_cast<int32_t>(raw < 0 ? 0 : raw > a.T ? a.T : raw);
    m[2] = max(m[2], v);
    if (i <= e + 1) m[1] = max(m[1], v);
    if (i <= e) m[0] = max(m[0], v);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    m[i] = __reduce_max_sync(kAll, m[i]);
    if (lane == 0) most[i][warp] = m[i];
  }
  if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(a.fault, kFaultOffsets);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int w = 0; w < kWarpCount; ++w) m[i] = max(m[i], most[i][w]);
  lo = m[0], hi = m[1], last = m[2];
  const int64_t raw = at(0);
  first = static_cast<int32_t>(raw < 0 ? 0 : raw > a.T ? a.T : raw);
}

__device__ __forceinline__ void store_out(const ProductArgs& a, int32_t t, int32_t n, float v) {
  const int64_t i = t * a.ldo + n;
  if (a.out_f32)
    static_cast<float*>(a.out)[i] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(v);
}

template <int G, int NT>
__global__ void __launch_bounds__(kThreads) int4_product_kernel(const __grid_constant__ ProductArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t barrier;
  constexpr int TT = 8 * NT, GROUPS = 128 / G, STEPS = G / 32;
  const Layout l = layout_of(G, a.R, a.slab, a.x_rows, TT);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x), n0 = static_cast<int>(blockIdx.y) * a.R, e = static_cast<int>(blockIdx.z);
  const int rows = min(a.R, a.N - n0), k0 = rank * a.slab, length = min(a.slab, a.K - k0);
  int32_t lo = 0, hi = a.T;
  if (a.offsets != nullptr) {
    int32_t first, last;
    group_rows(a, e, lo, hi, first, last);
    if (rank == 0) {  // rows of no group are zero
      auto zero = [&](int32_t from, int32_t to) {
        const int64_t count = static_cast<int64_t>(to - from) * rows;
        for (int64_t i = tid; i < count; i += kThreads)
          store_out(a, from + static_cast<int32_t>(i / rows), n0 + static_cast<int32_t>(i % rows), 0.0f);
      };
      if (e == 0) zero(0, first);
      if (e == a.E - 1) zero(last, a.T);
    }
  }
  if (lo >= hi) return;  // (the whole cluster)
  const uint32_t bar = smem_addr(&barrier), base = smem_addr(smem);
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int64_t row0 = static_cast<int64_t>(e) * a.N + n0;
  if (warp == 0) {
    if (lane == 0) mbar_expect_tx(bar, static_cast<uint32_t>(rows) * (length / 2));
    __syncwarp();
    for (int r = lane; r < rows; r += 32)
      bulk_load(base + r * l.code_stride, a.q + (row0 + r) * (a.K / 2) + k0 / 2, length / 2, bar);
  }
  float* scale = reinterpret_cast<float*>(smem + l.scale);
  uint16_t* zero = reinterpret_cast<uint16_t*>(smem + l.zero);
  {
    const int groups = a.K / G, g0 = k0 / G;
    for (int i = tid; i < a.R * l.groups; i += kThreads) {
      const int r = i / l.groups, g = g0 + i % l.groups;
      float s = 0.0f;
      uint32_t z = 8;
      if (r < rows && g < groups) {
        const int64_t at = (row0 + r) * groups + g;
        s = a.s_f32 ? __ldg(static_cast<const float*>(a.s) + at)
                    : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.s) + at)) << 16);
        if (a.z != nullptr) z = __ldg(a.z + at) & 15u;
      }
      scale[i % l.groups * a.R + r] = s;  // [group][row]: the rows that a warp reads at a time lie side by side
      zero[i % l.groups * a.R + r] = static_cast<uint16_t>(0x4300u | z);
    }
  }
  const int tiles = a.R / 16, ways = kWarpCount / tiles;  // the warps' 16-row tiles, and how many share a tile's slab
  const int tile = warp % tiles, way = warp / tiles, g = lane >> 2, t = lane & 3;
  const int blocks = (length + 127) / 128;
  float* red = reinterpret_cast<float*>(smem + l.red);
  bool loaded = false;
  for (int32_t tok = lo; tok < hi; tok += TT) {
    const int count = min(TT, hi - tok);
    // x, in the order of the codes' pairs; zeros behind the contraction's end
    for (int i = tid; i < count * (blocks * 16); i += kThreads) {
      const int r = i / (blocks * 16), c = i % (blocks * 16);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (c * 8 < length)
        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + (tok + r) * a.ldx + k0 + c * 8));
      uint4 p;
      p.x = __byte_perm(v.x, v.z, 0x5410);
      p.y = __byte_perm(v.x, v.z, 0x7632);
      p.z = __byte_perm(v.y, v.w, 0x5410);
      p.w = __byte_perm(v.y, v.w, 0x7632);
      *reinterpret_cast<uint4*>(smem + l.x + r * l.x_stride + (c >> 4) * 256 + chunk_place<G>(c & 15) * 16) = p;
    }
    if (!loaded) {
      loaded = true;
      if (!mbar_wait(bar, 0, a.wait_ns)) {
        atomicOr(a.fault, kFaultProducerWait);
        mbar_wait(bar, 0, a.wait_ns);
      }
    }
    __syncthreads();
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
    const uint8_t* codes = smem + (tile * 16 + g) * l.code_stride + t * (G / 8);
    const uint8_t* xs = smem + l.x + g * l.x_stride + t * 16;
    for (int blk = way; blk < blocks; blk += ways) {
#pragma unroll
      for (int grp = 0; grp < GROUPS; ++grp) {
        const int gi = blk * GROUPS + grp;
        uint32_t wa[STEPS], wb[STEPS];
        const uint8_t* p = codes + gi * (G / 2);
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          wa[j] = reinterpret_cast<const uint32_t*>(p)[j];
          wb[j] = reinterpret_cast<const uint32_t*>(p + 8 * l.code_stride)[j];
        }
        const int at = gi * a.R + tile * 16 + g;
        const uint32_t za = zero[at] * 0x10001u, zb = zero[at + 8] * 0x10001u;
        const float fa = scale[at], fb = scale[at + 8];
        float c[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          uint4 x[NT];
#pragma unroll
          for (int i = 0; i < NT; ++i)
            x[i] = i * 8 + g < count ? *reinterpret_cast<const uint4*>(xs + i * 8 * l.x_stride + blk * 256 + (grp * STEPS + j) * 64)
                                     : make_uint4(0, 0, 0, 0);
          const uint32_t a0 = code_pair(wa[j], 0, za), a1 = code_pair(wb[j], 0, zb), a2 = code_pair(wa[j], 1, za),
                         a3 = code_pair(wb[j], 1, zb);
          const uint32_t a4 = code_pair(wa[j], 2, za), a5 = code_pair(wb[j], 2, zb), a6 = code_pair(wa[j], 3, za),
                         a7 = code_pair(wb[j], 3, zb);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma_16x8x16(c[i], a0, a1, a2, a3, x[i].x, x[i].y);
            mma_16x8x16(c[i], a4, a5, a6, a7, x[i].z, x[i].w);
          }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[i][0] = fmaf(c[i][0], fa, acc[i][0]);
          acc[i][1] = fmaf(c[i][1], fa, acc[i][1]);
          acc[i][2] = fmaf(c[i][2], fb, acc[i][2]);
          acc[i][3] = fmaf(c[i][3], fb, acc[i][3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float* d = red + (way * TT + i * 8 + 2 * t) * l.red_stride + tile * 16 + g;
      d[0] = acc[i][0];
      d[l.red_stride] = acc[i][1];
      d[8] = acc[i][2];
      d[l.red_stride + 8] = acc[i][3];
    }
    __syncthreads();
    // the ways in order; then, where the contraction has more slabs, the cluster's ranks in order
    for (int i = tid; i < count * a.R; i += kThreads) {
      const int r = i / a.R, n = i % a.R;
      float s = red[r * l.red_stride + n];
      for (int w = 1; w < ways; ++w) s += red[(w * TT + r) * l.red_stride + n];
      if (a.slabs > 1)
        red[r * l.red_stride + n] = s;
      else if (n < rows)
        store_out(a, tok + r, n0 + n, s);
    }
    if (a.slabs > 1) {
      cluster_sync();
      const uint32_t mine = smem_addr(red);
      for (int i = rank * kThreads + tid; i < count * a.R; i += a.slabs * kThreads) {
        const int r = i / a.R, n = i % a.R;
        float s = 0.0f;
        for (int w = 0; w < a.slabs; ++w) s += ld_float_cluster(map_shared_rank(mine + (r * l.red_stride + n) * 4, w));
        if (n < rows) store_out(a, tok + r, n0 + n, s);
      }
      cluster_sync();
    } else {
      __syncthreads();
    }
  }
}

// ---------------------------------------------------- quantisation, expansion

struct CodeArgs {
  const void* w;
  int64_t ldw;
  uint8_t* q;
  void* s;
  uint8_t* z;
  int s_f32;
  int64_t rows;
  int32_t K, G;
  void* out;
  int64_t ldo;
};

constexpr float kTinyScale = 1e-30f;  // a group of zeros still has a scale to divide by

// A thread takes 8 neighbouring values, the G / 8 threads of a group share their range.
template <bool WF32>
__global__ void __launch_bounds__(256) int4_quantize_kernel(const __grid_constant__ CodeArgs a) {
  const int per_row = a.K / 8, lane = static_cast<int>(threadIdx.x) & 31, width = a.G / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const bool live = i < a.rows * per_row;  // (a row is whole groups: the threads of a group live together)
  const int64_t row = live ? i / per_row : 0;
  const int at = static_cast<int>(live ? i % per_row : 0) * 8;
  float w[8];
  if (live) {
    load8<WF32>(a.w, row * a.ldw + at, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.0f;
  }
  float lo = 0.0f, hi = 0.0f;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, w[j]);
    hi = fmaxf(hi, w[j]);
    nan = nan || w[j] != w[j];
  }
  for (int d = 1; d < width; d <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(kAll, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(kAll, hi, d));
    nan = __shfl_xor_sync(kAll, static_cast<int>(nan), d) || nan;
  }
  float s = a.z != nullptr ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(-lo, hi), 7.0f);
  s = nan ? __uint_as_float(0x7FC00000u) : fmaxf(s, kTinyScale);
  if (!a.s_f32) s = __bfloat162float(__float2bfloat16_rn(s));
  float z = 8.0f;
  if (a.z != nullptr) z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
  if (!live) return;
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float c = fminf(fmaxf(rintf(__fdiv_rn(w[j], s)) + z, 0.0f), 15.0f);  // (NaN: 0)
    word |= static_cast<uint32_t>(c) << (4 * j);
  }
  *reinterpret_cast<uint32_t*>(a.q + (row * a.K + at) / 2) = word;
  if (lane % width == 0) {
    const int64_t g = row * (a.K / a.G) + at / a.G;
    if (a.s_f32)
      static_cast<float*>(a.s)[g] = s;
    else
      static_cast<__nv_bfloat16*>(a.s)[g] = __float2bfloat16_rn(s);
    if (a.z != nullptr) a.z[g] = static_cast<uint8_t>(z);
  }
}

template <bool OF32>
__global__ void __launch_bounds__(256) int4_expand_kernel(const __grid_constant__ CodeArgs a) {
  const int per_row = a.K / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.rows * per_row) return;
  const int64_t row = i / per_row;
  const int at = static_cast<int>(i % per_row) * 8;
  const int64_t g = row * (a.K / a.G) + at / a.G;
  const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(a.q + (row * a.K + at) / 2));
  const float s = a.s_f32 ? __ldg(static_cast<const float*>(a.s) + g)
                          : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.s) + g)) << 16);
  const float z = a.z != nullptr ? static_cast<float>(__ldg(a.z + g) & 15) : 8.0f;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (static_cast<float>((word >> (4 * j)) & 15u) - z) * s;
  store8<OF32>(a.out, row * a.ldo + at, v);
}

// ----------------------------------------------------------------------- host

template <typename F>
void by_group(int64_t G, F f) {
  if (G == 32)
    f(std::integral_constant<int, 32>());
  else if (G == 64)
    f(std::integral_constant<int, 64>());
  else
    f(std::integral_constant<int, 128>());
}

template <typename F>
void by_tokens(int nt, F f) {
  if (nt == 1)
    f(std::integral_constant<int, 1>());
  else if (nt == 2)
    f(std::integral_constant<int, 2>());
  else
    f(std::integral_constant<int, 4>());
}

constexpr int kMaxShared = 227 * 1024 - 1024;

struct Int4Plan {
  int nt, R, slab, slabs, x_rows, bytes;
};

// How a product is cut: tokens a pass, rows of weights and contraction elements a CTA.
Int4Plan plan_int4(int64_t E, int64_t T, int64_t N, int64_t K, int64_t G, bool grouped) {
  Int4Plan p;
  const int64_t tokens = grouped ? (T + E - 1) / E : T;
  p.nt = tokens <= 8 ? 1 : tokens <= 16 ? 2 : 4;
  p.R = 16;
  int64_t slabs = std::min<int64_t>(kMaxSlabs, (K + 2047) / 2048);
  for (;;) {
    p.slab = static_cast<int>(((K + slabs - 1) / slabs + 127) / 128 * 128);
    p.slabs = static_cast<int>((K + p.slab - 1) / p.slab);
    p.x_rows = static_cast<int>(std::min<int64_t>(T, 8 * p.nt));
    p.bytes = layout_of(static_cast<int>(G), p.R, p.slab, p.x_rows, 8 * p.nt).bytes;
    if (p.bytes <= kMaxShared) return p;
    if (slabs < kMaxSlabs)
      ++slabs;
    else
      p.nt /= 2;
  }
}

bool flag(int v) { return v == 0 || v == 1; }

dp_status check_codes(const void* q, const void* s, const void* z, int s_f32, int64_t rows, int64_t K, int64_t G) {
  if (!flag(s_f32) || rows < 0 || K < 1) return DP_ERR_INVALID_ARG;
  if ((G != 32 && G != 64 && G != 128) || K % G != 0 || K > 0x7FFFFF00) return DP_ERR_UNSUPPORTED;
  if (rows > 0 && (q == nullptr || s == nullptr)) return DP_ERR_INVALID_ARG;
  if (!is_aligned16(q) || (reinterpret_cast<uintptr_t>(s) & (s_f32 ? 3 : 1)) != 0) return DP_ERR_ALIGNMENT;
  return DP_OK;
}

dp_status run_product(const void* x, int64_t ldx, const void* q, const void* s, int s_f32, const void* z, int64_t G,
                      const void* offsets, int offset_bits, void* out, int64_t ldo, int64_t E, int64_t T, int64_t N, int64_t K,
                      int out_f32, dp_stream stream) {
  if (!flag(out_f32) || E < 0 || T < 0 || N < 1 || K < 1) return DP_ERR_INVALID_ARG;
  if (offset_bits != 32 && offset_bits != 64) return DP_ERR_INVALID_ARG;
  dp_status st = check_codes(q, s, z, s_f32, E * N, K, G);
  if (st != DP_OK) return st;
  if (N % 8 != 0 || N > 0x7FFFF || K > kMaxInt4K || E > kMaxInt4Experts || T > 0x7FFFFFFF - 256) return DP_ERR_UNSUPPORTED;
  if ((st = check_operand(x, T, K, &ldx, 2)) != DP_OK) return st;
  if ((st = check_operand(out, T, N, &ldo, out_f32 ? 4 : 2)) != DP_OK) return st;
  if ((reinterpret_cast<uintptr_t>(offsets) & (offset_bits / 8 - 1)) != 0) return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (E == 0) {
    const size_t size = out_f32 ? 4 : 2;
    return cudaMemset2DAsync(out, ldo * size, 0, N * size, T, str) == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
  }
  const Int4Plan p = plan_int4(E, T, N, K, G, offsets != nullptr);
  ProductArgs a = {};
  a.x = x, a.ldx = ldx, a.q = static_cast<const uint8_t*>(q), a.s = s, a.z = static_cast<const uint8_t*>(z), a.s_f32 = s_f32;
  a.offsets = offsets, a.offsets64 = offset_bits == 64;
  a.E = static_cast<int32_t>(E), a.T = static_cast<int32_t>(T), a.N = static_cast<int32_t>(N), a.K = static_cast<int32_t>(K);
  a.R = p.R, a.slab = p.slab, a.slabs = p.slabs, a.x_rows = p.x_rows;
  a.out = out, a.ldo = ldo, a.out_f32 = out_f32, a.fault = ctx.fault, a.wait_ns = kWaitLimitNs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.slabs, static_cast<unsigned>((N + p.R - 1) / p.R), static_cast<unsigned>(E));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.bytes;
  cfg.stream = str;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.slabs, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t err = cudaSuccess;
  by_group(G, [&](auto g) {
    by_tokens(p.nt, [&](auto nt) {
      err = cudaLaunchKernelEx(&cfg, int4_product_kernel<decltype(g)::value, decltype(nt)::value>, a);
    });
  });
  return err == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

}  // namespace

cudaError_t set_attributes_int4() {
  cudaError_t e = cudaSuccess;
  for (int G = 32; G <= 128; G *= 2)
    by_group(G, [&](auto g) {
      for (int n = 1; n <= 4; n *= 2)
        by_tokens(n, [&](auto nt) {
          if (e == cudaSuccess)
            e = cudaFuncSetAttribute(int4_product_kernel<decltype(g)::value, decltype(nt)::value>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
        });
    });
  return e;
}

}  // namespace dp

extern "C" dp_status dp_int4_quantize(const void* w, int64_t ldw, int w_f32, int64_t rows, int64_t K, int64_t group, void* q,
                                      void* s, int s_f32, void* z, dp_stream stream) {
  using namespace dp;
  if (!flag(w_f32)) return DP_ERR_INVALID_ARG;
  dp_status st = check_codes(q, s, z, s_f32, rows, K, group);
  if (st == DP_OK) st = check_operand(w, rows, K, &ldw, w_f32 ? 4 : 2);
  if (st != DP_OK) return st;
  const int64_t blocks = (rows * (K / 8) + 255) / 256;
  if (blocks > 0x7FFFFFFF) return DP_ERR_UNSUPPORTED;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (rows == 0) return DP_OK;
  CodeArgs a = {};
  a.w = w, a.ldw = ldw, a.q = static_cast<uint8_t*>(q), a.s = s, a.z = static_cast<uint8_t*>(z), a.s_f32 = s_f32;
  a.rows = rows, a.K = static_cast<int32_t>(K), a.G = static_cast<int32_t>(group);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (w_f32)
    int4_quantize_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, str>>>(a);
  else
    int4_quantize_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, str>>>(a);
  return cudaGetLastError() == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

extern "C" dp_status dp_int4_dequantize(const void* q, const void* s, int s_f32, const void* z, int64_t rows, int64_t K,
                                        int64_t group, void* w, int64_t ldw, dp_out_dtype out, dp_stream stream) {
  using namespace dp;
  const int code = static_cast<int>(out);
  if (!flag(code)) return DP_ERR_INVALID_ARG;
  dp_status st = check_codes(q, s, z, s_f32, rows, K, group);
  if (st == DP_OK) st = check_operand(w, rows, K, &ldw, code ? 4 : 2);
  if (st != DP_OK) return st;
  const int64_t blocks = (rows * (K / 8) + 255) / 256;
  if (blocks > 0x7FFFFFFF) return DP_ERR_UNSUPPORTED;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (rows == 0) return DP_OK;
  CodeArgs a = {};
  a.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q)), a.s = const_cast<void*>(s);
  a.z = const_cast<uint8_t*>(static_cast<const uint8_t*>(z)), a.s_f32 = s_f32;
  a.rows = rows, a.K = static_cast<int32_t>(K), a.G = static_cast<int32_t>(group), a.out = w, a.ldo = ldw;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (code)
    int4_expand_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, str>>>(a);
  else
    int4_expand_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, str>>>(a);
  return cudaGetLastError() == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

extern "C" dp_status dp_gemm_fwd_int4(const void* X, int64_t ldx, const void* Wq, const void* Ws, int s_f32, const void* Wz,
                                      int64_t group, void* Y, int64_t ldy, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                                      dp_stream stream) {
  return dp::run_product(X, ldx, Wq, Ws, s_f32, Wz, group, nullptr, 32, Y, ldy, 1, T, N, K, static_cast<int>(out), stream);
}

extern "C" dp_status dp_gemm_fwd_int4_grouped(const void* X, int64_t ldx, const void* Wq, const void* Ws, int s_f32,
                                              const void* Wz, int64_t group, const void* offsets, int offset_bits, void* Y,
                                              int64_t ldy, int64_t E, int64_t T, int64_t N, int64_t K, dp_out_dtype out,
                                              dp_stream stream) {
  if (offsets == nullptr && E > 0) return DP_ERR_INVALID_ARG;
  return dp::run_product(X, ldx, Wq, Ws, s_f32, Wz, group, offsets, offset_bits, Y, ldy, E, T, N, K, static_cast<int>(out), stream);
}

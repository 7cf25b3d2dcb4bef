// What the kernels that go over rows share: eight neighbouring elements a thread (16 bytes of
// BF16, 32 of FP32) as FP32 values, and sums over the threads of a row.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace dp {

// Eight elements as they lie in memory.
template <bool F32>
struct Raw8 {
  uint4 v[F32 ? 2 : 1];
};

// (COHERENT: behind pdl_wait.  Loads of read-only data ask that nobody writes it while the kernel lives, and the grid before
// may, up to there.)
template <bool F32, bool COHERENT = false>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* base, int64_t at) {
  Raw8<F32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.v[i] = COHERENT ? p[i] : __ldg(p + i);
  return r;
}

template <bool F32>
__device__ __forceinline__ Raw8<F32> zero_raw8() {
  Raw8<F32> r;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.v[i] = make_uint4(0, 0, 0, 0);
  return r;
}

template <bool F32>
__device__ __forceinline__ void store_raw8(void* base, int64_t at, const Raw8<F32>& r) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) p[i] = r.v[i];
}

template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float (&x)[8]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F32) {
      x[2 * i] = __uint_as_float(w[2 * i]);
      x[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
    } else {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <bool F32, bool COHERENT = false>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
  unpack8<F32>(load_raw8<F32, COHERENT>(base, at), x);
}

// Eight FP32 values, rounded once to BF16 (nearest-even) or stored as they are.
template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&x)[8]) {
  uint4* p = reinterpret_cast<uint4*>(static_cast<char*>(base) + at * (F32 ? 4 : 2));
  if (F32) {
    p[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    p[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  } else {
    p[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
}

// Two FP32 values in one register pair, and the packed operations on them (each rounded as two
// ordinary ones).
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
  return {(static_cast<uint64_t>(__float_as_uint(hi)) << 32) | __float_as_uint(lo)};
}
__device__ __forceinline__ Two twice(float x) { return two(x, x); }
__device__ __forceinline__ float lo(Two a) { return __uint_as_float(static_cast<uint32_t>(a.v)); }
__device__ __forceinline__ float hi(Two a) { return __uint_as_float(static_cast<uint32_t>(a.v >> 32)); }
__device__ __forceinline__ Two operator+(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  Two d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, Two (&x)[4]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = F32 ? two(__uint_as_float(w[F32 ? 2 * i : 0]), __uint_as_float(w[F32 ? 2 * i + 1 : 0]))
               : two(__uint_as_float(w[F32 ? 0 : i] << 16), __uint_as_float(w[F32 ? 0 : i] & 0xFFFF0000u));
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t at, const Two (&x)[4]) {
  const float v[8] = {lo(x[0]), hi(x[0]), lo(x[1]), hi(x[1]), lo(x[2]), hi(x[2]), lo(x[3]), hi(x[3])};
  store8<F32>(base, at, v);
}

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Eight elements each of CH pieces of a thread's rows, DEPTH rows ahead, in shared memory that only
// its warp touches (so nobody waits at a barrier for them): [row][piece][unit][16 bytes of `stride` threads].  A piece's column is
// 8 t + 8 i threads-per-row.  FP32 pieces are 32 bytes: a warp's (or a shorter row's) threads copy the
// 16-byte units in their order, half of them at a time, so that each request is whole sectors
// (each thread its own 32 bytes asked twice for every sector: 3.9 TB/s in the forward pass of 1024
// columns), and their places are exchanged within every second eight, so that threads read
// their own two from different banks.
// (STRIDE: threads, 0 for the block's own: blocks of fewer than the most then leave room for others on their SM.)
template <bool F32, int CH, int DEPTH, int STRIDE>
struct Ahead {
  static constexpr int UNITS = F32 ? 2 : 1;
  uint4* base;
  int stride;
  const char* next;  // this thread's first 16 bytes of the row to ask for next
  int64_t step;
  uint32_t inside = 0;      // which of its units are inside the row
  int width, m, piece_bytes;  // threads that share a row, up to a warp; this one's place among them; from piece to piece

  // Rows of `cols` columns of x from `row` on, `rows` apart; t: this thread's place in its row.  What lies behind the columns is zero.
  __device__ __forceinline__ Ahead(float4* at, int tpr, int t, const void* x, int64_t ld, int64_t row, int64_t rows, int cols)
      : base(reinterpret_cast<uint4*>(at)), stride(STRIDE > 0 ? STRIDE : static_cast<int>(blockDim.x)), width(tpr < 32 ? tpr : 32), m(static_cast<int>(threadIdx.x) & (width - 1)) {
    constexpr int SIZE = F32 ? 4 : 2;
    base += (static_cast<int>(threadIdx.x) - m) * UNITS;
    const int first = F32 ? (t - m) * 8 + m * 4 : t * 8;
    next = static_cast<const char*>(x) + (row * ld + first) * SIZE;
    step = rows * ld * SIZE;
    piece_bytes = tpr * 8 * SIZE;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int h = 0; h < UNITS; ++h) {
        if (first + i * tpr * 8 + h * width * 4 < cols) {
          inside |= 1u << (i * UNITS + h);
        } else {
#pragma unroll
          for (int slot = 0; slot < DEPTH; ++slot) *unit(slot, i, h * width + m) = make_uint4(0, 0, 0, 0);
        }
      }
  }
  __device__ __forceinline__ int units() const { return DEPTH * CH * UNITS * stride; }
  __device__ __forceinline__ uint4* unit(int slot, int i, int u) const {
    return base + (slot * CH + i) * UNITS * stride + (F32 ? (u & ~7) | ((u ^ (u >> 3)) & 7) : u);
  }
  // Ask for piece i of the next row, if there is one.
  __device__ __forceinline__ void load(int slot, int i, bool row) const {
#pragma unroll
    for (int h = 0; h < UNITS; ++h)
      if (row && (inside >> (i * UNITS + h) & 1)) copy16_async(smem_addr(unit(slot, i, h * width + m)), next + (i * piece_bytes + h * width * 16));
  }
  __device__ __forceinline__ void advance() { next += step; }
  // (behind copies_wait and, FP32, __syncwarp)
  __device__ __forceinline__ Raw8<F32> take(int slot, int i) const {
    Raw8<F32> r;
#pragma unroll
    for (int h = 0; h < UNITS; ++h) r.v[h] = *unit(slot, i, UNITS * m + h);
    return r;
  }
};

// Sums of N values over groups of `tpr` consecutive threads (a power of two, or whole warps; all threads of a
// group call this).  Groups of more than a warp meet in `part`
// [2][32][N], used by turns, and at a barrier of their own: one a sum, and groups do not wait for others.
template <int N>
struct GroupSum {
  float (*part)[32][N];
  int tpr, warps, from, turn = 0;  // from: the warp whose sum this lane takes, or -1
  uint32_t barrier;
  __device__ __forceinline__ GroupSum(float (*p)[32][N], int threads_per_row) : part(p), tpr(threads_per_row), warps(tpr >> 5) {
    const int group = static_cast<int>(threadIdx.x) / tpr;
    int span = 1;
    while (span < warps) span *= 2;
    from = static_cast<int>(threadIdx.x) & (span - 1);
    from = from < warps ? group * warps + from : -1;
    barrier = 1 + group;
  }
  __device__ __forceinline__ void operator()(float (&v)[N]) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      if (d >= tpr) break;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    }
    if (tpr <= 32) return;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[turn][threadIdx.x >> 5][i] = v[i];
    }
    named_sync(barrier, static_cast<uint32_t>(tpr));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = from < 0 ? 0.0f : part[turn][from][i];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      if (d >= warps) break;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    }
    turn ^= 1;
  }
};

}  // namespace dp

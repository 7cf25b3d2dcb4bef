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

template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw8(const void* base, int64_t at) {
  Raw8<F32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.v[i] = __ldg(p + i);
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

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&x)[8]) {
  unpack8<F32>(load_raw8<F32>(base, at), x);
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

// Sums of N values over groups of `tpr` consecutive threads (a power of two; the block's threads
// are a multiple of it and all call this).  Groups of more than a warp meet in `part`
// [2][32][N], used by turns: one barrier a sum.
template <int N>
struct GroupSum {
  float (*part)[32][N];
  int tpr, turn = 0;
  __device__ __forceinline__ GroupSum(float (*p)[32][N], int threads_per_row) : part(p), tpr(threads_per_row) {}
  __device__ __forceinline__ void operator()(float (&v)[N]) {
    const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
    const int width = tpr < 32 ? tpr : 32;
    for (int d = 1; d < width; d <<= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    }
    if (tpr <= 32) return;
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) part[turn][warp][i] = v[i];
    }
    __syncthreads();
    const int warps = tpr >> 5, from = warp / warps * warps + lane % warps;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = part[turn][from][i];
    for (int d = 1; d < warps; d <<= 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
    }
    turn ^= 1;
  }
};

}  // namespace dp

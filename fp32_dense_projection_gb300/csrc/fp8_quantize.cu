// Quantisation to 8-bit floating point with one scale per 128 values:
//   a = max(max |x| over the block, 1e-30),  s = a / top,  q = rn(x * (top / a)),
// top the format's largest value (448 E4M3, 57344 E5M2).  A block is 128 values of a row
// (scales for contractions along the row), of a column (contractions along the rows: the
// weight gradient), or 128 x 128 (weights).  Row and column blocks together come from one
// read of x.
//
// Bound: HBM bytes (2 or 4 read, 1 or 2 written per value).  One CTA takes a 128 x 128 tile
// and keeps it in registers (64 values a thread: 16 rows x 4 columns), so x is read once
// whatever the blocks; a thread's 16 loads are in flight together.  A row's maximum is a
// shuffle reduction of one warp, a column's a maximum over the warps in shared memory.
//
// Maxima are taken on the bits of |x| as integers: that order puts NaN above infinity, so
// a block with a NaN gets a NaN scale (and one with an infinity an infinite scale, whose
// products are NaN) instead of hiding it.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_internal.h"
#include "ptx.cuh"

namespace dp {
namespace {

constexpr float kTinyMax = 1e-30f;  // keeps top / a finite for blocks of zeros

struct QuantArgs {
  const void* x;
  int64_t ldx;
  int32_t rows, cols, blk_cols;  // blk_cols = ceil(cols / 128)
  uint8_t* q;                    // row or 128 x 128 blocks
  int64_t ldq;
  float* s;
  int64_t s_row, s_col;          // strides of the row / 128 x 128 scales: [rows or row blocks][column blocks]
  uint8_t* qc;                   // column blocks
  int64_t ldqc;
  float* sc;
  int64_t sc_row;                // stride between row blocks of the column scales [row blocks][cols]
};

enum QuantMode { kRow = 0, kCol = 1, kBlock = 2, kBoth = 3 };

template <bool E5M2>
__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  if (E5M2) {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  } else {
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  }
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The block's maximum with its lower bound (a NaN stays).
__device__ __forceinline__ float block_max(uint32_t bits) {
  const float a = __uint_as_float(bits);
  return a < kTinyMax ? kTinyMax : a;
}

template <int MODE, bool F32, bool E5M2>
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantArgs a) {
  constexpr float kTop = E5M2 ? 57344.0f : 448.0f;
  constexpr bool COL = MODE == kCol || MODE == kBoth, ROW = MODE == kRow || MODE == kBoth;
  __shared__ uint32_t part[8][128];
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int cb = static_cast<int>(blockIdx.x) % a.blk_cols, rb = static_cast<int>(blockIdx.x) / a.blk_cols;
  const int col = cb * 128 + lane * 4, row0 = rb * 128 + warp * 16;
  const bool col_ok = col < a.cols;  // (cols is a multiple of 16: a thread's four columns exist together)
  float v[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.0f;
    if (col_ok && row0 + i < a.rows) {
      const int64_t at = (row0 + i) * a.ldx + col;
      if (F32) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + at));
        v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
      } else {
        const uint2 x = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.x) + at));
        v[i][0] = __uint_as_float(x.x << 16), v[i][1] = __uint_as_float(x.x & 0xFFFF0000u);
        v[i][2] = __uint_as_float(x.y << 16), v[i][3] = __uint_as_float(x.y & 0xFFFF0000u);
      }
    }
  }
  if (ROW) {
    float mine = 0.0f;  // lane i keeps row i's scale
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      uint32_t m = max(max(abs_bits(v[i][0]), abs_bits(v[i][1])), max(abs_bits(v[i][2]), abs_bits(v[i][3])));
      m = __reduce_max_sync(0xffffffffu, m);
      const float top = block_max(m), f = __fdiv_rn(kTop, top);
      if (lane == i) mine = __fdiv_rn(top, kTop);
      if (col_ok && row0 + i < a.rows)
        *reinterpret_cast<uint32_t*>(a.q + (row0 + i) * a.ldq + col) =
            cvt4<E5M2>(__fmul_rn(v[i][0], f), __fmul_rn(v[i][1], f), __fmul_rn(v[i][2], f), __fmul_rn(v[i][3], f));
    }
    if (lane < 16 && row0 + lane < a.rows) a.s[(row0 + lane) * a.s_row + cb * a.s_col] = mine;
  }
  if (MODE != kRow) {
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = max(m[j], abs_bits(v[i][j]));
    if (MODE == kBlock) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, max(max(m[0], m[1]), max(m[2], m[3])));
      if (lane == 0) part[0][warp] = w;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) all = max(all, part[0][k]);
      const float top = block_max(all), f = __fdiv_rn(kTop, top);
      if (threadIdx.x == 0) a.s[rb * a.s_row + cb * a.s_col] = __fdiv_rn(top, kTop);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (col_ok && row0 + i < a.rows)
          *reinterpret_cast<uint32_t*>(a.q + (row0 + i) * a.ldq + col) =
              cvt4<E5M2>(__fmul_rn(v[i][0], f), __fmul_rn(v[i][1], f), __fmul_rn(v[i][2], f), __fmul_rn(v[i][3], f));
    }
    if (COL) {
      *reinterpret_cast<uint4*>(&part[warp][lane * 4]) = make_uint4(m[0], m[1], m[2], m[3]);
      __syncthreads();
      float f[4];
      float4 sc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t all = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) all = max(all, part[k][lane * 4 + j]);
        const float top = block_max(all);
        f[j] = __fdiv_rn(kTop, top);
        (&sc.x)[j] = __fdiv_rn(top, kTop);
      }
      if (warp == 0 && col_ok) *reinterpret_cast<float4*>(a.sc + rb * a.sc_row + col) = sc;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (col_ok && row0 + i < a.rows)
          *reinterpret_cast<uint32_t*>(a.qc + (row0 + i) * a.ldqc + col) = cvt4<E5M2>(
              __fmul_rn(v[i][0], f[0]), __fmul_rn(v[i][1], f[1]), __fmul_rn(v[i][2], f[2]), __fmul_rn(v[i][3], f[3]));
    }
  }
}

template <bool F32, bool E5M2>
void launch_quantize(int mode, const QuantArgs& a, unsigned grid, cudaStream_t stream) {
  switch (mode) {
    case kRow:
      quantize_kernel<kRow, F32, E5M2><<<grid, 256, 0, stream>>>(a);
      break;
    case kCol:
      quantize_kernel<kCol, F32, E5M2><<<grid, 256, 0, stream>>>(a);
      break;
    case kBlock:
      quantize_kernel<kBlock, F32, E5M2><<<grid, 256, 0, stream>>>(a);
      break;
    default:
      quantize_kernel<kBoth, F32, E5M2><<<grid, 256, 0, stream>>>(a);
      break;
  }
}

}  // namespace
}  // namespace dp

extern "C" dp_status dp_fp8_quantize(const void* x, int64_t ldx, int x_f32, int64_t rows, int64_t cols,
                                     dp_fp8_scaling scaling, dp_fp8_format format, void* q, int64_t ldq, float* s,
                                     int64_t s_row, int64_t s_col, void* q_col, int64_t ldq_col, float* s_colwise,
                                     int64_t sc_row, dp_stream stream) {
  using namespace dp;
  const int mode = static_cast<int>(scaling), fmt = static_cast<int>(format);
  if (mode < 0 || mode > 3 || fmt < 0 || fmt > 1 || (x_f32 != 0 && x_f32 != 1)) return DP_ERR_INVALID_ARG;
  if (rows < 0 || cols < 1) return DP_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows > 0x7FFFFF00 || cols > 0x7FFFFF00) return DP_ERR_UNSUPPORTED;
  dp_status st = check_operand(x, rows, cols, &ldx, x_f32 ? 4 : 2);
  if (st != DP_OK) return st;
  if (mode != kCol) {
    if ((st = check_operand(q, rows, cols, &ldq, 1)) != DP_OK) return st;
    if (rows > 0 && s == nullptr) return DP_ERR_INVALID_ARG;
    if (s_row < 0 || s_col < 0) return DP_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(s) & 3) != 0) return DP_ERR_ALIGNMENT;
  }
  if (mode == kCol || mode == kBoth) {
    if ((st = check_operand(q_col, rows, cols, &ldq_col, 1)) != DP_OK) return st;
    if (rows > 0 && s_colwise == nullptr) return DP_ERR_INVALID_ARG;
    if (sc_row < cols) return DP_ERR_INVALID_ARG;
    if (!is_aligned16(s_colwise) || sc_row % 4 != 0) return DP_ERR_ALIGNMENT;
  }
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (rows == 0) return DP_OK;
  QuantArgs a;
  a.x = x;
  a.ldx = ldx;
  a.rows = static_cast<int32_t>(rows);
  a.cols = static_cast<int32_t>(cols);
  a.blk_cols = static_cast<int32_t>((cols + 127) / 128);
  a.q = static_cast<uint8_t*>(q);
  a.ldq = ldq;
  a.s = s;
  a.s_row = s_row;
  a.s_col = s_col;
  a.qc = static_cast<uint8_t*>(q_col);
  a.ldqc = ldq_col;
  a.sc = s_colwise;
  a.sc_row = sc_row;
  const int64_t tiles = (rows + 127) / 128 * a.blk_cols;
  if (tiles > 0x7FFFFFFF) return DP_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(tiles);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (x_f32)
    fmt ? launch_quantize<true, true>(mode, a, grid, str) : launch_quantize<true, false>(mode, a, grid, str);
  else
    fmt ? launch_quantize<false, true>(mode, a, grid, str) : launch_quantize<false, false>(mode, a, grid, str);
  return cudaGetLastError() == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

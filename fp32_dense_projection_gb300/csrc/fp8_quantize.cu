// Quantisation to 8-bit floating point with one scale per 128 values:
//   a = max(max |x| over the block, 1e-30),  s = a / top,  q = rn(x * (top / a)),
// top the format's largest value (448 E4M3, 57344 E5M2).  A block is 128 values of a row
// (scales for contractions along the row), of a column (contractions along the rows: the
// weight gradient), or 128 x 128 (weights).  Row and column blocks together come from one
// read of x.
//
// Bound: HBM bytes (2 or 4 read, 1 or 2 written per value): 16384 x 4096 BF16, rows and columns,
// takes 43 us or 6.2 TB/s, FP32 63 us or 6.4 TB/s.  One CTA takes a 128 x 128 tile and keeps it in
// registers (BF16 pairs packed), so x is read once whatever the blocks; a thread's loads are in
// flight together and several CTAs share an SM, so that one tile's loads run beside another's
// stores.  What stands beside the bytes is instructions: the first form (FP32 in registers, a
// division per lane and row) took 32 a value and 107 us for that BF16 tensor, this one 15.  A
// row's maximum is a shuffle reduction of two rows at a time, a column's a maximum over the
// warps in shared memory.
//
// Maxima are taken on the bits of |x| as integers (two BF16 at a time): that order puts NaN
// above infinity, so a block with a NaN gets a NaN scale (and one with an infinity an
// infinite scale, whose products are NaN) instead of hiding it.
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

// The block's maximum with its lower bound (a NaN stays).
__device__ __forceinline__ float block_max(uint32_t bits) {
  const float a = __uint_as_float(bits);
  return a < kTinyMax ? kTinyMax : a;
}

// Maxima of |x| as bits: one 32-bit word per FP32 value, or two BF16 in the halves of a word.
template <bool F32>
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t x) {
  return F32 ? max(m, x & 0x7FFFFFFFu) : __vmaxu2(m, x & 0x7FFF7FFFu);
}

// Warps of a CTA: FP32 tiles take 16 warps of 8 rows and two CTAs an SM, BF16 tiles, half as many
// bytes, 8 warps of 16 rows and four CTAs, so that the same bytes are in flight and fewer
// warps wait at a tile's barriers (16384 x 4096 BF16, rows and columns: 50.8 us with 16 warps, 43.1
// with 8; FP32: 63.1 with 16, 64.8 with 8).
template <bool F32>
constexpr int kWarps = F32 ? 16 : 8;

// A thread holds 16 bytes (4 FP32 or 8 BF16 columns) of each of ITERS rows: a warp's load covers
// one FP32 row or two BF16 rows of the tile.
template <int MODE, bool F32, bool E5M2>
__global__ void __launch_bounds__(kWarps<F32> * 32, F32 ? 2 : 4) quantize_kernel(const __grid_constant__ QuantArgs a) {
  constexpr float kTop = E5M2 ? 57344.0f : 448.0f;
  constexpr bool COL = MODE == kCol || MODE == kBoth, ROW = MODE == kRow || MODE == kBoth;
  constexpr int CPL = F32 ? 4 : 8, LPR = 128 / CPL, RPI = 32 / LPR, WARPS = kWarps<F32>, ROWS = 128 / WARPS,
                ITERS = ROWS / RPI;
  __shared__ __align__(16) uint32_t part[COL ? WARPS * RPI : 1][COL ? LPR * 4 : 32];
  __shared__ __align__(16) float factors[COL ? 128 : 4];
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int cb = static_cast<int>(blockIdx.x) % a.blk_cols, rb = static_cast<int>(blockIdx.x) / a.blk_cols;
  const int tcol = lane % LPR * CPL, col = cb * 128 + tcol;
  const int row0 = rb * 128 + warp * ROWS + lane / LPR;  // this thread's rows: row0 + RPI * i
  // (cols is a multiple of 16: a thread's columns exist together)
  const int rows = col < a.cols ? a.rows - row0 : 0;
  uint32_t v[ITERS][4];
  {
    const int esize = F32 ? 4 : 2;
    const char* p = static_cast<const char*>(a.x) + (row0 * a.ldx + col) * esize;
#pragma unroll
    for (int i = 0; i < ITERS; ++i, p += RPI * a.ldx * esize) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (RPI * i < rows) x = __ldg(reinterpret_cast<const uint4*>(p));
      v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
    }
  }
  auto value = [&](int i, int j) {
    if (F32) return __uint_as_float(v[i][j & 3]);
    return __uint_as_float(j & 1 ? v[i][j >> 1] & 0xFFFF0000u : v[i][j >> 1] << 16);
  };
  // row i's codes: values times factors (one for the row, or one per column)
  auto store = [&](uint8_t* p, int i, auto factor) {
    if (RPI * i >= rows) return;
    uint32_t w[CPL / 4];
#pragma unroll
    for (int j = 0; j < CPL; j += 4)
      w[j / 4] = cvt4<E5M2>(__fmul_rn(value(i, j), factor(j)), __fmul_rn(value(i, j + 1), factor(j + 1)),
                            __fmul_rn(value(i, j + 2), factor(j + 2)), __fmul_rn(value(i, j + 3), factor(j + 3)));
    if (F32)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[CPL / 4 - 1]);
  };
  // (Quotients are IEEE divisions of ~10 instructions: each is taken once and passed on.)
  if (ROW) {
    uint32_t m[ITERS];
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
      m[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m[i] = max_bits<F32>(m[i], v[i][j]);
    }
    uint32_t mine = 0;  // the maximum of row row0 + RPI * (lane % ITERS)
    if (F32) {
#pragma unroll
      for (int i = 0; i < ITERS; ++i) {
        const uint32_t r = __reduce_max_sync(0xffffffffu, m[i]);
        if (lane % ITERS == i) mine = r;
      }
    } else {
      // two rows' maxima in the halves of a word, reduced over the 16 lanes of a row
#pragma unroll
      for (int i = 0; i < ITERS; i += 2) {
        const uint32_t lo = __vmaxu2(m[i], m[i] >> 16) & 0xFFFFu, hi = __vmaxu2(m[i + 1], m[i + 1] << 16) & 0xFFFF0000u;
        uint32_t r = lo | hi;
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) r = __vmaxu2(r, __shfl_xor_sync(0xffffffffu, r, d));
        if (lane % ITERS == i) mine = r << 16;
        if (lane % ITERS == i + 1) mine = r & 0xFFFF0000u;
      }
    }
    const float top = block_max(mine), f = __fdiv_rn(kTop, top);
    const int srow = row0 + RPI * (lane % ITERS);
    if (lane % LPR < ITERS && srow < a.rows) a.s[srow * a.s_row + cb * a.s_col] = __fdiv_rn(top, kTop);
    uint8_t* p = a.q + row0 * a.ldq + col;
#pragma unroll
    for (int i = 0; i < ITERS; ++i, p += RPI * a.ldq) {
      const float fi = __shfl_sync(0xffffffffu, f, lane / LPR * LPR + i);
      store(p, i, [&](int) { return fi; });
    }
  }
  if (MODE != kRow) {
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < ITERS; ++i) m[j] = max_bits<F32>(m[j], v[i][j]);
    }
    if (MODE == kBlock) {
#pragma unroll
      for (int j = 1; j < 4; ++j) m[0] = max_bits<F32>(m[0], m[j]);
      if (!F32) m[0] = max(m[0] << 16, m[0] & 0xFFFF0000u);
      const uint32_t w = __reduce_max_sync(0xffffffffu, m[0]);
      if (lane == 0) part[0][warp] = w;
      __syncthreads();
      const float top = block_max(__reduce_max_sync(0xffffffffu, part[0][lane % WARPS])), f = __fdiv_rn(kTop, top);
      if (threadIdx.x == 0) a.s[rb * a.s_row + cb * a.s_col] = __fdiv_rn(top, kTop);
      uint8_t* p = a.q + row0 * a.ldq + col;
#pragma unroll
      for (int i = 0; i < ITERS; ++i, p += RPI * a.ldq) store(p, i, [&](int) { return f; });
    }
    if (COL) {
      *reinterpret_cast<uint4*>(&part[warp * RPI + lane / LPR][lane % LPR * 4]) = make_uint4(m[0], m[1], m[2], m[3]);
      __syncthreads();
      // one thread per word of maxima: 1 FP32 or 2 BF16 columns and their factors
      if (threadIdx.x < LPR * 4) {
        const int t = static_cast<int>(threadIdx.x);
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < WARPS * RPI; ++k) w = max_bits<F32>(w, part[k][t]);
        constexpr int PER = CPL / 4;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int c = t * PER + j;
          const float top = block_max(F32 ? w : j ? w & 0xFFFF0000u : w << 16);
          factors[c] = __fdiv_rn(kTop, top);
          if (cb * 128 + c < a.cols) a.sc[rb * a.sc_row + cb * 128 + c] = __fdiv_rn(top, kTop);
        }
      }
      __syncthreads();
      float f[CPL];
#pragma unroll
      for (int j = 0; j < CPL; ++j) f[j] = factors[tcol + j];
      uint8_t* p = a.qc + row0 * a.ldqc + col;
#pragma unroll
      for (int i = 0; i < ITERS; ++i, p += RPI * a.ldqc) store(p, i, [&](int j) { return f[j]; });
    }
  }
}

template <bool F32, bool E5M2>
void launch_quantize(int mode, const QuantArgs& a, unsigned grid, cudaStream_t stream) {
  switch (mode) {
    case kRow:
      quantize_kernel<kRow, F32, E5M2><<<grid, kWarps<F32> * 32, 0, stream>>>(a);
      break;
    case kCol:
      quantize_kernel<kCol, F32, E5M2><<<grid, kWarps<F32> * 32, 0, stream>>>(a);
      break;
    case kBlock:
      quantize_kernel<kBlock, F32, E5M2><<<grid, kWarps<F32> * 32, 0, stream>>>(a);
      break;
    default:
      quantize_kernel<kBoth, F32, E5M2><<<grid, kWarps<F32> * 32, 0, stream>>>(a);
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

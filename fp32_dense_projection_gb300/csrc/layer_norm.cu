// Layer norm over the rows of x [T][C]:
//   mu = mean(x),  rs = 1 / sqrt(mean((x - mu)^2) + eps),  h = (x - mu) rs,  y = h w + b
// and its backward pass, with g = dy w:
//   dx = rs (g - mean(g) - h mean(g h)),   dw = sum_t dy h,   db = sum_t dy
//
// Bound: HBM bytes (x read, y written; backward x and dy read, dx written).  A row's elements stay
// in the registers of the threads that share it, so each is read once; the variance is the mean
// of squared distances from the row's own mean, not a difference of two large sums.  dw and db are
// summed in FP32 registers over the rows that a block visits, in row order; each block writes its
// sums to the workspace, and a second launch adds them in block order: no atomics, the same bits
// every time.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_internal.h"
#include "row_ops.cuh"

namespace dp {
namespace {

constexpr int64_t kMaxCols = 16384;

struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* w;  // null: 1
  const void* b;  // null: 0
  int w_f32;
  float eps;
  int64_t T;
  int32_t C, tpr;  // columns; threads per row
  float inv_c;
  void* y;  // forward: y; backward: dx
  int64_t ldy;
  float* mean;
  float* rstd;
  const void* dy;
  int64_t ldg;
  float* partial;  // [blocks][2][C]: each block's sums for dw and db (null: no weight)
};

__device__ __forceinline__ void load_param(const void* p, int f32, int at, float other, float (&v)[8]) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = other;
  } else if (f32) {
    load8<true>(p, at, v);
  } else {
    load8<false>(p, at, v);
  }
}

template <bool XF32, bool YF32, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_fwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][32][1];
  const int t = static_cast<int>(threadIdx.x) % a.tpr, sub = static_cast<int>(threadIdx.x) / a.tpr;
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  GroupSum<1> sum(part, a.tpr);
  float w[CH][8], b[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int col = (t + i * a.tpr) * 8;
    if (col < a.C) {
      load_param(a.w, a.w_f32, col, 1.0f, w[i]);
      load_param(a.b, a.w_f32, col, 0.0f, b[i]);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  Raw8<XF32> next[CH];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * a.tpr) * 8;
      next[i] = row < a.T && col < a.C ? load_raw8<XF32>(a.x, row * a.ldx + col) : zero_raw8<XF32>();
    }
  };
  fetch(static_cast<int64_t>(blockIdx.x) * rows + sub);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows; base < a.T; base += step) {
    const int64_t row = base + sub;
    float x[CH][8], s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      unpack8<XF32>(next[i], x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += x[i][j];
    }
    fetch(row + step);
    sum(s);
    const float mean = s[0] * a.inv_c;
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((t + i * a.tpr) * 8 >= a.C) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[i][j] -= mean;
        q[0] = fmaf(x[i][j], x[i][j], q[0]);
      }
    }
    sum(q);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], a.inv_c, a.eps));
    if (row >= a.T) continue;
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * a.tpr) * 8;
      if (col >= a.C) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = fmaf(x[i][j] * rstd, w[i][j], b[i][j]);
      store8<YF32>(a.y, row * a.ldy + col, x[i]);
    }
  }
}

template <bool XF32, bool GF32, bool DF32, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][32][2];
  extern __shared__ float shared_sums[];  // [2][C], where a block has more than one row at a time
  const int t = static_cast<int>(threadIdx.x) % a.tpr, sub = static_cast<int>(threadIdx.x) / a.tpr;
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  GroupSum<2> sum(part, a.tpr);
  float dw[CH][8], db[CH][8], w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int col = (t + i * a.tpr) * 8;
    if (col < a.C) load_param(a.w, a.w_f32, col, 1.0f, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.0f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rows; base < a.T; base += step) {
    const int64_t row = base + sub;
    const bool live = row < a.T;
    const float mean = live ? a.mean[row] : 0.0f, rstd = live ? a.rstd[row] : 0.0f;
    float h[CH][8], g[CH][8], s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * a.tpr) * 8;
      if (!live || col >= a.C) continue;
      load8<XF32>(a.x, row * a.ldx + col, h[i]);
      load8<GF32>(a.dy, row * a.ldg + col, g[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = (h[i][j] - mean) * rstd;
        dw[i][j] = fmaf(g[i][j], h[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= w[i][j];
        s[0] += g[i][j];
        s[1] = fmaf(g[i][j], h[i][j], s[1]);
      }
    }
    sum(s);
    if (!live) continue;
    const float m0 = s[0] * a.inv_c, m1 = s[1] * a.inv_c;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * a.tpr) * 8;
      if (col >= a.C) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = (g[i][j] - m0 - h[i][j] * m1) * rstd;
      store8<DF32>(a.y, row * a.ldy + col, g[i]);
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
  // the rows that the block had at a time are added in their order
  for (int r = 0; r < rows; ++r) {
    if (sub == r) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int col = (t + i * a.tpr) * 8;
        if (col >= a.C) continue;
        if (r > 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[i][j] += shared_sums[col + j], db[i][j] += shared_sums[a.C + col + j];
        }
        if (r == rows - 1) {
          store8<true>(out, col, dw[i]);
          store8<true>(out, a.C + col, db[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) shared_sums[col + j] = dw[i][j], shared_sums[a.C + col + j] = db[i][j];
        }
      }
    }
    if (r < rows - 1) __syncthreads();
  }
}

// dw and db: the blocks' sums in block order (8 runs of blocks, then the runs).
__global__ void __launch_bounds__(256) norm_sum_kernel(const float* partial, int blocks, int C, float* dw, float* db) {
  __shared__ float runs[8][32];
  const int lane = static_cast<int>(threadIdx.x) & 31, run = static_cast<int>(threadIdx.x) >> 5;
  const int col = static_cast<int>(blockIdx.x) * 32 + lane;  // of 2 C
  const int per = (blocks + 7) / 8;
  float s = 0.0f;
  if (col < 2 * C)
    for (int k = run * per; k < blocks && k < (run + 1) * per; ++k) s += partial[static_cast<int64_t>(k) * 2 * C + col];
  runs[run][lane] = s;
  __syncthreads();
  if (run != 0 || col >= 2 * C) return;
  for (int k = 1; k < 8; ++k) s += runs[k][lane];
  if (col < C)
    dw[col] = s;
  else
    db[col - C] = s;
}

// Threads per row: a power of two that leaves a thread at most two pieces of eight columns.
int threads_per_row(int64_t C) {
  int tpr = 4;
  while (tpr * 16 < C) tpr *= 2;
  return tpr;
}

struct Shape {
  int tpr, threads, rows, pieces;
  int64_t blocks;
};

Shape shape_of(int64_t T, int64_t C, int sm_count, int per_sm) {
  Shape s;
  s.tpr = threads_per_row(C);
  s.threads = std::max(256, s.tpr);
  s.rows = s.threads / s.tpr;
  s.pieces = C > 8 * s.tpr ? 2 : 1;
  const int64_t most = static_cast<int64_t>(sm_count) * std::max(1, per_sm * 256 / s.threads);
  s.blocks = std::min(most, (T + s.rows - 1) / s.rows);
  return s;
}

constexpr int kFwdPerSm = 4, kBwdPerSm = 2;  // blocks of 256 threads an SM

template <typename F>
void by_bool(bool v, F f) {
  v ? f(std::true_type()) : f(std::false_type());
}

dp_status check_vector(const void* p) { return is_aligned16(p) ? DP_OK : DP_ERR_ALIGNMENT; }

dp_status check_norm(int64_t T, int64_t C) {
  if (T < 0 || C < 1) return DP_ERR_INVALID_ARG;
  if (C % 8 != 0 || C > kMaxCols || T > 0x7FFFFFFF) return DP_ERR_UNSUPPORTED;
  return DP_OK;
}

int64_t bwd_bytes(int64_t T, int64_t C, int sm_count) { return shape_of(T, C, sm_count, kBwdPerSm).blocks * 2 * C * 4; }

bool flag(int v) { return v == 0 || v == 1; }

}  // namespace
}  // namespace dp

extern "C" dp_status dp_layer_norm_workspace_size(int64_t T, int64_t C, int sm_count, size_t* bytes) {
  using namespace dp;
  if (bytes == nullptr) return DP_ERR_INVALID_ARG;
  dp_status st = check_norm(T, C);
  if (st != DP_OK) return st;
  if (sm_count <= 0) {
    DeviceContext ctx;
    if ((st = device_context(&ctx)) != DP_OK) return st;
    sm_count = ctx.sm_count;
  }
  *bytes = static_cast<size_t>(bwd_bytes(T, C, sm_count));
  return DP_OK;
}

extern "C" dp_status dp_layer_norm_fwd(const void* x, int64_t ldx, int x_f32, const void* weight, const void* bias,
                                       int weight_f32, double eps, void* y, int64_t ldy, dp_out_dtype out, float* mean,
                                       float* rstd, int64_t T, int64_t C, dp_stream stream) {
  using namespace dp;
  const int code = static_cast<int>(out);
  if (!flag(x_f32) || !flag(weight_f32) || !flag(code) || !(eps >= 0.0)) return DP_ERR_INVALID_ARG;
  dp_status st = check_norm(T, C);
  if (st == DP_OK) st = check_operand(x, T, C, &ldx, x_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(y, T, C, &ldy, code ? 4 : 2);
  if (st == DP_OK) st = check_vector(weight);
  if (st == DP_OK) st = check_vector(bias);
  if (st != DP_OK) return st;
  if (T > 0 && (mean == nullptr || rstd == nullptr)) return DP_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd)) & 3) != 0) return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return DP_OK;
  const Shape s = shape_of(T, C, ctx.sm_count, kFwdPerSm);
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.w = weight, a.b = bias, a.w_f32 = weight_f32, a.eps = static_cast<float>(eps);
  a.T = T, a.C = static_cast<int32_t>(C), a.tpr = s.tpr, a.inv_c = 1.0f / static_cast<float>(C);
  a.y = y, a.ldy = ldy, a.mean = mean, a.rstd = rstd;
  const unsigned grid = static_cast<unsigned>(s.blocks);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  by_bool(x_f32, [&](auto xf) {
    by_bool(code, [&](auto yf) {
      constexpr bool X = decltype(xf)::value, Y = decltype(yf)::value;
      if (s.threads > 256)
        norm_fwd_kernel<X, Y, 2, 1024><<<grid, s.threads, 0, str>>>(a);
      else if (s.pieces == 2)
        norm_fwd_kernel<X, Y, 2, 256><<<grid, s.threads, 0, str>>>(a);
      else
        norm_fwd_kernel<X, Y, 1, 256><<<grid, s.threads, 0, str>>>(a);
    });
  });
  return cudaGetLastError() == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

extern "C" dp_status dp_layer_norm_bwd(const void* dy, int64_t ldg, int dy_f32, const void* x, int64_t ldx, int x_f32,
                                       const float* mean, const float* rstd, const void* weight, int weight_f32, void* dx,
                                       int64_t ld_dx, dp_out_dtype out, float* dw, float* db, int64_t T, int64_t C,
                                       void* workspace, size_t workspace_bytes, dp_stream stream) {
  using namespace dp;
  const int code = static_cast<int>(out);
  if (!flag(x_f32) || !flag(dy_f32) || !flag(weight_f32) || !flag(code)) return DP_ERR_INVALID_ARG;
  dp_status st = check_norm(T, C);
  if (st == DP_OK) st = check_operand(dy, T, C, &ldg, dy_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(x, T, C, &ldx, x_f32 ? 4 : 2);
  if (st == DP_OK) st = check_operand(dx, T, C, &ld_dx, code ? 4 : 2);
  if (st == DP_OK) st = check_vector(weight);
  if (st != DP_OK) return st;
  if (T > 0 && (mean == nullptr || rstd == nullptr)) return DP_ERR_INVALID_ARG;
  if ((dw == nullptr) != (db == nullptr)) return DP_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(mean) | reinterpret_cast<uintptr_t>(rstd) | reinterpret_cast<uintptr_t>(dw) |
        reinterpret_cast<uintptr_t>(db)) & 3) != 0)
    return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (dw == nullptr) return DP_OK;
    const bool ok = cudaMemsetAsync(dw, 0, C * 4, str) == cudaSuccess && cudaMemsetAsync(db, 0, C * 4, str) == cudaSuccess;
    return ok ? DP_OK : DP_ERR_LAUNCH;
  }
  const Shape s = shape_of(T, C, ctx.sm_count, kBwdPerSm);
  if (dw != nullptr) {
    if (workspace == nullptr || workspace_bytes < static_cast<size_t>(bwd_bytes(T, C, ctx.sm_count))) return DP_ERR_WORKSPACE;
    if (!is_aligned16(workspace)) return DP_ERR_ALIGNMENT;
  }
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.w = weight, a.w_f32 = weight_f32;
  a.T = T, a.C = static_cast<int32_t>(C), a.tpr = s.tpr, a.inv_c = 1.0f / static_cast<float>(C);
  a.y = dx, a.ldy = ld_dx, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.dy = dy, a.ldg = ldg, a.partial = dw ? static_cast<float*>(workspace) : nullptr;
  const unsigned grid = static_cast<unsigned>(s.blocks);
  const size_t smem = s.rows > 1 && dw ? static_cast<size_t>(C) * 8 : 0;  // (at most 2048 columns: 16 KB)
  by_bool(x_f32, [&](auto xf) {
    by_bool(dy_f32, [&](auto gf) {
      by_bool(code, [&](auto df) {
        constexpr bool X = decltype(xf)::value, G = decltype(gf)::value, D = decltype(df)::value;
        if (s.threads > 256)
          norm_bwd_kernel<X, G, D, 2, 1024><<<grid, s.threads, smem, str>>>(a);
        else if (s.pieces == 2)
          norm_bwd_kernel<X, G, D, 2, 256><<<grid, s.threads, smem, str>>>(a);
        else
          norm_bwd_kernel<X, G, D, 1, 256><<<grid, s.threads, smem, str>>>(a);
      });
    });
  });
  if (cudaGetLastError() != cudaSuccess) return DP_ERR_LAUNCH;
  if (dw == nullptr) return DP_OK;
  norm_sum_kernel<<<static_cast<unsigned>((2 * C + 31) / 32), 256, 0, str>>>(a.partial, static_cast<int>(s.blocks),
                                                                             static_cast<int>(C), dw, db);
  return cudaGetLastError() == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

// Layer norm over the rows of x [T][C]:
//   mu = mean(x),  rs = 1 / sqrt(mean((x - mu)^2) + eps),  h = (x - mu) rs,  y = h w + b
// and its backward pass, with g = dy w:
//   dx = rs (g - mean(g) - h mean(g h)),   dw = sum_t dy h,   db = sum_t dy
//
// Bound: HBM bytes (x read, y written; backward x and dy read, dx written), and beside them the instructions
// of a row's sums, which a row's every warp spends.  Each row is read from memory once; the variance is the
// mean of squared distances from the row's own mean, not a difference of two large sums.  A thread's own
// pieces of the next rows are on their way into shared memory meanwhile (asynchronous copies that
// nobody else waits for); one row ahead in registers reached 3.6 TB/s in the backward pass.  Arithmetic
// is packed, two FP32 values an instruction; weight and bias lie in shared memory in FP32.  dw and db
// are summed in FP32 registers over the rows that a block visits, in row order; each block writes its sums
// to the workspace, and a second launch adds them in block order: no atomics, the same bits every time.
// The shape depends on C and the types alone, so that a row's result does not depend on how many there are.
//
// Four pieces of eight columns a thread halve the warps of a row against two (with 96 MB of x, four / two, us):
//   forward, BF16     256 columns 32.6 / 41.9, 1024 37.7 / 47.6, 4096 44.4 / 53.9, 5120 50.0 / 84.0, 8192 50.3 / 65.2: always four;
//   forward, FP32     256 25.4 / 26.9, 1024 29.1 / 30.8, 4096 34.1 / 34.6, 5120 33.3 / 46.9, 8192 32.8 / 39.6: four above 4096 (two
//                     leave shorter tails of few rows: 16173 x 1024 forward and backward 57, 60 with four);
//   backward, BF16    1024 59.6 / 53.8, 4096 61.5 / 55.2, 5120 63.7 / 69.7, 8192 63.3 / 60.8: four above 4096;
//   backward, FP32 x  1024 51.2 / 36.4, 4096 54.0 / 39.8, 5120 49.1 / 46.8, 8192 49.2 / 44.4: two up to 8192.
// Above 8192 columns four it is (one thread of 512 has no more than four): 3000 rows of 16384 in BF16 backward 71.5 us (with 1024
// threads that held dw and db in shared memory 1.8 times that).  16384 x 4096 in BF16 backward: 72.7 us, 5.5 TB/s.
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
  int y_f32;
  float* mean;
  float* rstd;
  int few;  // (forward) a block has one row, or one for each group of threads: weight and bias come straight from memory
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

__device__ __forceinline__ void store_row8(const NormArgs& a, int64_t at, const Two (&v)[4]) {
  if (a.y_f32)
    store8<true>(a.y, at, v);
  else
    store8<false>(a.y, at, v);
}

// A vector over the columns in FP32, each thread's own pieces: [piece][half][thread of the row].
__device__ __forceinline__ void keep_param(float4* kept, const NormArgs& a, const void* p, float other) {
  for (int c = static_cast<int>(threadIdx.x); c < a.C / 8; c += static_cast<int>(blockDim.x)) {
    float v[8];
    load_param(p, a.w_f32, c * 8, other, v);
    float4* at = kept + c / a.tpr * 2 * a.tpr + c % a.tpr;
    at[0] = make_float4(v[0], v[1], v[2], v[3]);
    at[a.tpr] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void take_param(const float4* kept, int tpr, int t, int i, Two (&v)[4]) {
  const float4 p = kept[2 * i * tpr + t], q = kept[(2 * i + 1) * tpr + t];
  v[0] = two(p.x, p.y), v[1] = two(p.z, p.w), v[2] = two(q.x, q.y), v[3] = two(q.z, q.w);
}

__device__ __forceinline__ void read_param(const void* p, int f32, int col, float other, Two (&w)[4]) {
  float v[8];
  load_param(p, f32, col, other, v);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = two(v[2 * j], v[2 * j + 1]);
}

// Rows in shared memory: as many as it holds beside the blocks that share an SM.
constexpr int fwd_depth(int threads, bool f32) { return threads == 512 && f32 ? 1 : 2; }
constexpr int bwd_depth(int pieces, bool x_f32, bool g_f32) {
  return pieces == 4 ? (x_f32 || g_f32 ? 1 : 2) : x_f32 && g_f32 ? 2 : 3;
}
constexpr int fwd_pieces(bool x_f32, int threads) { return x_f32 && threads == 256 ? 2 : 4; }
// Threads from piece to piece in shared memory (0: the block's): a constant where a block has the SM to itself and many
// pieces (16384 columns backward, BF16 rows and FP32 gradients: 96 us, 114 with the block's).
constexpr int ring_stride(int pieces, int threads) { return pieces == 4 && threads == 512 ? threads : 0; }
constexpr int fwd_per_sm(int threads) { return threads == 256 ? 3 : 1; }
constexpr int bwd_per_sm(int threads) { return threads == 256 ? 2 : 1; }

template <bool XF32, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS, fwd_per_sm(THREADS))
    norm_fwd_kernel(const __grid_constant__ NormArgs a) {
  constexpr int DEPTH = fwd_depth(THREADS, XF32);
  __shared__ float part[2][32][1];
  extern __shared__ float4 shared[];  // rows ahead, weight and bias
  const int t = static_cast<int>(threadIdx.x) % a.tpr, sub = static_cast<int>(threadIdx.x) / a.tpr;
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  GroupSum<1> sum(part, a.tpr);
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows, first = static_cast<int64_t>(blockIdx.x) * rows;
  Ahead<XF32, CH, DEPTH, ring_stride(CH, THREADS)> ahead(shared, a.tpr, t, a.x, a.ldx, first + sub, step, a.C);
  float4* const w_kept = shared + ahead.units();
  float4* const b_kept = w_kept + 2 * CH * a.tpr;
  auto fetch = [&](int slot, int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) ahead.load(slot, i, row < a.T);
    ahead.advance();
    copies_commit();
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(d, first + sub + d * step);
  if (!a.few) {
    keep_param(w_kept, a, a.w, 1.0f);
    keep_param(b_kept, a, a.b, 0.0f);
    __syncthreads();
  }
  int slot = 0;
  for (int64_t base = first; base < a.T; base += step) {
    const int64_t row = base + sub;
    Two x[CH][4], s2 = twice(0.0f);
    copies_wait<DEPTH - 1>();
    if (XF32) __syncwarp();
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      unpack8<XF32>(ahead.take(slot, i), x[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s2 = s2 + x[i][j];
    }
    float s[1] = {lo(s2) + hi(s2)};
    if (XF32) __syncwarp();
    fetch(slot, row + DEPTH * step);
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    sum(s);
    const float mean = s[0] * a.inv_c;
    Two q2 = twice(0.0f);
    const Two minus = twice(-mean);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((t + i * a.tpr) * 8 >= a.C) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = x[i][j] + minus;
        q2 = fma2(x[i][j], x[i][j], q2);
      }
    }
    float q[1] = {lo(q2) + hi(q2)};
    sum(q);
    const float rstd = __frsqrt_rn(fmaf(q[0], a.inv_c, a.eps));
    if (row >= a.T) continue;
    if (t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    const Two scale = twice(rstd);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * a.tpr) * 8;
      if (col >= a.C) continue;
      Two w[4], b[4];
      if (a.few) {
        read_param(a.w, a.w_f32, col, 1.0f, w);
        read_param(a.b, a.w_f32, col, 0.0f, b);
      } else {
        take_param(w_kept, a.tpr, t, i, w);
        take_param(b_kept, a.tpr, t, i, b);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = fma2(x[i][j] * scale, w[j], b[j]);
      store_row8(a, row * a.ldy + col, x[i]);
    }
  }
}

// Four pieces a thread leave no registers for the row: it is read from shared memory again for dx.
template <bool XF32, bool GF32, int CH, int THREADS>
__global__ void __launch_bounds__(THREADS, bwd_per_sm(THREADS)) norm_bwd_kernel(const __grid_constant__ NormArgs a) {
  constexpr bool TWICE = CH == 4;
  constexpr int DEPTH = bwd_depth(CH, XF32, GF32);
  __shared__ float part[2][32][2];
  extern __shared__ float4 shared[];  // rows ahead (x, then dy), the weight
  const int t = static_cast<int>(threadIdx.x) % a.tpr, sub = static_cast<int>(threadIdx.x) / a.tpr;
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  pdl_launch_dependents();  // (the sums' kernel may take its place; it waits for this one)
  GroupSum<2> sum(part, a.tpr);
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows, first = static_cast<int64_t>(blockIdx.x) * rows;
  Ahead<XF32, CH, DEPTH, ring_stride(CH, THREADS)> ahead_x(shared, a.tpr, t, a.x, a.ldx, first + sub, step, a.C);
  Ahead<GF32, CH, DEPTH, ring_stride(CH, THREADS)> ahead_g(shared + ahead_x.units(), a.tpr, t, a.dy, a.ldg, first + sub, step, a.C);
  float4* const kept = shared + ahead_x.units() + ahead_g.units();
  Two dw[CH][4], db[CH][4];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = twice(0.0f);
  }
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto fetch_stats = [&](int64_t row) {
    if (row < a.T) next_mean = __ldg(a.mean + row), next_rstd = __ldg(a.rstd + row);
  };
  auto fetch_piece = [&](int slot, int i, int64_t row) {
    ahead_x.load(slot, i, row < a.T);
    ahead_g.load(slot, i, row < a.T);
  };
  auto fetched = [&] {
    ahead_x.advance();
    ahead_g.advance();
    copies_commit();
  };
  auto fetch = [&](int slot, int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) fetch_piece(slot, i, row);
    fetched();
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(d, first + sub + d * step);
  fetch_stats(first + sub);
  keep_param(kept, a, a.w, 1.0f);
  __syncthreads();
  int slot = 0;
  for (int64_t base = first; base < a.T; base += step) {
    const int64_t row = base + sub;
    const bool live = row < a.T;
    const float mean = next_mean, rstd = next_rstd;
    fetch_stats(row + step);
    Two h[TWICE ? 1 : CH][4], g[TWICE ? 1 : CH][4], s0 = twice(0.0f), s1 = twice(0.0f);
    const Two minus = twice(-mean), scale = twice(rstd);
    copies_wait<DEPTH - 1>();
    if (XF32 || GF32) __syncwarp();
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      Two(&hx)[4] = h[TWICE ? 0 : i], (&gi)[4] = g[TWICE ? 0 : i];
      unpack8<XF32>(ahead_x.take(slot, i), hx);
      unpack8<GF32>(ahead_g.take(slot, i), gi);
      if (!live || (t + i * a.tpr) * 8 >= a.C) continue;
      Two w[4];
      take_param(kept, a.tpr, t, i, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        hx[j] = (hx[j] + minus) * scale;
        dw[i][j] = fma2(gi[j], hx[j], dw[i][j]);
        db[i][j] = db[i][j] + gi[j];
        gi[j] = gi[j] * w[j];
        s0 = s0 + gi[j];
        s1 = fma2(gi[j], hx[j], s1);
      }
    }
    if (!TWICE) {
      if (XF32 || GF32) __syncwarp();
      fetch(slot, row + DEPTH * step);
      slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }
    float s[2] = {lo(s0) + hi(s0), lo(s1) + hi(s1)};
    sum(s);
    // h is held, dx = g rs + (h c1 + c0); or, from x - mu and with as many operations, ((x - mu) c1 + (dy w + c0)) rs.  (c1 has rs once:
    // its square could leave FP32's range.)
    const Two c0 = twice(-s[0] * a.inv_c * (TWICE ? 1.0f : rstd)), c1 = twice(-s[1] * a.inv_c * rstd);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = (t + i * a.tpr) * 8;
      Two(&hx)[4] = h[TWICE ? 0 : i], (&gi)[4] = g[TWICE ? 0 : i];
      if (TWICE) {
        unpack8<XF32>(ahead_x.take(slot, i), hx);
        unpack8<GF32>(ahead_g.take(slot, i), gi);
        if (XF32 || GF32) __syncwarp();
        fetch_piece(slot, i, row + DEPTH * step);
      }
      if (!live || col >= a.C) continue;
      if (TWICE) {
        Two w[4];
        take_param(kept, a.tpr, t, i, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) gi[j] = fma2(hx[j] + minus, c1, fma2(gi[j], w[j], c0)) * scale;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) gi[j] = fma2(gi[j], scale, fma2(hx[j], c1, c0));
      }
      store_row8(a, row * a.ldy + col, gi);
    }
    if (TWICE) {
      fetched();
      slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.C;
  // the rows that the block had at a time are added in their order (the rows ahead have been used up)
  copies_wait<0>();
  __syncthreads();
  float* const held = reinterpret_cast<float*>(shared);
  for (int r = 0; r < rows; ++r) {
    if (sub == r) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int col = (t + i * a.tpr) * 8;
        if (col >= a.C) continue;
        if (r > 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dw[i][j] = dw[i][j] + two(held[col + 2 * j], held[col + 2 * j + 1]);
            db[i][j] = db[i][j] + two(held[a.C + col + 2 * j], held[a.C + col + 2 * j + 1]);
          }
        }
        float* const to = r == rows - 1 ? out : held;
        store8<true>(to, col, dw[i]);
        store8<true>(to, a.C + col, db[i]);
      }
    }
    if (r < rows - 1) __syncthreads();
  }
}

// dw and db: the blocks' sums in block order (32 runs of blocks, then the runs).  Few loads a thread, all in
// flight: with 8 runs this took 10 us for 304 blocks of 4096 columns.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float* partial, int blocks, int C, float* dw, float* db) {
  __shared__ float runs[32][33];
  const int lane = static_cast<int>(threadIdx.x) & 31, run = static_cast<int>(threadIdx.x) >> 5;
  const int col = static_cast<int>(blockIdx.x) * 32 + lane;  // of 2 C
  const int per = (blocks + 31) / 32, end = min(blocks, (run + 1) * per);
  pdl_wait();
  float s = 0.0f;
  if (col < 2 * C) {
    const float* p = partial + static_cast<int64_t>(run * per) * 2 * C + col;
#pragma unroll 10
    for (int k = run * per; k < end; ++k, p += 2 * C) s += __ldcg(p);
  }
  runs[run][lane] = s;
  __syncthreads();
  // warp r adds the runs of column r: lanes meet pairwise
  s = runs[lane][run];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const int mine = static_cast<int>(blockIdx.x) * 32 + run;
  if (lane != 0 || mine >= 2 * C) return;
  if (mine < C)
    dw[mine] = s;
  else
    db[mine - C] = s;
}

struct Shape {
  int pieces, threads;  // of eight columns a thread; the most threads of a block
  int tpr, rows, block;
  size_t smem;
  int64_t blocks;
};

// Threads per row: a power of two up to a warp, or whole warps.
Shape shape_of(int64_t C, int pieces, int threads) {
  Shape s = {pieces, threads};
  const int n = static_cast<int>((C / 8 + pieces - 1) / pieces);
  s.tpr = 4;
  while (s.tpr < 32 && s.tpr < n) s.tpr *= 2;
  if (n > 32) s.tpr = (n + 31) / 32 * 32;
  s.rows = threads / s.tpr;
  s.block = s.rows * s.tpr;
  return s;
}

constexpr int kMaxShared = 226 * 1024;

void set_blocks(Shape* s, int64_t T, int sm_count, int per_sm, size_t smem) {
  s->smem = smem;
  int most = per_sm * s->threads / s->block;
  if (smem > 0) most = std::min(most, static_cast<int>(228 * 1024 / (smem + 1536)));
  s->blocks = std::min((T + s->rows - 1) / s->rows, static_cast<int64_t>(sm_count) * std::max(1, most));
}

int threads_of(int64_t C) { return C > 4096 ? 512 : 256; }

Shape fwd_shape(int64_t T, int64_t C, bool x_f32, int sm_count) {
  const int threads = threads_of(C), pieces = fwd_pieces(x_f32, threads);
  Shape s = shape_of(C, pieces, threads);
  const int units = fwd_depth(threads, x_f32) * pieces * (x_f32 ? 2 : 1);
  set_blocks(&s, T, sm_count, fwd_per_sm(threads), static_cast<size_t>(units) * std::max(s.block, ring_stride(pieces, threads)) * 16 + static_cast<size_t>(s.tpr) * pieces * 64);
  return s;
}

Shape bwd_base(int64_t C, bool f32) { return shape_of(C, C > (f32 ? 8192 : 4096) ? 4 : 2, threads_of(C)); }

Shape bwd_shape(int64_t T, int64_t C, bool x_f32, bool g_f32, int sm_count) {
  Shape s = bwd_base(C, x_f32 || g_f32);
  const int units = bwd_depth(s.pieces, x_f32, g_f32) * s.pieces * ((x_f32 ? 2 : 1) + (g_f32 ? 2 : 1));
  // (a block's sums of several rows at a time take the place of the rows ahead: 64 bytes a thread and piece, of two threads or more)
  set_blocks(&s, T, sm_count, bwd_per_sm(s.threads), static_cast<size_t>(units) * std::max(s.block, ring_stride(s.pieces, s.threads)) * 16 + static_cast<size_t>(s.tpr) * s.pieces * 32);
  return s;
}

template <typename F>
void by_bool(bool v, F f) {
  v ? f(std::true_type()) : f(std::false_type());
}

// (pieces, threads) of the forward pass
template <typename F>
void by_fwd_shape(int threads, bool x_f32, F f) {
  by_bool(x_f32, [&](auto xf) {
    by_bool(threads == 512, [&](auto large) {
      constexpr bool X = decltype(xf)::value, LARGE = decltype(large)::value;
      f(xf, std::integral_constant<int, fwd_pieces(X, LARGE ? 512 : 256)>(), std::integral_constant<int, LARGE ? 512 : 256>());
    });
  });
}

// (pieces, threads) of the backward pass; F32: of FP32 rows or gradients, which alone take two pieces above 4096 columns
template <bool F32, typename F>
void by_bwd_shape(const Shape& s, F f) {
  if (s.threads == 256) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 256>());
  if constexpr (F32)
    if (s.pieces == 2) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 512>());
  f(std::integral_constant<int, 4>(), std::integral_constant<int, 512>());
}

dp_status check_vector(const void* p) { return is_aligned16(p) ? DP_OK : DP_ERR_ALIGNMENT; }

dp_status check_norm(int64_t T, int64_t C) {
  if (T < 0 || C < 1) return DP_ERR_INVALID_ARG;
  if (C % 8 != 0 || C > kMaxCols || T > 0x7FFFFFFF) return DP_ERR_UNSUPPORTED;
  return DP_OK;
}

// (for any types: as many blocks as registers allow)
int64_t bwd_bytes(int64_t T, int64_t C, int sm_count) {
  int64_t blocks = 0;
  for (bool f32 : {false, true}) {
    Shape s = bwd_base(C, f32);
    set_blocks(&s, T, sm_count, bwd_per_sm(s.threads), 0);
    blocks = std::max(blocks, s.blocks);
  }
  return blocks * 2 * C * 4;
}

bool flag(int v) { return v == 0 || v == 1; }

}  // namespace

cudaError_t set_attributes_layer_norm() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void* kernel) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
  };
  for (int i = 0; i < 4; ++i)
    by_fwd_shape(i & 2 ? 512 : 256, i & 1, [&](auto xf, auto pieces, auto threads) {
      set(reinterpret_cast<const void*>(&norm_fwd_kernel<decltype(xf)::value, decltype(pieces)::value, decltype(threads)::value>));
    });
  for (int i = 0; i < 12; ++i) {
    Shape s = {};
    s.pieces = i / 4 == 2 ? 4 : 2, s.threads = i / 4 == 0 ? 256 : 512;
    by_bool(i & 1, [&](auto xf) {
      by_bool(i & 2, [&](auto gf) {
        constexpr bool X = decltype(xf)::value, G = decltype(gf)::value;
        by_bwd_shape<X || G>(s, [&](auto pieces, auto threads) {
          set(reinterpret_cast<const void*>(&norm_bwd_kernel<X, G, decltype(pieces)::value, decltype(threads)::value>));
        });
      });
    });
  }
  return e;
}

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
  const Shape s = fwd_shape(T, C, x_f32, ctx.sm_count);
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.w = weight, a.b = bias, a.w_f32 = weight_f32, a.eps = static_cast<float>(eps);
  a.T = T, a.C = static_cast<int32_t>(C), a.tpr = s.tpr, a.inv_c = 1.0f / static_cast<float>(C);
  a.y = y, a.ldy = ldy, a.mean = mean, a.rstd = rstd;
  a.few = T <= s.blocks * s.rows;
  a.y_f32 = code;
  const unsigned grid = static_cast<unsigned>(s.blocks);
  cudaStream_t str = static_cast<cudaStream_t>(stream);
  by_fwd_shape(s.threads, x_f32, [&](auto xf, auto pieces, auto threads) {
    norm_fwd_kernel<decltype(xf)::value, decltype(pieces)::value, decltype(threads)::value><<<grid, s.block, s.smem, str>>>(a);
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
  const Shape s = bwd_shape(T, C, x_f32, dy_f32, ctx.sm_count);
  if (dw != nullptr) {
    if (workspace == nullptr || workspace_bytes < static_cast<size_t>(bwd_bytes(T, C, ctx.sm_count))) return DP_ERR_WORKSPACE;
    if (!is_aligned16(workspace)) return DP_ERR_ALIGNMENT;
  }
  NormArgs a = {};
  a.x = x, a.ldx = ldx, a.w = weight, a.w_f32 = weight_f32;
  a.T = T, a.C = static_cast<int32_t>(C), a.tpr = s.tpr, a.inv_c = 1.0f / static_cast<float>(C);
  a.y = dx, a.ldy = ld_dx, a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.dy = dy, a.ldg = ldg, a.partial = dw ? static_cast<float*>(workspace) : nullptr;
  a.y_f32 = code;
  const unsigned grid = static_cast<unsigned>(s.blocks);
  by_bool(x_f32, [&](auto xf) {
    by_bool(dy_f32, [&](auto gf) {
      constexpr bool X = decltype(xf)::value, G = decltype(gf)::value;
      by_bwd_shape<X || G>(s, [&](auto pieces, auto threads) {
        constexpr int CH = decltype(pieces)::value, N = decltype(threads)::value;
        norm_bwd_kernel<X, G, CH, N><<<grid, s.block, s.smem, str>>>(a);
      });
    });
  });
  if (cudaGetLastError() != cudaSuccess) return DP_ERR_LAUNCH;
  if (dw == nullptr) return DP_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((2 * C + 31) / 32));
  cfg.blockDim = dim3(1024);
  cfg.stream = str;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_sum_kernel, static_cast<const float*>(a.partial), static_cast<int>(s.blocks),
                                           static_cast<int>(C), dw, db);
  return e == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

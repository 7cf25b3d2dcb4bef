// C ABI of the products grouped by expert and of the 8-bit products (declared in
// include/dp_gemm.h): argument checks, tile width, tensor maps, one launch.  Nothing here
// allocates device memory, copies or synchronises.
#include <algorithm>
#include <atomic>
#include <cstring>

#include "api_internal.h"
#include "promoted_gemm.cuh"

namespace {

using namespace dp;

constexpr int64_t kMaxInt = 0x7FFFFFFF;
constexpr int64_t kPairRows = 384;  // rows per expert, on average, from which pairs pay

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile width: the widest that gives the SMs `least` tiles.  Wide tiles read A less often and keep
// the tensor cores fed: a 128 x 256 tile needs 96 bytes of operands per cycle, a 128 x 64 tile
// 192 (16384 rows over 64 experts, 4096 -> 2048: 263 us at 256 columns, 299 at 128, 408 at 64).
// One tile per SM is enough for them, two where a few rows stream their experts' weights and
// the last tiles' share of the SMs counts (64 rows over 64 experts, 4096 -> 1024: 74 us at 256
// columns, 53 to 68 at 128 by how many experts have rows, 69 at 64).
int tile_width(int64_t tiles_m, int64_t gn, int64_t least) {
  for (int bn = 256; bn > 64; bn /= 2)
    if (tiles_m * cdiv(gn, bn) >= least) return bn;
  return 64;
}

// Row tiles per raster group: as many rows of A as fill a share of L2 beside the weights.
int raster_rows(int64_t tile_rows, int64_t k_bytes) {
  const int64_t rows = (int64_t{48} << 20) / std::max<int64_t>(1, tile_rows * k_bytes);
  return static_cast<int>(std::min<int64_t>(64, std::max<int64_t>(4, rows)));
}

// Rows of A a load brings: where there are fewer than a tile's 128, just those, in whole swizzle
// rows of 8 (the accumulator's other rows come from stale shared memory and are not stored).
int rows_loaded(int64_t rows) { return static_cast<int>(std::min<int64_t>(128, cdiv(rows, 8) * 8)); }

dp_status zero_rows(void* out, int64_t rows, int64_t cols, int64_t ld, int esize, cudaStream_t stream) {
  if (rows == 0) return DP_OK;
  return cudaMemset2DAsync(out, static_cast<size_t>(ld) * esize, 0, static_cast<size_t>(cols) * esize,
                           static_cast<size_t>(rows), stream) == cudaSuccess
             ? DP_OK
             : DP_ERR_LAUNCH;
}

// ------------------------------------------------ how an 8-bit product is launched

struct Fp8Plan {
  int bn, form, split;  // bn 0: no form meets the overrides
};

// Clusters that run at one time, asked once per kernel, size and device.
int cluster_capacity(int dev, int kind, int bn, int split) {
  static std::atomic<int> known[kMaxDevices][3][2][9];  // capacity + 1; 0: not asked yet
  std::atomic<int>& entry = known[dev][kind - kFp8KK][bn == 256][split];
  int n = entry.load(std::memory_order_relaxed);
  if (n == 0) {
    n = max_clusters_fp8(kind, bn, split) + 1;
    entry.store(n, std::memory_order_relaxed);
  }
  return n - 1;
}

// The form of least modelled time.  A CTA's time is its blocks (128 contraction elements) at
// the rate measured for its tile, whole waves of tiles counted.  Measured on GB300 (forced
// forms, 34 shapes), ns a block: 128 x 128 215, 128 x 256 405, pairs of 256 x 256 440 while one
// wave suffices; with more waves 255 / 410 / 400, as narrow tiles then wait for L2 and pairs,
// which load least, do not (16384 x 12288 -> 4096: 795 / 559 / 537 us; 4031 x 4096 -> 4096: 62.0 /
// 57.5 / 57.8).  With column scales, whose promotion takes twice the operations and reads every
// column's scale, it is 350 / 595 / 585 for both.  A split adds its exchange: barriers of the
// cluster, and the tile's rows through its shared memory.  DP_FORCE_BN, DP_FORCE_PAIR and
// DP_FORCE_SPLITS leave only the forms that they name (a split then need not run in one wave).
Fp8Plan plan_fp8(int kind, int64_t gm, int64_t gn, int64_t nkb, const DeviceContext& ctx) {
  struct Rates {
    double one_wave, more;
  };
  const bool cols = kind == kFp8MM;
  const int sm_count = ctx.sm_count;
  const Rates r128 = cols ? Rates{350, 350} : Rates{215, 255}, r256 = cols ? Rates{595, 595} : Rates{405, 410},
              r_pair = cols ? Rates{585, 585} : Rates{440, 400};
  const int want_bn = tuning_override("DP_FORCE_BN", 0), want_pair = tuning_override("DP_FORCE_PAIR", -1),
            want_split = tuning_override("DP_FORCE_SPLITS", 0);
  Fp8Plan best = {0, kPlain, 1};
  double least = 1e30;
  auto offer = [&](int bn, int form, int split, int64_t tiles, int64_t slots, const Rates& r) {
    if ((want_bn > 0 && bn != want_bn) || (want_pair >= 0 && (form == kPair) != (want_pair != 0)) ||
        (want_split > 0 && split != want_split))
      return;
    const int64_t waves = cdiv(tiles, slots);
    double t = static_cast<double>(waves * cdiv(nkb, split)) * (waves == 1 ? r.one_wave : r.more);
    if (form == kSplit) t += 2300.0 + 200.0 * split + 12.0 * static_cast<double>(std::min<int64_t>(gm, 128)) * bn / 256;
    if (t < least) least = t, best = {bn, form, split};
  };
  offer(256, kPair, 1, cdiv(gm, 256) * cdiv(gn, 256), sm_count / 2, r_pair);
  for (int bn = 256; bn >= 128; bn /= 2) {
    const int64_t tiles = cdiv(gm, 128) * cdiv(gn, bn);
    const Rates& r = bn == 256 ? r256 : r128;
    offer(bn, kPlain, 1, tiles, sm_count, r);
    for (int split = 2; split <= 8 && split <= nkb; ++split) {
      if (want_split == 0 && tiles * split > sm_count) break;
      const int64_t room = cluster_capacity(ctx.device, kind, bn, split);
      if (want_split > 0 ? room > 0 : tiles <= room) offer(bn, kSplit, split, tiles, std::max<int64_t>(1, std::min(tiles, room)), r);
    }
  }
  return best;
}

enum GroupedOp { kFwd, kDgrad, kWgrad };

// fwd:   a = X [T][K],  b = W,        out = Y [T][N]
// dgrad: a = dY [T][N], b = W,        out = dX [T][K]
// wgrad: a = dY [T][N], b = X [T][K], out = dW
// W and dW: [E][N][K], or [E][K][N] with kn.
dp_status run_grouped(GroupedOp op, const void* a, int64_t lda, const void* b, int64_t ldb, int64_t bsb,
                      const void* offsets, int offset_bits, void* out, int64_t ldo, int64_t bso, int kn, int64_t E,
                      int64_t T, int64_t N, int64_t K, int out_f32, cudaStream_t stream) {
  if (out_f32 != DP_OUT_BF16 && out_f32 != DP_OUT_F32) return DP_ERR_INVALID_ARG;
  if ((kn != 0 && kn != 1) || E < 0 || T < 0 || N < 1 || K < 1 || bsb < 0 || bso < 0) return DP_ERR_INVALID_ARG;
  if (offset_bits != 32 && offset_bits != 64) return DP_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0) return DP_ERR_UNSUPPORTED;
  if (E > kMaxExperts || T > kMaxInt - 256 || N > kMaxInt - 256 || K > kMaxInt - 256) return DP_ERR_UNSUPPORTED;
  const int osize = out_f32 ? 4 : 2;
  const int64_t a_cols = op == kFwd ? K : N;
  const int64_t w_rows = kn ? K : N, w_cols = kn ? N : K;
  const int64_t out_rows = op == kWgrad ? w_rows : T, out_cols = op == kFwd ? N : op == kDgrad ? K : w_cols;
  dp_status st = check_operand(a, T, a_cols, &lda, 2);
  if (st == DP_OK) st = op == kWgrad ? check_operand(b, T, K, &ldb, 2) : check_operand(b, E * w_rows, w_cols, &ldb, 2);
  if (st == DP_OK) st = check_operand(out, op == kWgrad ? E * out_rows : out_rows, out_cols, &ldo, osize);
  if (st != DP_OK) return st;
  if (offsets == nullptr && E > 0) return DP_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(offsets) & (offset_bits / 8 - 1)) != 0) return DP_ERR_ALIGNMENT;
  if (bsb == 0) bsb = w_rows * ldb;
  if (bso == 0) bso = w_rows * ldo;
  if (op != kWgrad && bsb * 2 % 16 != 0) return DP_ERR_ALIGNMENT;
  if (op == kWgrad && bso * osize % 16 != 0) return DP_ERR_ALIGNMENT;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (E == 0) return op == kWgrad ? DP_OK : zero_rows(out, T, out_cols, ldo, osize, stream);
  if (T == 0) {
    if (op != kWgrad) return DP_OK;
    for (int64_t e = 0; e < E; ++e)
      if ((st = zero_rows(static_cast<char*>(out) + e * bso * osize, out_rows, out_cols, ldo, osize, stream)) != DP_OK)
        return st;
    return DP_OK;
  }

  PgLaunch l;
  std::memset(&l, 0, sizeof(l));
  PgArgs& g = l.args;
  g.rows = static_cast<int32_t>(T);
  g.experts = static_cast<int32_t>(E);
  g.offsets = offsets;
  g.offsets64 = offset_bits == 64;
  g.out = out;
  g.ldo = ldo;
  g.out_gstride = bso;
  g.out_f32 = out_f32;
  g.fault = ctx.fault;
  g.wait_ns = kWaitLimitNs;
  const auto bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  int kind, bn, form = kPlain;
  int64_t tiles;
  bool ok;
  if (op == kWgrad) {
    // dW[n][k] with A = dY, B = X; dW stored [K][N]: A = X, B = dY
    const int64_t gm = w_rows, gn = w_cols;
    kind = kGroupMM;
    g.gm = static_cast<int32_t>(gm);
    g.gn = static_cast<int32_t>(gn);
    bn = tile_width(E * cdiv(gm, 128), gn, ctx.sm_count);
    g.tiles_m = static_cast<int32_t>(cdiv(gm, 128));
    g.tiles_n = static_cast<int32_t>(cdiv(gn, bn));
    g.group_m = 8;
    tiles = E * g.tiles_m * g.tiles_n;
    const void *pa = kn ? b : a, *pb = kn ? a : b;
    const int64_t la = kn ? ldb : lda, lb = kn ? lda : ldb;
    ok = encode_operand(&l.tmA, pa, bf16, 2, T, gm, la, 0, 0, 64, 64) &&
         encode_operand(&l.tmB, pb, bf16, 2, T, gn, lb, 0, 0, 64, 64);
  } else {
    const int64_t gk = a_cols, gn = out_cols;
    const bool b_mn = (op == kFwd) == (kn != 0);  // W's rows are contraction rows
    kind = b_mn ? kGroupKM : kGroupKK;
    g.gn = static_cast<int32_t>(gn);
    g.gk = static_cast<int32_t>(gk);
    // (the groups' sizes are known on the device only: at most one partial tile per group)
    // Pairs of SMs on tiles of 256 rows load a third less per SM and keep six stages in flight
    // instead of four, but round every group up to 256 rows (16384 rows, 4096 -> 4096: over 8
    // experts 311 us against 332 on single SMs, over 32 386 against 402; over 64 at 4096 -> 2048
    // no difference, over 128 at 2048 -> 2048 205 against 199).
    const bool pair = T >= kPairRows * E && cdiv(T, 256) * cdiv(gn, 256) >= ctx.sm_count / 2;
    form = pair ? kPair : kPlain;
    const int64_t tiles_m = T / (pair ? 256 : 128) + std::min(E, T);
    bn = pair ? 256 : tile_width(std::max(cdiv(T, 128), std::min(E, T)), gn,
                                 T <= 32 * E ? 2 * ctx.sm_count : ctx.sm_count);
    g.tiles_n = static_cast<int32_t>(cdiv(gn, bn));
    g.group_m = raster_rows(pair ? 256 : 128, gk * 2);
    tiles = tiles_m * g.tiles_n;
    g.a_rows = rows_loaded(T);
    ok = encode_operand(&l.tmA, a, bf16, 2, T, gk, lda, 0, 0, 64, static_cast<uint32_t>(g.a_rows)) &&
         (b_mn ? encode_operand(&l.tmB, b, bf16, 2, w_rows, w_cols, ldb, E, bsb, 64, 64)
               : encode_operand(&l.tmB, b, bf16, 2, w_rows, w_cols, ldb, E, bsb, 64, static_cast<uint32_t>(pair ? bn / 2 : bn)));
  }
  if (!ok) return DP_ERR_LAUNCH;
  if (tiles > kMaxInt) return DP_ERR_UNSUPPORTED;
  g.idesc = idesc_bf16_f32(form == kPair ? 256 : 128, bn, kind == kGroupMM, kind != kGroupKK);
  l.grid = static_cast<int>(form == kPair ? 2 * std::min<int64_t>(ctx.sm_count / 2, tiles)
                                          : std::min<int64_t>(ctx.sm_count, tiles));
  return launch_grouped(kind, bn, form, l, stream) == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

struct Scales {
  const float* p;
  int64_t row, blk;
};

dp_status check_scales(const Scales& s) {
  if (s.p == nullptr || s.row < 0 || s.blk < 0) return DP_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(s.p) & 3) != 0 ? DP_ERR_ALIGNMENT : DP_OK;
}

dp_status run_fp8(GroupedOp op, const void* a, int64_t lda, int a_fmt, Scales sa, const void* b, int64_t ldb, int b_fmt,
                  Scales sb, void* out, int64_t ldo, int64_t T, int64_t N, int64_t K, int out_f32,
                  cudaStream_t stream) {
  if (out_f32 != DP_OUT_BF16 && out_f32 != DP_OUT_F32) return DP_ERR_INVALID_ARG;
  if (a_fmt < DP_FP8_E4M3 || a_fmt > DP_FP8_E5M2 || b_fmt < DP_FP8_E4M3 || b_fmt > DP_FP8_E5M2)
    return DP_ERR_INVALID_ARG;
  if (T < 0 || N < 1 || K < 1) return DP_ERR_INVALID_ARG;
  if (N % 16 != 0 || K % 16 != 0) return DP_ERR_UNSUPPORTED;
  if (T > kMaxInt - 256 || N > kMaxInt - 256 || K > kMaxInt - 256) return DP_ERR_UNSUPPORTED;
  const int osize = out_f32 ? 4 : 2;
  const int64_t gm = op == kWgrad ? N : T, gn = op == kFwd ? N : K, gk = op == kFwd ? K : op == kDgrad ? N : T;
  dp_status st = check_operand(a, T, op == kFwd ? K : N, &lda, 1);
  if (st == DP_OK) st = op == kWgrad ? check_operand(b, T, K, &ldb, 1) : check_operand(b, N, K, &ldb, 1);
  if (st == DP_OK) st = check_operand(out, gm, gn, &ldo, osize);
  if (st != DP_OK) return st;
  if (T > 0) {
    if ((st = check_scales(sa)) != DP_OK || (st = check_scales(sb)) != DP_OK) return st;
  }
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  if (T == 0) return op == kWgrad ? zero_rows(out, gm, gn, ldo, osize, stream) : DP_OK;

  PgLaunch l;
  std::memset(&l, 0, sizeof(l));
  PgArgs& g = l.args;
  const int kind = op == kFwd ? kFp8KK : op == kDgrad ? kFp8KM : kFp8MM;
  const Fp8Plan plan = plan_fp8(kind, gm, gn, cdiv(gk, 128), ctx);
  if (plan.bn == 0) return DP_ERR_UNSUPPORTED;
  const int bn = plan.bn, tm = plan.form == kPair ? 256 : 128;
  g.rows = static_cast<int32_t>(gm);
  g.gm = static_cast<int32_t>(gm);
  g.gn = static_cast<int32_t>(gn);
  g.gk = static_cast<int32_t>(gk);
  g.experts = 1;
  g.out = out;
  g.ldo = ldo;
  g.out_f32 = out_f32;
  g.tiles_m = static_cast<int32_t>(cdiv(gm, tm));
  g.tiles_n = static_cast<int32_t>(cdiv(gn, bn));
  g.split = plan.split;
  g.a_rows = plan.form == kPair ? 128 : rows_loaded(gm);
  g.group_m = raster_rows(tm, gk);
  g.idesc = idesc_fp8_f32(tm, std::min(bn, 128), kind == kFp8MM, kind != kFp8KK, a_fmt == DP_FP8_E5M2, b_fmt == DP_FP8_E5M2);
  g.sa = sa.p;
  g.sa_row = sa.row;
  g.sa_blk = sa.blk;
  g.sb = sb.p;
  // (input gradient: the contraction runs along W's rows, so their block index is the chunk)
  g.sb_row = op == kDgrad ? sb.blk : sb.row;
  g.sb_blk = op == kDgrad ? sb.row : sb.blk;
  g.fault = ctx.fault;
  g.wait_ns = kWaitLimitNs;
  const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const bool ok =
      (kind == kFp8MM ? encode_operand(&l.tmA, a, u8, 1, gk, gm, lda, 0, 0, 128, 128)
                      : encode_operand(&l.tmA, a, u8, 1, gm, gk, lda, 0, 0, 128, static_cast<uint32_t>(g.a_rows))) &&
      (kind == kFp8KK ? encode_operand(&l.tmB, b, u8, 1, gn, gk, ldb, 0, 0, 128, static_cast<uint32_t>(plan.form == kPair ? bn / 2 : bn))
                      : encode_operand(&l.tmB, b, u8, 1, gk, gn, ldb, 0, 0, 128, 128));
  if (!ok) return DP_ERR_LAUNCH;
  const int64_t tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
  if (tiles * plan.split > kMaxInt) return DP_ERR_UNSUPPORTED;
  l.grid = static_cast<int>(plan.form == kPair    ? 2 * std::min<int64_t>(ctx.sm_count / 2, tiles)
                            : plan.form == kSplit ? tiles * plan.split
                                                  : std::min<int64_t>(ctx.sm_count, tiles));
  return launch_fp8(kind, bn, plan.form, l, stream) == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

}  // namespace

extern "C" {

dp_status dp_gemm_fwd_grouped(const void* X, int64_t ldx, const void* W, int64_t ldw, int64_t bsw, int weight_kn,
                              const void* offsets, int offset_bits, void* Y, int64_t ldy, int64_t E, int64_t T,
                              int64_t N, int64_t K, dp_out_dtype out, dp_stream stream) {
  return run_grouped(kFwd, X, ldx, W, ldw, bsw, offsets, offset_bits, Y, ldy, 0, weight_kn, E, T, N, K,
                     static_cast<int>(out), static_cast<cudaStream_t>(stream));
}

dp_status dp_gemm_dgrad_grouped(const void* dY, int64_t ldg, const void* W, int64_t ldw, int64_t bsw, int weight_kn,
                                const void* offsets, int offset_bits, void* dX, int64_t ldx, int64_t E, int64_t T,
                                int64_t N, int64_t K, dp_out_dtype out, dp_stream stream) {
  return run_grouped(kDgrad, dY, ldg, W, ldw, bsw, offsets, offset_bits, dX, ldx, 0, weight_kn, E, T, N, K,
                     static_cast<int>(out), static_cast<cudaStream_t>(stream));
}

dp_status dp_gemm_wgrad_grouped(const void* dY, int64_t ldg, const void* X, int64_t ldx, const void* offsets,
                                int offset_bits, void* dW, int64_t ldw, int64_t bsw, int weight_kn, int64_t E,
                                int64_t T, int64_t N, int64_t K, dp_out_dtype out, dp_stream stream) {
  return run_grouped(kWgrad, dY, ldg, X, ldx, 0, offsets, offset_bits, dW, ldw, bsw, weight_kn, E, T, N, K,
                     static_cast<int>(out), static_cast<cudaStream_t>(stream));
}

dp_status dp_gemm_fwd_fp8(const void* Xq, int64_t ldx, dp_fp8_format x_format, const float* Xs, int64_t xs_row,
                          int64_t xs_blk, const void* Wq, int64_t ldw, dp_fp8_format w_format, const float* Ws,
                          int64_t ws_row, int64_t ws_col, void* Y, int64_t ldy, int64_t T, int64_t N, int64_t K,
                          dp_out_dtype out, dp_stream stream) {
  return run_fp8(kFwd, Xq, ldx, static_cast<int>(x_format), {Xs, xs_row, xs_blk}, Wq, ldw, static_cast<int>(w_format),
                 {Ws, ws_row, ws_col}, Y, ldy, T, N, K, static_cast<int>(out), static_cast<cudaStream_t>(stream));
}

dp_status dp_gemm_dgrad_fp8(const void* dYq, int64_t ldg, dp_fp8_format dy_format, const float* dYs, int64_t gs_row,
                            int64_t gs_blk, const void* Wq, int64_t ldw, dp_fp8_format w_format, const float* Ws,
                            int64_t ws_row, int64_t ws_col, void* dX, int64_t ldx, int64_t T, int64_t N, int64_t K,
                            dp_out_dtype out, dp_stream stream) {
  return run_fp8(kDgrad, dYq, ldg, static_cast<int>(dy_format), {dYs, gs_row, gs_blk}, Wq, ldw,
                 static_cast<int>(w_format), {Ws, ws_row, ws_col}, dX, ldx, T, N, K, static_cast<int>(out),
                 static_cast<cudaStream_t>(stream));
}

dp_status dp_gemm_wgrad_fp8(const void* dYq, int64_t ldg, dp_fp8_format dy_format, const float* dYs, int64_t gs_blk,
                            int64_t gs_col, const void* Xq, int64_t ldx, dp_fp8_format x_format, const float* Xs,
                            int64_t xs_blk, int64_t xs_col, void* dW, int64_t ldw, int64_t T, int64_t N, int64_t K,
                            dp_out_dtype out, dp_stream stream) {
  return run_fp8(kWgrad, dYq, ldg, static_cast<int>(dy_format), {dYs, gs_col, gs_blk}, Xq, ldx,
                 static_cast<int>(x_format), {Xs, xs_col, xs_blk}, dW, ldw, T, N, K, static_cast<int>(out),
                 static_cast<cudaStream_t>(stream));
}

}  // extern "C"

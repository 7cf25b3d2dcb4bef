// Persistent tensor-core GEMM whose accumulators are promoted into registers:
//     D[m][n] = sum over chunks c of  sa(m, c) sb(n, c)  sum_{k in c} A(m, k) B(n, k)
// for the products grouped by expert (BF16, scales 1) and the 8-bit products with a
// scale per 128 contraction elements (a chunk is then one 128-element block).
//
// One CTA per SM walks the list of output tiles (128 x BN), 384 threads:
//   warp 0       TMA loads of A    (stages of 128 bytes x 128 rows, 128-byte swizzle)
//   warp 1       TMEM allocation and tcgen05.mma; for ragged contractions it also zeroes
//                the rows of the last block that belong to the next group
//   warp 2       TMA loads of B
//   warp 3       8-bit products: the chunks' scales, through registers into a ring
//   warps 4..11  promotion and epilogue: read a finished chunk's accumulator from TMEM,
//                add it (scaled) to FP32 registers; after the last chunk, round once and
//                store.  Warp w holds rows 32 (w % 4) .. + 32 and one half of the columns.
// A chunk's accumulator is one of two TMEM buffers of the tile's width (8-bit tiles of 256
// columns: two of four halves, each promoted by its own four warps), so the promotion of one
// chunk runs beside the MMAs of the next.
//
// What bounds it, measured on GB300:
//   grouped, few rows: the experts' weights from HBM (64 rows over 64 experts, 4096 -> 1024: 59-67 us,
//     5.1-5.8 TB/s, by where the weights lie; 4031 rows over 32: 60 us);
//   grouped, training: HBM and MMAs about equally (16384 rows over 64 experts, 4096 -> 2048: input
//     gradient 250-275 us, 1.0-1.1 PFLOP/s beside 4.6-5.1 TB/s), the weight gradient its FP32 output
//     (407-430 us, 5.5-5.8 TB/s; shared-memory bandwidth 79% busy with the operands);
//   8-bit: the promotion.  A 128 x 256 block's MMAs take 512 cycles; reading its sums from TMEM (145
//     cycles), adding them (256 at the FP32 pipe's rate) and the waits around them one after
//     another about 690, with column scales and their second multiplication 1100 (T = 16384,
//     12288 -> 4096: 591-622 us, 2.7 PFLOP/s; weight gradient T = 16173, 1024 x 4096: 80 us).  Asking
//     for the next chunk before adding this one took 4 to 7% off; more promoting warps, reading
//     the next chunk's first columns early and spinning waits took nothing.
//
// Why promotion: (1) the scale of a 128-element block multiplies that block's sum only,
// so it cannot be applied after the whole contraction; (2) the tensor core rounds every
// FP32 accumulate toward zero, an error that grows with the length of one accumulator
// (relative RMS 1.9e-5 at 16384 elements, measured in tests of the dense path), while the
// register sums round to nearest: BF16 chunks of 512 elements keep it at 4.8e-7 whatever the
// length (2048: 2.1e-6; 256: 2.4e-7, but 2 to 5% slower from 256 rows a group on).
//
// Groups (experts): their row ranges come from an offsets array in device memory that the
// host never reads.  Every CTA turns it into a table in shared memory (clamped to [0, T]
// and to a running maximum, so no content of the array leads out of bounds) and finds its
// tiles there by binary search.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"

namespace dp {

// Operand forms.  G: BF16 grouped by expert; F: 8-bit with block scales.  Then A's and
// B's majorness: K (rows of contraction elements) or M (contraction rows).
enum PgKind : int {
  kGroupKK = 0,  // A row-grouped [T][gk], B [E][gn][gk]
  kGroupKM = 1,  // A row-grouped [T][gk], B [E][gk][gn]
  kGroupMM = 2,  // contraction grouped: A [T][gm], B [T][gn], D [E][gm][gn]
  kFp8KK = 3,    // A [gm][gk] (scale per row and block), B [gn][gk] (scale per 128 x 128)
  kFp8KM = 4,    // A as above, B [gk][gn] (scale per 128 x 128)
  kFp8MM = 5,    // A [gk][gm], B [gk][gn] (scale per column and block, both)
};

constexpr int kMaxExperts = 1024;
constexpr int kScaleAhead = 3;  // 8-bit products: how many chunks ahead scales are loaded
constexpr int kPgChunk = 8;   // BF16: contraction blocks of 64 per accumulator

struct PgArgs {
  int32_t rows;        // T: rows of A and D (row-grouped), contraction rows (contraction-grouped)
  int32_t gm, gn, gk;  // dense sizes; row-grouped: gm unused; contraction-grouped: gk unused
  int32_t experts;     // groups (8-bit products: 1)
  int32_t offsets64;   // offsets are int64
  const void* offsets; // [experts + 1]
  void* out;
  int64_t ldo, out_gstride;  // elements; out_gstride: between experts' outputs (contraction-grouped)
  int32_t out_f32;
  int32_t tiles_m, tiles_n;  // (row-grouped: tiles_m unused)
  int32_t group_m;           // raster: row tiles that share a column tile's operand in L2
  int32_t a_rows;            // rows of A a load brings (K-major A; 128, or all rows where there are fewer)
  int32_t split;             // kSplit: CTAs that share a tile (2..8)
  uint32_t idesc;
  const float* sa;           // 8-bit products: scale of row m, block c at sa[m * sa_row + c * sa_blk]
  int64_t sa_row, sa_blk;
  const float* sb;           // of column (or 128-column block) n, block c
  int64_t sb_row, sb_blk;
  uint32_t* fault;
  uint64_t wait_ns;
};

// Forms of a launch.  kSplit: clusters of `split` CTAs share a tile's contraction, one range of
// blocks each, and the first sums the others' tiles from their shared memory in rank order:
// for few tiles, whose operands one CTA each would stream too slowly.
// kPair: a cluster of two CTAs computes one tile of 256 x BN.  Each loads its 128 rows of A
// and half of the tile's columns of B, the leader (rank 0) issues the MMAs over both, and each
// promotes its 128 x BN half of the accumulator: a third less operand traffic per SM.
enum PgForm : int { kPlain = 0, kPair = 1, kSplit = 2 };

template <int BN, int KIND, int FORM = kPlain>
struct PgCfg {
  static constexpr bool PAIR = FORM == kPair, SPLIT = FORM == kSplit;
  static constexpr int TM = PAIR ? 256 : 128;     // rows of a tile
  static constexpr int BNL = PAIR ? BN / 2 : BN;  // columns of B a CTA loads
  static constexpr bool FP8 = KIND >= kFp8KK;
  static constexpr bool A_MN = KIND == kGroupMM || KIND == kFp8MM;
  static constexpr bool B_MN = KIND != kGroupKK && KIND != kFp8KK;
  static constexpr bool ROW_GROUPS = KIND == kGroupKK || KIND == kGroupKM;
  static constexpr bool K_GROUPS = KIND == kGroupMM;
  static constexpr int BM = 128;
  static constexpr int BK = FP8 ? 128 : 64;  // contraction elements per stage (128 bytes of a K-major row)
  static constexpr int MN = FP8 ? 128 : 64;  // columns of one MN-major box (128 bytes)
  static constexpr int SLICE = FP8 ? 32 : 16;  // contraction elements of one MMA
  static constexpr int A_BYTES = BM * 128;
  static constexpr int B_BYTES = BNL * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = (192 * 1024) / STAGE_BYTES < 8 ? (192 * 1024) / STAGE_BYTES : 8;
  // Accumulator buffers.  8-bit products commit every block: their MMAs are 128 columns wide
  // (as fast as 256) into four buffers, so that the tensor cores go on while two blocks are
  // promoted; with two buffers of 256 the promotion of a block had to end within the MMAs of the
  // next one.  At 256 columns the two groups of epilogue warps take one half each.
  static constexpr int SUB = FP8 && BN == 256 ? 128 : BN;  // columns of one MMA
  static constexpr int NSUB = BN / SUB;
  static constexpr int NBUF = FP8 ? 4 : 2;
  static constexpr int EPI_ARRIVALS = (NSUB == 2 ? 4 : 8) * (PAIR ? 2 : 1);  // per buffer
  static constexpr int HALF = BN / 2;  // columns of one epilogue warp
  static constexpr int EPI_BYTES = 8 * 2048;
  // 8-bit products: a ring of the chunks' scales, filled by warp 3: for each of the 128 rows its
  // scale times that of the tile's first and second 128 columns (128 x 128 blocks of B), or
  // the scales of the rows and then of the BN columns.
  static constexpr bool COL_SCALES = KIND == kFp8MM;
  // A promoting thread holds pairs of columns of four rows (16x256b) instead of one row.
  static constexpr bool QUADS = COL_SCALES || K_GROUPS;
  static constexpr int SCALE_FLOATS = COL_SCALES ? 128 + BN : 256;
  static constexpr int SCALE_SLOTS = !FP8 ? 1 : NSUB == 2 ? 8 : 16;
  static constexpr int SCALE_BYTES = FP8 ? SCALE_SLOTS * SCALE_FLOATS * 4 : 0;
  static constexpr int TABLE_BYTES = (ROW_GROUPS || K_GROUPS) ? 2 * (kMaxExperts + 4) * 4 : 0;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NBUF + 1;
  static constexpr int TMEM_COLS = NBUF * SUB;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + EPI_BYTES + SCALE_BYTES + TABLE_BYTES + NUM_BARS * 8 + 256;
  static constexpr int THREADS = 384;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(BN == 64 || BN == 128 || BN == 256, "tile width");
  static_assert(!SPLIT || FP8, "split contractions are built for the 8-bit products");
  static_assert(!SPLIT || STAGES * STAGE_BYTES >= BM * BN * 4, "a split tile passes through the operand ring");
  static_assert(!(PAIR && K_GROUPS), "the leader zeroes ragged rows in its own shared memory only");
  static_assert(!(FP8 && B_MN) || BNL >= 128, "8-bit MN-major boxes are 128 columns wide");
};

// tcgen05.mma on operands given by the halves of their shared-memory descriptors.  The low
// half holds the start address >> 4 and the leading offset, the high half (constant over a
// kernel) the stride and the layout: stepping through stages and slices is one 32-bit add, which
// stays in uniform registers.  (8-bit operands: E4M3 or E5M2 each, as the instruction
// descriptor says.)
template <bool FP8, bool PAIR>
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
#define DP_MMA(GROUP, TYPE)                                                                      \
  asm volatile(                                                                                  \
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"                                              \
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"                                       \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                \
      "tcgen05.mma.cta_group::" GROUP ".kind::" TYPE " [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem), \
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)                    \
      : "memory")
  if (FP8 && PAIR)
    DP_MMA("2", "f8f6f4");
  else if (FP8)
    DP_MMA("1", "f8f6f4");
  else if (PAIR)
    DP_MMA("2", "f16");
  else
    DP_MMA("1", "f16");
#undef DP_MMA
}

// Instruction descriptor, kind::f8f6f4 with FP32 D: as idesc_bf16_f32, formats 0 = E4M3, 1 = E5M2.
constexpr uint32_t idesc_fp8_f32(int m, int n, bool a_mn, bool b_mn, bool a_e5m2, bool b_e5m2) {
  return (1u << 4) | ((a_e5m2 ? 1u : 0u) << 7) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// One output tile of the list.
struct PgTile {
  int e;       // expert
  int row0;    // first row in A (row-grouped) / first contraction row (contraction-grouped)
  int tm, tn;  // tile coordinates inside the group's output
  int m_left;  // rows of the tile that exist (may exceed 128)
  int nkb;     // contraction blocks
  int k_left;  // contraction elements
  int kb0;     // first contraction block (of this CTA's share)
};

template <int N>
struct Int {
  static constexpr int value = N;
};

template <int BN, int KIND, int FORM>
struct PgWalk {
  using C = PgCfg<BN, KIND, FORM>;
  const PgArgs& a;
  const int32_t* start;  // [experts + 1] first row of each group
  const int32_t* first;  // [experts + 1] first tile of each group (row-grouped)
  __device__ __forceinline__ int units() const {
    if (C::ROW_GROUPS) return first[a.experts];
    return a.tiles_m * a.tiles_n * (C::K_GROUPS ? a.experts : C::SPLIT ? a.split : 1);
  }
  // Tiles are rastered in groups of group_m row tiles, row tiles fastest: the CTAs that run
  // at one time share the column tile's operand and the group's rows in L2.
  __device__ __forceinline__ PgTile at(int u) const {
    PgTile t;
    int local, tiles_m;
    if (C::ROW_GROUPS) {
      int lo = 0, hi = a.experts - 1;  // the last group whose first tile is <= u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      t.e = lo;
      local = u - first[lo];
      const int cnt = start[lo + 1] - start[lo];
      tiles_m = (cnt + C::TM - 1) / C::TM;
      t.m_left = cnt;
      t.row0 = start[lo];
      t.k_left = a.gk;
    } else if (C::K_GROUPS) {
      const int per = a.tiles_m * a.tiles_n;
      t.e = u / per;
      local = u - t.e * per;
      tiles_m = a.tiles_m;
      t.m_left = a.gm;
      t.row0 = start[t.e];
      t.k_left = start[t.e + 1] - start[t.e];
    } else {
      t.e = 0;
      local = C::SPLIT ? u / a.split : u;
      tiles_m = a.tiles_m;
      t.m_left = a.gm;
      t.row0 = 0;
      t.k_left = a.gk;
    }
    const int per_group = a.group_m * a.tiles_n;
    const int g = local / per_group;
    const int m0 = g * a.group_m;
    const int width = min(a.group_m, tiles_m - m0);
    const int l2 = local - g * per_group;
    t.tm = m0 + l2 % width;
    t.tn = l2 / width;
    t.m_left -= t.tm * C::TM;
    if (C::ROW_GROUPS) t.row0 += t.tm * C::TM;
    t.nkb = (t.k_left + C::BK - 1) / C::BK;
    t.kb0 = 0;
    if (C::SPLIT) {
      const int s = u % a.split;
      t.kb0 = s * t.nkb / a.split;
      t.nkb = (s + 1) * t.nkb / a.split - t.kb0;
    }
    return t;
  }
};

// The groups' table: start[i] = running maximum of the offsets, clamped to [0, rows], and
// (row-grouped) first[i] = tiles of the groups before i.  Offsets that decrease or leave
// [0, rows] set kFaultOffsets.  All 384 threads call it; each takes `per` consecutive entries.
template <int BN, int KIND, int FORM>
__device__ __forceinline__ void build_group_table(const PgArgs& a, int32_t* start, int32_t* first, int32_t* scan) {
  using C = PgCfg<BN, KIND, FORM>;
  constexpr int NW = C::THREADS / 32;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int n = a.experts + 1;
  const int per = (n + C::THREADS - 1) / C::THREADS;  // 1..3
  int32_t v[3];
  bool bad = false;
  int32_t top = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    v[j] = 0;
    const int i = tid * per + j;
    if (j < per && i < n) {
      const int64_t raw = a.offsets64 ? static_cast<const int64_t*>(a.offsets)[i]
                                      : static_cast<const int32_t*>(a.offsets)[i];
      bad = bad || raw < 0 || raw > a.rows;
      v[j] = static_cast<int32_t>(raw < 0 ? 0 : raw > a.rows ? a.rows : raw);
      bad = bad || v[j] < top;
      top = max(top, v[j]);
      v[j] = top;
    }
  }
  int32_t incl = top;  // inclusive maximum over the threads
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl = max(incl, o);
  }
  int32_t excl = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) excl = 0;
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  for (int w = 0; w < warp; ++w) excl = max(excl, scan[w]);
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int i = tid * per + j;
    if (j < per && i < n) {
      bad = bad || v[j] < excl;  // (a later entry below an earlier thread's maximum)
      start[i] = max(v[j], excl);
    }
  }
  if (bad) atomicOr(a.fault, kFaultOffsets);
  __syncthreads();
  if (!C::ROW_GROUPS) return;
  int32_t tiles[3], sum = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int i = tid * per + j;
    tiles[j] = 0;
    if (j < per && i < a.experts) tiles[j] = (start[i + 1] - start[i] + C::TM - 1) / C::TM * a.tiles_n;
    sum += tiles[j];
  }
  int32_t tot = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, tot, d);
    if (lane >= d) tot += o;
  }
  int32_t before = tot - sum;
  if (lane == 31) scan[NW + warp] = tot;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += scan[NW + w];
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const int i = tid * per + j;
    if (j < per && i < n) first[i] = before;
    before += tiles[j];
  }
  __syncthreads();
}

// Pairs of FP32 values in one 64-bit register: one instruction for two operations.  Volatile,
// so that they stay behind the wait for the TMEM loads whose values they take (passing the
// values through the wait instead costs a register copy each).
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  return (static_cast<uint64_t>(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t pack_u32x2(uint32_t lo, uint32_t hi) { return (static_cast<uint64_t>(hi) << 32) | lo; }
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm volatile("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm volatile("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void st_shared_f2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
__device__ __forceinline__ float2 ld_shared_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint64_t ld_shared_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
// From a CTA of the cluster (a shared::cluster address).
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Registers move between the warpgroups: 384 x 168 at launch = 128 x 88 + 256 x 208.
template <int N>
__device__ __forceinline__ void regs_give() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The sum of a split tile: the cluster's CTAs share its columns in groups of eight; each of
// their 256 epilogue threads adds a row's eight values of all ranks, in rank order, and stores
// them.  `base`: where every CTA keeps its partial tile, [pair of columns][row].
template <int BN>
__device__ __forceinline__ void sum_split(const PgArgs& a, const PgTile& t, uint32_t base, int thread) {
  const int rank = static_cast<int>(cluster_rank()), rows = min(128, t.m_left);
  const int g0 = rank * (BN / 8) / a.split, g1 = (rank + 1) * (BN / 8) / a.split;
  for (int i = thread; i < (g1 - g0) * rows; i += 256) {
    const int g = g0 + i / rows, row = i % rows, col = t.tn * BN + 8 * g;
    if (col >= a.gn) break;  // (gn is a multiple of 16; later items lie further right)
    uint64_t sum[4] = {0, 0, 0, 0};
    for (int r = 0; r < a.split; ++r) {
      const uint32_t from = map_shared_rank(base + static_cast<uint32_t>(4 * g * 128 + row) * 8, static_cast<uint32_t>(r));
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] = add_f32x2(sum[j], ld_cluster_u64(from + j * (128 * 8)));
    }
    const int64_t at = (static_cast<int64_t>(t.tm) * 128 + row) * a.ldo + col;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[2 * j] = static_cast<uint32_t>(sum[j]), w[2 * j + 1] = static_cast<uint32_t>(sum[j] >> 32);
    if (a.out_f32) {
      uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(a.out) + at);
      p[0] = make_uint4(w[0], w[1], w[2], w[3]);
      p[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      auto pack = [&](int j) { return pack_bf16x2(__uint_as_float(w[j]), __uint_as_float(w[j + 1])); };
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) = make_uint4(pack(0), pack(2), pack(4), pack(6));
    }
  }
}

template <int BN, int KIND, int FORM>
__global__ void __launch_bounds__(PgCfg<BN, KIND, FORM>::THREADS, 1)
    promoted_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ PgArgs args) {
  using C = PgCfg<BN, KIND, FORM>;
  constexpr bool PAIR = C::PAIR;
  constexpr int STAGES = C::STAGES;
  constexpr int CHUNK = C::FP8 ? 1 : kPgChunk;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // the 128-byte swizzle wants 1024-byte alignment
  uint8_t* base_ptr = smem_raw + (base - raw);
  const uint32_t ebase = base + STAGES * C::STAGE_BYTES;
  const uint32_t scbase = ebase + C::EPI_BYTES;
  uint8_t* tail_ptr = base_ptr + STAGES * C::STAGE_BYTES + C::EPI_BYTES + C::SCALE_BYTES;
  int32_t* start = reinterpret_cast<int32_t*>(tail_ptr);
  int32_t* first = start + kMaxExperts + 4;
  uint8_t* bar_ptr = tail_ptr + C::TABLE_BYTES;
  const uint32_t bar0 = base + static_cast<uint32_t>(bar_ptr - base_ptr);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_ptr + C::NUM_BARS * 8);
  int32_t* scan = reinterpret_cast<int32_t*>(tmem_slot + 2);  // [24]

  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + C::NBUF + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 2 * C::NBUF);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 2);  // one expect-tx arrival from each producer
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < C::NBUF; ++b) {
      mbar_init(tfull_bar(b), C::FP8 ? 2 : 1);  // the MMAs' commit and, 8-bit, the scales
      mbar_init(tempty_bar(b), C::EPI_ARRIVALS);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
  }
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_addr(tmem_slot), C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR)
    cluster_sync();  // both CTAs' barriers are initialised before either signals the other
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (C::ROW_GROUPS || C::K_GROUPS) build_group_table<BN, KIND, FORM>(args, start, first, scan);
  const PgWalk<BN, KIND, FORM> walk{args, start, first};
  const int units = walk.units();
  const int unit0 = static_cast<int>(blockIdx.x) / (PAIR ? 2 : 1);
  const int step = static_cast<int>(gridDim.x) / (PAIR ? 2 : 1);

  // (Narrower tiles need fewer registers than every thread has at launch.)
  if (warp < 4) {
    if (BN == 256) regs_give<88>();
    if (warp == 0 || warp == 2) {
      // -------------------------------------------------------------- producers
      if (lane == 0) {
        const bool load_a = warp == 0;
        int stage = 0;
        uint32_t phase = 0, issued = 0, issued_phase = 0;
        bool ok = true;
        for (int u = unit0; ok && u < units; u += step) {
          const PgTile t = walk.at(u);
          for (int kb = 0; kb < t.nkb; ++kb) {
            if (!mbar_wait<PAIR>(empty_bar(stage), phase ^ 1u, args.wait_ns)) {
              atomicOr(args.fault, kFaultProducerWait);
              ok = false;
              break;
            }
            // (a pair's loads all complete on the leader's barrier)
            const uint32_t fb = PAIR ? map_shared_rank(full_bar(stage), 0) : full_bar(stage);
            const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
            auto load2 = [&](uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y) {
              if (PAIR)
                tma_load_2d_pair(dst, map, fb, x, y);
              else
                tma_load_2d(dst, map, fb, x, y);
            };
            auto load3 = [&](uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z) {
              if (PAIR)
                tma_load_3d_pair(dst, map, fb, x, y, z);
              else
                tma_load_3d(dst, map, fb, x, y, z);
            };
            const int kx = (C::SPLIT ? t.kb0 + kb : kb) * C::BK;
            const int k0 = (C::K_GROUPS ? t.row0 : 0) + kx;
            const int a_bytes = C::A_MN ? C::A_BYTES : args.a_rows * 128;
            if (rank == 0) mbar_expect_tx(full_bar(stage), (PAIR ? 2 : 1) * (load_a ? a_bytes : C::B_BYTES));
            if (load_a) {
              const int m0 = t.tm * C::TM + static_cast<int>(rank) * C::BM;
              if (C::A_MN) {
#pragma unroll
                for (int g = 0; g < C::BM / C::MN; ++g) load2(sa + g * (C::BK * 128), &tmA, m0 + g * C::MN, k0);
              } else {
                load2(sa, &tmA, kx, C::ROW_GROUPS ? t.row0 + static_cast<int>(rank) * C::BM : m0);
              }
            } else {
              const int n0 = t.tn * BN + static_cast<int>(rank) * C::BNL;
              if (C::B_MN) {
#pragma unroll
                for (int g = 0; g < C::BNL / C::MN; ++g) {
                  if (C::ROW_GROUPS)
                    load3(sb + g * (C::BK * 128), &tmB, n0 + g * C::MN, k0, t.e);
                  else
                    load2(sb + g * (C::BK * 128), &tmB, n0 + g * C::MN, k0);
                }
              } else if (C::ROW_GROUPS) {
                load3(sb, &tmB, kx, n0, t.e);
              } else {
                load2(sb, &tmB, kx, n0);
              }
            }
            issued |= 1u << stage;
            issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // every load has landed before the CTA may exit (a pair's: the MMAs that read it are done)
        for (int s = 0; s < STAGES; ++s)
          if ((issued >> s) & 1u)
            if (!mbar_wait<PAIR>(PAIR ? empty_bar(s) : full_bar(s), (issued_phase >> s) & 1u, args.wait_ns))
              atomicOr(args.fault, kFaultDrainWait);
      }
    } else if (warp == 1) {
      if (rank == 0) {
        // ------------------------------------------------------------- MMA issuer
        // One elected thread walks the list (297 cycles a block with nothing to wait for, against
        // 415 where the whole warp walks it, votes and elects for each block: a block's MMAs take
        // 512).  Ragged contractions need the warp: its lanes zero the rows of a last block.
        constexpr bool SOLO = !C::K_GROUPS;
        if (!SOLO || elect_one()) {
          auto all = [](bool in) { return SOLO ? in : __all_sync(0xffffffffu, in) != 0; };
          auto one = []() { return SOLO || elect_one(); };
          auto give_up = [&]() {
            if (SOLO || lane == 0) atomicOr(args.fault, kFaultMmaWait);
            return false;
          };
          int stage = 0, buf = 0;
          uint32_t phase = 0, bphase = 0;
          bool ok = true;
          // descriptors of stage 0 and their step per slice: K-major 32 bytes along the swizzled row,
          // MN-major SLICE rows of 128 bytes (see sdesc_sw128)
          constexpr uint32_t A_STEP = C::A_MN ? C::SLICE * 8 : 2, B_STEP = C::B_MN ? C::SLICE * 8 : 2;
          // B of the second 128-column MMA: 128 K-major rows further, or the next MN-major box.  A
          // pair's MMA takes 64 of its columns from each CTA: 64 rows further, or 64 bytes along the
          // rows of the one box (see tile_col for the columns this makes).
          constexpr uint32_t SUB_STEP = !PAIR ? 128 * 128 / 16 : C::B_MN ? 64 / 16 : 64 * 128 / 16;
          const uint64_t a_desc = sdesc_sw128(base, C::A_MN ? C::BK * 128 : 16, 1024);
          const uint64_t b_desc = sdesc_sw128(base + C::A_BYTES, C::B_MN ? C::BK * 128 : 16, 1024);
          const uint32_t a_lo = static_cast<uint32_t>(a_desc), a_hi = static_cast<uint32_t>(a_desc >> 32);
          const uint32_t b_lo = static_cast<uint32_t>(b_desc), b_hi = static_cast<uint32_t>(b_desc >> 32);
          for (int u = unit0; ok && u < units; u += step) {
            const PgTile t = walk.at(u);
            for (int c0 = 0; ok && c0 < t.nkb; c0 += CHUNK) {
              const int c1 = min(c0 + CHUNK, t.nkb);
              auto wait_empty = [&](int b) {
                return all(mbar_wait_soon<PAIR>(tempty_bar(b), bphase ^ 1u, args.wait_ns)) || give_up();
              };
              if (!(ok = wait_empty(buf))) break;
              for (int kb = c0; kb < c1; ++kb) {
                if (!all(mbar_wait_soon<PAIR>(full_bar(stage), phase, args.wait_ns))) {
                  ok = give_up();
                  break;
                }
                int slices = C::BK / C::SLICE;
                if (C::K_GROUPS) {
                  // the last block's rows past the group's end belong to the next group: contract
                  // whole slices only, and zero the rest of the last one in both operands (a
                  // product with an infinity or NaN there would not vanish)
                  const int valid = t.k_left - kb * C::BK;
                  if (valid < C::BK) {
                    slices = (valid + C::SLICE - 1) / C::SLICE;
                    const int rows = slices * C::SLICE - valid;  // 0..15 rows of 128 bytes in each box
                    constexpr int BOXES = (C::BM + BN) / C::MN;
                    for (int i = lane; i < rows * 8 * BOXES; i += 32) {
                      const int box = i / (rows * 8), j = i - box * (rows * 8);
                      const int at = box * (C::BK * 128) + (valid + (j >> 3)) * 128 + (j & 7) * 16;
                      st_shared_u4(base + stage * C::STAGE_BYTES + at, make_uint4(0, 0, 0, 0));
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                  }
                }
#pragma unroll
                for (int sub = 0; sub < C::NSUB; ++sub) {
                  if (sub > 0 && !(ok = wait_empty(buf + sub))) break;
                  tc_fence_after();
                  if (one()) {
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>((buf + sub) * C::SUB);
                    const uint32_t at = static_cast<uint32_t>(stage) * (C::STAGE_BYTES >> 4);
                    auto issue = [&](int kk) {
                      mma_lo<C::FP8, PAIR>(d_tmem, a_lo + at + kk * A_STEP, a_hi, b_lo + at + sub * SUB_STEP + kk * B_STEP, b_hi,
                                           args.idesc, (kb > c0 || kk > 0) ? 1u : 0u);
                    };
                    if (C::K_GROUPS && slices < C::BK / C::SLICE) {
                      for (int kk = 0; kk < slices; ++kk) issue(kk);
                    } else {
#pragma unroll
                      for (int kk = 0; kk < C::BK / C::SLICE; ++kk) issue(kk);
                    }
                    auto commit = [&](uint32_t bar) {  // (in both CTAs of a pair)
                      if (PAIR)
                        mma_commit_pair_multicast(bar, 0x3);
                      else
                        mma_commit(bar);
                    };
                    if (sub == C::NSUB - 1) commit(empty_bar(stage));
                    if (kb + 1 == c1) commit(tfull_bar(buf + sub));
                  }
                  if (!SOLO) __syncwarp();
                }
                if (!ok) break;
                if (++stage == STAGES) {
                  stage = 0;
                  phase ^= 1u;
                }
              }
              if (!ok) break;
              if ((buf += C::NSUB) == C::NBUF) {
                buf = 0;
                bphase ^= 1u;
              }
            }
          }
          // every MMA has finished before TMEM is freed (a commit covers the MMAs of the thread that
          // issues it: the elected one is the same throughout)
          if (one()) {
            if (PAIR)
              mma_commit_pair(drain_bar);
            else
              mma_commit(drain_bar);
            if (!mbar_wait(drain_bar, 0, args.wait_ns)) atomicOr(args.fault, kFaultDrainWait);
          }
        }
        __syncwarp();
      }
    } else if (C::FP8) {
      // ------------------------------------------------------------------ scales
      // A chunk's accumulator barriers take an arrival of this warp beside the MMAs' commit, so the
      // epilogue waits once for the sums and their scales.  The arrival may be made once the
      // barrier's phase before is over (the chunk NBUF / NSUB earlier); the loads run kScaleAhead
      // chunks ahead of it, in registers.  A ring slot's last readers are done by then: they gave
      // back the accumulator of a later chunk, which the MMAs of that earlier phase overwrote.
      static_assert(!C::FP8 || C::SCALE_SLOTS > 2 * C::NBUF / C::NSUB, "scale ring");
      constexpr int NB = C::COL_SCALES ? BN / 32 : 2, NV = 4 + NB;
      float v[kScaleAhead][NV];
      int lu = unit0, left = 0;  // tile of the next load, chunks left in it
      const float* at[NV];
      bool in[NV];
      // (rows and columns past the edges have zero operands: their scale is zero)
      auto load = [&](float (&x)[NV]) {
        if (left == 0) {
          if (lu >= units) return;
          const PgTile t = walk.at(lu);
          lu += step;
          left = t.nkb;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int m = t.tm * C::TM + static_cast<int>(rank) * C::BM + 32 * j + lane;
            in[j] = m < args.gm;
            at[j] = args.sa + (in[j] ? m * args.sa_row + t.kb0 * args.sa_blk : 0);
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int n = t.tn * BN + (C::COL_SCALES ? 32 * j + lane : 128 * j);
            in[4 + j] = n < args.gn;
            at[4 + j] = args.sb + (in[4 + j] ? (C::COL_SCALES ? n : n / 128) * args.sb_row + t.kb0 * args.sb_blk : 0);
          }
        }
        --left;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          x[j] = in[j] ? __ldg(at[j]) : 0.0f;
          at[j] += j < 4 ? args.sa_blk : args.sb_blk;
        }
      };
#pragma unroll
      for (int i = 0; i < kScaleAhead; ++i) load(v[i]);
      // (every tile has the same number of blocks; a split launch gives each CTA one share)
      const int nkb = C::SPLIT ? walk.at(unit0).nkb : (args.gk + C::BK - 1) / C::BK;
      const int total = unit0 < units ? ((units - unit0 + step - 1) / step) * nkb : 0;
      bool ok = true;
      for (int i0 = 0; ok && i0 < total; i0 += kScaleAhead) {
#pragma unroll
        for (int k = 0; k < kScaleAhead; ++k) {
          const int i = i0 + k;
          if (i >= total) break;
          const int b = i * C::NSUB % C::NBUF;
          const uint32_t parity = ((i * C::NSUB / C::NBUF) & 1) ^ 1;
          bool free = mbar_wait_soon<PAIR>(tfull_bar(b), parity, args.wait_ns);
          if (C::NSUB == 2) free = free && mbar_wait_soon<PAIR>(tfull_bar(b + 1), parity, args.wait_ns);
          if (!__all_sync(0xffffffffu, free)) {
            if (lane == 0) atomicOr(args.fault, kFaultProducerWait);
            ok = false;
            break;
          }
          const uint32_t dst = scbase + static_cast<uint32_t>(i % C::SCALE_SLOTS) * (C::SCALE_FLOATS * 4);
          if (C::COL_SCALES) {
#pragma unroll
            for (int j = 0; j < NV; ++j) st_shared_f32(dst + (32 * j + lane) * 4, v[k][j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) st_shared_f2(dst + (32 * j + lane) * 8, v[k][j] * v[k][4], v[k][j] * v[k][5]);
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(tfull_bar(b));
            if (C::NSUB == 2) mbar_arrive(tfull_bar(b + 1));
          }
          load(v[k]);
        }
      }
    }
    if (C::SPLIT) {  // (the epilogue warps' exchange)
      cluster_sync();
      cluster_sync();
    }
  } else {
    // -------------------------------------------------- promotion and epilogue
    if (BN == 256) regs_take<208>();
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                               static_cast<uint32_t>(C::NSUB == 2 ? 0 : h * C::HALF);
    const uint32_t ebuf = ebase + static_cast<uint32_t>(warp - 4) * 2048u;
    // The tile's column of this warp's accumulator c.  A pair's 128-column MMA h has 64 columns
    // from the first and 64 from the second half of the tile.
    constexpr bool MIXED = PAIR && C::NSUB == 2;
    auto tile_col = [&](int c) { return !MIXED ? h * C::HALF + c : 64 * h + c + (c < 64 ? 0 : 64); };
    // (Beside 128 accumulators registers are short: one counter gives every ring position, and
    // the tile is decoded again for the store.)
    uint32_t it = 0;  // chunks done by this CTA
    bool exchanged = false;
    bool ok = true, ready = false;
    for (int u = unit0; u < units; u += step) {
      uint64_t acc[C::HALF / 2];  // pairs of columns
#pragma unroll
      for (int j = 0; j < C::HALF / 2; ++j) acc[j] = 0;
      for (int left = (walk.at(u).nkb + CHUNK - 1) / CHUNK; left > 0; --left, ++it) {
        auto buffer = [&](uint32_t i) { return C::NSUB == 2 ? 2 * (i & 1u) + static_cast<uint32_t>(h) : i % C::NBUF; };
        auto parity = [&](uint32_t i) { return (i * C::NSUB / C::NBUF) & 1u; };
        const uint32_t buf = buffer(it);
        if (!ready && !__all_sync(0xffffffffu, mbar_wait_soon<PAIR>(tfull_bar(buf), parity(it), args.wait_ns))) {
          if (lane == 0) atomicOr(args.fault, kFaultEpilogueWait);
          ok = false;
          break;
        }
        const uint32_t sc = scbase + (it % C::SCALE_SLOTS) * (C::SCALE_FLOATS * 4);
        // This thread's factors: of its row and, in a pair, of the second 64 columns; with column
        // scales, of its four rows.
        uint64_t s0 = 0, s1 = 0, srow[4] = {0, 0, 0, 0};
        if (C::COL_SCALES) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f = ld_shared_f32(sc + (q * 32 + 8 * k + lane / 4) * 4);
            srow[k] = pack_f32x2(f, f);
          }
        } else if (C::FP8) {
          const float2 f = ld_shared_f2(sc + (q * 32 + lane) * 8);
          const float f0 = !PAIR && C::NSUB == 2 && h == 1 ? f.y : f.x;
          s0 = pack_f32x2(f0, f0), s1 = pack_f32x2(f.y, f.y);
        }
        tc_fence_after();
        const uint32_t t_addr = lane_addr + buf * C::SUB;
        // 32 columns at a time through two register blocks: both are loaded, then each is refilled
        // as soon as its columns are added, so that a chunk waits for TMEM twice at most.
        auto add32 = [&](uint32_t (&v)[32], int c) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            uint64_t lo = pack_u32x2(v[j], v[j + 1]), hi = pack_u32x2(v[j + 2], v[j + 3]);
            uint64_t& a0 = acc[(c + j) / 2];
            uint64_t& a1 = acc[(c + j) / 2 + 1];
            const uint64_t s = MIXED && c >= 64 ? s1 : s0;
            a0 = C::FP8 ? fma_f32x2(lo, s, a0) : add_f32x2(lo, a0);
            a1 = C::FP8 ? fma_f32x2(hi, s, a1) : add_f32x2(hi, a1);
          }
        };
        auto release = [&]() {  // the accumulator is read: later MMAs may use the buffer
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (PAIR)
              mbar_arrive_remote(map_shared_rank(tempty_bar(buf), 0));
            else
              mbar_arrive(tempty_bar(buf));
          }
          // (whether the next chunk is there is asked here, beside the additions that follow)
          const uint32_t next = tfull_bar(buffer(it + 1));
          ready = __all_sync(0xffffffffu, PAIR ? mbar_peek_cluster(next, parity(it + 1)) : mbar_peek(next, parity(it + 1)));
        };
        if (C::QUADS) {
          // A thread takes pairs of columns of four rows.  With column scales a warp then reads a
          // chunk's as 16 words of 8 bytes a thread and not as 32 broadcasts of 16; without, the
          // output goes straight from registers (below).  The registers are filled in turn.
          using Block = uint32_t[2][16];
          auto load32 = [&](Block& v, int c) {
            tmem_ld_16x256b_x4(t_addr + c, v[0]);
            tmem_ld_16x256b_x4(t_addr + c + (16u << 16), v[1]);
          };
          auto add_cols32 = [&](Block& v, int c) {
            const uint32_t x = sc + (128 + tile_col(c) + 2 * (lane & 3)) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t col = C::COL_SCALES ? ld_shared_u64(x + 32 * i) : 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint64_t& a0 = acc[c / 2 + 4 * i + k];
                const uint32_t* r = &v[k >> 1][4 * i + 2 * (k & 1)];
                const uint64_t p = pack_u32x2(r[0], r[1]);
                a0 = C::COL_SCALES ? fma_f32x2(mul_f32x2(p, col), srow[k], a0) : add_f32x2(p, a0);
              }
            }
          };
          Block v0, v1;
          load32(v0, 0);
          if (C::HALF >= 64) load32(v1, 32);
          tmem_wait_ld();
          if (C::HALF <= 64) release();
          add_cols32(v0, 0);
          if (C::HALF == 128) load32(v0, 64);
          if (C::HALF >= 64) add_cols32(v1, 32);
          if (C::HALF == 128) {
            load32(v1, 96);
            tmem_wait_ld();
            release();
            add_cols32(v0, 64);
            add_cols32(v1, 96);
          }
        } else {
          uint32_t r0[32], r1[32];
          tmem_ld_32x32b_x32(t_addr, r0);
          if (C::HALF >= 64) tmem_ld_32x32b_x32(t_addr + 32, r1);
          tmem_wait_ld();
          if (C::HALF <= 64) release();
          add32(r0, 0);
          if (C::HALF == 128) tmem_ld_32x32b_x32(t_addr + 64, r0);
          if (C::HALF >= 64) add32(r1, 32);
          if (C::HALF == 128) {
            tmem_ld_32x32b_x32(t_addr + 96, r1);
            tmem_wait_ld();
            release();
            add32(r0, 64);
            add32(r1, 96);
          }
        }
      }
      if (!ok) break;
      int us = u;
      asm volatile("" : "+r"(us));
      const PgTile t = walk.at(us);
      const int n0 = t.tn * BN;
      if (C::SPLIT) {
        // This rank's partial tile, [pair of columns][row], into the operand ring.  Its loads and MMAs
        // have to be done: where a block takes two MMAs, the warps of the first half have waited for
        // the first one's commit only, so they wait for the last block's second one here.
        if (C::NSUB == 2 && h == 0) {
          const uint32_t last = it - 1;
          if (!__all_sync(0xffffffffu, mbar_wait_soon<PAIR>(tfull_bar(2 * (last & 1u) + 1), (last * C::NSUB / C::NBUF) & 1u,
                                                            args.wait_ns))) {
            if (lane == 0) atomicOr(args.fault, kFaultEpilogueWait);
            break;
          }
        }
        if (C::COL_SCALES) {
          const uint32_t at = base + static_cast<uint32_t>((h * (C::HALF / 2) + (lane & 3)) * C::BM + q * 32 + lane / 4) * 8;
#pragma unroll
          for (int j = 0; j < C::HALF / 2; ++j)
            st_shared_u64(at + (j / 16 * 16 + (j % 16) / 4 * 4) * (C::BM * 8) + (j & 3) * 64, acc[j]);
        } else if (q * 32 + lane < t.m_left) {
          const uint32_t at = base + static_cast<uint32_t>(h * (C::HALF / 2) * C::BM + q * 32 + lane) * 8;
#pragma unroll
          for (int j = 0; j < C::HALF / 2; ++j) st_shared_u64(at + j * (C::BM * 8), acc[j]);
        }
        cluster_sync();
        sum_split<BN>(args, t, base, static_cast<int>(threadIdx.x) - 128);
        cluster_sync();  // (no CTA leaves while its tile may be read)
        exchanged = true;
        break;
      }
      // Store 32 rows x HALF columns through the warp's 2 KB block, a pass of 16 rows of 128 bytes
      // (32 rows of 64 where HALF is 32 BF16 columns), 16-byte chunks XOR-swizzled by row, read
      // back so that eight (four) lanes write consecutive bytes of a row.
      const int half_row = static_cast<int>(rank) * C::BM + q * 32;  // of the tile's rows
      const int rows_left = t.m_left - half_row;
      const int64_t row = (C::ROW_GROUPS ? static_cast<int64_t>(t.row0) : static_cast<int64_t>(t.tm) * C::TM) + half_row;
      const int esize = args.out_f32 ? 4 : 2;
      char* out = static_cast<char*>(args.out) +
                  ((C::K_GROUPS ? t.e * args.out_gstride : int64_t{0}) + row * args.ldo) * esize;
      auto lo32 = [&](int j) { return static_cast<uint32_t>(acc[j]); };
      auto hi32 = [&](int j) { return static_cast<uint32_t>(acc[j] >> 32); };
      auto bf16x2 = [&](int j) { return pack_bf16x2(__uint_as_float(lo32(j)), __uint_as_float(hi32(j))); };
      if (C::QUADS) {
        // Straight from registers: neighbouring lanes swap a pair of columns, so that four lanes
        // hold 16 consecutive columns of a row (64 bytes of FP32, 32 of BF16).
        const bool odd = (lane & 1) != 0;
        auto swap32 = [&](uint32_t a, uint32_t b) { return __shfl_xor_sync(0xffffffffu, odd ? a : b, 1); };
#pragma unroll
        for (int j = 0; j < C::HALF / 2; j += j % 4 == 3 ? 5 : 1) {  // columns c..c+7, and c+8..c+15 at j + 4
          const int r = 8 * (j & 3) + lane / 4;
          const int col = n0 + tile_col(j / 16 * 32) + (j % 16) / 4 * 8 + 2 * (lane & 2) + (odd ? 8 : 0);
          const bool in = r < rows_left && col < args.gn;
          char* p = out + (r * args.ldo + col) * esize;
          if (args.out_f32) {
            const uint32_t x = swap32(lo32(j), lo32(j + 4)), y = swap32(hi32(j), hi32(j + 4));
            const uint4 w = odd ? make_uint4(x, y, lo32(j + 4), hi32(j + 4)) : make_uint4(lo32(j), hi32(j), x, y);
            if (in) *reinterpret_cast<uint4*>(p) = w;
          } else {
            const uint32_t a = bf16x2(j), b = bf16x2(j + 4), x = swap32(a, b);
            if (in) *reinterpret_cast<uint2*>(p) = odd ? make_uint2(x, b) : make_uint2(a, x);
          }
        }
      } else {
        auto put = [&](auto chunks, int col0, int per_chunk, auto chunk) {
          constexpr int CH = decltype(chunks)::value, ROWS = 128 / CH, SHIFT = CH == 8 ? 0 : 1;
          const int ch = lane % CH, r0 = lane / CH, mine = lane % ROWS;
          const int col = col0 + ch * per_chunk;
          char* p = out + (r0 * args.ldo + col) * esize;
          const int64_t down = 32 / CH * args.ldo * esize;
#pragma unroll
          for (int pass = 0; pass < 32 / ROWS; ++pass) {
            __syncwarp();
            if (lane / ROWS == pass) {
#pragma unroll
              for (int j = 0; j < CH; ++j)
                st_shared_u4(ebuf + mine * (CH * 16) + ((j ^ ((mine >> SHIFT) & (CH - 1))) << 4), chunk(j));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i, p += down) {
              const int r = 32 / CH * i + r0;
              const uint4 x = ld_shared_u4(ebuf + r * (CH * 16) + ((ch ^ ((r >> SHIFT) & (CH - 1))) << 4));
              if (col < args.gn && pass * ROWS + r < rows_left) *reinterpret_cast<uint4*>(p) = x;
            }
          }
        };
        if (args.out_f32) {
#pragma unroll
          for (int c = 0; c < C::HALF; c += 32)
            put(Int<8>(), n0 + tile_col(c), 4, [&](int j) {
              const int k = c / 2 + 2 * j;
              return make_uint4(lo32(k), hi32(k), lo32(k + 1), hi32(k + 1));
            });
        } else {
          constexpr int CH = C::HALF >= 64 ? 8 : 4;
#pragma unroll
          for (int c = 0; c < C::HALF; c += CH * 8)
            put(Int<CH>(), n0 + tile_col(c), 8, [&](int j) {
              const int k = c / 2 + 4 * j;
              return make_uint4(bf16x2(k), bf16x2(k + 1), bf16x2(k + 2), bf16x2(k + 3));
            });
        }
      }
    }
    if (C::SPLIT && !exchanged) {  // (a wait ran out: the others still meet this CTA twice)
      cluster_sync();
      cluster_sync();
    }
    // Rows before the first group and after the last one belong to no expert: zeros.
    if (C::ROW_GROUPS) {
      const int lo = start[0], hi = start[args.experts], esize = args.out_f32 ? 4 : 2;
      const int64_t idle = static_cast<int64_t>(lo) + (args.rows - hi);
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (warp - 4); i < idle; i += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t r = i < lo ? i : hi + (i - lo);
        char* p = static_cast<char*>(args.out) + r * args.ldo * esize;
        const int64_t bytes = static_cast<int64_t>(args.gn) * esize;
        for (int64_t b = lane * 16; b < bytes; b += 512) *reinterpret_cast<uint4*>(p + b) = make_uint4(0, 0, 0, 0);
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  if (PAIR)
    cluster_sync();  // neither CTA leaves while the other may still signal it or read its operands
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else
      tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side

struct PgLaunch {
  CUtensorMap tmA, tmB;
  PgArgs args;
  int grid;
};

// gemm_grouped.cu / gemm_fp8.cu: one launch of the kernel of that kind, tile width and form.
cudaError_t launch_grouped(int kind, int bn, int form, const PgLaunch& l, cudaStream_t stream);
cudaError_t launch_fp8(int kind, int bn, int form, const PgLaunch& l, cudaStream_t stream);
cudaError_t set_attributes_grouped();
cudaError_t set_attributes_fp8();
int max_clusters_fp8(int kind, int bn, int split);

template <int BN, int KIND, int FORM = kPlain>
cudaError_t launch_pg(const PgLaunch& l, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(l.grid), 1, 1);
  cfg.blockDim = dim3(PgCfg<BN, KIND, FORM>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = PgCfg<BN, KIND, FORM>::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = FORM == kSplit ? static_cast<unsigned>(l.args.split) : 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = FORM == kPlain ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, promoted_gemm_kernel<BN, KIND, FORM>, l.tmA, l.tmB, l.args);
}

template <int BN, int KIND, int FORM>
int max_clusters_pg(int split) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
  cfg.blockDim = dim3(PgCfg<BN, KIND, FORM>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = PgCfg<BN, KIND, FORM>::SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, promoted_gemm_kernel<BN, KIND, FORM>, &cfg) != cudaSuccess) {
    cudaGetLastError();  // clear: no split launches
    return 0;
  }
  return n;
}

template <int BN, int KIND, int FORM = kPlain>
cudaError_t set_attr_pg() {
  const auto kernel = promoted_gemm_kernel<BN, KIND, FORM>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PgCfg<BN, KIND, FORM>::SMEM_BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (BN == 256 && e == cudaSuccess) {
    // the warpgroups trade exactly the registers of a launch at 168 a thread (regs_take
    // would wait for ever on fewer): refuse to run a build that launches with another count
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, kernel);
    if (e == cudaSuccess && f.numRegs < 168) e = cudaErrorInvalidConfiguration;
  }
  return e;
}

}  // namespace dp

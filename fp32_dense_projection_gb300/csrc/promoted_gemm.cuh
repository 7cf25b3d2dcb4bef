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
//   warp 3       8-bit products: the chunks' scales, by asynchronous copies into a ring
//   warps 4..11  promotion and epilogue: read a finished chunk's accumulator from TMEM,
//                add it (scaled) to FP32 registers; after the last chunk, round once and
//                store.  Warp w holds rows 32 (w % 4) .. + 32 and one half of the columns.
// A chunk's accumulator is one of two TMEM buffers, so the promotion of one chunk runs
// beside the MMAs of the next.
//
// Why promotion: (1) the scale of a 128-element block multiplies that block's sum only,
// so it cannot be applied after the whole contraction; (2) the tensor core rounds every
// FP32 accumulate toward zero, an error that grows with the length of one accumulator
// (relative RMS 1.9e-5 at 16384 elements, measured in tests of the dense path), while the
// register sums round to nearest: BF16 chunks of 2048 elements keep it near 2e-6.
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
constexpr int kScaleSlots = 8;  // 8-bit products: chunks whose scales are in shared memory
constexpr int kPgChunk = 32;  // BF16: contraction blocks of 64 per accumulator

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
  uint32_t idesc;
  const float* sa;           // 8-bit products: scale of row m, block c at sa[m * sa_row + c * sa_blk]
  int64_t sa_row, sa_blk;
  const float* sb;           // of column (or 128-column block) n, block c
  int64_t sb_row, sb_blk;
  uint32_t* fault;
  uint64_t wait_ns;
};

template <int BN, int KIND>
struct PgCfg {
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
  static constexpr int B_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = (192 * 1024) / STAGE_BYTES < 8 ? (192 * 1024) / STAGE_BYTES : 8;
  static constexpr int HALF = BN / 2;  // columns of one epilogue warp
  static constexpr int EPI_BYTES = 8 * 2048;
  // 8-bit products: a ring of the scales of a chunk's 128 rows and BN columns (one value per
  // 128 columns where blocks of 128 x 128 cover them)
  static constexpr bool COL_SCALES = KIND == kFp8MM;
  static constexpr int SCALE_SLOTS = FP8 ? kScaleSlots : 0;
  static constexpr int SCALE_FLOATS = 128 + (COL_SCALES ? BN : 4);
  static constexpr int SCALE_BYTES = SCALE_SLOTS * SCALE_FLOATS * 4;
  static constexpr int TABLE_BYTES = (ROW_GROUPS || K_GROUPS) ? 2 * (kMaxExperts + 4) * 4 : 0;
  static constexpr int NUM_BARS = 2 * STAGES + 5 + 2 * SCALE_SLOTS;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + EPI_BYTES + SCALE_BYTES + TABLE_BYTES + NUM_BARS * 8 + 256;
  static constexpr int THREADS = 384;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(BN == 64 || BN == 128 || BN == 256, "tile width");
  static_assert(!(FP8 && B_MN) || BN >= 128, "8-bit MN-major boxes are 128 columns wide");
};

// tcgen05.mma on operands given by the halves of their shared-memory descriptors.  The low
// half holds the start address >> 4 and the leading offset, the high half (constant over a
// kernel) the stride and the layout: stepping through stages and slices is one 32-bit add, which
// stays in uniform registers.  (8-bit operands: E4M3 or E5M2 each, as the instruction
// descriptor says.)
template <bool FP8>
__device__ __forceinline__ void mma_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  if (FP8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
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
};

template <int BN, int KIND>
struct PgWalk {
  using C = PgCfg<BN, KIND>;
  const PgArgs& a;
  const int32_t* start;  // [experts + 1] first row of each group
  const int32_t* first;  // [experts + 1] first tile of each group (row-grouped)
  __device__ __forceinline__ int units() const {
    if (C::ROW_GROUPS) return first[a.experts];
    return a.tiles_m * a.tiles_n * (C::K_GROUPS ? a.experts : 1);
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
      tiles_m = (cnt + C::BM - 1) / C::BM;
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
      local = u;
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
    t.m_left -= t.tm * C::BM;
    if (C::ROW_GROUPS) t.row0 += t.tm * C::BM;
    t.nkb = (t.k_left + C::BK - 1) / C::BK;
    return t;
  }
};

// The groups' table: start[i] = running maximum of the offsets, clamped to [0, rows], and
// (row-grouped) first[i] = tiles of the groups before i.  Offsets that decrease or leave
// [0, rows] set kFaultOffsets.  All 384 threads call it; each takes `per` consecutive entries.
template <int BN, int KIND>
__device__ __forceinline__ void build_group_table(const PgArgs& a, int32_t* start, int32_t* first, int32_t* scan) {
  using C = PgCfg<BN, KIND>;
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
    if (j < per && i < a.experts) tiles[j] = (start[i + 1] - start[i] + C::BM - 1) / C::BM * a.tiles_n;
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

// Four bytes from global to shared memory without a register; zero where !valid.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrive on `bar` when this thread's copies so far have landed (counted among the
// arrivals the barrier was initialised with).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
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

template <int BN, int KIND>
__global__ void __launch_bounds__(PgCfg<BN, KIND>::THREADS, 1)
    promoted_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ PgArgs args) {
  using C = PgCfg<BN, KIND>;
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
  auto tempty_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
  auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + s); };
  auto sempty_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + C::SCALE_SLOTS + s); };

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) / 32, 0);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 2);  // one expect-tx arrival from each producer
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull_bar(b), 1);
      mbar_init(tempty_bar(b), 8);  // one arrival per epilogue warp
    }
    for (int s = 0; s < C::SCALE_SLOTS; ++s) {
      mbar_init(sfull_bar(s), 32);  // every lane's copies
      mbar_init(sempty_bar(s), 8);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (C::ROW_GROUPS || C::K_GROUPS) build_group_table<BN, KIND>(args, start, first, scan);
  const PgWalk<BN, KIND> walk{args, start, first};
  const int units = walk.units();
  const int step = static_cast<int>(gridDim.x);

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
      for (int u = static_cast<int>(blockIdx.x); ok && u < units; u += step) {
        const PgTile t = walk.at(u);
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, args.wait_ns)) {
            atomicOr(args.fault, kFaultProducerWait);
            ok = false;
            break;
          }
          const uint32_t fb = full_bar(stage);
          const uint32_t sa = base + stage * C::STAGE_BYTES, sb = sa + C::A_BYTES;
          if (load_a) {
            mbar_expect_tx(fb, C::A_BYTES);
            if (C::A_MN) {
              const int k0 = (C::K_GROUPS ? t.row0 : 0) + kb * C::BK;
#pragma unroll
              for (int g = 0; g < C::BM / C::MN; ++g)
                tma_load_2d(sa + g * (C::BK * 128), &tmA, fb, t.tm * C::BM + g * C::MN, k0);
            } else {
              tma_load_2d(sa, &tmA, fb, kb * C::BK, C::ROW_GROUPS ? t.row0 : t.tm * C::BM);
            }
          } else {
            mbar_expect_tx(fb, C::B_BYTES);
            const int n0 = t.tn * BN;
            if (C::B_MN) {
              const int k0 = (C::K_GROUPS ? t.row0 : 0) + kb * C::BK;
#pragma unroll
              for (int g = 0; g < BN / C::MN; ++g) {
                if (C::ROW_GROUPS)
                  tma_load_3d(sb + g * (C::BK * 128), &tmB, fb, n0 + g * C::MN, k0, t.e);
                else
                  tma_load_2d(sb + g * (C::BK * 128), &tmB, fb, n0 + g * C::MN, k0);
              }
            } else if (C::ROW_GROUPS) {
              tma_load_3d(sb, &tmB, fb, kb * C::BK, n0, t.e);
            } else {
              tma_load_2d(sb, &tmB, fb, kb * C::BK, n0);
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
      // every load has landed before the CTA may exit
      for (int s = 0; s < STAGES; ++s)
        if ((issued >> s) & 1u)
          if (!mbar_wait(full_bar(s), (issued_phase >> s) & 1u, args.wait_ns)) atomicOr(args.fault, kFaultDrainWait);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    // (the whole warp walks the list: its lanes zero the rows of a ragged last block)
    int stage = 0, buf = 0;
    uint32_t phase = 0, bphase = 0;
    bool ok = true;
    // descriptors of stage 0 and their step per slice: K-major 32 bytes along the swizzled row,
    // MN-major SLICE rows of 128 bytes (see sdesc_sw128)
    constexpr uint32_t A_STEP = C::A_MN ? C::SLICE * 8 : 2, B_STEP = C::B_MN ? C::SLICE * 8 : 2;
    const uint64_t a_desc = sdesc_sw128(base, C::A_MN ? C::BK * 128 : 16, 1024);
    const uint64_t b_desc = sdesc_sw128(base + C::A_BYTES, C::B_MN ? C::BK * 128 : 16, 1024);
    const uint32_t a_lo = static_cast<uint32_t>(a_desc), a_hi = static_cast<uint32_t>(a_desc >> 32);
    const uint32_t b_lo = static_cast<uint32_t>(b_desc), b_hi = static_cast<uint32_t>(b_desc >> 32);
    for (int u = static_cast<int>(blockIdx.x); ok && u < units; u += step) {
      const PgTile t = walk.at(u);
      for (int c0 = 0; ok && c0 < t.nkb; c0 += CHUNK) {
        const int c1 = min(c0 + CHUNK, t.nkb);
        if (!__all_sync(0xffffffffu, mbar_wait(tempty_bar(buf), bphase ^ 1u, args.wait_ns))) {
          if (lane == 0) atomicOr(args.fault, kFaultMmaWait);
          ok = false;
          break;
        }
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * BN);
        for (int kb = c0; kb < c1; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(full_bar(stage), phase, args.wait_ns))) {
            if (lane == 0) atomicOr(args.fault, kFaultMmaWait);
            ok = false;
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
                st_shared_u4(base + stage * C::STAGE_BYTES + box * (C::BK * 128) + (valid + (j >> 3)) * 128 + (j & 7) * 16, make_uint4(0, 0, 0, 0));
              }
              fence_proxy_async_shared();
              __syncwarp();
            }
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t at = static_cast<uint32_t>(stage) * (C::STAGE_BYTES >> 4);
            auto issue = [&](int kk) {
              mma_lo<C::FP8>(d_tmem, a_lo + at + kk * A_STEP, a_hi, b_lo + at + kk * B_STEP, b_hi, args.idesc,
                             (kb > c0 || kk > 0) ? 1u : 0u);
            };
            if (C::K_GROUPS && slices < C::BK / C::SLICE) {
              for (int kk = 0; kk < slices; ++kk) issue(kk);
            } else {
#pragma unroll
              for (int kk = 0; kk < C::BK / C::SLICE; ++kk) issue(kk);
            }
            mma_commit(empty_bar(stage));
            if (kb + 1 == c1) mma_commit(tfull_bar(buf));
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (++buf == 2) {
          buf = 0;
          bphase ^= 1u;
        }
      }
    }
    // every MMA has finished before TMEM is freed (each commit covers the MMAs of the lane
    // that issues it: the elected lane is the same one throughout)
    if (elect_one()) {
      mma_commit(drain_bar);
      if (!mbar_wait(drain_bar, 0, args.wait_ns)) atomicOr(args.fault, kFaultDrainWait);
    }
    __syncwarp();
  } else if (C::FP8) {
    // ------------------------------------------------------------------ scales
    int slot = 0;
    uint32_t sphase = 0;
    bool ok = true;
    for (int u = static_cast<int>(blockIdx.x); ok && u < units; u += step) {
      const PgTile t = walk.at(u);
      // (rows and columns past the edges have zero operands: their scale is zero)
      const float* pa[4];
      bool in_a[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = t.tm * C::BM + 32 * j + lane;
        in_a[j] = m < args.gm;
        pa[j] = args.sa + (in_a[j] ? m * args.sa_row : 0);
      }
      constexpr int NB = C::COL_SCALES ? BN / 32 : 1;
      const float* pb[NB];
      bool in_b[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int n = t.tn * BN + (C::COL_SCALES ? 32 * j + lane : 128 * lane);
        in_b[j] = n < args.gn;
        pb[j] = args.sb + (in_b[j] ? (C::COL_SCALES ? n : n / 128) * args.sb_row : 0);
      }
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(sempty_bar(slot), sphase ^ 1u, args.wait_ns))) {
          if (lane == 0) atomicOr(args.fault, kFaultProducerWait);
          ok = false;
          break;
        }
        const uint32_t dst = scbase + static_cast<uint32_t>(slot) * (C::SCALE_FLOATS * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cp_async4(dst + (32 * j + lane) * 4, pa[j], in_a[j]);
          pa[j] += in_a[j] ? args.sa_blk : 0;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          if (C::COL_SCALES || lane < (BN + 127) / 128) cp_async4(dst + (128 + 32 * j + lane) * 4, pb[j], in_b[j]);
          pb[j] += in_b[j] ? args.sb_blk : 0;
        }
        cp_async_arrive(sfull_bar(slot));
        if (++slot == C::SCALE_SLOTS) {
          slot = 0;
          sphase ^= 1u;
        }
      }
    }
    // one empty slot past the last chunk: the epilogue looks one ahead
    if (ok && __all_sync(0xffffffffu, mbar_wait(sempty_bar(slot), sphase ^ 1u, args.wait_ns)))
      cp_async_arrive(sfull_bar(slot));
    cp_async_wait_all();
  }
  } else {
    // -------------------------------------------------- promotion and epilogue
    if (BN == 256) regs_take<208>();
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(h * C::HALF);
    const uint32_t ebuf = ebase + static_cast<uint32_t>(warp - 4) * 2048u;
    // (Beside 128 accumulators registers are short: one counter gives every ring position, and
    // the tile is decoded again for the store.)
    uint32_t it = 0;  // chunks done by this CTA
    bool ok = true;
    float next = 1.0f;  // this row's factor for chunk `it`, read one chunk ahead
    auto read_scale = [&](uint32_t i) {
      const bool in = mbar_wait(sfull_bar(i % kScaleSlots), (i / kScaleSlots) & 1u, args.wait_ns);
      const uint32_t at = scbase + (i % kScaleSlots) * (C::SCALE_FLOATS * 4);
      next = ld_shared_f32(at + (q * 32 + lane) * 4);
      if (!C::COL_SCALES) next *= ld_shared_f32(at + (128 + (BN == 256 ? h : 0)) * 4);
      return in;
    };
    if (C::FP8) ok = read_scale(0);
    for (int u = static_cast<int>(blockIdx.x); u < units; u += step) {
      uint64_t acc[C::HALF / 2];  // pairs of columns
#pragma unroll
      for (int j = 0; j < C::HALF / 2; ++j) acc[j] = 0;
      for (int left = (walk.at(u).nkb + CHUNK - 1) / CHUNK; left > 0; --left, ++it) {
        const uint64_t s = pack_f32x2(next, next);
        const uint32_t xcol = scbase + (it % kScaleSlots) * (C::SCALE_FLOATS * 4) + (128 + h * C::HALF) * 4;
        if (C::FP8) ok = read_scale(it + 1) && ok;
        ok = mbar_wait(tfull_bar(it & 1u), (it >> 1) & 1u, args.wait_ns) && ok;
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) atomicOr(args.fault, kFaultEpilogueWait);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t_addr = lane_addr + (it & 1u) * BN;
        // 32 columns at a time.  Where the registers allow it the next 32 are on their way from
        // TMEM while these are added; beside 128 accumulators they do not (the pairs would be
        // copied to make room: 107 moves a chunk, 85 against 61 us at T = 4031, 4096 -> 4096),
        // and the other warp of the SM sub-partition adds while this one loads.
        constexpr int AHEAD = C::HALF <= 64 ? 1 : 0;
        uint32_t r[1 + AHEAD][32];
        if (AHEAD) tmem_ld_32x32b_x32(t_addr, r[0]);
#pragma unroll
        for (int c = 0; c < C::HALF; c += 32) {
          uint32_t(&v)[32] = r[AHEAD ? (c / 32) & 1 : 0];
          if (!AHEAD) tmem_ld_32x32b_x32(t_addr + c, v);
          tmem_wait_ld();
          if (c + 32 < C::HALF) {
            if (AHEAD) tmem_ld_32x32b_x32(t_addr + c + 32, r[(c / 32 + 1) & 1]);
          } else {  // the accumulator is read: the next chunk but one may use it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(it & 1u));
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            uint64_t lo = pack_u32x2(v[j], v[j + 1]), hi = pack_u32x2(v[j + 2], v[j + 3]);
            uint64_t& a0 = acc[(c + j) / 2];
            uint64_t& a1 = acc[(c + j) / 2 + 1];
            if (C::COL_SCALES) {
              const float4 x = ld_shared_f4(xcol + (c + j) * 4);
              lo = mul_f32x2(lo, pack_f32x2(x.x, x.y));
              hi = mul_f32x2(hi, pack_f32x2(x.z, x.w));
            }
            a0 = C::FP8 ? fma_f32x2(lo, s, a0) : add_f32x2(lo, a0);
            a1 = C::FP8 ? fma_f32x2(hi, s, a1) : add_f32x2(hi, a1);
          }
        }
        if (C::FP8) {
          __syncwarp();  // every lane has read its scales
          if (lane == 0) mbar_arrive(sempty_bar(it % kScaleSlots));
        }
      }
      if (!ok) break;
      int us = u;
      asm volatile("" : "+r"(us));
      const PgTile t = walk.at(us);
      const int n0 = t.tn * BN + h * C::HALF;  // this warp's first column
      // Store 32 rows x HALF columns through the warp's 2 KB block: 64-byte rows (32 BF16 or
      // 16 FP32 columns), 16-byte chunks XOR-swizzled by row, read back so that four lanes
      // write 64 consecutive bytes of a row.
      const int rows_left = t.m_left - q * 32;
      const int64_t row = (C::ROW_GROUPS ? static_cast<int64_t>(t.row0) : static_cast<int64_t>(t.tm) * C::BM) + q * 32;
      const int esize = args.out_f32 ? 4 : 2;
      char* out = static_cast<char*>(args.out) +
                  ((C::K_GROUPS ? t.e * args.out_gstride : int64_t{0}) + row * args.ldo) * esize;
      const int ch = lane & 3, r0 = lane >> 2;
      auto flush = [&](int col0, int per_chunk) {
        const int col = col0 + ch * per_chunk;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + r0;
          const uint4 x = ld_shared_u4(ebuf + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
          if (col < args.gn && r < rows_left)
            *reinterpret_cast<uint4*>(out + (r * args.ldo + col) * esize) = x;
        }
      };
      auto lo32 = [&](int j) { return static_cast<uint32_t>(acc[j]); };
      auto hi32 = [&](int j) { return static_cast<uint32_t>(acc[j] >> 32); };
      auto bf16x2 = [&](int j) { return pack_bf16x2(__uint_as_float(lo32(j)), __uint_as_float(hi32(j))); };
      if (args.out_f32) {
#pragma unroll
        for (int c = 0; c < C::HALF; c += 16) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_u4(ebuf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4),
                         make_uint4(lo32(c / 2 + 2 * j), hi32(c / 2 + 2 * j), lo32(c / 2 + 2 * j + 1), hi32(c / 2 + 2 * j + 1)));
          __syncwarp();
          flush(n0 + c, 4);
        }
      } else {
#pragma unroll
        for (int c = 0; c < C::HALF; c += 32) {
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            st_shared_u4(ebuf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4),
                         make_uint4(bf16x2(c / 2 + 4 * j), bf16x2(c / 2 + 4 * j + 1), bf16x2(c / 2 + 4 * j + 2),
                                    bf16x2(c / 2 + 4 * j + 3)));
          __syncwarp();
          flush(n0 + c, 8);
        }
      }
    }
    // Rows before the first group and after the last one belong to no expert: zeros.
    if (C::ROW_GROUPS) {
      const int lo = start[0], hi = start[args.experts], esize = args.out_f32 ? 4 : 2;
      const int64_t idle = static_cast<int64_t>(lo) + (args.rows - hi);
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (warp - 4); i < idle; i += static_cast<int64_t>(step) * 8) {
        const int64_t r = i < lo ? i : hi + (i - lo);
        char* p = static_cast<char*>(args.out) + r * args.ldo * esize;
        for (int b = lane * 16; b < args.gn * esize; b += 512) *reinterpret_cast<uint4*>(p + b) = make_uint4(0, 0, 0, 0);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side

struct PgLaunch {
  CUtensorMap tmA, tmB;
  PgArgs args;
  int grid;
};

// gemm_grouped.cu / gemm_fp8.cu: one launch of the kernel of that kind and tile width.
cudaError_t launch_grouped(int kind, int bn, const PgLaunch& l, cudaStream_t stream);
cudaError_t launch_fp8(int kind, int bn, const PgLaunch& l, cudaStream_t stream);
cudaError_t set_attributes_grouped();
cudaError_t set_attributes_fp8();

template <int BN, int KIND>
cudaError_t launch_pg(const PgLaunch& l, cudaStream_t stream) {
  promoted_gemm_kernel<BN, KIND><<<static_cast<unsigned>(l.grid), PgCfg<BN, KIND>::THREADS, PgCfg<BN, KIND>::SMEM_BYTES,
                                   stream>>>(l.tmA, l.tmB, l.args);
  return cudaGetLastError();
}

template <int BN, int KIND>
cudaError_t set_attr_pg() {
  cudaError_t e = cudaFuncSetAttribute(promoted_gemm_kernel<BN, KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PgCfg<BN, KIND>::SMEM_BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(promoted_gemm_kernel<BN, KIND>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (BN == 256 && e == cudaSuccess) {
    // the warpgroups trade exactly the registers of a launch at 168 a thread (regs_take
    // would wait for ever on fewer): refuse to run a build that launches with another count
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, promoted_gemm_kernel<BN, KIND>);
    if (e == cudaSuccess && f.numRegs < 168) e = cudaErrorInvalidConfiguration;
  }
  return e;
}

}  // namespace dp

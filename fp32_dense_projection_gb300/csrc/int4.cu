// Weights in 4 bits with a scale per group of G = 32, 64 or 128 values along the contraction:
//   w[n][k] = (q - z) s,   q in 0..15, two to a byte (the even k in the low half)
// z is 8, or a zero point of the group's own.
//
// Products of few rows, plain or grouped by expert:  Y[t][n] = sum over groups of s sum x[t][k] (q - z)
//
// Bound: the codes' bytes from HBM, and beside them the instructions that unpack them (118 a block
// of 16 x 128 codes).  64 experts of 1024 x 4096 with 64 rows: 23.8 us, 3.8 TB/s (24.4 with codes read word by word; 26.4 and, with groups of 32, 78 in place of 41
// when scales were loaded one by one three stages ahead, in registers that spilled).  A unit of work is
// 16 rows of weights (the MMA's rows) times the tokens of their group (its 8 columns, once or twice).
// One CTA an SM goes over a contiguous range of units, so the tokens stay in shared memory while the
// codes stream past.  Teams of warps take the units in turn (four teams of four warps, or one of sixteen
// where an SM has few units), each team through a ring of its own: a ring that they shared would be
// read by one team or another, and a barrier's parity does not tell a round from the one after next.
// A team's warps take blocks of 128 in turn and once a unit add their sums in order.  Four more
// warps ask for the codes by TMA, as far ahead as the rings reach, and bring scales and zero points into
// the form that the products read.  (A bulk copy for each row, 1 KB at a time, reached 3.1 TB/s without
// any products behind it.)
// - four bits at the low end of a BF16's mantissa, or the four above them, are the subnormal (or
//   first normal) number q 2^-133 or q 2^-129: one AND and one exact fused multiply-add make
//   (q - z) / 64 of two codes;
// - the MMA's sums run over one group and meet the group's scale in FP32, so the product is as
//   exact as with weights expanded in FP32 (sums below 2^-120 lose bits to the factor 64).
// The threads of a CTA leave 96 registers each.  With one MMA a step nothing spills; with two (9 to 16 tokens) 44 to 144 bytes a
// thread are loaded back (groups of 32: 144 as one team, 124 as four; of 64: 44, 56; of 128: none, 48).
// The order of the contraction within a group is free as long as both operands agree: the four threads
// of a row take G / 4 neighbouring codes each, in one load, and each reads pairs (i, i + 4) of a word of 8 with one mask;
// x is laid out in shared memory in their order.
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
constexpr int kUserWarps = 16, kHelpers = 4;  // the warps that multiply, and those that load for them
constexpr int kUsers = kUserWarps * 32, kThreads = kUsers + kHelpers * 32, kWarps = kThreads / 32;
constexpr int kRows = 16;    // of weights in a unit
constexpr int kPiece = 256;  // contraction elements in 128 bytes of codes, the width of a swizzled row
constexpr int kPieceBytes = kRows * 128;
constexpr int kRedStride = kRows + 4;
constexpr int kMostStages = 8;  // of a ring
// Contraction elements of a stage: one or two blocks of 128 a warp (one with groups of 32, whose scales are many).
constexpr int least_chunk(int teams) { return kUserWarps / teams * 128; }
constexpr int most_chunk(int teams, int G) { return teams == 1 || G == 32 ? least_chunk(teams) : 2 * least_chunk(teams); }
constexpr uint32_t kAll = 0xffffffffu;

struct ProductArgs {
  const void* x;
  int64_t ldx;
  const void* s;     // [E][N][K / G]
  const uint8_t* z;  // the same shape, or null
  int s_f32;
  int wide;    // scales and zero points lie so that several of a row are loaded at once
  int pieces;  // 1: the codes' map is [rows][K / 2], 128 bytes wide boxes; else [pieces][rows][128] with a stage a box
  const void* offsets;  // null: one group of all T rows
  int offsets64;
  int32_t E, T, N, K;
  int32_t x_rows, chunk, stages;  // tokens a pass; contraction elements of a stage, stages of a ring
  int32_t tiles;                  // ceil(N / 16)
  void* out;
  int64_t ldo;
  int out_f32;
  uint32_t* fault;
  uint64_t wait_ns;
};

// Shared memory of a CTA, from a multiple of 1024 on: codes of all rings' stages ([piece][16 rows][128
// bytes], swizzled by TMA, so that a piece's 16 bytes of 8 rows lie in different banks), their scales, x, sums, table.
struct Layout {
  int32_t code_bytes, meta, meta_bytes;  // of a stage
  int32_t x_stride, x, red, table, bytes;
};

__host__ __device__ inline Layout layout_of(int G, int K, int teams, int chunk, int stages, int x_rows, int tokens, int experts) {
  Layout l;
  l.code_bytes = chunk / kPiece * kPieceBytes;
  l.meta_bytes = chunk / G * (kRows + 1) * 8;
  l.x_stride = (K + 127) / 128 * 256 + 64;  // (what a warp reads of two rows at a time lies in different banks)
  l.meta = teams * stages * l.code_bytes;
  l.x = (l.meta + teams * stages * l.meta_bytes + 15) / 16 * 16;
  l.red = l.x + x_rows * l.x_stride;
  l.table = l.red + kUserWarps * tokens * kRedStride * 4;
  l.bytes = l.table + (experts > 0 ? (experts + 1) * 8 + experts * 2 : 0);
  return l;
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_16x8x16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Twice -z / 64 in BF16.
__device__ __forceinline__ uint32_t minus_zero(uint32_t z) { return fma_bf16x2((z & 15u) * 0x10001u, 0xFF00FF00u, 0); }

// (q - z) / 64 for the codes i and i + 4 of a word of 8, as pairs p[i] (`zero`: twice -z / 64 in BF16).
__device__ __forceinline__ void code_pairs(uint32_t word, uint32_t zero, uint32_t (&p)[4]) {
  constexpr uint32_t kLow = 0x7F007F00u, kHigh = 0x7D007D00u;  // 2^127, 2^123
  const uint32_t upper = word >> 8;
  p[0] = fma_bf16x2(word & 0x000F000Fu, kLow, zero);
  p[1] = fma_bf16x2(word & 0x00F000F0u, kHigh, zero);
  p[2] = fma_bf16x2(upper & 0x000F000Fu, kLow, zero);
  p[3] = fma_bf16x2(upper & 0x00F000F0u, kHigh, zero);
}

// N words of shared memory at once.
template <int N>
__device__ __forceinline__ void take_words(uint32_t* w, const uint8_t* p) {
  if (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// The groups' table: start[i], offset i clamped to [0, T] and to the running maximum; list, the experts
// that have rows; passes[i], the passes over tokens of those before the i-th (and of all, behind
// the last).  What had to be clamped is reported.  All threads call it.  Returns all passes.
struct Table {
  int32_t *start, *passes;
  uint16_t* list;
  int live;
};

__device__ __forceinline__ int build_table(const ProductArgs& a, Table& tab) {
  __shared__ int32_t most[kWarps], rows[kWarps], count[kWarps];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  int32_t carry = 0;
  for (int i0 = 0; i0 <= a.E; i0 += kThreads) {
    const int i = i0 + tid;
    int32_t v = 0;
    if (i <= a.E) {
      const int64_t raw = a.offsets64 ? static_cast<const int64_t*>(a.offsets)[i] : static_cast<const int32_t*>(a.offsets)[i];
      v = static_cast<int32_t>(raw < 0 ? 0 : raw > a.T ? a.T : raw);
      bad = bad || raw != v;
    }
    int32_t top = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(kAll, top, d);
      if (lane >= d) top = max(top, o);
    }
    if (lane == 31) most[warp] = top;
    __syncthreads();
    top = max(top, carry);
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) top = max(top, most[w]);
      carry = max(carry, most[w]);
    }
    if (i <= a.E) {
      bad = bad || v < top;
      tab.start[i] = top;
    }
    __syncthreads();
  }
  if (bad && blockIdx.x == 0) atomicOr(a.fault, kFaultOffsets);
  int live = 0, total = 0;
  for (int e0 = 0; e0 < a.E; e0 += kThreads) {
    const int e = e0 + tid, n = e < a.E ? tab.start[e + 1] - tab.start[e] : 0;
    const int own = (n + a.x_rows - 1) / a.x_rows;
    const uint32_t mask = __ballot_sync(kAll, n > 0);
    int incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kAll, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) rows[warp] = __popc(mask), count[warp] = incl;
    __syncthreads();
    int at = live + __popc(mask & ((1u << lane) - 1)), before = total + incl - own;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += rows[w], before += count[w];
      live += rows[w], total += count[w];
    }
    if (n > 0) tab.list[at] = static_cast<uint16_t>(e), tab.passes[at] = before;
    __syncthreads();
  }
  if (tid == 0) tab.passes[live] = total;
  tab.live = live;
  return total;
}

// A CTA's range of units: passes (one over the tokens of an expert, x_rows at a time) and, of each, tiles.
struct Pass {
  int index, tile, end;        // the pass; its tiles in the range
  int last_index, last_end;    // the range's last pass, and where in it the range ends
  int at, e, tok, count;       // the expert's place in the list, the expert, the pass's first token and their number

  __device__ __forceinline__ void enter(const ProductArgs& a, const Table& tab) {
    end = index == last_index ? last_end : a.tiles;
    int from = 0, hi = a.T, done = index;
    e = 0;
    if (a.offsets != nullptr) {
      e = tab.list[at];
      from = tab.start[e], hi = tab.start[e + 1];
      done = index - tab.passes[at];
    }
    tok = from + done * a.x_rows;
    count = min(a.x_rows, hi - tok);
  }
  __device__ __forceinline__ Pass(const ProductArgs& a, const Table& tab, int64_t from, int64_t to) {
    index = static_cast<int>(from / a.tiles), tile = static_cast<int>(from % a.tiles);
    last_index = static_cast<int>((to - 1) / a.tiles), last_end = static_cast<int>((to - 1) % a.tiles) + 1;
    at = 0;
    if (a.offsets != nullptr)
      for (int step = 512; step > 0; step >>= 1)  // (at most 1024 experts)
        if (at + step < tab.live && tab.passes[at + step] <= index) at += step;
    enter(a, tab);
  }
  __device__ __forceinline__ bool done() const { return index > last_index; }
  __device__ __forceinline__ void next(const ProductArgs& a, const Table& tab) {
    tile = 0;
    if (++index > last_index) return;
    if (a.offsets != nullptr && index == tab.passes[at + 1]) ++at;
    enter(a, tab);
  }
};

// A place in a ring: stage and parity.
struct Place {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void advance(int stages) {
    if (++slot == stages) slot = 0, parity ^= 1;
  }
};

__device__ __forceinline__ void store_out(const ProductArgs& a, int32_t t, int32_t n, float v) {
  const int64_t i = t * a.ldo + n;
  if (a.out_f32)
    static_cast<float*>(a.out)[i] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[i] = __float2bfloat16_rn(v);
}

// N neighbouring words in as few loads as their alignment (that of all of them, up to 16 bytes) allows.
template <int N, int M>
__device__ __forceinline__ void load_words(uint32_t (&v)[M], const uint32_t* p) {
  if (N == 1) {
    v[0] = __ldg(p);
  } else if (N == 2) {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = t.x, v[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 t = __ldg(reinterpret_cast<const uint4*>(p) + i);
      v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
    }
  }
}

template <int G, int NT, int TEAMS>
__global__ void __launch_bounds__(kThreads, 1)
    int4_product_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ CUtensorMap codes_map) {
  extern __shared__ __align__(1024) uint8_t raw_smem[];
  uint8_t* smem = raw_smem + (0u - smem_addr(raw_smem)) % 1024;
  __shared__ __align__(8) uint64_t barriers[2][TEAMS * kMostStages];
  constexpr int WAYS = kUserWarps / TEAMS, TEAM = WAYS * 32, HELPERS = kHelpers / TEAMS;  // warps and threads of a team, helpers of a ring
  constexpr int TT = 8 * NT, GROUPS = 128 / G, STEPS = G / 32, CHUNK = most_chunk(TEAMS, G);
  const Layout l = layout_of(G, a.K, TEAMS, a.chunk, a.stages, a.x_rows, TT, a.offsets != nullptr ? a.E : 0);
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  // ring r's stage i is number r * stages + i
  const uint32_t full = smem_addr(barriers[0]), empty = smem_addr(barriers[1]);
  if (tid < TEAMS * a.stages) {
    mbar_init(full + 8 * tid, 1 + HELPERS);  // the codes (bytes), and each helper's scales
    mbar_init(empty + 8 * tid, WAYS);        // the team's warps
    fence_mbar_init();
  }
  if (tid == kUsers) tma_prefetch_map(&codes_map);
  Table tab;
  tab.start = reinterpret_cast<int32_t*>(smem + l.table), tab.passes = tab.start + a.E + 1;
  tab.list = reinterpret_cast<uint16_t*>(tab.passes + a.E + 1), tab.live = 0;
  int passes = (a.T + a.x_rows - 1) / a.x_rows;
  if (a.offsets != nullptr) {
    passes = build_table(a, tab);
    // rows of no group are zero
    auto zero = [&](int32_t from, int32_t to) {
      const int64_t count = static_cast<int64_t>(to - from) * a.N;
      for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + tid; i < count; i += static_cast<int64_t>(gridDim.x) * kThreads)
        store_out(a, from + static_cast<int32_t>(i / a.N), static_cast<int32_t>(i % a.N), 0.0f);
    };
    zero(0, tab.start[0]);
    zero(tab.start[a.E], a.T);
  }
  const int64_t units = static_cast<int64_t>(passes) * a.tiles;
  const int64_t from = units * blockIdx.x / gridDim.x, to = units * (blockIdx.x + 1) / gridDim.x;
  __syncthreads();
  if (from >= to) return;
  Pass pass(a, tab, from, to);
  // A wait that runs out is recorded; the warp then waits no more, and a helper stops.
  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    const bool ok = dead || mbar_wait_idle(bar, parity, a.wait_ns);
    if (__all_sync(kAll, ok)) return;
    dead = true;
    atomicOr(a.fault, kFaultProducerWait);
  };
  Place at;
  int phase = 0;  // units of the passes before, modulo the teams

  if (warp >= kUserWarps) {
    // --------------------------------------------------- codes, scales and zero points of a ring
    // Scales are [group][row] (scale, twice -z / 64), some rows a helper; a lane has PER neighbouring groups of one row, in
    // one or two loads where they lie so, and the next stage's are on their way.  (Two stages: spills, 47 us for 41 with groups
    // of 32.  Helpers that took stages by turns could be two rounds from a barrier.)
    constexpr int ROWS = kRows / HELPERS, PER = CHUNK / G * ROWS / 32;
    const int team = (warp - kUserWarps) / HELPERS, helper = (warp - kUserWarps) % HELPERS;
    const int groups = a.K / G, in_stage = a.chunk / G;  // (a power of two)
    const int shift = 31 - __clz(in_stage);
    uint32_t held_s[PER], held_z[PER];  // of the next stage, as they come: a conversion would wait for them
    int held_row = 0, held_k0 = 0;
    int k0 = 0, pending = 0, tile = 0;
    const int own_r = (lane * PER) >> shift, own_g = (lane * PER) & (in_stage - 1);
    const bool wide = a.wide && groups % PER == 0;
    auto settle = [&]() {  // the ring's next unit, from this pass on
      while (!pass.done() && tile >= pass.end) {
        phase = (phase + pass.end - pass.tile) % TEAMS;
        pass.next(a, tab);
        tile = pass.tile + (team - phase + TEAMS) % TEAMS;
      }
    };
    auto fetch = [&]() {  // the next stage's, if there is one
      if (pass.done()) return;
      const int n0 = tile * kRows + helper * ROWS, g0 = k0 / G;
      held_row = pass.e * a.N + tile * kRows, held_k0 = k0;
#pragma unroll
      for (int i = 0; i < PER; ++i) held_s[i] = 0, held_z[i] = wide ? 0x08080808 : 8;
      if (own_r < ROWS && n0 + own_r < a.N && g0 + own_g < groups) {
        const int64_t p = static_cast<int64_t>(pass.e * a.N + n0 + own_r) * groups + g0 + own_g;
        const uint16_t* const s16 = static_cast<const uint16_t*>(a.s) + p;
        const uint32_t* const s32 = static_cast<const uint32_t*>(a.s) + p;
        if (wide) {
          if (a.s_f32)
            load_words<PER>(held_s, s32);
          else
            load_words<PER / 2>(held_s, reinterpret_cast<const uint32_t*>(s16));
          if (a.z != nullptr) {
            if (PER >= 4)
              load_words<PER / 4>(held_z, reinterpret_cast<const uint32_t*>(a.z + p));
            else
              held_z[0] = __ldg(reinterpret_cast<const uint16_t*>(a.z + p));
          }
        } else {
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if (g0 + own_g + i >= groups) continue;
            held_s[i] = a.s_f32 ? __ldg(s32 + i) : __ldg(s16 + i);
            if (a.z != nullptr) held_z[i] = __ldg(a.z + p + i);
          }
        }
      }
      ++pending;
      k0 += a.chunk;
      if (k0 >= a.K) {
        k0 = 0;
        tile += TEAMS;
        settle();
      }
    };
    auto load_codes = [&](int stage, int row, int from_k) {  // (a box may reach into the next expert's rows: they are not used)
      if (helper != 0) return;
      const uint32_t bar = full + 8 * stage, dst = smem_addr(smem) + stage * l.code_bytes;
      if (lane == 0) mbar_expect_tx(bar, l.code_bytes);
      __syncwarp();
      if (a.pieces == 1) {
        if (lane < a.chunk / kPiece) tma_load_2d(dst + lane * kPieceBytes, &codes_map, bar, from_k / 2 + lane * 128, row);
      } else if (lane == 0) {
        tma_load_3d(dst, &codes_map, bar, 0, row, from_k / kPiece);
      }
    };
    tile = pass.tile + team;
    settle();
    fetch();
    while (pending > 0 && !dead) {
      const int stage = team * a.stages + at.slot;
      wait(empty + 8 * stage, at.parity ^ 1);
      if (dead) break;
      load_codes(stage, held_row, held_k0);
      uint2* meta = reinterpret_cast<uint2*>(smem + l.meta + stage * l.meta_bytes) + own_g * (kRows + 1) + helper * ROWS + own_r;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        uint32_t sc = held_s[i], z = held_z[i];
        if (wide) z = held_z[i / 4] >> (8 * (i % 4));
        if (!a.s_f32) sc = !wide ? sc << 16 : i % 2 ? held_s[i / 2] & 0xFFFF0000u : held_s[i / 2] << 16;
        if (own_r < ROWS) meta[i * (kRows + 1)] = make_uint2(sc, minus_zero(z));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * stage);
      at.advance(a.stages);
      --pending;
      fetch();
    }
    // (a CTA does not end before its copies: without a fault the team has waited for them all)
    for (int i = 0; dead && i < a.stages; ++i)  // stages before this place were filled in its round, the others in the one before
      mbar_wait(full + 8 * (team * a.stages + i), i < at.slot ? at.parity : at.parity ^ 1, a.wait_ns);
    return;
  }
  // ------------------------------------------------------------------ products
  const int team = warp / WAYS, way = warp % WAYS, g = lane >> 2, t = lane & 3;
  float* red = reinterpret_cast<float*>(smem + l.red) + team * (WAYS * TT * kRedStride);
  // Of a group's bytes each thread of a row takes neighbouring ones, in one load.  The MMA's row g is the unit's row
  // (0, 4, 2, 6, 1, 5, 3, 7)[g] (and g + 8 that + 8), so that what the threads of two or four rows read at a time
  // lies in different banks of a swizzled piece (a warp's blocks are all a piece's first or second half).
  const int row_g = (g & 1) << 2 | (g & 2) | g >> 2;
  int32_t word[GROUPS];
#pragma unroll
  for (int i = 0; i < GROUPS; ++i)
    word[i] = way / 2 * kPieceBytes + row_g * 128 + (((way % 2 * 4 + i * STEPS + t * STEPS / 4) ^ row_g) << 4) + t * STEPS % 4 * 4;
  for (; !pass.done(); phase = (phase + pass.end - pass.tile) % TEAMS, pass.next(a, tab)) {
    const int count = pass.count;
    int32_t x_row[NT];  // this thread's rows of x (columns behind the last token: its row again, their sums are not used)
#pragma unroll
    for (int i = 0; i < NT; ++i) x_row[i] = l.x + min(i * 8 + g, count - 1) * l.x_stride + t * 16 + way * 256;
    // the pass's tokens, in the order of the codes' pairs; zeros behind the contraction's end
    named_sync(1, kUsers);
    for (int c = tid; c < (a.K + 127) / 128 * 16; c += kUsers) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.x) + pass.tok * a.ldx) + c;
      // chunk (group, thread, step) of a block of 128 stands where that step's load of that thread finds it
      const int to = (c & ~(4 * STEPS - 1)) + c % STEPS * 4 + c / STEPS % 4;
      for (int r0 = 0; r0 < count; r0 += 8) {
        uint4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          v[r] = r0 + r < count && c * 8 < a.K ? __ldg(src + (r0 + r) * (a.ldx / 8)) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r0 + r < count)
            *reinterpret_cast<uint4*>(smem + l.x + (r0 + r) * l.x_stride + to * 16) =
                make_uint4(__byte_perm(v[r].x, v[r].z, 0x5410), __byte_perm(v[r].x, v[r].z, 0x7632),
                           __byte_perm(v[r].y, v[r].w, 0x5410), __byte_perm(v[r].y, v[r].w, 0x7632));
      }
    }
    named_sync(1, kUsers);
    for (int tile = pass.tile + (team - phase + TEAMS) % TEAMS; tile < pass.end; tile += TEAMS) {
      float acc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
      uint32_t xs = 0;
      for (int k0 = 0; k0 < a.K; k0 += a.chunk) {
        const int stage = team * a.stages + at.slot;
        wait(full + 8 * stage, at.parity);
        const uint2* meta = reinterpret_cast<const uint2*>(smem + l.meta + stage * l.meta_bytes) + way * (GROUPS * (kRows + 1)) + row_g;
        const uint8_t* codes = smem + stage * l.code_bytes;
        const int left = min(a.chunk, a.K - k0);
        for (int k = way * 128; k < left; k += WAYS * 128) {
          uint32_t wa[4], wb[4];
#pragma unroll
          for (int i = 0; i < GROUPS; ++i) {
            take_words<STEPS>(wa + i * STEPS, codes + word[i]);
            take_words<STEPS>(wb + i * STEPS, codes + word[i] + 8 * 128);
          }
#pragma unroll
          for (int grp = 0; grp < GROUPS; ++grp) {
            const uint2 ma = meta[grp * (kRows + 1)], mb = meta[grp * (kRows + 1) + 8];
            float c[NT][4];
#pragma unroll
            for (int j = grp * STEPS; j < (grp + 1) * STEPS; ++j) {
              uint32_t pa[4], pb[4];
              code_pairs(wa[j], ma.y, pa);
              code_pairs(wb[j], mb.y, pb);
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(smem + (x_row[i] + xs) + j * 64);
                if (j == grp * STEPS)
                  mma_16x8x16_zero(c[i], pa[0], pb[0], pa[1], pb[1], x.x, x.y);
                else
                  mma_16x8x16(c[i], pa[0], pb[0], pa[1], pb[1], x.x, x.y);
                mma_16x8x16(c[i], pa[2], pb[2], pa[3], pb[3], x.z, x.w);
              }
            }
            const float fa = __uint_as_float(ma.x), fb = __uint_as_float(mb.x);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              acc[i][0] = fmaf(c[i][0], fa, acc[i][0]);
              acc[i][1] = fmaf(c[i][1], fa, acc[i][1]);
              acc[i][2] = fmaf(c[i][2], fb, acc[i][2]);
              acc[i][3] = fmaf(c[i][3], fb, acc[i][3]);
            }
          }
          codes += WAYS / 2 * kPieceBytes;
          meta += WAYS * GROUPS * (kRows + 1);
          xs += WAYS * 256;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + 8 * stage);
        at.advance(a.stages);
      }
      named_sync(2 + team, TEAM);  // (the sums of the team's last unit have been read)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float* d = red + (way * TT + i * 8 + 2 * t) * kRedStride + row_g;
        d[0] = acc[i][0];
        d[kRedStride] = acc[i][1];
        d[8] = acc[i][2];
        d[kRedStride + 8] = acc[i][3];
      }
      named_sync(2 + team, TEAM);
      // the warps' sums in order
      const int n0 = tile * kRows;
      for (int i = tid % TEAM; i < count * kRows; i += TEAM) {
        const int r = i / kRows, n = i % kRows;
        float s = red[r * kRedStride + n];
#pragma unroll
        for (int w = 1; w < WAYS; ++w) s += red[(w * TT + r) * kRedStride + n];
        if (n0 + n < a.N) store_out(a, pass.tok + r, n0 + n, s * 64.0f);
      }
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
  int32_t K, G;
  uint32_t pieces, per_row;  // of 8 values: below 2^31, and K / 8
  uint32_t mul, shift;       // n / per_row = (umulhi(n, mul) + n) >> shift
  int group_shift;           // log2 of a group's pieces
  void* out;
  int64_t ldo;
};

constexpr float kTinyScale = 1e-30f;  // a group of zeros still has a scale to divide by
constexpr int kPerThread = 4;         // pieces: their loads are in flight together

// Maxima that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A group's scale, zero point and the scale's reciprocal from its largest value and its largest negated one.
struct Scale {
  float s, z, inverse;
};

__device__ __forceinline__ Scale scale_of(const CodeArgs& a, float hi, float minus_lo) {
  Scale v;
  v.s = a.z != nullptr ? __fdiv_rn(hi + minus_lo, 15.0f) : __fdiv_rn(max_nan(hi, minus_lo), 7.0f);
  v.s = max_nan(v.s, kTinyScale);
  if (!a.s_f32) v.s = __bfloat162float(__float2bfloat16_rn(v.s));
  v.z = 8.0f;
  if (a.z != nullptr) v.z = fminf(fmaxf(rintf(__fdiv_rn(minus_lo, v.s)), 0.0f), 15.0f);
  v.inverse = __frcp_rn(v.s);
  return v;
}

__device__ __forceinline__ void put_scale(const CodeArgs& a, uint32_t group, const Scale& v) {
  if (a.s_f32)
    static_cast<float*>(a.s)[group] = v.s;
  else
    static_cast<__nv_bfloat16*>(a.s)[group] = __float2bfloat16_rn(v.s);
  if (a.z != nullptr) a.z[group] = static_cast<uint8_t>(v.z);
}

// The codes of 8 values, rn(rn(w / s)) + z.  The quotient is w times the rounded reciprocal, corrected twice by its remainder: the
// first makes it one of its two neighbours in FP32, whose remainder is exact, the second the rounded quotient (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, 1990).  The reciprocal is normal below 1e37,
// and a remainder that underflows belongs to a quotient below 1/4 (s is 1e-30 at least).  Quotients halfway between
// two integers are common where w and s are BF16: a product by the reciprocal alone, and divisions next to a border, took 30 us
// in place of 24 for 12288 x 4096.
__device__ __forceinline__ uint32_t codes_of(const CodeArgs& a, const Two (&w)[4], const Scale& v) {
  constexpr float kRound = 12582912.0f;  // 1.5 2^23: adding it leaves the nearest integer, to even between two
  constexpr float kInteger = 8388608.0f;  // 2^23: an integer's bits
  float low = 0.0f, high = 0.0f;  // codes 0 to 3 and 4 to 7 as one number
  auto add = [&](int j, Two q) {
    const Two c = (q + twice(kRound)) + twice(v.z - kRound);
    float c0 = lo(c), c1 = dp::hi(c);
    // (at least 0: rn(-lo / s) = -rn(lo / s); above 15 only where both ends of a range are rounded up)
    if (a.z != nullptr) c0 = fminf(c0, 15.0f), c1 = fminf(c1, 15.0f);
    float& sum = j < 2 ? low : high;
    const float weight = j % 2 ? 256.0f : 1.0f;
    sum = fmaf(c1, 16.0f * weight, fmaf(c0, weight, sum));
  };
  if (v.s < 1e37f) {
    const Two y = twice(v.inverse), minus_s = twice(-v.s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      Two q = w[j] * y;
      q = fma2(fma2(q, minus_s, w[j]), y, q);
      add(j, fma2(fma2(q, minus_s, w[j]), y, q));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) add(j, two(__fdiv_rn(lo(w[j]), v.s), __fdiv_rn(dp::hi(w[j]), v.s)));
  }
  return __byte_perm(__float_as_uint(low + kInteger), __float_as_uint(high + kInteger), 0x5410);
}

// BF16: a thread takes 32 neighbouring values, the WIDTH = G / 32 threads of a group share their range.  Their loads, 16 bytes
// of every 64, meet in L1.  Bound: HBM bytes and instructions; 12288 x 4096 with zero points, groups of 128:
// 24 us, 5.3 TB/s (8 to 14 us more with 8 values of each of four places a thread, whose ranges go over 16 threads; 100 so
// with a division for every value).
template <int WIDTH>
__global__ void __launch_bounds__(256) int4_quantize_bf16_kernel(const __grid_constant__ CodeArgs a) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x, n = 4 * i;
  const uint32_t r = (__umulhi(n, a.mul) + n) >> a.shift;
  const bool in = n < a.pieces;  // (a row is whole groups: the threads of a group are in range together)
  Raw8<false> raw[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    raw[k] = in ? load_raw8<false>(a.w, r * a.ldw + (n - r * a.per_row) * 8 + k * 8) : zero_raw8<false>();
  uint32_t up = 0, down = 0;  // two at a time
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) up = max_nan2(up, w[j]), down = min_nan2(down, w[j]);
  }
  down ^= 0x80008000u;
  uint32_t both = max_nan2(__byte_perm(up, down, 0x5410), __byte_perm(up, down, 0x7632));  // both maxima in one word
#pragma unroll
  for (int d = 1; d < WIDTH; d <<= 1) both = max_nan2(both, __shfl_xor_sync(kAll, both, d));
  const Scale v = scale_of(a, __uint_as_float(both << 16), __uint_as_float(both & 0xFFFF0000u));
  uint32_t word[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    Two w[4];
    unpack8<false>(raw[k], w);
    word[k] = codes_of(a, w, v);
  }
  if (!in) return;
  reinterpret_cast<uint4*>(a.q)[i] = make_uint4(word[0], word[1], word[2], word[3]);
  if ((threadIdx.x & (WIDTH - 1)) == 0) put_scale(a, i / WIDTH, v);
}

// FP32: a thread takes 8 neighbouring values of kPerThread places, the WIDTH = G / 8 threads of a group share their range.
// Bound: HBM bytes; 12288 x 4096 with zero points, groups of 128: 38 us, 6.0 TB/s.
template <int WIDTH>
__global__ void __launch_bounds__(256, 4) int4_quantize_f32_kernel(const __grid_constant__ CodeArgs a) {
  const uint32_t first = blockIdx.x * (256u * kPerThread) + threadIdx.x;
  Raw8<true> raw[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const uint32_t i = first + k * 256, r = (__umulhi(i, a.mul) + i) >> a.shift;
    raw[k] = i < a.pieces ? load_raw8<true>(a.w, r * a.ldw + (i - r * a.per_row) * 8) : zero_raw8<true>();
  }
  // Of a group's first four threads (and every four after them), each divides for one of the places.
  static_assert(kPerThread == 4, "places are shared among four threads");
  float its_hi = 0.0f, its_minus_lo = 0.0f;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[k]);
    float hi = 0.0f, minus_lo = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = __uint_as_float(w[j]);
      hi = max_nan(hi, x);
      minus_lo = max_nan(minus_lo, -x);
    }
#pragma unroll
    for (int d = 1; d < WIDTH; d <<= 1) {
      hi = max_nan(hi, __shfl_xor_sync(kAll, hi, d));
      minus_lo = max_nan(minus_lo, __shfl_xor_sync(kAll, minus_lo, d));
    }
    if ((threadIdx.x & 3) == k) its_hi = hi, its_minus_lo = minus_lo;
  }
  const Scale its = scale_of(a, its_hi, its_minus_lo);
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int from = static_cast<int>(threadIdx.x & 28) + k;
    const Scale v = {__shfl_sync(kAll, its.s, from), __shfl_sync(kAll, its.z, from), __shfl_sync(kAll, its.inverse, from)};
    Two w[4];
    unpack8<true>(raw[k], w);
    const uint32_t word = codes_of(a, w, v), i = first + k * 256;
    if (i >= a.pieces) continue;
    reinterpret_cast<uint32_t*>(a.q)[i] = word;
    if ((threadIdx.x & (WIDTH - 1)) == 0) put_scale(a, i / WIDTH, v);
  }
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Bound: HBM bytes and instructions.  PAIRS (BF16 scales and weights): the products' pairs of codes, times 64 and times s two at a
// time, each product of a code and a scale rounded once.  12288 x 4096 to BF16 with zero points: 22 us, 5.7 TB/s
// (23 through FP32).
template <bool OF32, bool PAIRS>
__global__ void __launch_bounds__(256) int4_expand_kernel(const __grid_constant__ CodeArgs a) {
  const uint32_t first = blockIdx.x * (256u * kPerThread) + threadIdx.x;
  uint32_t word[kPerThread], s[kPerThread], z[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const uint32_t i = first + k * 256;
    word[k] = s[k] = 0, z[k] = 8;
    if (i >= a.pieces) continue;
    word[k] = __ldg(reinterpret_cast<const uint32_t*>(a.q) + i);
    const uint32_t g = i >> a.group_shift;  // (rows are whole groups, and packed)
    s[k] = a.s_f32 ? __ldg(static_cast<const uint32_t*>(a.s) + g) : __ldg(static_cast<const uint16_t*>(a.s) + g);
    if (a.z != nullptr) z[k] = __ldg(a.z + g);
  }
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const uint32_t i = first + k * 256;
    if (i >= a.pieces) continue;
    const uint32_t r = (__umulhi(i, a.mul) + i) >> a.shift;
    const int64_t at = r * a.ldo + (i - r * a.per_row) * 8;
    if (PAIRS) {
      uint32_t p[4];
      code_pairs(word[k], minus_zero(z[k]), p);
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] = mul_bf16x2(mul_bf16x2(p[j], 0x42804280u), s[k] * 0x10001u);
      Raw8<false> out;
      out.v[0] = make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410), __byte_perm(p[0], p[1], 0x7632),
                            __byte_perm(p[2], p[3], 0x7632));
      store_raw8<false>(a.out, at, out);
      continue;
    }
    // (2^23 + a code is the code's bits under that exponent)
    const Two scale = twice(__uint_as_float(a.s_f32 ? s[k] : s[k] << 16));
    const Two zero = twice(-8388608.0f - static_cast<float>(z[k] & 15u));
    Two v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = (two(__uint_as_float(((word[k] >> (8 * j)) & 15u) | 0x4B000000u),
                  __uint_as_float(((word[k] >> (8 * j + 4)) & 15u) | 0x4B000000u)) + zero) * scale;
    store8<OF32>(a.out, at, v);
  }
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
void by_form(int nt, int teams, F f) {
  if (nt == 1)
    teams == 1 ? f(std::integral_constant<int, 1>(), std::integral_constant<int, 1>())
               : f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
  else
    teams == 1 ? f(std::integral_constant<int, 2>(), std::integral_constant<int, 1>())
               : f(std::integral_constant<int, 2>(), std::integral_constant<int, 4>());
}

constexpr int kMaxShared = 225 * 1024;

struct Int4Plan {
  int nt, teams, x_rows, chunk, stages, bytes, grid;
};

// Tokens a pass: as many as shared memory holds beside two stages a ring, at most two MMAs' (16); one MMA's (8) where groups
// have four and fewer on average, whose passes seldom need more.
// Teams: one where an SM has fewer than two units (eight where a pass has more than 8 tokens, whose room the rings lose),
// which four teams would share unevenly and whose sums they would begin late.  One team / four (us):
//   one token, groups of 128: 6144 x 4096 (2.5 units an SM) 7.0 / 6.2, 12288 x 4096 10.8 / 9.5; of 32: 4096 x 4096 (1.7) 6.4 / 7.9
//   8 tokens, groups of 64: 6144 x 4096 7.8 / 7.0, 4096 x 12288 (1.7) 21.1 / 24.2
//   16 tokens: 12288 x 4096 (5.1) 15.3 / 17.7, 16384 x 4096 (6.7) 17.0 / 18.6, 24576 x 2048 (10.1) 15.9 / 12.5
//   64 experts of 1024 x 4096 with 64 rows (17) 30.7 / 24.3
Int4Plan plan_int4(int64_t E, int64_t T, int64_t N, int64_t K, int64_t G, bool grouped, int sm_count) {
  Int4Plan p;
  const int64_t tokens = grouped ? (T + E - 1) / E : T, tiles = (N + kRows - 1) / kRows;
  const int64_t units = tiles * (grouped ? std::min(E, T) : (T + 15) / 16);  // about
  const int want = tuning_override("DP_FORCE_INT4_TOKENS", 0), want_teams = tuning_override("DP_FORCE_INT4_TEAMS", 0);
  const int experts = grouped ? static_cast<int>(E) : 0, g = static_cast<int>(G), k = static_cast<int>(K);
  p.teams = want_teams == 1 || want_teams == 4 ? want_teams : units < (tokens <= 8 ? 2 : 8) * sm_count ? 1 : 4;
  p.x_rows = static_cast<int>(std::min<int64_t>(T, want > 0 && want <= 16 ? want : tokens <= 4 && grouped ? 8 : 16));
  for (;; p.x_rows = (p.x_rows + 1) / 2) {
    p.nt = p.x_rows <= 8 ? 1 : 2;
    for (p.chunk = most_chunk(p.teams, g); p.chunk >= least_chunk(p.teams); p.chunk /= 2) {
      const Layout none = layout_of(g, k, p.teams, p.chunk, 0, p.x_rows, 8 * p.nt, experts);
      p.stages = std::min(kMostStages, (kMaxShared - 1024 - none.bytes) / (p.teams * (none.code_bytes + none.meta_bytes)));
      if (p.stages >= (p.chunk > least_chunk(p.teams) ? 3 : 2)) {
        p.bytes = layout_of(g, k, p.teams, p.chunk, p.stages, p.x_rows, 8 * p.nt, experts).bytes + 1024;
        p.grid = static_cast<int>(std::min<int64_t>(tiles * (grouped ? std::min(E, T) : 1) * ((T + p.x_rows - 1) / p.x_rows), sm_count));
        return p;
      }
    }
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
  if (!flag(out_f32) || !flag(s_f32) || E < 0 || T < 0 || N < 1 || K < 1) return DP_ERR_INVALID_ARG;
  if (offset_bits != 32 && offset_bits != 64) return DP_ERR_INVALID_ARG;
  if (N % 8 != 0 || N > 0x7FFFF || K > kMaxInt4K || E > kMaxInt4Experts || T > 0x7FFFFFFF - 256) return DP_ERR_UNSUPPORTED;
  dp_status st = check_codes(q, s, z, s_f32, E * N, K, G);  // (each held to its range: the product fits)
  if (st != DP_OK) return st;
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
  const Int4Plan p = plan_int4(E, T, N, K, G, offsets != nullptr, ctx.sm_count);
  ProductArgs a = {};
  a.x = x, a.ldx = ldx, a.s = s, a.z = static_cast<const uint8_t*>(z), a.s_f32 = s_f32;
  a.wide = is_aligned16(s) && is_aligned16(z);
  a.offsets = offsets, a.offsets64 = offset_bits == 64;
  a.E = static_cast<int32_t>(E), a.T = static_cast<int32_t>(T), a.N = static_cast<int32_t>(N), a.K = static_cast<int32_t>(K);
  a.x_rows = p.x_rows, a.chunk = p.chunk, a.stages = p.stages, a.tiles = static_cast<int32_t>((N + kRows - 1) / kRows);
  a.out = out, a.ldo = ldo, a.out_f32 = out_f32, a.fault = ctx.fault, a.wait_ns = kWaitLimitNs;
  a.pieces = K % kPiece == 0 ? p.chunk / kPiece : 1;
  CUtensorMap map;
  if (!encode_bytes(&map, q, E * N, K / 2, kRows, a.pieces)) return DP_ERR_LAUNCH;
  by_group(G, [&](auto g) {
    by_form(p.nt, p.teams, [&](auto nt, auto teams) {
      int4_product_kernel<decltype(g)::value, decltype(nt)::value, decltype(teams)::value><<<p.grid, kThreads, p.bytes, str>>>(a, map);
    });
  });
  return cudaGetLastError() == cudaSuccess ? DP_OK : DP_ERR_LAUNCH;
}

}  // namespace

cudaError_t set_attributes_int4() {
  cudaError_t e = cudaSuccess;
  for (int G = 32; G <= 128; G *= 2)
    by_group(G, [&](auto g) {
      for (int form = 0; form < 4; ++form)
        by_form(1 + form % 2, form / 2 ? 4 : 1, [&](auto nt, auto teams) {
          if (e == cudaSuccess)
            e = cudaFuncSetAttribute(int4_product_kernel<decltype(g)::value, decltype(nt)::value, decltype(teams)::value>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared);
        });
    });
  return e;
}

}  // namespace dp

namespace dp {
namespace {

// Launches over rows of K values, so many at a time that their pieces can be counted in 31 bits.
template <typename F>
dp_status run_codes(CodeArgs a, int64_t rows, int w_size, int s_size, F launch) {
  a.per_row = static_cast<uint32_t>(a.K / 8);
  a.group_shift = a.G == 32 ? 2 : a.G == 64 ? 3 : 4;
  a.shift = 0;
  while ((uint64_t{1} << a.shift) < a.per_row) ++a.shift;
  a.mul = static_cast<uint32_t>((((uint64_t{1} << a.shift) - a.per_row) << 32) / a.per_row + 1);
  int64_t most = 0x7FFFFF00 / a.per_row;
  if (const int want = tuning_override("DP_FORCE_INT4_ROWS", 0); want > 0) most = std::min<int64_t>(most, want);
  for (int64_t row = 0; row < rows; row += most) {
    const int64_t n = std::min(most, rows - row);
    a.pieces = static_cast<uint32_t>(n * a.per_row);
    launch(a, static_cast<unsigned>((a.pieces + 256u * kPerThread - 1) / (256u * kPerThread)));
    if (cudaGetLastError() != cudaSuccess) return DP_ERR_LAUNCH;
    const int64_t groups = n * (a.K / a.G);
    if (a.w != nullptr) a.w = static_cast<const char*>(a.w) + n * a.ldw * w_size;
    if (a.out != nullptr) a.out = static_cast<char*>(a.out) + n * a.ldo * w_size;
    a.q += n * (a.K / 2);
    a.s = static_cast<char*>(a.s) + groups * s_size;
    if (a.z != nullptr) a.z += groups;
  }
  return DP_OK;
}

}  // namespace
}  // namespace dp

extern "C" dp_status dp_int4_quantize(const void* w, int64_t ldw, int w_f32, int64_t rows, int64_t K, int64_t group, void* q,
                                      void* s, int s_f32, void* z, dp_stream stream) {
  using namespace dp;
  if (!flag(w_f32)) return DP_ERR_INVALID_ARG;
  dp_status st = check_codes(q, s, z, s_f32, rows, K, group);
  if (st == DP_OK) st = check_operand(w, rows, K, &ldw, w_f32 ? 4 : 2);
  if (st != DP_OK) return st;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  CodeArgs a = {};
  a.w = w, a.ldw = ldw, a.q = static_cast<uint8_t*>(q), a.s = s, a.z = static_cast<uint8_t*>(z), a.s_f32 = s_f32;
  a.K = static_cast<int32_t>(K), a.G = static_cast<int32_t>(group);
  static_assert(kPerThread == 4, "32 values a thread, of one place or of four");
  return run_codes(a, rows, w_f32 ? 4 : 2, s_f32 ? 4 : 2, [&](const CodeArgs& part, unsigned grid) {
    by_group(group, [&](auto g) {
      constexpr int G = decltype(g)::value;
      if (w_f32)
        int4_quantize_f32_kernel<G / 8><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(part);
      else
        int4_quantize_bf16_kernel<G / 32><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(part);
    });
  });
}

extern "C" dp_status dp_int4_dequantize(const void* q, const void* s, int s_f32, const void* z, int64_t rows, int64_t K,
                                        int64_t group, void* w, int64_t ldw, dp_out_dtype out, dp_stream stream) {
  using namespace dp;
  const int code = static_cast<int>(out);
  if (!flag(code)) return DP_ERR_INVALID_ARG;
  dp_status st = check_codes(q, s, z, s_f32, rows, K, group);
  if (st == DP_OK) st = check_operand(w, rows, K, &ldw, code ? 4 : 2);
  if (st != DP_OK) return st;
  DeviceContext ctx;
  if ((st = device_context(&ctx)) != DP_OK) return st;
  CodeArgs a = {};
  a.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q)), a.s = const_cast<void*>(s);
  a.z = const_cast<uint8_t*>(static_cast<const uint8_t*>(z)), a.s_f32 = s_f32;
  a.K = static_cast<int32_t>(K), a.G = static_cast<int32_t>(group), a.out = w, a.ldo = ldw;
  return run_codes(a, rows, code ? 4 : 2, s_f32 ? 4 : 2, [&](const CodeArgs& part, unsigned grid) {
    if (code)
      int4_expand_kernel<true, false><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(part);
    else if (part.s_f32)
      int4_expand_kernel<false, false><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(part);
    else
      int4_expand_kernel<false, true><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(part);
  });
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

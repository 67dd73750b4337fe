// Large tiles of the products grouped by expert (ragged.hip has the formulas
// and the form for any alignment): operands whose rows start on 16 bytes.
//
// One workgroup per CU walks output tiles of 64 FA x 256; 4 waves, 2 x 2, each
// 32 FA x 128.  Operands go from memory to LDS without passing registers (buffer
// loads to LDS, 16 bytes a lane), in stages of 128 contraction bytes (64 values of
// 16 bits, 128 of 8) in two slots.
//
// Two kinds of operand:
//  * contraction contiguous (X and W in NT, dY in NN): a stage is [rows][128 B],
//    16-byte chunk c of row r at chunk c ^ ((r >> 1) & 7): two rows fill the
//    256 bytes of the banks, and the 16 rows that one LDS access phase reads use
//    16 different places there.
//  * contraction over rows (W in NN, dY and X in TN): a stage is [64][512 B],
//    chunk c of row r at chunk c ^ {0, 4, 10, 14}[r & 3] ^ 2 (r / 8 % 2).  Fragments
//    come through the transposing LDS read: in each group of 16 lanes, lane l
//    hands in the address of 4 columns of contraction row l / 4 and gets 4
//    contraction rows of column l.  The 8 rows (two groups of 4, 8 apart) x 16
//    columns of 32 lanes lie in 256 different bytes of bank space.
// What lies outside an operand (rows past an expert's in TN, past N in
// NN, past K in a last stage, row indexes out of range) is zero because the
// buffer loads are bounded: such a lane's offset fails the range check and the
// load writes zeros.  Rows of other experts that a tile of NT or NN takes along
// reach only result rows that are not stored.
//
// The matrix instructions are the 16 x 16 ones: for each product they read and write
// half as many accumulators as the 32 x 32 ones, and under this load the chip's
// clock goes by the power it draws.  Measured in turn on 8 x 4096 x 14336: forward
// 1.67 ms with 32 x 32 and 1.59 with 16 x 16, int8 0.93 and 0.90.  They take the
// column operand first, so that a lane holds 4 consecutive columns of one row and
// stores 16 bytes at a time.
#pragma once

#include <type_traits>

#include "ragged_common.h"

namespace mx {

constexpr int kTileN = 256;
constexpr int kStageK = 128;                     // contraction bytes of a stage
constexpr uint32_t kOut = 0xFFFFFF00u;           // a lane offset that no range check passes

typedef __attribute__((address_space(3))) const u32x4_t lds_u32x4_t;
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Buffer load to LDS: lane i writes LDS bytes [lds + 16 i, lds + 16 i + 16) (4 for
// the dword form) from rsrc's base + voff + soff, zeros where the range check
// fails.  Inline assembly so that the compiler's counters do not see it: the
// explicit waits below order the copies.  One wait state between the write of
// M0 and its use.
__device__ __forceinline__ void copy16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds),
               "v"(voff), "s"(rsrc), "s"(soff)
               : "m0", "memory");
}
__device__ __forceinline__ void copy4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds),
               "v"(voff), "s"(rsrc), "s"(soff)
               : "m0", "memory");
}

__device__ __forceinline__ i32x4 bounded(const void* base, int64_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint64_t n = bytes < 0 ? 0 : ((uint64_t)bytes < kSpan ? (uint64_t)bytes : kSpan);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xFFFFu));
  r[2] = __builtin_amdgcn_readfirstlane((int)(uint32_t)n);
  r[3] = 0x00020000;
  return r;
}

// The same range for the compiler's buffer loads and stores.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const uint64_t n = bytes < 0 ? 0 : ((uint64_t)bytes < kSpan ? (uint64_t)bytes : kSpan);
  const uint64_t u = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)b);
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)u, 0,
                                           __builtin_amdgcn_readfirstlane((int)(uint32_t)n), 0x00020000);
}

// The range check goes by dwords: one that the last value fills half of counts.
__device__ __forceinline__ int64_t whole_dwords(int64_t bytes) { return (bytes + 3) & ~(int64_t)3; }

// The same value in every lane, in scalar registers.
template <typename V>
__device__ __forceinline__ V uniform(V v) {
  const uint64_t b = (uint64_t)v;
  return (V)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32) |
             (uint32_t)__builtin_amdgcn_readfirstlane((int)b));
}

template <int N, int I = 0, typename F>
__device__ __forceinline__ void unroll(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    unroll<N, I + 1>(f);
  }
}

__device__ __forceinline__ uint32_t hide(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}
constexpr int vm_wait(int n) { return 0x0F70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xC07F;

// Prefix sums of the experts' row tiles and rows.
struct RaggedTable {
  int32_t tiles[kRaggedMaxGroups + 1];
  int32_t rows[kRaggedMaxGroups + 1];
};
template <int THREADS = 256>
__device__ __forceinline__ void build_ragged_table(const int64_t* m_splits, int G, int64_t R,
                                                   int tile, RaggedTable* t, int32_t* scan) {
  const int tid = threadIdx.x, wave = tid >> 6;
  constexpr int per = kRaggedMaxGroups / THREADS;
  const uint32_t most = (uint32_t)R;
  uint32_t rows[per], own = 0;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    rows[i] = g < G ? (uint32_t)split_rows(m_splits, g, R) : 0;
    own = min(own + rows[i], most);
  }
  const uint32_t upto = wave_sums<true>(own, most);
  if ((tid & 63) == 63) scan[wave] = (int32_t)upto;
  __syncthreads();
  // the rows of the lanes before (wave_shr: 1) and of the waves before
  uint32_t off[per + 1];
  off[0] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)upto, 0x138, 0xF, 0xF, false);
  for (int w = 0; w < wave; ++w) off[0] = min(off[0] + (uint32_t)scan[w], most);
  uint32_t tiles = 0;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    off[i + 1] = min(off[i] + rows[i], most);
    tiles += (off[i + 1] - off[i] + (uint32_t)tile - 1) / (uint32_t)tile;
  }
  const uint32_t tiles_upto = wave_sums<false>(tiles, 0);
  if ((tid & 63) == 63) scan[THREADS / 64 + wave] = (int32_t)tiles_upto;
  __syncthreads();
  uint32_t t0 = tiles_upto - tiles;
  for (int w = 0; w < wave; ++w) t0 += (uint32_t)scan[THREADS / 64 + w];
#pragma unroll
  for (int i = 0; i < per; ++i) {
    t->tiles[tid * per + i] = (int32_t)t0;
    t->rows[tid * per + i] = (int32_t)off[i];
    t0 += (off[i + 1] - off[i] + (uint32_t)tile - 1) / (uint32_t)tile;
  }
  if (tid == THREADS - 1) {
    t->tiles[kRaggedMaxGroups] = (int32_t)t0;
    t->rows[kRaggedMaxGroups] = (int32_t)off[per];
  }
  __syncthreads();
}

// Units of work of a launch.  Tiles that fill whole rounds of the grid are one unit
// each; where the rest fills less than half of a round, each of its tiles is
// split along the contraction into `parts` units, whose sums go to the
// workspace and are joined by ragged_join_kernel.
constexpr int kMinPart = 4;   // stages of a part
struct Units {
  uint32_t full, rem, parts;
};
__host__ __device__ __forceinline__ Units units_of(uint32_t ntiles, uint32_t grid, int64_t stages, bool ws) {
  Units u;
  u.full = ntiles / grid * grid;
  u.rem = ntiles - u.full;
  u.parts = 1;
  if (ws && u.rem > 0) {
    // A part's sums cost a write and a read of a tile each, for all `rem` tiles as
    // long as about rem / 7 stages of one: with p parts the round takes about
    // stages / p + p rem / 7.
    const uint32_t most = (uint32_t)(stages / kMinPart < 1 ? 1 : stages / kMinPart);
    const uint32_t best = (uint32_t)sqrtf(7.f * (float)stages / (float)u.rem);
    const uint32_t fit = grid / u.rem, p = fit < most ? fit : most;
    u.parts = p < best ? p : best;
    if (u.parts < 1) u.parts = 1;
  }
  return u;
}
// Row and column tile of tile `at`: 8 row tiles by all column tiles at a
// time, columns outermost.
__device__ __forceinline__ void tile_order(uint32_t at, uint32_t rtiles, uint32_t ctiles, int32_t* mt,
                                           int32_t* nt) {
  const uint32_t per = 8u * ctiles, grp = at / per, in = at % per;
  const uint32_t wide = min(8u, rtiles - 8u * grp);
  *mt = (int32_t)(8u * grp + in % wide);
  *nt = (int32_t)(in / wide);
}
// Stages of the contraction that the number of parts goes by: all of it, or the
// rows of an expert on average.
__device__ __forceinline__ int64_t part_stages(int layout, const RaggedArgs& p, int esize) {
  const int64_t con = layout == 2 ? p.R / p.G : p.con;
  return (con * esize + kStageK - 1) / kStageK;
}

// 4 consecutive columns of each of two blocks of 16 (words 0, 1 and 2, 3), in rows l % 16, to 8
// consecutive columns a lane, and back: its own inverse.
__device__ __forceinline__ u32x4_t swap_blocks(u32x4_t v) {
  const auto s0 = __builtin_amdgcn_permlane16_swap(v[0], v[2], false, false);
  const auto s1 = __builtin_amdgcn_permlane16_swap(v[1], v[3], false, false);
  return u32x4_t{(uint32_t)s0[0], (uint32_t)s1[0], (uint32_t)s0[1], (uint32_t)s1[1]};
}
// Two such runs of 16 rows by 32 columns (a: columns 0.., b: columns 32..) to two of 8 rows by 64, and
// back: whole 128-byte lines.  Lanes of rows 8.. trade their a for the b of the row 8 above.
__device__ __forceinline__ void whole_lines(u32x4_t& a, u32x4_t& b) {
  const bool low = (threadIdx.x & 8) == 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t give = low ? b[k] : a[k];
    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0x128, 0xF, 0xF, false);   // row_ror:8
    a[k] = low ? a[k] : got;
    b[k] = low ? got : b[k];
  }
}
// Row (of 16) and column (of 64) where lane ln's 8 columns of a, after that, belong; b: 8 rows on.
__device__ __forceinline__ int line_row(int ln) { return ln & 7; }
__device__ __forceinline__ int line_col(int ln) {
  return 32 * ((ln >> 3) & 1) + 16 * ((ln >> 4) & 1) + 8 * (ln >> 5);
}

// A wave's 32 FA rows by 64 gate columns (accumulators 0..3 of a row block) and their up
// columns (4..7): the activation and, KEEP, both projections, in whole lines.
template <typename O, int FA, bool KEEP, typename Acc>
__device__ __forceinline__ void store_gated(const RaggedArgs& p, Acc (&acc)[2 * FA][8], int32_t m0, int32_t n0,
                                            int32_t rows, int wm, int wn, int ln) {
  const int64_t F = p.N / 2;
  const uint32_t ec = (uint32_t)(p.ldc * 2), eh = (uint32_t)(F * 4);
  const int right = (int)min((int64_t)(kTileN / 2), F - n0);
  const auto out = make_rsrc((uint16_t*)p.c + (int64_t)m0 * p.ldc + n0, (int64_t)(rows - 1) * ec + (F - n0) * 2);
  const auto gate = make_rsrc((uint16_t*)p.h + (int64_t)m0 * 2 * F + n0, (int64_t)(rows - 1) * eh + (F - n0) * 2);
  const auto up = make_rsrc((uint16_t*)p.h + (int64_t)m0 * 2 * F + F + n0, (int64_t)(rows - 1) * eh + (F - n0) * 2);
  const int n = wn * 64 + line_col(ln);
#pragma unroll
  for (int i = 0; i < 2 * FA; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) asm volatile("" : "+a"(acc[i][j]));
    const int m = wm * 32 * FA + 16 * i + line_row(ln);
    const bool in0 = (n < right) & (m < rows), in1 = (n < right) & (m + 8 < rows);
    auto put = [&](__amdgpu_buffer_rsrc_t to, uint32_t pitch, auto value) {
      u32x4_t w[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[b][k] = (uint32_t)O::cvt(value(2 * b + (k >> 1), 2 * (k & 1))) |
                    ((uint32_t)O::cvt(value(2 * b + (k >> 1), 2 * (k & 1) + 1)) << 16);
        w[b] = swap_blocks(w[b]);
      }
      whole_lines(w[0], w[1]);
      const uint32_t at = (uint32_t)m * pitch + (uint32_t)n * 2u;
      __builtin_amdgcn_raw_buffer_store_b128(w[0], to, in0 ? at : kOut, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(w[1], to, in1 ? at + 8 * pitch : kOut, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    put(out, ec, [&](int b, int e) { return gated(acc[i][b][e], acc[i][b + 4][e]); });
    if constexpr (KEEP) {
      put(gate, eh, [&](int b, int e) { return acc[i][b][e]; });
      put(up, eh, [&](int b, int e) { return acc[i][b + 4][e]; });
    }
  }
}

// A wave's 32 FA rows by 128 columns of da: both projections are read (16 rows ahead of their
// use), their gradients and the activation written, in whole lines.
template <typename T, typename O, int FA, typename Acc>
__device__ __forceinline__ void store_gated_bwd(const RaggedArgs& p, Acc (&acc)[2 * FA][8], int32_t m0,
                                                int32_t n0, int32_t rows, int wm, int wn, int ln) {
  const int64_t F = p.K;
  const uint32_t eh = (uint32_t)(F * 4), ea = (uint32_t)(F * 2);
  const int right = (int)min((int64_t)kTileN, F - n0);
  const int64_t at0 = (int64_t)m0 * 2 * F + n0, room = (int64_t)(rows - 1) * eh + (F - n0) * 2;
  const auto hg = make_rsrc((const uint16_t*)p.h + at0, room), hu = make_rsrc((const uint16_t*)p.h + at0 + F, room);
  const auto dg = make_rsrc((uint16_t*)p.c + at0, room), du = make_rsrc((uint16_t*)p.c + at0 + F, room);
  const auto act = make_rsrc((uint16_t*)p.act + (int64_t)m0 * F + n0,
                             p.act == nullptr ? 0 : (int64_t)(rows - 1) * ea + (F - n0) * 2);
  // columns 64 c + .., rows 16 i + 8 b + ..
  auto col = [&](int c) { return wn * 128 + 64 * c + line_col(ln); };
  auto row = [&](int i, int b) { return wm * 32 * FA + 16 * i + 8 * b + line_row(ln); };
  auto place = [&](int i, int b, int c, uint32_t pitch) {
    return ((col(c) < right) & (row(i, b) < rows)) ? (uint32_t)row(i, b) * pitch + (uint32_t)col(c) * 2u : kOut;
  };
  u32x4_t g[2][4], u[2][4];
  auto load = [&](int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t at = place(i, q & 1, q >> 1, eh);
      g[i & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(hg, at, 0, 0);
      u[i & 1][q] = __builtin_amdgcn_raw_buffer_load_b128(hu, at, 0, 0);
    }
  };
  load(0);
#pragma unroll
  for (int i = 0; i < 2 * FA; ++i) {
    if (i + 1 < 2 * FA) load(i + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      u32x4_t vg[2] = {g[i & 1][2 * c], g[i & 1][2 * c + 1]}, vu[2] = {u[i & 1][2 * c], u[i & 1][2 * c + 1]};
      whole_lines(vg[0], vg[1]);
      whole_lines(vu[0], vu[1]);
      u32x4_t og[2], ou[2], oa[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int j = 4 * c + 2 * b;
        asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
        vg[b] = swap_blocks(vg[b]);
        vu[b] = swap_blocks(vu[b]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          GatedGrad r[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            r[e] = gated_grad(acc[i][j + (k >> 1)][2 * (k & 1) + e], widen<T>((uint16_t)(vg[b][k] >> (16 * e))),
                              widen<T>((uint16_t)(vu[b][k] >> (16 * e))));
          og[b][k] = (uint32_t)O::cvt(r[0].gate) | ((uint32_t)O::cvt(r[1].gate) << 16);
          ou[b][k] = (uint32_t)O::cvt(r[0].up) | ((uint32_t)O::cvt(r[1].up) << 16);
          oa[b][k] = (uint32_t)O::cvt(r[0].act) | ((uint32_t)O::cvt(r[1].act) << 16);
        }
        og[b] = swap_blocks(og[b]);
        ou[b] = swap_blocks(ou[b]);
        oa[b] = swap_blocks(oa[b]);
      }
      whole_lines(og[0], og[1]);
      whole_lines(ou[0], ou[1]);
      whole_lines(oa[0], oa[1]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t at = place(i, b, c, eh);
        __builtin_amdgcn_raw_buffer_store_b128(og[b], dg, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(ou[b], du, at, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(oa[b], act, place(i, b, c, ea), 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Column tiles of a launch; a gated tile holds 128 gate columns and their 128 up columns.
template <int LAYOUT, int EPI>
__host__ __device__ __forceinline__ uint32_t column_tiles(const RaggedArgs& p) {
  if (EPI == kGated || EPI == kGatedKeep) return (uint32_t)((p.N / 2 + kTileN / 2 - 1) / (kTileN / 2));
  return (uint32_t)(((LAYOUT == 0 ? p.N : p.K) + kTileN - 1) / kTileN);
}

template <typename T, typename O, int LAYOUT, int FA, bool GATHER, int EPI = kPlain>
__global__ __launch_bounds__(256, 1) void ragged_tile_kernel(RaggedArgs p) {
  typedef typename T::elem E;
  constexpr bool kIsGated = EPI == kGated || EPI == kGatedKeep;
  static_assert(EPI == kPlain || (sizeof(typename O::elem) == 2 && sizeof(E) == 2), "");
  static_assert(kIsGated ? LAYOUT == 0 : (EPI != kGatedBwd || LAYOUT == 1), "");
  constexpr bool kInt8 = sizeof(E) == 1;
  constexpr bool kColA = LAYOUT == 2, kColB = LAYOUT != 0;   // contraction over rows
  constexpr int kTileM = 64 * FA;
  constexpr int kOffB = kTileM * kStageK;
  constexpr int kStage = kOffB + kTileN * kStageK;
  constexpr int kPartsA = 2 * FA, kParts = kPartsA + 8;      // copies of a wave for a stage
  constexpr int kRowsF = 2 * FA;                             // fragments of 16 rows; 8 of 16 columns
  constexpr int kMfma = 8 * kRowsF;                          // of a half stage: 64 contraction bytes
  constexpr int kReads = kRowsF + 8;
  constexpr int kEarly = 3 * kParts / 8;                     // copies in the first half
  // (at least: a wait that counts fewer than there are waits for some of them)
  constexpr int kStores = EPI == kGated ? 4 * FA : EPI == kGatedKeep ? 12 * FA :
                          sizeof(typename O::elem) == 4 || EPI == kGatedBwd ? 16 * FA : 8 * FA;
  static_assert(!kColA || FA == 4, "");
  // row indexes, per wave: TN the 64 of each of 8 stages, NT the wave's rows of
  // the next tile
  constexpr int kRing = !GATHER ? 16 : (kColA ? 4 * 8 * 256 : 4 * 256);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  __shared__ __attribute__((aligned(16))) uint8_t ring[kRing];
  // int8: scales of the rows and columns of two tiles
  __shared__ __attribute__((aligned(16))) float scales[2][2][kInt8 ? 256 : 4];
  __shared__ RaggedTable table;
  // What only the start and the end of a tile need is kept in LDS, not in
  // scalar registers: they would spill.
  __shared__ RaggedArgs args;
  __shared__ struct {
    uint32_t full, rem, parts, rtiles, ctiles, band;
  } plan;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  build_ragged_table(p.m_splits, p.G, p.R, kTileM, &table, (int32_t*)smem);

  uint32_t nunits;
  {
    const uint32_t ctiles = column_tiles<LAYOUT, EPI>(p);
    const uint32_t band = (uint32_t)((p.N + kTileM - 1) / kTileM);       // TN: row tiles of an expert
    const uint32_t rtiles = kColA ? (uint32_t)p.G * band : (uint32_t)table.tiles[kRaggedMaxGroups];
    // tiles: below 2^31 (checked by the caller)
    const Units u =
        units_of(rtiles * ctiles, gridDim.x, part_stages(LAYOUT, p, sizeof(E)), p.ws != nullptr);
    nunits = (uint32_t)__builtin_amdgcn_readfirstlane((int)(u.full + u.rem * u.parts));
    if (tid == 0) {
      plan.full = u.full;
      plan.rem = u.rem;
      plan.parts = u.parts;
      plan.rtiles = rtiles;
      plan.ctiles = ctiles;
      plan.band = band;
      copy_args(args, p);
    }
  }
  __syncthreads();

  // Order of the tiles (tile_order); of each full round of the grid, XCD x
  // (workgroups x, x + 8, ...) takes consecutive ones, so that its 32 workgroups
  // share 8 row and 4 column panels in its L2.
  auto place = [&](uint32_t i) -> uint32_t {
    const uint32_t n = gridDim.x;
    if (n % 8 != 0 || i >= plan.full) return i;   // a last round that is not full as it comes
    const uint32_t b = i % n;
    return i - b + (b & 7) * (n / 8) + (b >> 3);
  };

  struct Tile {
    i32x4 sa, sb;        // bounded operands at contraction 0
    int64_t na, nb;      // contraction over rows: bytes left of each operand
    const uint8_t *pa, *pb;
    int32_t ns;          // stages
    int32_t len;         // contraction length (TN)
    int32_t lo;          // first row of the expert (TN), of the tile (NT, NN)
    int32_t rows;        // rows to store
    int32_t n0;          // first column
    int32_t m0;          // first result row
    int32_t g;
    int32_t split;       // a part: its number among the units that store partial sums, or -1
    int32_t last;        // its last stage is the contraction's
  };
  // row strides in bytes: 256 of them lie within 32 bits
  const uint32_t ea = (uint32_t)(p.lda * (int64_t)sizeof(E)), eb = (uint32_t)(p.ldb * (int64_t)sizeof(E));
  auto describe = [&](uint32_t i) {
    Tile t;
    const RaggedArgs& p = args;
    const uint32_t ctiles = plan.ctiles, rtiles = plan.rtiles, band = plan.band;
    const uint32_t ufull = plan.full, urem = plan.rem, uparts = plan.parts;
    const int64_t con = p.con;   // NT, NN
    const int64_t la = ea, lb = eb;
    const bool part = i >= ufull && uparts > 1;
    const uint32_t v = i - ufull;
    const uint32_t at = part ? ufull + v % urem : place(i);
    int32_t mt, nt;
    t.split = part ? (int32_t)v : -1;
    if (kColA) {
      const uint32_t all = band * ctiles;
      t.g = __builtin_amdgcn_readfirstlane((int32_t)(at / all));
      tile_order(at % all, band, ctiles, &mt, &nt);
      t.lo = table.rows[t.g];
      t.len = table.rows[t.g + 1] - t.lo;
      t.m0 = mt * kTileM;
      t.rows = (int32_t)min((int64_t)kTileM, p.N - t.m0);
      t.n0 = nt * kTileN;
      t.ns = (int32_t)(((int64_t)t.len * sizeof(E) + kStageK - 1) / kStageK);
      // columns m0.. of dY and n0.. of X, the expert's rows
      t.pa = (const uint8_t*)p.a + (int64_t)t.lo * la + (int64_t)t.m0 * sizeof(E);
      t.na = t.len == 0 ? 0 : (int64_t)(t.len - 1) * la + whole_dwords((p.N - t.m0) * (int64_t)sizeof(E));
      if (GATHER) {
        t.pb = (const uint8_t*)p.b + (int64_t)t.n0 * sizeof(E);
        t.nb = p.S == 0 ? 0 : (p.S - 1) * lb + whole_dwords((p.K - t.n0) * (int64_t)sizeof(E));
      } else {
        t.pb = (const uint8_t*)p.b + (int64_t)t.lo * lb + (int64_t)t.n0 * sizeof(E);
        t.nb = t.len == 0 ? 0 : (int64_t)(t.len - 1) * lb + whole_dwords((p.K - t.n0) * (int64_t)sizeof(E));
      }
    } else {
      tile_order(at, rtiles, ctiles, &mt, &nt);
      int lo = 0, hi = p.G;   // tiles[lo] <= mt < tiles[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.tiles[mid] <= mt) lo = mid; else hi = mid;
      }
      t.g = lo;
      t.lo = table.rows[lo] + (mt - table.tiles[lo]) * kTileM;
      t.m0 = t.lo;
      t.rows = min(kTileM, table.rows[lo + 1] - t.lo);
      t.n0 = nt * (kIsGated ? kTileN / 2 : kTileN);
      t.len = 0;
      t.ns = (int32_t)((con * (int64_t)sizeof(E) + kStageK - 1) / kStageK);
      if (GATHER) {
        t.pa = (const uint8_t*)p.a;
        t.na = p.S == 0 ? 0 : (p.S - 1) * la + con * (int64_t)sizeof(E);
      } else {
        t.pa = (const uint8_t*)p.a + (int64_t)t.lo * la;
        t.na = (p.R - 1 - t.lo) * la + con * (int64_t)sizeof(E);
      }
      const uint8_t* w = (const uint8_t*)p.b + (int64_t)t.g * p.N * lb;
      if (LAYOUT == 0) {
        t.pb = w + (int64_t)t.n0 * lb;
        t.nb = (p.N - 1 - t.n0) * lb + con * (int64_t)sizeof(E);
      } else {
        t.pb = w + (int64_t)t.n0 * sizeof(E);
        t.nb = (p.N - 1) * lb + whole_dwords((p.K - t.n0) * (int64_t)sizeof(E));
      }
    }
    t.last = 1;
    if (part) {   // stages [s0, s1)
      const int32_t which = (int32_t)(v / urem), n = (int32_t)uparts;
      const int32_t each = t.ns / n, more = t.ns % n;   // the first `more` parts have one stage more
      const int32_t s0 = which * each + min(which, more), s1 = s0 + each + (which < more ? 1 : 0);
      t.last = s1 == t.ns;
      t.ns = s1 - s0;
      const int64_t da = kColA ? (int64_t)s0 * 64 * la : (int64_t)s0 * kStageK;
      const int64_t db = kColB ? (int64_t)s0 * 64 * lb : (int64_t)s0 * kStageK;
      t.pa += da;
      t.na -= da;
      if (!(GATHER && kColA)) {   // gathered rows move with their indexes
        t.pb += db;
        t.nb -= db;
      }
      if (kColA) {
        t.lo += s0 * 64;
        t.len -= s0 * 64;
      }
    }
    t.sa = bounded(t.pa, t.na);
    t.sb = bounded(t.pb, t.nb);
    if (kColA) t.pa = uniform(t.pa), t.na = uniform(t.na);
    if (kColB) t.pb = uniform(t.pb), t.nb = uniform(t.nb);
    t.split = __builtin_amdgcn_readfirstlane(t.split);
    t.last = __builtin_amdgcn_readfirstlane(t.last);
    t.ns = __builtin_amdgcn_readfirstlane(t.ns);
    t.len = __builtin_amdgcn_readfirstlane(t.len);
    t.lo = __builtin_amdgcn_readfirstlane(t.lo);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
    t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    return t;
  };

  // Lane offsets of the copies.  Contiguous: part j copies rows 8 (parts wave + j)
  // + lane / 8, chunk position lane % 8.  Over rows: part j copies contraction
  // rows 16 wave + 2 j + lane / 32, chunk position lane % 32.
  auto chunk_k = [&](int j) { return (uint32_t)((lane & 7) ^ (4 * (j & 1) + (lane >> 4))) * 16; };
  auto chunk_c = [&](int j) {
    const int r = 2 * (j & 1) + (lane >> 5);
    const int x = ((r & 1) * 4 + (r >> 1) * 10) ^ (2 * (j >> 2));   // row 2 j + .. of 16
    return (uint32_t)((lane & 31) ^ x) * 16;
  };
  uint32_t va[kPartsA], vb[8];
#pragma unroll
  for (int j = 0; j < kPartsA; ++j)
    va[j] = kColA ? (uint32_t)((16 * wave + 2 * j + (lane >> 5)) * ea) + chunk_c(j)
                  : (uint32_t)((8 * (kPartsA * wave + j) + (lane >> 3)) * ea) + chunk_k(j);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    vb[j] = kColB ? (uint32_t)((16 * wave + 2 * j + (lane >> 5)) * eb) + chunk_c(j)
                  : (uint32_t)((kIsGated ? 64 * (wave >> 1) + 8 * j : 8 * (8 * wave + j)) + (lane >> 3)) * eb +
                        chunk_k(j);
  // gated: rows 64 (2 c + u) .. of the stage are gate (u = 0) and up (u = 1) rows of wave column c
  if constexpr (kIsGated) {
    const uint32_t up = (wave & 1) ? (uint32_t)(p.N / 2) * eb : 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) vb[j] += up;
  }
  // contiguous contraction: lanes past its end in the last stage
  const uint32_t last_bytes =
      (uint32_t)((p.con * (int64_t)sizeof(E) - 1) % kStageK) + 1;
  uint32_t past[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) past[j] = !kColA && chunk_k(j) >= last_bytes ? kOut : 0u;

  // Address of the first fragment of each half of a stage.  Contiguous: fragment i
  // 16 rows (2048 bytes) on.  Over rows: columns 16 i on, address bits 5..7 changed
  // by 32 i; the halves 32 contraction rows apart.
  uint32_t ra[2], rb[2];
  {
    const int xr = (((lane >> 2) & 1) * 4 + ((lane >> 3) & 1) * 10) ^ (2 * ((lane >> 4) & 1));
    auto col = [&](int first, int h) {
      return (uint32_t)((32 * h + 8 * (lane >> 4) + ((lane >> 2) & 3)) * 512 +
                        (((first >> 3) + ((lane >> 1) & 1)) ^ xr) * 16 + (lane & 1) * 8);
    };
    auto row = [&](int first, int h) {
      return (uint32_t)((first + (lane & 15)) * kStageK +
                        (((4 * h + (lane >> 4)) ^ ((lane >> 1) & 7)) * 16));
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      ra[h] = lds0 + (kColA ? col(wm * 32 * FA, h) : row(wm * 32 * FA, h));
      rb[h] = lds0 + kOffB + (kColB ? col(wn * 128, h) : row(wn * 128, h));
    }
  }
  auto transposed = [](uint32_t at) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 2048));
    const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
    return u32x4_t{a[0], a[1], b[0], b[1]};
  };

  typename T::acc16 acc[kRowsF][8];
  u32x4_t fa[2][kRowsF], fb[2][8];

  Tile t;              // the tile whose operands are copied
  int slot0 = 0;       // slot of the computed tile's stage 0
  int ring_at = 0;     // place of its stage 0 in the ring of row indexes

  // Row indexes of the gathered operand go to LDS beside the stages: no load
  // of theirs is waited for.
  const uint32_t ring0 = (uint32_t)(uintptr_t)ring + (uint32_t)(wave * (kColA ? 2048 : 256));
  auto copy_index = [&](const Tile& n, int st, int at) {   // TN: stage st of n
    const i32x4 si = bounded(p.row_index + n.lo + 64 * st, ((int64_t)n.len - 64 * st) * 4);
    copy4(si, (uint32_t)(lane * 4), 0u, ring0 + (uint32_t)(at & 7) * 256u);
  };
  auto copy_rows = [&](const Tile& n) {   // NT: the wave's rows of n
    const i32x4 si = bounded(p.row_index + n.lo, (int64_t)n.rows * 4);
    copy4(si, (uint32_t)(lane * 4 + wave * 8 * kPartsA * 4), 0u, ring0);
  };
  auto take_rows = [&](const Tile& n) {   // NT: lane offsets from them
#pragma unroll
    for (int j = 0; j < kPartsA; ++j) {
      const uint32_t r = (uint32_t)(8 * j + (lane >> 3));
      const uint32_t row = *(__attribute__((address_space(3))) const uint32_t*)(ring0 + r * 4);
      const bool ok = ((int)(8 * kPartsA * wave + r) < n.rows) & (row < (uint32_t)p.S);
      va[j] = (row * ea + chunk_k(j)) | (ok ? 0u : kOut);
    }
  };

  // int8: scales of tile n's rows (this wave's and on, as copy_rows
  // brought their indexes) and columns (64) to LDS, with the copies; zeros outside.
  int side = 0;   // place of the computed tile's
  auto copy_scales = [&](const Tile& n, int at) {
    const RaggedArgs& p = args;
    // (with fewer than 64 rows a wave, waves write rows of the next one too, the
    // same values)
    const uint32_t to = (uint32_t)(uintptr_t)scales + (uint32_t)(at * 2048);
    const uint32_t r = (uint32_t)(8 * kPartsA * wave + lane),
                   c = (uint32_t)(64 * wave + lane);
    uint32_t row = r;
    if (GATHER) row = *(__attribute__((address_space(3))) const uint32_t*)(ring0 + (uint32_t)lane * 4);
    const i32x4 rs = GATHER ? bounded(p.sa, p.S * 4) : bounded(p.sa + n.lo, (int64_t)n.rows * 4);
    const bool ok = ((int)r < n.rows) & (!GATHER | (row < (uint32_t)p.S));
    const i32x4 cs = bounded(p.sb + (int64_t)n.g * p.N + n.n0, (p.N - n.n0) * 4);
    copy4(rs, (row * 4u) | (ok ? 0u : kOut), 0u,
          __builtin_amdgcn_readfirstlane(to + (uint32_t)(wave * kPartsA * 32)));
    copy4(cs, c * 4u, 0u, __builtin_amdgcn_readfirstlane(to + 1024u + (uint32_t)(wave * 256)));
  };

  struct Stage {
    int st, len, at;
    uint32_t soff, lds, kill[2];
    i32x4 sa, sb;
  };
  // Stage st of the copied tile; v: its number counted from the computed tile's
  // stage 0.
  auto stage = [&](int st, int v) {
    const Tile& n = t;
    // A stage past the last copies zeros: every lane out of range.  The range
    // check takes soff from the range, so soff must not pass it: it is 0 there,
    // and within a row otherwise.
    const bool none = st >= n.ns;
    Stage s;
    s.st = st;
    s.len = none ? 0 : n.len;
    s.at = ring_at + v;
    s.lds = lds0 + (uint32_t)(((slot0 + v) & 1) * kStage);
    s.soff = none ? 0u : (uint32_t)st * kStageK;
#pragma unroll
    for (int j = 0; j < 2; ++j) s.kill[j] = none ? kOut : (st == n.ns - 1 && n.last ? past[j] : 0u);
    s.sa = n.sa;
    s.sb = n.sb;
    if (kColA)
      s.sa = bounded(n.pa + (uint64_t)(64u * (uint32_t)st) * ea,
                     none ? 0 : n.na - (int64_t)((uint64_t)(64u * (uint32_t)st) * ea));
    if (kColB && !(GATHER && kColA))
      s.sb = bounded(n.pb + (uint64_t)(64u * (uint32_t)st) * eb,
                     none ? 0 : n.nb - (int64_t)((uint64_t)(64u * (uint32_t)st) * eb));
    // the same in every lane, which the compiler does not always see
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s.sa[i] = __builtin_amdgcn_readfirstlane(s.sa[i]);
      s.sb[i] = __builtin_amdgcn_readfirstlane(s.sb[i]);
    }
    s.lds = __builtin_amdgcn_readfirstlane(s.lds);
    s.soff = __builtin_amdgcn_readfirstlane(s.soff);
    return s;
  };
  // TN: the row indexes of this lane's contraction rows in a stage, from the
  // ring: read together ahead of the stage's copies, so that no copy waits.
  uint32_t rows_at[8];
  auto read_index = [&](const Stage& s) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      rows_at[j] = *(__attribute__((address_space(3))) const uint32_t*)(
          ring0 + (uint32_t)(s.at & 7) * 256u + (uint32_t)(16 * wave + 2 * j + (lane >> 5)) * 4u);
  };
  // Copy c of a stage (A and B parts in turn, then what is left of B): its addresses first, behind a matrix instruction of their
  // own, then the copy behind the next (all five instructions behind one are more
  // than its 16 cycles hide: 8 x 4096 x 14336 forward 1.59 ms, so 1.55).
  struct Part {
    uint32_t off, at;
  } part[kParts];
  auto prepare = [&](const Stage& s, auto C) {
    constexpr int c = decltype(C)::value;
    constexpr bool isA = c < 2 * kPartsA && c % 2 == 0;
    constexpr int j = isA ? c / 2 : (c < 2 * kPartsA ? c / 2 : c - kPartsA);
    uint32_t off;
    if constexpr (isA) {
      off = kColA ? va[j] : (va[j] | s.kill[j & 1]);
    } else if constexpr (GATHER && kColA) {
      const int r = 16 * wave + 2 * j + (lane >> 5);
      const bool ok = (s.st * 64 + r < s.len) & (rows_at[j] < (uint32_t)p.S);
      off = (rows_at[j] * eb + chunk_c(j)) | (ok ? 0u : kOut);
    } else {
      off = kColB ? vb[j] : (vb[j] | s.kill[j & 1]);
    }
    uint32_t at = s.lds + (isA ? (uint32_t)(wave * kPartsA * 1024 + j * 1024)
                               : kOffB + (uint32_t)(wave * 8192 + j * 1024));
    asm volatile("" : "+s"(at));
    part[c] = {hide(off), at};
  };
  auto copy = [&](const Stage& s, auto C) {
    constexpr int c = decltype(C)::value;
    constexpr bool isA = c < 2 * kPartsA && c % 2 == 0;
    if constexpr (isA) copy16(s.sa, part[c].off, kColA ? 0u : s.soff, part[c].at);
    else copy16(s.sb, part[c].off, kColB ? 0u : s.soff, part[c].at);
  };
  // fragment r (0 .. kReads) of half h of a stage into register set h
  struct Base {
    uint32_t a, b;
  };
  auto base = [&](int slot, auto H) {
    constexpr int h = decltype(H)::value;
    const uint32_t off = (uint32_t)slot * kStage;
    return Base{hide(ra[h] + off), hide(rb[h] + off)};
  };
  auto read = [&](const Base& x, auto H, auto R) {
    constexpr int h = decltype(H)::value, r = decltype(R)::value;
    constexpr bool isA = r < 2 * kRowsF && r % 2 == 0;
    constexpr int i = r < 2 * kRowsF ? r / 2 : r - kRowsF;
    if constexpr (isA) {
      if constexpr (kColA) fa[h][i] = transposed(x.a ^ (uint32_t)(32 * i));
      else fa[h][i] = *(lds_u32x4_t*)(x.a + i * 2048);
    } else {
      if constexpr (kColB) fb[h][i] = transposed(x.b ^ (uint32_t)(32 * i));
      else fb[h][i] = *(lds_u32x4_t*)(x.b + i * 2048);
    }
  };
  auto mma = [&](auto H, auto Q) {
    constexpr int h = decltype(H)::value, q = decltype(Q)::value;
    constexpr int i = q / 8, j = q % 8;
    acc[i][j] = T::mma16(fb[h][j], fa[h][i], acc[i][j]);
    asm volatile("" : "+a"(acc[i][j]));
    __builtin_amdgcn_sched_barrier(0);
  };
  using H0 = std::integral_constant<int, 0>;
  using H1 = std::integral_constant<int, 1>;

  // A tile from the start: its first two stages (and the indexes before them),
  // waited for, and its first fragments.
  auto start = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (GATHER && kColA) {
#pragma unroll
      for (int st = 0; st < 4; ++st) copy_index(t, st, ring_at + st);
      __builtin_amdgcn_s_waitcnt(vm_wait(0));
    }
    if constexpr (GATHER && !kColA) {
      copy_rows(t);
      __builtin_amdgcn_s_waitcnt(vm_wait(0));
      take_rows(t);
    }
    if constexpr (kInt8) copy_scales(t, side);
    __builtin_amdgcn_sched_barrier(0);
    for (int st = 0; st < 2; ++st) {   // a stage past the last copies zeros
      const Stage s = stage(st, st);
      if constexpr (GATHER && kColA) read_index(s);
      unroll<kParts>([&](auto C) {
        prepare(s, C);
        copy(s, C);
      });
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(vm_wait(0));
    __syncthreads();
    const Base x = base(slot0 & 1, H0{});
    unroll<kReads>([&](auto R) { read(x, H0{}, R); });
  };

  // First half of a stage: matrix instructions on set 0; the second half's
  // fragments are read in their first half, then the slot is free (each wave
  // has waited for its reads) and the copies of the stage two ahead begin.
  auto first_half = [&](int st, const Stage& cp) {
    const Base x = base((slot0 + st) & 1, H1{});
    if constexpr (GATHER && kColA) read_index(cp);
    __builtin_amdgcn_sched_barrier(0);
    unroll<kMfma>([&](auto Q) {
      constexpr int q = decltype(Q)::value, m = kMfma / 2;
      mma(H0{}, Q);
      unroll<kReads>([&](auto R) {
        if constexpr (decltype(R)::value * m / kReads == q) read(x, H1{}, R);
      });
      if constexpr (q == m) {
        __builtin_amdgcn_s_waitcnt(kLgkmWait0);
        __syncthreads();
      }
      unroll<kEarly>([&](auto C) {
        constexpr int at = m + 1 + decltype(C)::value * (m - 1) / kEarly;
        if constexpr (at - 1 == q) prepare(cp, C);
        if constexpr (at == q) copy(cp, C);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // Second half: the next stage has landed (only the copies just begun, and the
  // stores of the tile before, may be in flight), its first fragments are read,
  // the rest of the copies go out.
  auto second_half = [&](int st, const Stage& cp, bool stores) {
    if (stores) __builtin_amdgcn_s_waitcnt(vm_wait(kStores + kEarly < 63 ? kStores + kEarly : 63));
    else __builtin_amdgcn_s_waitcnt(vm_wait(kEarly));
    __syncthreads();
    const Base x = base((slot0 + st + 1) & 1, H0{});
    __builtin_amdgcn_sched_barrier(0);
    unroll<kMfma>([&](auto Q) {
      constexpr int q = decltype(Q)::value, left = kParts - kEarly;
      mma(H1{}, Q);
      unroll<kReads>([&](auto R) {
        if constexpr (decltype(R)::value * kMfma / kReads == q) read(x, H0{}, R);
      });
      unroll<left>([&](auto C) {
        constexpr int at = decltype(C)::value * (kMfma / 4) / left * 4 + 2;   // between two reads
        using Part_ = std::integral_constant<int, decltype(C)::value + kEarly>;
        if constexpr (at - 1 == q) prepare(cp, Part_{});
        if constexpr (at == q) copy(cp, Part_{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  uint32_t tile = blockIdx.x;
  if (tile >= nunits) return;
  t = describe(tile);
  start();
  bool chained = false;   // the previous tile's last stages carried this one's first two

  for (;;) {
    const int ns = t.ns;
    // what the stores need of this tile
    const int32_t rows = t.rows, n0 = t.n0, m0 = t.m0, g = t.g, split = t.split;
    const uint32_t next = tile + gridDim.x;
    // Chain: the last two stages of a tile carry the copies of the next tile's
    // first two and read its first fragments, as if the contraction went on.
    // Otherwise they copy nothing (an empty range) and the next tile starts
    // anew.  The indexes of gathered rows go ahead, from four stages before
    // the end; int8's scales take the place that the previous tile's had, so a
    // barrier of this tile lies between.
    bool chain = next < nunits && ns >= (GATHER ? 4 : (kInt8 ? 3 : 2));
#pragma unroll
    for (int i = 0; i < kRowsF; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        acc[i][j] = typename T::acc16{0, 0, 0, 0};
        asm volatile("" : "+a"(acc[i][j]));
      }
    for (int st = 0; st < ns; ++st) {
      int from = st + 2;
      if (st >= ns - 2) {
        from -= ns;
        if (st == ns - 2 || ns == 1) {
          if (chain) {
            t = describe(next);
            chain = t.ns >= 2;
            if constexpr (GATHER && !kColA) take_rows(t);
            if constexpr (kInt8) copy_scales(t, side ^ 1);
          }
          if (!chain) t.ns = 0;
        }
      }
      const Stage cp = stage(from, st + 2);
      first_half(st, cp);
      second_half(st, cp, chained && st == 0);
      if constexpr (GATHER) {
        if constexpr (kColA) {
          if (st + 4 < ns) copy_index(t, st + 4, ring_at + st + 4);
        }
        if (chain && st == ns - 4) {
          const Tile n = describe(next);
          if constexpr (kColA) {
#pragma unroll
            for (int s = 0; s < 4; ++s) copy_index(n, s, ring_at + ns + s);
          } else {
            copy_rows(n);
          }
        }
      }
    }

    // the lane number anew for each tile: addresses formed from it would otherwise
    // be kept, and spilled, through the whole loop
    const int ln = (int)hide((uint32_t)lane);
    const RaggedArgs& p = args;
    if (split >= 0) {
      // a part (the last unit of its workgroup): the accumulators as they lie
      const auto ws = make_rsrc((const uint8_t*)p.ws + (int64_t)split * (kTileM * kTileN * 4),
                                kTileM * kTileN * 4);
#pragma unroll
      for (int i = 0; i < kRowsF; ++i) {
        if (wm * 32 * FA + 16 * i >= rows) continue;   // not read by the join either
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // (values of this branch's own: moved ahead of the branch, all 256
          // accumulators would be spilled)
          asm volatile("" : "+a"(acc[i][j]));
          __builtin_amdgcn_raw_buffer_store_b128(
              __builtin_bit_cast(u32x4_t, acc[i][j]), ws,
              (uint32_t)(((wave * kRowsF + i) * 8 + j) * 1024 + ln * 16), 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
    float srow[kRowsF];
    if constexpr (kInt8) {
#pragma unroll
      for (int i = 0; i < kRowsF; ++i) srow[i] = scales[side][0][wm * 32 * FA + 16 * i + (ln & 15)];
    }

    // Stores, bounded like the loads: lanes past the tile's rows or columns get an
    // offset that stores nothing, so that every tile issues the same stores
    // (the waits count on it).
    typedef typename O::elem OE;
    if constexpr (kIsGated) {
      store_gated<O, FA, EPI == kGatedKeep>(p, acc, m0, n0, rows, wm, wn, ln);
    } else if constexpr (EPI == kGatedBwd) {
      store_gated_bwd<T, O, FA>(p, acc, m0, n0, rows, wm, wn, ln);
    } else {
    OE* c = (OE*)p.c + ((kColA ? (int64_t)g * p.N : 0) + m0) * p.ldc + n0;
    const uint32_t ec = (uint32_t)(p.ldc * sizeof(OE));
    const int64_t room = (int64_t)(rows - 1) * ec + (p.ccols - n0) * (int64_t)sizeof(OE);
    const auto out = make_rsrc(c, room);
    const int right = (int)min((int64_t)kTileN, p.ccols - n0);   // columns to store
    auto value = [&](int i, int j, int e) {
      if constexpr (kInt8)
        return scaled<O>(acc[i][j][e], srow[i], scales[side][1][wn * 128 + 16 * j + 4 * (ln >> 4) + e]);
      else
        return acc[i][j][e];
    };
    // Accumulator e of block (i, j) in lane l: row 16 i + l % 16, column
    // 16 j + 4 (l / 16) + e.
#pragma unroll
    for (int i = 0; i < kRowsF; ++i) {
      const int m = wm * 32 * FA + 16 * i + (ln & 15);
      const uint32_t roff = m < rows ? (uint32_t)m * ec : kOut;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        asm volatile("" : "+a"(acc[i][j]), "+a"(acc[i][j + 1]));
        if constexpr (sizeof(OE) == 4) {
#pragma unroll
          for (int k = j; k < j + 2; ++k) {
            const int n = wn * 128 + 16 * k + 4 * (ln >> 4);
            const u32x4_t v = {__float_as_uint(value(i, k, 0)), __float_as_uint(value(i, k, 1)),
                               __float_as_uint(value(i, k, 2)), __float_as_uint(value(i, k, 3))};
            const uint32_t off = ((n < right) & (m < rows)) ? roff + (uint32_t)n * 4u : kOut;
            __builtin_amdgcn_raw_buffer_store_b128(v, out, off, 0, 0);
          }
        } else {
          // 8 consecutive columns a lane: rows of 16 lanes trade, so that rows 0 and 2
          // of lanes take block j (columns 0.. and 8..), rows 1 and 3 block j + 1
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = (uint32_t)O::cvt(value(i, j + (k >> 1), 2 * (k & 1))) |
                   ((uint32_t)O::cvt(value(i, j + (k >> 1), 2 * (k & 1) + 1)) << 16);
          const auto s0 = __builtin_amdgcn_permlane16_swap(w[0], w[2], false, false);
          const auto s1 = __builtin_amdgcn_permlane16_swap(w[1], w[3], false, false);
          const u32x4_t v = {(uint32_t)s0[0], (uint32_t)s1[0], (uint32_t)s0[1], (uint32_t)s1[1]};
          const int n = wn * 128 + 16 * (j + ((ln >> 4) & 1)) + 8 * (ln >> 5);
          const uint32_t off = ((n < right) & (m < rows)) ? roff + (uint32_t)n * 2u : kOut;
          __builtin_amdgcn_raw_buffer_store_b128(v, out, off, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    }
    if (next >= nunits) return;
    slot0 = (slot0 + ns) & 1;
    ring_at += ns;
    if (kInt8) side ^= 1;
    chained = chain;
    tile = next;
    if (!chain) {
      // this wave's copies (of nothing) are done, every wave has read the
      // last fragments: both slots are free
      __builtin_amdgcn_s_waitcnt(vm_wait(0));
      __builtin_amdgcn_s_waitcnt(kLgkmWait0);
      __syncthreads();
      t = describe(tile);
      start();
    }
  }
}

// Sums of the parts of split tiles, in order, with the conversion and stores of the kernel above.
// Workgroup b takes strips b, b + grid, ... of the split tiles (strip: a wave's 16 rows).
template <typename T, typename O, int LAYOUT, int FA, int EPI = kPlain>
__global__ __launch_bounds__(256) void ragged_join_kernel(RaggedArgs p, uint32_t tile_grid) {
  constexpr bool kInt8 = sizeof(typename T::elem) == 1;
  constexpr bool kIsGated = EPI == kGated || EPI == kGatedKeep;
  constexpr int kTileM = 64 * FA;
  constexpr int kRowsF = 2 * FA, kStrips = 4 * kRowsF;
  const int lane = threadIdx.x & 63;
  const int64_t cols = LAYOUT == 0 ? p.N : p.K;
  const uint32_t ctiles = column_tiles<LAYOUT, EPI>(p);
  const uint32_t band = (uint32_t)((p.N + kTileM - 1) / kTileM);
  uint32_t rtiles = (uint32_t)p.G * band;
  if (LAYOUT != 2)
    rtiles = (uint32_t)wave_row_tile(p.m_splits, p.G, p.R, kTileM, -1, true).total;
  const Units u = units_of(rtiles * ctiles, tile_grid, part_stages(LAYOUT, p, sizeof(typename T::elem)), true);
  if (u.parts < 2) return;
  for (uint32_t b = blockIdx.x; b < u.rem * kStrips; b += gridDim.x) {
    const uint32_t v = b / kStrips, strip = b % kStrips, at = u.full + v;
    const int wave = (int)strip / kRowsF, i = (int)strip % kRowsF;
    int32_t mt, nt, g;
    int64_t m0, rows;
    if (LAYOUT == 2) {
      g = (int32_t)(at / (band * ctiles));
      tile_order(at % (band * ctiles), band, ctiles, &mt, &nt);
      m0 = (int64_t)mt * kTileM;
      rows = min((int64_t)kTileM, p.N - m0);
    } else {
      tile_order(at, rtiles, ctiles, &mt, &nt);
      const RowSpan s = wave_row_tile(p.m_splits, p.G, p.R, kTileM, mt, false);
      g = s.g;
      m0 = s.row0;
      rows = s.rows;
    }
    if ((wave >> 1) * 32 * FA + 16 * i >= rows) continue;
    // blocks threadIdx.x / 64 and 4 on of the strip's 8
    typedef typename T::acc16 V;
    V sum[2];
    for (uint32_t part = 0; part < u.parts; ++part) {
      const uint8_t* ws = (const uint8_t*)p.ws + (int64_t)(part * u.rem + v) * (kTileM * kTileN * 4) +
                          ((wave * kRowsF + i) * 8 + (threadIdx.x >> 6)) * 1024 + lane * 16;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const V x = *(const V*)(ws + q * 4096);
        if (part == 0) sum[q] = x;
        else sum[q] += x;
      }
    }
    const int m = (wave >> 1) * 32 * FA + 16 * i + (lane & 15);
    if (m >= rows) continue;
    float sa = 0.f;
    if (kInt8) {
      const int64_t row = p.row_index != nullptr ? p.row_index[m0 + m] : m0 + m;
      if (row >= 0 && row < p.S) sa = p.sa[row];
    }
    typedef typename O::elem OE;
    if constexpr (kIsGated) {
      // the two blocks are a gate and its up block; columns come in eights
      const int64_t F = p.N / 2;
      const int64_t n = (int64_t)nt * (kTileN / 2) + (wave & 1) * 64 + 16 * (int)(threadIdx.x >> 6) + 4 * (lane >> 4);
      if (n >= F) continue;
      OE o[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[0][e] = O::cvt(gated(sum[0][e], sum[1][e]));
        o[1][e] = O::cvt(sum[0][e]);
        o[2][e] = O::cvt(sum[1][e]);
      }
      __builtin_memcpy(__builtin_assume_aligned((OE*)p.c + (m0 + m) * p.ldc + n, 8), o[0], 8);
      if constexpr (EPI == kGatedKeep) {
        OE* h = (OE*)p.h + (m0 + m) * 2 * F + n;
        __builtin_memcpy(__builtin_assume_aligned(h, 8), o[1], 8);
        __builtin_memcpy(__builtin_assume_aligned(h + F, 8), o[2], 8);
      }
      continue;
    }
    if constexpr (EPI == kGatedBwd) {
      const int64_t F = p.K;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t n = (int64_t)nt * kTileN + (wave & 1) * 128 + 16 * (int)(threadIdx.x >> 6) + 64 * q +
                          4 * (lane >> 4);
        if (n >= F) continue;
        const int64_t at = (m0 + m) * 2 * F + n;
        OE o[3][4], hg[4], hu[4];
        __builtin_memcpy(hg, __builtin_assume_aligned((const OE*)p.h + at, 8), 8);
        __builtin_memcpy(hu, __builtin_assume_aligned((const OE*)p.h + at + F, 8), 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const GatedGrad r = gated_grad((float)sum[q][e], widen<T>(hg[e]), widen<T>(hu[e]));
          o[0][e] = O::cvt(r.gate);
          o[1][e] = O::cvt(r.up);
          o[2][e] = O::cvt(r.act);
        }
        __builtin_memcpy(__builtin_assume_aligned((OE*)p.c + at, 8), o[0], 8);
        __builtin_memcpy(__builtin_assume_aligned((OE*)p.c + at + F, 8), o[1], 8);
        if (p.act != nullptr)
          __builtin_memcpy(__builtin_assume_aligned((OE*)p.act + (m0 + m) * F + n, 8), o[2], 8);
      }
      continue;
    }
    OE* c = (OE*)p.c + ((LAYOUT == 2 ? (int64_t)g * p.N : 0) + m0 + m) * p.ldc;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t n = (int64_t)nt * kTileN + (wave & 1) * 128 + 16 * (int)(threadIdx.x >> 6) + 64 * q +
                        4 * (lane >> 4);
      if (n >= p.ccols) continue;   // columns come in fours (rows are multiples of 16 bytes)
      OE o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = (float)sum[q][e];
        if constexpr (kInt8)
          x = n + e < cols ? scaled<O>(sum[q][e], sa, p.sb[(int64_t)g * p.N + n + e]) : 0.f;
        o[e] = O::cvt(x);
      }
      __builtin_memcpy(__builtin_assume_aligned(c + n, sizeof(o)), o, sizeof(o));
    }
  }
}

}  // namespace mx

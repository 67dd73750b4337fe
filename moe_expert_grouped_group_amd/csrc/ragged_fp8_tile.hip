// Large tiles of the products in 8-bit floating point with a scale for each block of 128 (ragged_fp8.hip
// has the formula), for results of 16 bits and operands whose rows start on 16 bytes.
//
// One workgroup per CU walks output tiles of 32 RF x 256; 8 waves, 2 x 4, each 16 RF x 64.  Operands go
// from memory to LDS without passing registers, in stages of 128 contraction bytes: one block of scales
// (two slots, rows and chunks laid out as in ragged_tile.h).  A stage's sums start from zero for each
// 16 x 16 block of the result; times the two scales they are added to the fp32 sums by vector
// instructions, which run beside the next matrix instructions.  Those cannot reach the accumulation
// registers: eight waves of 128 sums each in ordinary registers, not four of 256.
//
// The sums of a stage (FAST chooses):
//  * fp32: four 16 x 16 x 32 bf16 matrix instructions on widened codes.  A wave widens what it has read
//    from LDS, in registers: 12 conversions for 8 matrix instructions (16 cycles each), the rows of the
//    next group beside the last block of this one, the columns of a stage beside a block of the last group
//    before it and the first three of its own.  Widened once into LDS instead, the tile would be read at
//    twice the bytes: LDS busy for three quarters of the time that a stage's matrix instructions take, with the
//    widening's reads and writes on top.
//    8 x 4096 x 14336, 16384 rows: 1500 to 1660 us by the machine's clock, 1.16 to 1.28 PFLOP/s (matrix cores
//    busy 57 % at 1.64 GHz; the bf16 product of ragged_tile.h 1594 to 1624: the power is spent alike).  128 x 128
//    tiles through registers (ragged_fp8.hip) take 2440.
//  * 8-bit (the caller asked for them): one 16 x 16 x 128 instruction, which keeps 13 bits below the
//    largest of 8 consecutive products (1.5e-5 of a block's sum on normal values, where bf16 has 9e-9; the 16 x 16 x
//    32 one for 8-bit operands the same).  It runs at twice the rate: 950 to 1060 us by the machine's clock, 1.8
//    to 2.0 PFLOP/s, where the MXFP8 product of this package, whose scales the matrix instruction applies
//    itself, takes 929 (zeros: 920; matrix cores busy 51 % at 1.86 GHz).  Without its copies to LDS the kernel
//    takes 870, with every copy hitting L2 1045, without the scaling 1081 beside 1157 at the time.  All of
//    a wave's copies at once instead of one to a block cost 4 %, one to two or three 2 and 5 %; a second
//    meeting half way, so that three quarters of the copies go out half a stage earlier, 0 to 1 %; the two
//    waves of a SIMD copying in turn 6 %.
#include <type_traits>

#include "fp8_tile_ranges.h"
#include "ragged_tile_launch.h"

namespace mx {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kF8Threads = 512;

template <typename O, int RF, bool FAST>
__global__ __launch_bounds__(kF8Threads, 1) void ragged_fp8_tile_kernel(RaggedArgs kernel_args) {
  constexpr int kTileM = 32 * RF;
  constexpr int kOffB = kTileM * kStageK, kStage = kOffB + kTileN * kStageK;
  constexpr int kCopiesA = RF / 2;                 // of a wave for a stage: 8 rows each; 4 of B
  constexpr int kGroup = 4;                        // blocks whose scales are copied together
  constexpr int kBlocks = 4 * RF;                  // blocks of a wave, each with its sums of a stage
  constexpr int kLag = FAST ? 3 : 1;               // blocks between one and the use of its sums
  static_assert(RF == 8 || RF == 4 || RF == 2, "");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  // scales of four blocks: [row][4], then [half of the columns][4], twice
  __shared__ __attribute__((aligned(16))) float scales[2][kTileM + 64][kGroup];
  __shared__ int32_t ring[2][kTileM];              // row indexes of two tiles
  __shared__ RaggedTable table;
  __shared__ RaggedArgs args;   // what only the start and end of a tile need: scalar registers are few
  __shared__ struct {
    uint32_t rtiles, ctiles, full, rem, parts;
  } plan;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem, scale0 = (uint32_t)(uintptr_t)scales;
  uint32_t nunits;
  int kb;
  bool gather;
  {
    const RaggedArgs& p = kernel_args;
    build_ragged_table<kF8Threads>(p.m_splits, p.G, p.R, kTileM, &table, (int32_t*)smem);
    const uint32_t ctiles = (uint32_t)((p.N + kTileN - 1) / kTileN);
    const uint32_t rtiles = (uint32_t)__builtin_amdgcn_readfirstlane(table.tiles[kRaggedMaxGroups]);
    kb = (int)((p.K + 127) / 128);
    const Units u = units_of(rtiles * ctiles, gridDim.x, kb, p.ws != nullptr);
    nunits = (uint32_t)__builtin_amdgcn_readfirstlane((int)(u.full + u.rem * u.parts));
    gather = p.row_index != nullptr;
    if (tid == 0) {
      copy_args(args, p);
      plan.rtiles = rtiles;
      plan.ctiles = ctiles;
      plan.full = u.full;
      plan.rem = u.rem;
      plan.parts = u.parts;
    }
  }
  uint32_t tile = blockIdx.x;
  if (tile >= nunits) return;
  __syncthreads();

  // A unit: a tile, or a part of one's stages (Units in ragged_tile.h; split: its number among the
  // parts, or -1).
  struct Tile {
    int32_t g, row0, rows, n0, first, end, split;
  };
  auto describe = [&](uint32_t i) {
    // of each full round of the grid an XCD takes consecutive tiles (as ragged_tile.h)
    const uint32_t n = gridDim.x;
    Tile t;
    t.first = 0;
    t.end = kb;
    t.split = -1;
    if (i < plan.full) {
      if (n % 8 == 0) i = i - i % n + (i % n & 7) * (n / 8) + (i % n >> 3);
    } else if (plan.parts > 1) {
      const uint32_t v = i - plan.full, which = v / plan.rem;
      const int32_t each = kb / (int32_t)plan.parts, more = kb % (int32_t)plan.parts;
      t.first = __builtin_amdgcn_readfirstlane((int32_t)which * each + min((int32_t)which, more));
      t.end = __builtin_amdgcn_readfirstlane(t.first + each + ((int32_t)which < more ? 1 : 0));
      t.split = __builtin_amdgcn_readfirstlane((int32_t)v);
      i = plan.full + v % plan.rem;
    }
    int32_t mt, nt;
    tile_order(i, plan.rtiles, plan.ctiles, &mt, &nt);
    int lo = 0, hi = args.G;   // tiles[lo] <= mt < tiles[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (table.tiles[mid] <= mt) lo = mid; else hi = mid;
    }
    t.g = __builtin_amdgcn_readfirstlane(lo);
    t.row0 = __builtin_amdgcn_readfirstlane(table.rows[lo] + (mt - table.tiles[lo]) * kTileM);
    t.rows = __builtin_amdgcn_readfirstlane(min(kTileM, table.rows[lo + 1] - t.row0));
    t.n0 = __builtin_amdgcn_readfirstlane(nt * kTileN);
    return t;
  };

  // Copies.  Part j of wave w: rows 8 (parts w + j) + lane / 8, chunk position lane % 8, which holds the
  // row's chunk (lane % 8) ^ (row / 2 % 8).  B's parts 2 and 3 go from 16 rows on in its memory.
  auto chunk = [&](int row8) {
    const int l = (int)hide((uint32_t)lane);   // anew where it is used, not kept
    return (uint32_t)((l & 7) ^ ((4 * (row8 & 1) + (l >> 4)) & 7)) * 16;
  };
  uint32_t va[kCopiesA], vb[2], vs;
  i32x4 sa, sb[2], ss;
#pragma unroll
  for (int j = 0; j < 2; ++j) vb[j] = (uint32_t)(32 * wave + 8 * j + (lane >> 3)) * (uint32_t)kernel_args.K + chunk(j);
  auto operands = [&](const Tile& t, int side) {
    const RaggedArgs& p = args;
    const uint32_t pitch = (uint32_t)p.lda;
    auto row = [&](int i) {   // row i of the tile as one of X, from its first or the tile's; -1: none
      if (i >= t.rows) return (int32_t)-1;
      if (!gather) return (int32_t)i;
      const int32_t x = ring[side][i];
      return x >= 0 && x < p.S ? x : (int32_t)-1;
    };
    const int64_t first = gather ? 0 : t.row0, count = (gather ? p.S : p.R) - first;
    sa = bounded((const uint8_t*)p.a + first * p.lda, rows_range(count, p.lda, p.K));
    const uint8_t* w = (const uint8_t*)p.b + ((int64_t)t.g * p.N + t.n0) * p.K;
    sb[0] = bounded(w, rows_range(p.N - t.n0, p.K, p.K));
    sb[1] = bounded(w + 16 * p.K, rows_range(p.N - t.n0 - 16, p.K, p.K));
#pragma unroll
    for (int j = 0; j < kCopiesA; ++j) {
      const int32_t r = row(8 * (kCopiesA * wave + j) + (lane >> 3));
      va[j] = r < 0 ? kOut : (uint32_t)r * pitch + chunk(kCopiesA * wave + j);
    }
    // waves of rows copy their scales; the next one those of the two halves of the columns
    if (64 * wave < kTileM) {
      const int32_t r = row(64 * wave + lane);
      ss = bounded(p.sa + first * kb, rows_range(count, kb * 4, kb * 4));
      vs = r < 0 ? kOut : (uint32_t)r * (uint32_t)kb * 4u;
    } else {
      const int64_t nb = (p.N + 127) / 128, b0 = t.n0 / 128;
      ss = bounded(p.sb + ((int64_t)t.g * nb + b0) * kb, rows_range(nb - b0, kb * 4, kb * 4));
      vs = lane < 2 ? (uint32_t)lane * (uint32_t)kb * 4u : kOut;
    }
  };
  auto copy_rows = [&](const Tile& t, int side) {   // its row indexes
    if (!gather || 64 * wave >= kTileM) return;
    const uint32_t to = (uint32_t)(uintptr_t)ring + (uint32_t)(side * kTileM * 4 + wave * 256);
    copy4(bounded(args.row_index + t.row0, (int64_t)t.rows * 4), (uint32_t)((64 * wave + lane) * 4), 0u,
          __builtin_amdgcn_readfirstlane(to));
  };

  // What is copied runs two stages ahead of what is computed, from tile to tile, and the row
  // indexes a tile ahead of that.  Past the last tile the ranges are empty: zeros, never used.
  constexpr int kCopies = kCopiesA + 4;
  uint32_t ctile = tile;
  int cst = 0, cslot = 0, cside = 0, cring = 0;   // stage, its slot, the place of its scales, of its rows
  uint32_t scales_off = 0;
  Tile ct, after;
  uint32_t to_stage = 0, to_scales = 0, soff = 0, past[2] = {0, 0};
  bool with_scales = false;
  auto next_stage = [&]() {
    if (cst == ct.end) {
      ctile += gridDim.x;
      if (ctile < nunits) {
        cring ^= 1;
        ct = after;
        operands(ct, cring);
        if (ctile + gridDim.x < nunits) {
          after = describe(ctile + gridDim.x);
          copy_rows(after, cring ^ 1);
        }
        cst = ct.first;
      } else {
        ctile = nunits;
        cst = 0;
        ct.first = 0;
        ct.end = kb;
        sa[2] = sb[0][2] = sb[1][2] = ss[2] = 0;
      }
    }
    const uint32_t left = cst == kb - 1 ? (uint32_t)((args.K - 1) & 127) + 1 : 128u;
#pragma unroll
    for (int h = 0; h < 2; ++h) past[h] = chunk(h) >= left ? kOut : 0u;
    to_stage = __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)(cslot * kStage));
    soff = ctile < nunits ? (uint32_t)cst * kStageK : 0u;
    // the scales of a group of four blocks with the first of them that the unit has
    const bool opens = (cst & 3) == 0 || cst == ct.first;
    with_scales = opens && 64 * wave <= kTileM;
    scales_off = ctile < nunits ? (uint32_t)(cst & ~3) * 4u : 0u;
    to_scales = __builtin_amdgcn_readfirstlane(scale0 + (uint32_t)(cside * (int)sizeof(scales[0]) + wave * 1024));
    if (opens) cside ^= 1;
    ++cst;
    cslot ^= 1;
  };
  auto copy = [&](auto C) {   // copy c of that stage; the first with the scales
    constexpr int c = decltype(C)::value;
    // (what lies past a row's last block is not used)
    if (c == 0 && with_scales) copy16(ss, vs, scales_off, to_scales);
    if constexpr (c < kCopiesA)
      copy16(sa, va[c] | past[(kCopiesA * wave + c) & 1], soff, to_stage + (uint32_t)((kCopiesA * wave + c) * 1024));
    else
      copy16(sb[(c - kCopiesA) >> 1], vb[(c - kCopiesA) & 1] | past[(c - kCopiesA) & 1],
             c - kCopiesA < 2 ? soff : row_offset((uint32_t)sb[1][2], soff),
             to_stage + kOffB + (uint32_t)((4 * wave + c - kCopiesA) * 1024));
  };

  Tile t = describe(tile);
  ct = after = t;
  copy_rows(t, 0);
  if (tile + gridDim.x < nunits) {
    after = describe(tile + gridDim.x);
    copy_rows(after, 1);
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  __syncthreads();
  operands(t, 0);
  cst = t.first;
  __syncthreads();   // with one stage a tile, the second copies go on to the third tile's rows
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    next_stage();
    unroll<kCopies>([&](auto C) { copy(C); });
  }
  __builtin_amdgcn_s_waitcnt(vm_wait(0));
  __syncthreads();

  // Fragments: lane l row l % 16, chunks l / 16 and l / 16 + 4 of its 128 bytes (bit 6 of the address).
  const uint32_t lane_at = (uint32_t)((lane & 15) * kStageK + (((lane >> 4) ^ ((lane >> 1) & 7)) * 16));
  const uint32_t base_a = lds0 + (uint32_t)(wm * 16 * RF * kStageK), base_b = lds0 + kOffB + (uint32_t)(wn * 64 * kStageK);
  auto fragment = [&](uint32_t at, int imm) {
    const u32x4_t lo = *(lds_u32x4_t*)(at + imm), hi = *(lds_u32x4_t*)((at ^ 64u) + imm);
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  typedef __attribute__((address_space(3))) const float lds_f32_t;
  const uint32_t row_scale = scale0 + (uint32_t)((wm * 16 * RF + (lane & 15)) * kGroup * 4);
  const uint32_t col_scale = scale0 + (uint32_t)((kTileM + (wn >> 1)) * kGroup * 4);

  // A stage: RF groups of 16 rows, 4 blocks each, from zero.  Each one's sums are scaled and
  // added kLag blocks later, beside the instructions that run then; the next group's fragments are read
  // meanwhile.  Ahead of the last group every fragment of the stage is in registers: there the waves
  // meet (the next stage has landed, this one's slot is free), and the last group's instructions cover
  // the first reads of the next stage.  (!FAST: registers are few.  fb holds codes of two blocks of B on their
  // way to wb: 1 and 2 at a stage's start, with block 0 widened before it.)
  constexpr int kKept = kLag + 1;   // blocks whose sums are not added yet
  f32x4 acc[RF][4], part[kKept];
  float before = 0.f, mine = 0.f;   // scales of the group before and of this one
  int slot = 0, side = 0;           // of the stage computed
  i32x8 fa[FAST ? 2 : 1], fb[FAST ? 4 : 2];
  u32x4_t wa[4], wb[4][4];   // !FAST: runs of 32 of the contraction, in bf16
  auto widened = [](const i32x8& c, int s) { return widen_codes8((uint32_t)c[2 * s], (uint32_t)c[2 * s + 1]); };
  fa[0] = fragment(base_a + lane_at, 0);
  if constexpr (FAST) {
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[j] = fragment(base_b + lane_at, j * 2048);
  } else {
    fb[0] = fragment(base_b + lane_at, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      wa[s] = widened(fa[0], s);
      wb[0][s] = widened(fb[0], s);
    }
    fb[1] = fragment(base_b + lane_at, 2048);
    fb[0] = fragment(base_b + lane_at, 2 * 2048);
  }
  float row = *(lds_f32_t*)(row_scale + (uint32_t)((t.first & 3) * 4));
  float col = *(lds_f32_t*)(col_scale + (uint32_t)((t.first & 3) * 4));
  // the sums of block n - kLag of a stage (or of the stage before)
  auto add = [&](auto N, int from, int to) {
    constexpr int n = (decltype(N)::value + kBlocks - kLag) % kBlocks, i = n / 4, j = n % 4;
    constexpr bool same = decltype(N)::value / 4 == i;
    const float s = same ? mine : before;
#pragma unroll
    for (int e = from; e < to; ++e) acc[i][j][e] = __builtin_fmaf(part[n % kKept][e], s, acc[i][j][e]);
    // (held in place: the compiler would move all of a stage's sums behind its branches)
    asm volatile("" : "+v"(acc[i][j]));
  };

  for (;;) {
    const uint32_t next = tile + gridDim.x;
#pragma unroll
    for (int i = 0; i < RF; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kKept; ++j) part[j] = f32x4{0, 0, 0, 0};
    const int end = t.end;
    for (int st = t.first; st < end; ++st) {
      const uint32_t at_a = hide(lane_at + (base_a + (uint32_t)(slot * kStage)));
      const uint32_t at_row = hide(row_scale + (uint32_t)(side * (int)sizeof(scales[0])) + (uint32_t)((st & 3) * 4));
      uint32_t at_b = 0;
      unroll<RF>([&](auto I) {
        constexpr int i = decltype(I)::value;
        before = mine;
        mine = row * col;
        if constexpr (i + 1 < RF) {
          fa[FAST ? (i + 1) & 1 : 0] = fragment(at_a, (i + 1) * 2048);
          row = *(lds_f32_t*)(at_row + (uint32_t)((i + 1) * 16 * kGroup * 4));
        } else {
          __builtin_amdgcn_s_waitcnt(vm_wait(0));
          __builtin_amdgcn_s_waitcnt(kLgkmWait0);
          __syncthreads();
          next_stage();
          // (the unit that follows starts inside its tile only if it has four stages and more, so that it is
          // the one copied now)
          const int next_first = kb > 1 ? ct.first : 0;
          slot ^= 1;
          if ((st & 3) == 3 || st == end - 1) side ^= 1;
          const uint32_t to = (uint32_t)(side * (int)sizeof(scales[0])) +
                              (uint32_t)(((st == end - 1 ? next_first : st + 1) & 3) * 4);
          row = *(lds_f32_t*)hide(row_scale + to);
          col = *(lds_f32_t*)hide(col_scale + to);
          at_b = hide(lane_at + (base_b + (uint32_t)(slot * kStage)));
          if constexpr (!FAST) fa[0] = fragment(hide(lane_at + (base_a + (uint32_t)(slot * kStage))), 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        unroll<4>([&](auto J) {
          constexpr int j = decltype(J)::value;
          using N = std::integral_constant<int, 4 * i + j>;
          f32x4& sum = part[N::value % kKept];
          if constexpr (FAST) {
            sum = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i & 1], f32x4{0, 0, 0, 0}, 0, 0, 0, 127, 0,
                                                                   127);
            asm volatile("" : "+v"(sum));
            __builtin_amdgcn_sched_barrier(0);
            add(N{}, 0, 4);
            if constexpr (i == RF - 1) fb[j] = fragment(at_b, j * 2048);
          } else {
            unroll<4>([&](auto S) {
              constexpr int s = decltype(S)::value;
              sum = TypeBf16::mma16(wb[j][s], wa[s], s == 0 ? f32x4{0, 0, 0, 0} : sum);
              asm volatile("" : "+v"(sum));
              __builtin_amdgcn_sched_barrier(0);
              if constexpr (s == 1) add(N{}, 0, 2);
              if constexpr (s == 2) add(N{}, 2, 4);
              if constexpr (j == 3) wa[s] = widened(fa[0], s);
              if constexpr (i == 0 && j < 3) wb[j + 1][s] = widened(fb[(j + 1) & 1], s);
              if constexpr (i == RF - 1 && j == 2) wb[0][s] = widened(fb[0], s);
              __builtin_amdgcn_sched_barrier(0);
            });
            // the codes of B: the next stage's first two once a block of this one's is done
            if constexpr (i == RF - 1 && j == 0) fb[0] = fragment(at_b, 0), fb[1] = fragment(at_b, 2048);
            if constexpr (i == RF - 1 && j == 2) fb[0] = fragment(at_b, 2 * 2048);
            if constexpr (i == 0 && j == 0)
              fb[1] = fragment(hide(lane_at + (base_b + (uint32_t)(slot * kStage))), 3 * 2048);
          }
          // the copies of the stage two ahead go out one to a matrix instruction, from the last group on
          constexpr int at = ((i + 1) % RF) * 4 + j;
          if constexpr (at < kCopies) copy(std::integral_constant<int, at>{});
          __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (FAST && i == RF - 1) fa[0] = fragment(hide(lane_at + (base_a + (uint32_t)(slot * kStage))), 0);
      });
    }
    // the last kLag blocks
    before = mine;
    unroll<kLag>([&](auto N) { add(N, 0, 4); });
    mine = 0.f;

    if (t.split >= 0) {
      // a part (the last unit of its workgroup): the sums as they lie
      const auto ws = make_rsrc((const uint8_t*)args.ws + (int64_t)t.split * (kTileM * kTileN * 4), kTileM * kTileN * 4);
#pragma unroll
      for (int i = 0; i < RF; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, acc[i][j]), ws,
                                                 (uint32_t)(((wave * RF + i) * 4 + j) * 1024 + lane * 16), 0, 0);
      return;
    }

    // Stores, whole lines of 64 columns, bounded, as in ragged_tile.h.  Sum e of block (i, j) in lane l:
    // row 16 i + l % 16, column 16 j + 4 (l / 16) + e.
    typedef typename O::elem OE;
    const RaggedArgs& p = args;
    const int ln = (int)hide((uint32_t)lane);
    const uint32_t ec = (uint32_t)(p.ldc * sizeof(OE));
    const auto out = make_rsrc((OE*)p.c + (int64_t)t.row0 * p.ldc + t.n0,
                               (int64_t)(t.rows - 1) * ec + (p.N - t.n0) * (int64_t)sizeof(OE));
    const int right = (int)min((int64_t)kTileN, p.N - t.n0);
    const int n = wn * 64 + line_col(ln);
#pragma unroll
    for (int i = 0; i < RF; ++i) {
      const int m = wm * 16 * RF + 16 * i + line_row(ln);
      u32x4_t w[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[b][k] = (uint32_t)O::cvt(acc[i][2 * b + (k >> 1)][2 * (k & 1)]) |
                    ((uint32_t)O::cvt(acc[i][2 * b + (k >> 1)][2 * (k & 1) + 1]) << 16);
        w[b] = swap_blocks(w[b]);
      }
      whole_lines(w[0], w[1]);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t at = ((n < right) & (m + 8 * b < t.rows)) ? (uint32_t)(m + 8 * b) * ec + (uint32_t)n * 2u : kOut;
        __builtin_amdgcn_raw_buffer_store_b128(w[b], out, at, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (next >= nunits) return;
    tile = next;
    t = kb > 1 ? ct : describe(tile);
  }
}

// Sums of the parts of split tiles, in order.  Workgroup b takes strips b, b + grid, ... (a wave's 16 rows).
template <typename O, int RF>
__global__ __launch_bounds__(256) void ragged_fp8_join_kernel(RaggedArgs p, uint32_t tile_grid) {
  constexpr int kTileM = 32 * RF, kStrips = 8 * RF;
  const int lane = threadIdx.x & 63, j = threadIdx.x >> 6;
  const uint32_t ctiles = (uint32_t)((p.N + kTileN - 1) / kTileN);
  const uint32_t rtiles = (uint32_t)wave_row_tile(p.m_splits, p.G, p.R, kTileM, -1, true).total;
  const Units u = units_of(rtiles * ctiles, tile_grid, (p.K + 127) / 128, true);
  if (u.parts < 2) return;
  for (uint32_t b = blockIdx.x; b < u.rem * kStrips; b += gridDim.x) {
    const uint32_t v = b / kStrips, strip = b % kStrips;
    const int wave = (int)strip / RF, i = (int)strip % RF;
    int32_t mt, nt;
    tile_order(u.full + v, rtiles, ctiles, &mt, &nt);
    const RowSpan t = wave_row_tile(p.m_splits, p.G, p.R, kTileM, mt, false);
    const int m = (wave >> 2) * 16 * RF + 16 * i + (lane & 15);
    const int64_t n = (int64_t)nt * kTileN + (wave & 3) * 64 + 16 * j + 4 * (lane >> 4);
    if (m >= t.rows || n >= p.N) continue;   // columns come in eights
    f32x4 sum = {0, 0, 0, 0};
    for (uint32_t part = 0; part < u.parts; ++part)
      sum += *(const f32x4*)((const uint8_t*)p.ws + (int64_t)(part * u.rem + v) * (kTileM * kTileN * 4) +
                             ((wave * RF + i) * 4 + j) * 1024 + lane * 16);
    typename O::elem o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = O::cvt(sum[e]);
    __builtin_memcpy(__builtin_assume_aligned((typename O::elem*)p.c + (t.row0 + m) * p.ldc + n, sizeof(o)), o, sizeof(o));
  }
}

namespace {

template <typename O, int RF, bool FAST>
hipError_t launch_fp8_tile(const RaggedArgs& p, hipStream_t st) {
  const int64_t m = 32 * RF, tiles = ((p.N + kTileN - 1) / kTileN) * (p.R / m + std::min<int64_t>(p.G, p.R));
  const unsigned grid = (unsigned)(p.ws != nullptr ? compute_units() : std::min<int64_t>(tiles, compute_units()));
  ragged_fp8_tile_kernel<O, RF, FAST><<<dim3(grid), dim3(kF8Threads), 0, st>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.ws == nullptr) return e;
  // half the tiles of a round at most are split
  const unsigned strips = std::max(1u, grid / 2) * 8 * RF;
  ragged_fp8_join_kernel<O, RF><<<dim3(std::min(strips, 1024u)), dim3(256), 0, st>>>(p, grid);
  return hipGetLastError();
}

template <typename O, bool FAST>
hipError_t launch_fp8_tile_rows(int rows, const RaggedArgs& p, hipStream_t st) {
  if (rows == 64) return launch_fp8_tile<O, 2, FAST>(p, st);
  return rows == 128 ? launch_fp8_tile<O, 4, FAST>(p, st) : launch_fp8_tile<O, 8, FAST>(p, st);
}

// 8-bit sums.  Rows of a tile: low ones for experts of few rows and where high ones would leave CUs idle (half
// of an expert's last tile empty on average).  Measured (us, 64, 128 and 256 rows): 8 x 14336 x 4096, 32 rows an
// expert 106, 112, 126, 96 rows 179, 125, 134; 8 x 2048 x 2048, 128 rows 24, 25, 32, 512 rows 39 to 55, 29 to
// 46 (uneven), 36; 4 x 7168 x 4096, 192 rows 69, 52, 56, 256 rows 76, 52 to 79, 57.
int fast_rows(const RaggedArgs& p) {
  const int64_t groups = std::min<int64_t>(p.G, p.R), mean = p.R / groups;
  if (mean <= 32) return 64;
  return mean <= 96 || (p.R / 128 + groups / 2) * ((p.N + kTileN - 1) / kTileN) <= compute_units() ? 128 : 256;
}

// 8-bit sums.  Whether a launch may split tiles (the table in the kernel, which has the experts' rows, decides on
// how many parts): the stages saved, as units_of counts them, have to pay the second launch and the
// workspace, about 8 us or six stages, where experts' rows are even or on average over the numbers of
// tiles that uneven ones can make.  Measured (us, whole, split; on the same kernel with a
// slower start, 10 us on both): 1 x 4096 x 14336, 257 rows 168, 76;
// 8 x 4096 x 14336, 768 rows 191, 142, 2048 rows 229, 178; 8 x 2048 x 7168, 1024 rows 93, 77; 1 x 4096 x
// 4096, 200 rows 56, 44; and with nothing to split 8 x 2048 x 2048, 2048 rows 42, 50.
bool fast_splits(const RaggedArgs& p, int64_t m) {
  const int64_t groups = std::min<int64_t>(p.G, p.R), stages = (p.K + 127) / 128;
  const int64_t ctiles = (p.N + kTileN - 1) / kTileN;
  auto saved = [&](int64_t rtiles) -> int64_t {
    const Units u = units_of((uint32_t)std::min<int64_t>(rtiles * ctiles, 1 << 30), (uint32_t)compute_units(), stages, true);
    return u.parts > 1 ? stages - stages / u.parts - u.parts * u.rem / 7 : 0;
  };
  if (saved(groups * ((p.R / groups + m - 1) / m)) > 6) return true;
  const int64_t least = (p.R + m - 1) / m, most = p.R / m + groups;
  int64_t sum = 0;
  for (int i = 0; i < 8; ++i) sum += saved(least + (most - least) * i / 7);
  return sum > 6 * 8;
}

// fp32 sums.  About what a launch takes, in us, by the rows of its tiles: a stage while each CU has a tile, what
// comes once, a second launch where tiles may be split (half of it also if none is).  Half by the number of tiles
// of even experts, half by the mean over the numbers that uneven ones can make.  Measured, even experts and ones
// of 0.2 to 1.8 times the mean (64, 128 and 256 rows; s: may be split):
//   1 x 4096 x 4096    128 rows each  47  58  95, s  32  32  47    256:  47  59  96, s  50  40  49
//                              1024:  50  64  97, s  52  65  99
//   8 x 2048 x 2048    128 rows each  29  35  53, s  31  37  56    256:  29  36  54, s  32  39  57; uneven 50  37  55
//   4 x 4096 x 4096    192 rows each  52  61  96, s  54  65  99    512:  91  66  98; uneven 130 116 100, s 116  97 102
//   8 x 4096 x 7168     96 rows each  89 102 162                   256: 168 109 163; uneven 223 197 168, s 203 164 171
//   64 x 2048 x 1024    64 rows each  36  42  64; uneven  47  58  65;   128:  59  46  66; uneven  71  77  92
//   8 x 14336 x 4096    64 rows each 126 145 216; uneven 170 144 204;   128: 221 151 215; uneven 260 207 204
//                                                                       512: 705 466 416; uneven 709 506 493
Fp8Plan fp32_sums_plan(const RaggedArgs& p, bool can_split) {
  const int64_t groups = std::min<int64_t>(p.G, p.R), stages = (p.K + 127) / 128;
  const int64_t ctiles = (p.N + kTileN - 1) / kTileN, cus = compute_units();
  const struct { int rows; double stage, once; } kinds[] = {{64, 1.25, 7.0}, {128, 1.6, 8.0}, {256, 2.66, 10.5}};
  Fp8Plan best{0, false, 0.0};
  for (const auto& kind : kinds)
    for (int split = 0; split <= (can_split ? 1 : 0); ++split) {
      auto us = [&](int64_t rtiles) {
        const Units u = units_of((uint32_t)std::min<int64_t>(rtiles * ctiles, 1 << 30), (uint32_t)cus, stages, split != 0);
        const double last = u.rem == 0 ? 0.0 : u.parts > 1 ? (double)((stages + u.parts - 1) / u.parts) + 3.0 / kind.stage
                                                           : (double)stages;
        return kind.once + 3.0 * split + kind.stage * ((double)stages * (double)(u.full / cus) + last);
      };
      const int64_t least = (p.R + kind.rows - 1) / kind.rows, most = p.R / kind.rows + groups;
      double uneven = 0.0;
      for (int i = 0; i < 8; ++i) uneven += us(least + (most - least) * i / 7) / 8;
      const double both = 0.5 * (us(groups * ((p.R / groups + kind.rows - 1) / kind.rows)) + uneven);
      if (best.rows == 0 || both < best.us) best = Fp8Plan{kind.rows, split != 0, both};
    }
  // (reading the weights takes its time, however few the rows)
  best.us = std::max(best.us, 7.0 + 1e-6 * (double)groups * (double)p.N * (double)p.K / 4.7);
  return best;
}

}  // namespace

Fp8Plan ragged_fp8_plan(bool fast, bool can_split, const RaggedArgs& p) {
  if (!fast) return fp32_sums_plan(p, can_split);
  const int rows = fast_rows(p);
  return Fp8Plan{rows, can_split && fast_splits(p, rows), 0.0};
}

hipError_t launch_ragged_fp8_tile(int out, bool fast, const RaggedArgs& p, hipStream_t st) {
  const Fp8Plan plan = ragged_fp8_plan(fast, p.ws != nullptr, p);
  RaggedArgs q = p;
  if (!plan.split) q.ws = nullptr;
  if (fast)
    return out == 1 ? launch_fp8_tile_rows<OutBf16, true>(plan.rows, q, st)
                    : launch_fp8_tile_rows<OutF16, true>(plan.rows, q, st);
  return out == 1 ? launch_fp8_tile_rows<OutBf16, false>(plan.rows, q, st)
                  : launch_fp8_tile_rows<OutF16, false>(plan.rows, q, st);
}

}  // namespace mx

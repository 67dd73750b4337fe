// Forward products grouped by expert in 8-bit floating point (e4m3) with a scale for each block of
// 128 along the contraction (and of 128 output channels for the weights):
//
//   C[r, n] = sum over blocks b of  sa[i(r), b] sb[g, n / 128, b]  sum over k in b of q[i(r), k] w[g, n, k]
//
// The sum within a block is formed by matrix instructions, multiplied by the two scales and added
// to the result's fp32 sum.  Codes become bf16 on their way to the matrix instructions (exact: e4m3
// has 3 bits behind the leading one), because the 8-bit matrix instructions keep 13 bits below the
// largest of 8 consecutive products: 1.5e-5 of a block's sum on normal values, and all of it where large
// products cancel.  The large tiles (ragged_fp8_tile.hip), for results of 16 bits, take those instructions
// where the caller asked for fast sums; the forms here serve every type.
#include <algorithm>

#include "ragged_common.h"

namespace mx {

// 16 codes as two runs of 8 bf16 values.
struct Wide {
  u32x4_t lo, hi;
};
__device__ __forceinline__ Wide widen_codes(u32x4_t c) {
  return Wide{widen_codes8(c[0], c[1]), widen_codes8(c[2], c[3])};
}

// ---------------------------------------------------------------------------
// Any size, stride and alignment: 128 x 128 output tile, 4 waves of 64 x 64 (64 rows where tiles are few), a block at
// a time through registers to LDS, the next one's loads in flight meanwhile.
// ---------------------------------------------------------------------------
constexpr int kF8Tile = 128;
constexpr int kF8Pitch = 144;   // LDS row: 128 codes + 16 bytes, so that consecutive rows start in other banks

// TM: rows of a tile, 128 or 64.
template <typename O, int TM>
__global__ __launch_bounds__(256, 2) void ragged_fp8_any_kernel(RaggedArgs p, uint32_t first) {
  constexpr int MI = TM / 64, PA = TM / 32;   // blocks of 32 rows of a wave, rows of a thread
  __shared__ __attribute__((aligned(16))) uint8_t smem[(TM + kF8Tile) * kF8Pitch];
  __shared__ float srow[TM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t nt = (p.N + kF8Tile - 1) / kF8Tile, kb = (p.K + 127) / 128;
  const int64_t at = first + blockIdx.x, ct = at % nt;
  const int64_t n0 = ct * kF8Tile;
  const RowSpan t = wave_row_tile(p.m_splits, p.G, p.R, TM, at / nt, false);
  if (t.g < 0) return;
  const int g = t.g, rows = t.rows;
  const int64_t m0 = t.row0;

  // this thread's rows of both operands: (tid >> 3) + 32 i, 16 codes from 16 (tid & 7) on
  const int64_t k0 = (tid & 7) * 16;
  const uint8_t* a[PA];
  uint32_t there_a = 0, there_b = 0;   // bit i: row i is there; the others are rows of zeros
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = (tid >> 3) + 32 * i;
    there_b |= n0 + r < p.N ? 1u << i : 0u;
    if (i >= PA) continue;
    int64_t row = m0 + r;
    bool ok = r < rows;
    if (p.row_index != nullptr && ok) {
      row = p.row_index[row];
      ok = row >= 0 && row < p.S;
    }
    a[i] = (const uint8_t*)p.a + (ok ? row : 0) * p.lda + k0;
    there_a |= ok ? 1u << i : 0u;
  }
  const uint8_t* b = (const uint8_t*)p.b + ((int64_t)g * p.N + n0 + (tid >> 3)) * p.K + k0;
  // scales: thread r < 128 that of row r; the weights' is the tile's
  const float* sa = nullptr;
  if (tid < rows) {
    const int64_t row = p.row_index != nullptr ? p.row_index[m0 + tid] : m0 + tid;
    if (row >= 0 && row < p.S) sa = p.sa + row * kb;
  }
  const float* sb = p.sb + ((int64_t)g * nt + ct) * kb;

  u32x4_t ra[PA], rb[4];
  float next = 0.f;
  auto fetch = [&](int64_t block) {
    const int64_t k = block * 128, left = p.K - k0 - k;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < PA) ra[i] = chunk_end<uint8_t>(a[i] + k, (there_a >> i) & 1 ? left : 0);
      rb[i] = chunk_end<uint8_t>(b + 32 * i * p.K + k, (there_b >> i) & 1 ? left : 0);
    }
    next = (sa != nullptr ? sa[block] : 0.f) * sb[block];
  };
  uint8_t* la = smem;
  uint8_t* lb = smem + TM * kF8Pitch;
  typedef TypeBf16::acc Acc;
  Acc acc[MI][2];
  const Acc zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 2 * MI; ++i) acc[i >> 1][i & 1] = zero;
  const int wm = (wave >> 1) * 32 * MI, wn = (wave & 1) * 64;
  const uint8_t* fa = la + (wm + (lane & 31)) * kF8Pitch + (lane >> 5) * 16;
  const uint8_t* fb = lb + (wn + (lane & 31)) * kF8Pitch + (lane >> 5) * 16;

  fetch(0);
  for (int64_t block = 0; block < kb; ++block) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < PA) *(u32x4_t*)(la + ((tid >> 3) + 32 * i) * kF8Pitch + k0) = ra[i];
      *(u32x4_t*)(lb + ((tid >> 3) + 32 * i) * kF8Pitch + k0) = rb[i];
    }
    if (tid < TM) srow[tid] = next;
    __syncthreads();
    if (block + 1 < kb) fetch(block + 1);
    Acc part[MI][2];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Wide va[MI], vb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i < MI) va[i] = widen_codes(*(const u32x4_t*)(fa + i * 32 * kF8Pitch + s * 32));
        vb[i] = widen_codes(*(const u32x4_t*)(fb + i * 32 * kF8Pitch + s * 32));
      }
      // the weights first: a lane holds columns of one row
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          part[i][j] = TypeBf16::mma(vb[j].lo, va[i].lo, s == 0 ? zero : part[i][j]);
          part[i][j] = TypeBf16::mma(vb[j].hi, va[i].hi, part[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const float s = srow[wm + 32 * i + (lane & 31)];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(part[i][j][r], s, acc[i][j][r]);
    }
    __syncthreads();
  }

  // accumulator r of a 32 x 32 block in lane l: row l % 32, column 8 (r / 4) + 4 (l / 32) + r % 4
  typename O::elem* c = (typename O::elem*)p.c + m0 * p.ldc;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = wm + 32 * i + (lane & 31);
    if (m >= rows) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t n = n0 + wn + 32 * j + 8 * (r / 4) + 4 * (lane >> 5) + (r & 3);
        if (n < p.N) c[m * p.ldc + n] = O::cvt(acc[i][j][r]);
      }
  }
}

// ---------------------------------------------------------------------------
// Experts with few rows (decoding): bound by reading the weights, as ragged_few_kernel.  A workgroup
// takes up to 16 MR rows of an expert and 16 output columns; its waves split the blocks of the
// contraction in runs of U, weights go straight to the matrix instructions' registers.
// ---------------------------------------------------------------------------
// ODD: rows that do not start on 4 bytes.
template <typename O, int MR, int U, int WAVES, bool ODD>
__global__ __launch_bounds__(64 * WAVES) void ragged_fp8_few_kernel(RaggedArgs p, uint32_t first) {
  typedef f32x4 Acc;
  __shared__ Acc sums[WAVES][MR][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t ctiles = (uint32_t)((p.N + 15) / 16);
  const uint32_t tile = first + blockIdx.x;
  const int64_t n0 = (int64_t)(tile % ctiles) * 16;
  const RowSpan t = wave_row_tile(p.m_splits, p.G, p.R, 16 * MR, tile / ctiles, false);
  const int g = t.g, rows = t.rows;
  if (g < 0) return;

  const int64_t kb = (p.K + 127) / 128, nb = (p.N + 127) / 128;
  const int sub = lane >> 4;   // 16-code chunk of half a block
  const uint8_t* w = (const uint8_t*)p.b + ((int64_t)g * p.N + min(n0 + (lane & 15), p.N - 1)) * p.K + sub * 16;
  const float* sb = p.sb + ((int64_t)g * nb + n0 / 128) * kb;
  const uint8_t* x[MR];
  const float* sa[MR];
  bool there[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const int64_t r = t.row0 + min(16 * m + (lane & 15), rows - 1);
    const int64_t s = p.row_index != nullptr ? p.row_index[r] : r;
    there[m] = s >= 0 && s < p.S;
    // rows of zeros read the weights' (a place that is there) and drop it
    x[m] = there[m] ? (const uint8_t*)p.a + s * p.lda + sub * 16 : w;
    sa[m] = there[m] ? p.sa + s * kb : sb;
  }
  Acc acc[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) acc[m] = Acc{0, 0, 0, 0};
  // one block: its sum, times the scales
  auto block = [&](const u32x4_t (&wv)[2], const u32x4_t (&xv)[MR][2], const float (&va)[MR], float vb) {
    const Wide w0 = widen_codes(wv[0]), w1 = widen_codes(wv[1]);
#pragma unroll
    for (int m = 0; m < MR; ++m) {
      const u32x4_t none = {0, 0, 0, 0};
      const Wide x0 = widen_codes(there[m] ? xv[m][0] : none), x1 = widen_codes(there[m] ? xv[m][1] : none);
      Acc part = {0, 0, 0, 0};
      part = TypeBf16::mma16(w0.lo, x0.lo, part);
      part = TypeBf16::mma16(w0.hi, x0.hi, part);
      part = TypeBf16::mma16(w1.lo, x1.lo, part);
      part = TypeBf16::mma16(w1.hi, x1.hi, part);
      const float s = (there[m] ? va[m] : 0.f) * vb;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[m][e] = __builtin_fmaf(part[e], s, acc[m][e]);
    }
  };
  auto load = [](const uint8_t* at) {
    if constexpr (ODD) return load16_odd(at);
    u32x4_t v;
    __builtin_memcpy(&v, at, 16);
    return v;
  };
  const int64_t whole = p.K / 128, runs = whole / U;
  for (int64_t run = wave; run < runs; run += WAVES) {
    u32x4_t wv[U][2], xv[U][MR][2];
    float va[U][MR], vb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t b = run * U + i;
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[i][h] = load(w + b * 128 + h * 64);
#pragma unroll
      for (int m = 0; m < MR; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[i][m][h] = load(x[m] + b * 128 + h * 64);
        va[i][m] = sa[m][b];
      }
      vb[i] = sb[b];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) block(wv[i], xv[i], va[i], vb[i]);
  }
  // the blocks that are left, each to the next wave; the last may be short
  for (int64_t b = runs * U + (wave + WAVES - (int)(runs % WAVES)) % WAVES; b < kb; b += WAVES) {
    u32x4_t wv[2], xv[MR][2];
    float va[MR];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = b * 128 + h * 64, n = p.K - at - sub * 16;
      wv[h] = chunk_end<uint8_t>(w + at, n);
#pragma unroll
      for (int m = 0; m < MR; ++m) xv[m][h] = chunk_end<uint8_t>(x[m] + at, n);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) va[m] = sa[m][b];
    block(wv, xv, va, sb[b]);
  }

#pragma unroll
  for (int m = 0; m < MR; ++m) sums[wave][m][lane] = acc[m];
  __syncthreads();
  // token 16 m + lane % 16, columns 4 (lane / 16) + 0..3
  for (int m = wave; m < MR; m += WAVES) {
    Acc sum = sums[0][m][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) sum += sums[v][m][lane];
    const int r = 16 * m + (lane & 15);
    if (r >= rows) continue;
    typename O::elem* c = (typename O::elem*)p.c + (t.row0 + r) * p.ldc;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t n = n0 + 4 * sub + e;
      if (n < p.N) c[n] = O::cvt(sum[e]);
    }
  }
}

namespace {

template <typename O, int TM>
hipError_t launch_fp8_any_rows(const RaggedArgs& p, hipStream_t st) {
  const int64_t blocks = ((p.N + kF8Tile - 1) / kF8Tile) * (p.R / TM + std::min<int64_t>(p.G, p.R));
  return launch_in_parts(blocks, 256, [&](uint32_t first, uint32_t n) {
    ragged_fp8_any_kernel<O, TM><<<dim3(n), dim3(256), 0, st>>>(p, first);
  });
}
template <typename O>
hipError_t launch_fp8_any(const RaggedArgs& p, hipStream_t st) {
  // Low tiles while they add few to what a CU does (half of an expert's last tile empty on average).
  // Measured (us, 64 and 128 rows, by tiles of 128): 3 x 4099 x 1000, 99: 20, 24, 231: 30, 32, 429: 53, 46;
  // 8 x 2048 x 2048, 128: 27, 33, 320: 39, 47, 576: 68, 69; 8 x 4096 x 7168, 160: 76, 100, 384: 109, 124,
  // 640: 210, 161.
  const int64_t tiles = ((p.N + kF8Tile - 1) / kF8Tile) * (p.R / kF8Tile + std::min<int64_t>(p.G, p.R) / 2);
  return tiles <= 400 ? launch_fp8_any_rows<O, 64>(p, st) : launch_fp8_any_rows<O, 128>(p, st);
}

template <typename O, int MR, int U, int WAVES>
hipError_t launch_fp8_few(const RaggedArgs& p, hipStream_t st) {
  const int64_t blocks = (p.R / (16 * MR) + std::min<int64_t>(p.G, p.R)) * ((p.N + 15) / 16);
  // (8 x 4096 x 4098, 16 rows, took 66 us with plain loads, where 4100 took 27)
  const bool odd = (((uintptr_t)p.a | (uintptr_t)p.b) & 3) != 0 || p.K % 4 != 0 || p.lda % 4 != 0;
  return launch_in_parts(blocks, 64 * WAVES, [&](uint32_t first, uint32_t n) {
    if (odd) ragged_fp8_few_kernel<O, MR, U, WAVES, true><<<dim3(n), dim3(64 * WAVES), 0, st>>>(p, first);
    else ragged_fp8_few_kernel<O, MR, U, WAVES, false><<<dim3(n), dim3(64 * WAVES), 0, st>>>(p, first);
  });
}

// Measured (us) by blocks of a run and waves: 8 x 14336 x 4096, 16 rows  1 x 4: 95   2 x 2: 90   2 x 4: 95
// 3 x 4: 95   4 x 4: 99   8 x 4: 113;  128 x 2048 x 7168, 64 rows  123, 123, 121, 126, 133, 161;  4 x 4096 x
// 4096, 4 rows  16, 14, 18, 20, -, -.  Of two waves more fit on a CU.  Where weights are few, 8 waves share them.
template <typename O>
hipError_t launch_fp8_rows(const RaggedArgs& p, hipStream_t st) {
  const int64_t groups = std::min<int64_t>(p.G, p.R);
  const int64_t mean = (p.R + groups - 1) / groups;
  const bool many = groups * ((p.N + 15) / 16) >= 1024;
  if (mean <= 16) return many ? launch_fp8_few<O, 1, 2, 2>(p, st) : launch_fp8_few<O, 1, 2, 8>(p, st);
  if (mean <= 32) return many ? launch_fp8_few<O, 2, 2, 2>(p, st) : launch_fp8_few<O, 2, 2, 8>(p, st);
  return many ? launch_fp8_few<O, 4, 1, 2>(p, st) : launch_fp8_few<O, 4, 1, 8>(p, st);
}

bool fp8_tiles(int out, const RaggedArgs& p) {
  const int64_t osize = out == 0 ? 4 : 2, span = (int64_t)kSpan;
  auto on16 = [](const void* q, int64_t stride) { return (uintptr_t)q % 16 == 0 && stride % 16 == 0; };
  if (out == 0 || !on16(p.a, p.lda) || !on16(p.b, p.K) || !on16(p.c, p.ldc * osize) || p.N * osize % 16 != 0)
    return false;
  const int64_t rows = p.row_index != nullptr ? p.S : 256, kb4 = (p.K + 127) / 128 * 4;
  return 256 * p.K <= span && 256 * p.ldc * osize <= span && rows * p.lda <= span && rows * kb4 <= span && p.S > 0;
}

// Whether the few-rows form takes a product: bound by reading the weights, then by making bf16 of codes
// anew for every 16 columns, about 8 + W (0.08 + 0.0115 m) us for W MB of weights and m rows an expert.
// The large tiles take what their plan says (fp32 sums).  Measured, even experts (here, there):
//    17 (1 x 4096 x 4096)     m 64:  18,  24   96:  26,  32   192:  43,  33
//    34 (8 x 2048 x 2048)     m 32:  17,  27   48:  26,  27    64:  31,  27
//    67 (4 x 4096 x 4096)     m 24:  27,  47   32:  30,  47    48:  48,  47
//   117 (4 x 7168 x 4096)     m 16:  32,  47   24:  44,  47    32:  50,  47
//   134 (64 x 2048 x 1024)    m  8:  28,  33   12:  31,  33    16:  35,  33
//   235 (8 x 4096 x 7168)     m 12:  50,  77   16:  57,  78    32:  87,  78
//   470 (8 x 14336 x 4096)    m  8: 106, 120   12: 119, 120    16: 130, 120
// and with 8-bit sums:
//    17 (1 x 4096 x 4096)     m 32:  11,  20   64:  17,  24    96:  26,  24
//    34 (8 x 2048 x 2048)     m 32:  16,  21   48:  26,  24    96:  58,  24
//    67 (4 x 4096 x 4096)     m 24:  27,  35   32:  31,  35    48:  47,  40
//   117 (4 x 7168 x 4096)     m 12:  29,  37   16:  32,  37    24:  48,  37
//   134 (64 x 2048 x 1024)    m  8:  31,  28   12:  34,  28    16:  38,  28
//   470 (8 x 14336 x 4096)    m  8: 108, 104   12: 119, 120    16: 130, 105
// The any-size form takes about 1.15 us a block while its tiles have a CU each, and more in proportion;
// here, there:
//    12 (3 x 4099 x 1000)     m 48:  16,  17   64:  17,  18    96:  28,  20
//    17 (1 x 4096 x 4096)     m 96:  25,  38  128:  30,  39   192:  42,  39
//    34 (8 x 2048 x 2048)     m 32:  16,  25   48:  25,  26    64:  30,  27
//   235 (8 x 4096 x 7168)     m 16:  55,  76   32:  85,  77    64: 176,  80
bool fp8_few(const RaggedArgs& p, bool tiles, bool fast) {
  const int64_t groups = std::min<int64_t>(p.G, p.R);
  const double mean = (double)p.R / (double)groups, mb = 1e-6 * (double)groups * (double)p.N * (double)p.K;
  if (p.R >= (1 << 20) || mean > 256) return false;
  if (mean <= 8) return true;
  if (tiles && fast) return (mean - 8) * mb <= (mb < 125 ? 1250 : 300);
  const double blocks = (double)((p.N + kF8Tile - 1) / kF8Tile) * (double)(p.R / kF8Tile + groups);
  return 8 + mb * (0.08 + 0.0115 * mean) <=
         (tiles ? ragged_fp8_plan(false, true, p).us : 6 + 1.15 * (double)((p.K + 127) / 128) * std::max(1.0, blocks / 320));
}

}  // namespace

// For results of 16 bits and operands that are contiguous and on 16 bytes.
size_t ragged_fp8_workspace_bytes(int64_t R, int64_t S, int64_t N, int64_t K, int32_t G) {
  RaggedArgs p{};
  p.R = R;
  p.S = S;
  p.N = N;
  p.K = K;
  p.G = G;
  p.lda = K;
  p.ldc = N;
  if (R == 0 || !fp8_tiles(1, p)) return 0;
  for (const bool fast : {false, true})
    if (!fp8_few(p, true, fast) && ragged_fp8_plan(fast, true, p).split) return ragged_split_bytes();
  return 0;
}

hipError_t launch_ragged_gemm_fp8(int out, bool fast, const RaggedArgs& p, size_t ws_bytes, hipStream_t st) {
  const bool tiles = fp8_tiles(out, p);
  if (fp8_few(p, tiles, fast)) {
    if (out == 0) return launch_fp8_rows<OutF32>(p, st);
    return out == 1 ? launch_fp8_rows<OutBf16>(p, st) : launch_fp8_rows<OutF16>(p, st);
  }
  if (tiles) {
    RaggedArgs q = p;
    if (ws_bytes < ragged_split_bytes()) q.ws = nullptr;
    return launch_ragged_fp8_tile(out, fast, q, st);
  }
  if (out == 0) return launch_fp8_any<OutF32>(p, st);
  return out == 1 ? launch_fp8_any<OutBf16>(p, st) : launch_fp8_any<OutF16>(p, st);
}

}  // namespace mx

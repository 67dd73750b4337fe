// Forward products where experts have few rows (decoding): bound by reading
// the weights once.
//
// One workgroup takes up to 16 MR rows of one expert and 16 output columns; its
// waves split the contraction in runs of U 128-byte lines, so that few columns
// still give many loads in flight, and their sums are joined in LDS in a fixed
// order.  Weights go from memory straight to the registers of the matrix
// instruction, as its first operand (16 columns by 64 contraction bytes; rows of
// tokens are the second), at element alignment: no size or stride is special.
// 16 columns and runs of 1 KB read the weights fastest: 8 experts of 14336 x
// 4096 bf16, 16 rows, took 137 us (6.0 TB/s); 32 columns took 178, 64 took 175,
// runs of 512 B 140, and non-temporal loads 155.
#include <algorithm>

#include "ragged_common.h"

namespace mx {

// GATED: 16 gate columns and their 16 up columns, the activation of both (and the
// projections, where p.h is given).  ODD: rows that do not start on 4 bytes.
template <typename T, typename O, int MR, int U, int WAVES, bool GATED = false, bool ODD = false>
__global__ __launch_bounds__(64 * WAVES) void ragged_few_kernel(RaggedArgs p, uint32_t first) {
  typedef typename T::elem E;
  typedef typename T::acc16 Acc;
  constexpr bool kInt8 = sizeof(E) == 1;
  constexpr int NB = GATED ? 2 : 1;   // blocks of 16 weight rows
  static_assert(!GATED || !kInt8, "");
  __shared__ Acc part[WAVES][MR * NB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t cols = GATED ? p.N / 2 : p.N;
  const uint32_t ctiles = (uint32_t)((cols + 15) / 16);
  const uint32_t tile = first + blockIdx.x;
  const int64_t rt = tile / ctiles;
  const int64_t n0 = (int64_t)(tile % ctiles) * 16;

  const RowSpan at = wave_row_tile(p.m_splits, p.G, p.R, 16 * MR, rt, false);
  const int g = at.g, rows = at.rows;
  const int64_t row0 = at.row0;
  if (g < 0) return;

  const int64_t kb = p.K * (int64_t)sizeof(E);
  const int sub = lane >> 4;   // 16-byte chunk of a 64-byte step
  // this lane's weight row and token rows; rows past the end repeat the last
  const uint8_t* w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b)
    w[b] = (const uint8_t*)p.b +
           ((int64_t)g * p.N + b * cols + min(n0 + (lane & 15), cols - 1)) * kb + sub * 16;
  const uint8_t* x[MR];
  int64_t token[MR];   // -1: a row of zeros
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const int64_t r = row0 + min(16 * m + (lane & 15), rows - 1);
    const int64_t s = p.row_index != nullptr ? p.row_index[r] : r;
    token[m] = s >= 0 && s < p.S ? s : -1;
    // any readable row of K values does for a row of zeros: its sums are replaced below
    x[m] = token[m] >= 0 ? (const uint8_t*)p.a + s * p.lda * (int64_t)sizeof(E) + sub * 16 : w[0];
  }

  Acc acc[MR * NB];
#pragma unroll
  for (int m = 0; m < MR * NB; ++m) acc[m] = Acc{0, 0, 0, 0};
  // whole runs of U lines, wave by wave
  const int64_t runs = kb / (128 * U);
  for (int64_t run = wave; run < runs; run += WAVES) {
    u32x4_t wv[2 * U][NB], xv[2 * U][MR];
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) {
      const int64_t at = run * (128 * U) + i * 64;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (ODD) wv[i][b] = load16_odd(w[b] + at);
        else __builtin_memcpy(&wv[i][b], w[b] + at, 16);
      }
#pragma unroll
      for (int m = 0; m < MR; ++m) {
        if constexpr (ODD) xv[i][m] = load16_odd(x[m] + at);
        else __builtin_memcpy(&xv[i][m], x[m] + at, 16);
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * U; ++i)
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[m * NB + b] = T::mma16(wv[i][b], xv[i][m], acc[m * NB + b]);
  }
  // the lines that are left, each to the next wave; the last may be partial
  const int64_t lines = (kb + 127) / 128;
  for (int64_t l = runs * U + (wave + WAVES - (int)(runs % WAVES)) % WAVES; l < lines; l += WAVES) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = l * 128 + h * 64;
      const int64_t n = kb - at - sub * 16;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const u32x4_t wv = chunk_end<E>(w[b] + at, n);
#pragma unroll
        for (int m = 0; m < MR; ++m)
          acc[m * NB + b] = T::mma16(wv, chunk_end<E>(x[m] + at, n), acc[m * NB + b]);
      }
    }
  }

  // Rows of zeros: what they make of this wave's share of the weights, NaN where one
  // is infinite or NaN, in a pass of its own.  Clearing such rows' values in the loops
  // above instead costs every call: 64 rows of 2 x 4096 x 4096 in 8-bit integers took
  // 24.0 us so, 22.9 without.
  bool gone = false;
#pragma unroll
  for (int m = 0; m < MR; ++m) gone |= token[m] < 0;
  if (__ballot(gone) != 0) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      Acc none = {0, 0, 0, 0};
      if (!kInt8)
        for (int64_t l = wave; l < lines; l += WAVES)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t at = l * 128 + h * 64;
            none = T::mma16(chunk_end<E>(w[b] + at, kb - at - sub * 16), u32x4_t{0, 0, 0, 0}, none);
          }
#pragma unroll
      for (int m = 0; m < MR; ++m)
        if (token[m] < 0) acc[m * NB + b] = none;
    }
  }

#pragma unroll
  for (int m = 0; m < MR * NB; ++m) part[wave][m][lane] = acc[m];
  __syncthreads();
  // block m: token 16 m + lane % 16, columns 4 (lane / 16) + 0..3
  for (int m = wave; m < MR; m += WAVES) {
    Acc sum = part[0][m * NB][lane], up = part[0][m * NB + NB - 1][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) {
      sum += part[v][m * NB][lane];
      if constexpr (GATED) up += part[v][m * NB + 1][lane];
    }
    const int r = 16 * m + (lane & 15);
    if (r >= rows) continue;
    int64_t s = -1;
#pragma unroll
    for (int j = 0; j < MR; ++j)
      if (j == m) s = token[j];
    typename O::elem* c = (typename O::elem*)p.c + (row0 + r) * p.ldc;
    const float sa = kInt8 && s >= 0 ? p.sa[s] : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t n = n0 + 4 * sub + e;
      if (n >= cols) continue;
      if constexpr (GATED) {
        c[n] = O::cvt(gated(sum[e], up[e]));
        if (p.h != nullptr) {
          typename O::elem* h = (typename O::elem*)p.h + (row0 + r) * p.N + n;
          h[0] = O::cvt(sum[e]);
          h[cols] = O::cvt(up[e]);
        }
        continue;
      }
      float v = (float)sum[e];
      if constexpr (kInt8) v = scaled<O>(sum[e], sa, p.sb[(int64_t)g * p.N + n]);
      c[n] = O::cvt(v);
    }
  }
}

namespace {

template <typename T, typename O, int MR, int U, int WAVES, bool GATED = false, bool ODD = false>
hipError_t launch_few(const RaggedArgs& p, hipStream_t st) {
  const int64_t rt = p.R / (16 * MR) + std::min<int64_t>(p.G, p.R);
  const int64_t blocks = rt * (((GATED ? p.N / 2 : p.N) + 15) / 16);
  return launch_in_parts(blocks, 64 * WAVES, [&](uint32_t first, uint32_t n) {
    ragged_few_kernel<T, O, MR, U, WAVES, GATED, ODD><<<dim3(n), dim3(64 * WAVES), 0, st>>>(p, first);
  });
}

template <typename T, typename O>
hipError_t launch_rows(const RaggedArgs& p, hipStream_t st) {
  // rows of an expert on average, over experts that can have any
  const int64_t groups = std::min<int64_t>(p.G, p.R);
  const int64_t mean = (p.R + groups - 1) / groups;
  // Four workgroups of four waves for each CU fill it; with fewer workgroups
  // twice the waves share the contraction, in shorter runs.  Runs of 8 lines want
  // a contraction that has one for each wave.
  const bool many = groups * ((p.N + 15) / 16) >= 1024;
  const bool longk = p.K * (int64_t)sizeof(typename T::elem) >= 4 * 8 * 128;
  if (mean <= 16) {
    if (!many) return launch_few<T, O, 1, 2, 8>(p, st);
    return longk ? launch_few<T, O, 1, 8, 4>(p, st) : launch_few<T, O, 1, 2, 4>(p, st);
  }
  if (mean <= 32) return many ? launch_few<T, O, 2, 4, 4>(p, st) : launch_few<T, O, 2, 2, 8>(p, st);
  return many ? launch_few<T, O, 4, 2, 4>(p, st) : launch_few<T, O, 4, 2, 8>(p, st);
}

// Gated: twice the loads in flight for a row of tokens.  Measured (us, 2 to 8 lines by 4 or 8 waves):
//   8 x 28672 x 4096, 16 rows    2 x 4: 285   4 x 4: 294   8 x 4: 295   2 x 8: 276   3 x 8: 278   4 x 8: 285
//   64 x 2048 x 2048, 64 rows          99          108           98           118          109            96
// Four runs and more for a wave, or all of its share at once, read fastest; two runs wait for each other.
template <typename T, typename O, bool ODD>
hipError_t launch_rows_gated(const RaggedArgs& p, hipStream_t st) {
  const int64_t groups = std::min<int64_t>(p.G, p.R);
  const int64_t mean = (p.R + groups - 1) / groups;
  const bool many = groups * ((p.N / 2 + 15) / 16) >= 1024;
  const int64_t lines = p.K * (int64_t)sizeof(typename T::elem) / 128;
  if (mean <= 16) {
    if (!many || lines >= 4 * 2 * 8) return launch_few<T, O, 1, 2, 8, true, ODD>(p, st);
    return lines >= 4 * 8 ? launch_few<T, O, 1, 4, 8, true, ODD>(p, st) : launch_few<T, O, 1, 2, 4, true, ODD>(p, st);
  }
  if (mean <= 32) return many ? launch_few<T, O, 2, 2, 4, true, ODD>(p, st) : launch_few<T, O, 2, 2, 8, true, ODD>(p, st);
  return many ? launch_few<T, O, 4, 1, 4, true, ODD>(p, st) : launch_few<T, O, 4, 1, 8, true, ODD>(p, st);
}

}  // namespace

// Rows off 4 bytes: 8 x 8192 x 4097, 16 rows, took 220 us with plain loads, where 4098 took 124.
hipError_t launch_ragged_few_gated(bool f16, const RaggedArgs& p, hipStream_t st) {
  const bool odd = (((uintptr_t)p.a | (uintptr_t)p.b) & 3) != 0 || p.K % 2 != 0 || p.lda % 2 != 0;
  if (f16) return odd ? launch_rows_gated<TypeF16, OutF16, true>(p, st) : launch_rows_gated<TypeF16, OutF16, false>(p, st);
  return odd ? launch_rows_gated<TypeBf16, OutBf16, true>(p, st) : launch_rows_gated<TypeBf16, OutBf16, false>(p, st);
}

hipError_t launch_ragged_few(bool f16, int out, const RaggedArgs& p, hipStream_t st) {
  if (f16)
    return out == 0 ? launch_rows<TypeF16, OutF32>(p, st) : launch_rows<TypeF16, OutF16>(p, st);
  return out == 0 ? launch_rows<TypeBf16, OutF32>(p, st) : launch_rows<TypeBf16, OutBf16>(p, st);
}

hipError_t launch_ragged_few_int8(int out, const RaggedArgs& p, hipStream_t st) {
  if (out == 0) return launch_rows<TypeI8, OutF32>(p, st);
  if (out == 1) return launch_rows<TypeI8, OutBf16>(p, st);
  return launch_rows<TypeI8, OutF16>(p, st);
}

}  // namespace mx

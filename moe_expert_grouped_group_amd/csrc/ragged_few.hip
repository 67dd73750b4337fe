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

// 16 bytes at p, of which the contraction holds n (n <= 0: none): zeros behind.
template <typename E>
__device__ __forceinline__ u32x4_t chunk_end(const uint8_t* p, int64_t n) {
  u32x4_t v = {0, 0, 0, 0};
  if (n >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else if (n > 0) {
    E e[16 / sizeof(E)];
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(E)); ++i)
      e[i] = (int64_t)(i * sizeof(E)) < n ? ((const E*)p)[i] : (E)0;
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

template <typename T, typename O, int MR, int U, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void ragged_few_kernel(RaggedArgs p, uint32_t first) {
  typedef typename T::elem E;
  typedef typename T::acc16 Acc;
  constexpr bool kInt8 = sizeof(E) == 1;
  __shared__ Acc part[WAVES][MR][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t ctiles = (uint32_t)((p.N + 15) / 16);
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
  const uint8_t* w = (const uint8_t*)p.b +
                     ((int64_t)g * p.N + min(n0 + (lane & 15), p.N - 1)) * kb + sub * 16;
  const uint8_t* x[MR];
  int64_t token[MR];   // -1: a row of zeros
#pragma unroll
  for (int m = 0; m < MR; ++m) {
    const int64_t r = row0 + min(16 * m + (lane & 15), rows - 1);
    const int64_t s = p.row_index != nullptr ? p.row_index[r] : r;
    token[m] = s >= 0 && s < p.S ? s : -1;
    // any readable row of K values does for a row of zeros: its sums are replaced below
    x[m] = token[m] >= 0 ? (const uint8_t*)p.a + s * p.lda * (int64_t)sizeof(E) + sub * 16 : w;
  }

  Acc acc[MR];
#pragma unroll
  for (int m = 0; m < MR; ++m) acc[m] = Acc{0, 0, 0, 0};
  // whole runs of U lines, wave by wave
  const int64_t runs = kb / (128 * U);
  for (int64_t run = wave; run < runs; run += WAVES) {
    u32x4_t wv[2 * U], xv[2 * U][MR];
#pragma unroll
    for (int i = 0; i < 2 * U; ++i) {
      const int64_t at = run * (128 * U) + i * 64;
      __builtin_memcpy(&wv[i], w + at, 16);
#pragma unroll
      for (int m = 0; m < MR; ++m) __builtin_memcpy(&xv[i][m], x[m] + at, 16);
    }
#pragma unroll
    for (int i = 0; i < 2 * U; ++i)
#pragma unroll
      for (int m = 0; m < MR; ++m) acc[m] = T::mma16(wv[i], xv[i][m], acc[m]);
  }
  // the lines that are left, each to the next wave; the last may be partial
  const int64_t lines = (kb + 127) / 128;
  for (int64_t l = runs * U + (wave + WAVES - (int)(runs % WAVES)) % WAVES; l < lines; l += WAVES) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = l * 128 + h * 64;
      const int64_t n = kb - at - sub * 16;
      const u32x4_t wv = chunk_end<E>(w + at, n);
#pragma unroll
      for (int m = 0; m < MR; ++m) acc[m] = T::mma16(wv, chunk_end<E>(x[m] + at, n), acc[m]);
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
    Acc none = {0, 0, 0, 0};
    if (!kInt8)
      for (int64_t l = wave; l < lines; l += WAVES)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t at = l * 128 + h * 64;
          none = T::mma16(chunk_end<E>(w + at, kb - at - sub * 16), u32x4_t{0, 0, 0, 0}, none);
        }
#pragma unroll
    for (int m = 0; m < MR; ++m)
      if (token[m] < 0) acc[m] = none;
  }

#pragma unroll
  for (int m = 0; m < MR; ++m) part[wave][m][lane] = acc[m];
  __syncthreads();
  // block m: token 16 m + lane % 16, columns 4 (lane / 16) + 0..3
  for (int m = wave; m < MR; m += WAVES) {
    Acc sum = part[0][m][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) sum += part[v][m][lane];
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
      if (n >= p.N) continue;
      float v = (float)sum[e];
      if constexpr (kInt8) v = scaled<O>(sum[e], sa, p.sb[(int64_t)g * p.N + n]);
      c[n] = O::cvt(v);
    }
  }
}

namespace {

template <typename T, typename O, int MR, int U, int WAVES>
hipError_t launch_few(const RaggedArgs& p, hipStream_t st) {
  const int64_t rt = p.R / (16 * MR) + std::min<int64_t>(p.G, p.R);
  const int64_t blocks = rt * ((p.N + 15) / 16);
  return launch_in_parts(blocks, 64 * WAVES, [&](uint32_t first, uint32_t n) {
    ragged_few_kernel<T, O, MR, U, WAVES><<<dim3(n), dim3(64 * WAVES), 0, st>>>(p, first);
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

}  // namespace

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

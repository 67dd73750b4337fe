// Shared pieces of the products grouped by expert with ragged row counts
// (ragged.hip): element types, the expert lookup from the device splits, and
// the output conversion.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"

namespace mx {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRaggedMaxGroups = 1024;

// Workgroups 0 .. blocks - 1 (below 2^32) of `threads` threads.  A launch holds fewer than
// 2^32 threads, and one of more goes wrong without an error: larger grids go in parts, fn
// launching `n` workgroups from number `first` on.
template <typename F>
hipError_t launch_in_parts(int64_t blocks, int threads, F fn) {
  const int64_t most = 0xFFFFFFFFll / threads;
  for (int64_t first = 0; first < blocks; first += most) {
    fn((uint32_t)first, (uint32_t)std::min(most, blocks - first));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// The arguments of one product.  X, dY and W are row-major with a contiguous
// last dimension; strides are in elements.
struct RaggedArgs {
  const void* a;        // NT: X [S, K]; NN, TN: dY [R, N]
  const void* b;        // NT, NN: W [G, N, K]; TN: X [S, K]
  void* c;              // NT [R, N], NN [R, K], TN [G, N, K]
  int64_t lda, ldb, ldc;
  int64_t R, S;         // rows of the product; rows of X
  int64_t N, K;
  const int64_t* m_splits;
  const int32_t* row_index;   // NULL: row r of the product is row r of X
  const float* sa;      // int8: scale of each row of X [S]
  const float* sb;      // int8: scale of each output channel [G, N]
  int32_t G;
  // for the large tiles
  int64_t con;          // NT, NN: contraction with its zero padding
  int64_t ccols;        // columns that a row of C has room for
  void* ws;             // partial sums of split tiles (large tiles), or NULL
};

// Forward products of experts with few rows (ragged_few.hip).
hipError_t launch_ragged_few(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_few_int8(int out, const RaggedArgs& p, hipStream_t st);
// The large-tile form (ragged_tile.h), by layout.
hipError_t launch_ragged_tile_nt(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_nn(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_tn(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_int8(int out, const RaggedArgs& p, hipStream_t st);
size_t ragged_split_bytes();   // a partial 256 x 256 tile for each CU

// Longest range of a bounded operand (32-bit offsets, less what marks a lane that
// is out of it).
constexpr uint64_t kSpan = 0xFFFFFE00ull;

// Element types: every one is handled as 16-byte chunks of the contraction
// (8 values of 16 bits, 16 of 8), which is what one lane hands to one
// matrix instruction.  Which contraction indices a lane's chunk holds does not
// matter as long as both operands hold the same ones.
struct TypeBf16 {
  typedef uint16_t elem;
  typedef f32x16 acc;
  typedef __bf16 vec __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ acc mma(u32x4_t a, u32x4_t b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(vec, a),
                                                   __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
  // 16 x 16 results, 64 contraction bytes
  typedef f32x4 acc16;
  static __device__ __forceinline__ acc16 mma16(u32x4_t a, u32x4_t b, acc16 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vec, a),
                                                   __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
};
struct TypeF16 {
  typedef uint16_t elem;
  typedef f32x16 acc;
  typedef _Float16 vec __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ acc mma(u32x4_t a, u32x4_t b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(vec, a),
                                                  __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
  // 16 x 16 results, 64 contraction bytes
  typedef f32x4 acc16;
  static __device__ __forceinline__ acc16 mma16(u32x4_t a, u32x4_t b, acc16 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vec, a),
                                                  __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
};
// 8-bit integers: products and sums are exact in 32 bits for K <= 131071.
struct TypeI8 {
  typedef uint8_t elem;
  typedef i32x16 acc;
  static __device__ __forceinline__ acc mma(u32x4_t a, u32x4_t b, acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
  typedef i32x4 acc16;
  static __device__ __forceinline__ acc16 mma16(u32x4_t a, u32x4_t b, acc16 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

// Output conversion: one rounding (nearest even) of the fp32 value.
struct OutF32 {
  typedef float elem;
  static __device__ __forceinline__ float cvt(float v) { return v; }
};
struct OutBf16 {
  typedef uint16_t elem;
  static __device__ __forceinline__ uint16_t cvt(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
  }
};
struct OutF16 {
  typedef uint16_t elem;
  static __device__ __forceinline__ uint16_t cvt(float v) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  }
};

// 8-bit integers: an exact sum, rounded to fp32, times the row's and the channel's scale,
// rounded to fp32 before the output's conversion in every form and type.  Left to itself
// the compiler multiplies and converts to fp16 in one instruction, which rounds once: one
// result in 20000 differs in its last place.
template <typename O>
__device__ __forceinline__ float scaled(int sum, float row, float channel) {
  float v = (float)sum * row * channel;
  if (std::is_same<O, OutF16>::value) asm("" : "+v"(v));
  return v;
}

// A split as the kernels take it: negative ones count as empty, and none is
// longer than the R rows there are, so that sums cannot overflow.
__device__ __forceinline__ int64_t split_rows(const int64_t* m_splits, int g, int64_t R) {
  const int64_t m = m_splits[g];
  return m < 0 ? 0 : (m < R ? m : R);
}

// The expert, first row and row count of row tile rt (tiles of `tile` rows), by one
// wave; g = -1 past the last.  total: row tiles of all experts (only if asked for).
struct RowSpan {
  int g, rows;
  int64_t row0, total;
};
__device__ __forceinline__ RowSpan wave_row_tile(const int64_t* m_splits, int G, int64_t R, int tile,
                                                 int64_t rt, bool want_total) {
  const int lane = threadIdx.x & 63;
  RowSpan s;
  s.g = -1;
  s.rows = 0;
  s.row0 = 0;
  int64_t before_r = 0, before_t = 0;
  for (int base = 0; base < G; base += 64) {
    const int e = base + lane;
    const int64_t m = e < G ? split_rows(m_splits, e, R) : 0;
    // rows, then tiles, of the experts up to this one
    int64_t r = m;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t u = __shfl_up(r, d, 64);
      if (lane >= d) r += u;
    }
    const int64_t hi = min(before_r + r, R), lo = min(before_r + r - m, R);   // cut at R
    const int64_t t = (hi - lo + tile - 1) / tile;
    int64_t ts = t;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t u = __shfl_up(ts, d, 64);
      if (lane >= d) ts += u;
    }
    const int64_t first = before_t + ts - t;
    const uint64_t who = __ballot(rt >= first && rt < first + t);
    if (who != 0) {
      const int src = __builtin_ctzll(who);
      s.g = base + src;
      s.row0 = __shfl(lo + (rt - first) * tile, src, 64);
      s.rows = (int)min((int64_t)tile, __shfl(hi, src, 64) - s.row0);
      if (!want_total) break;
    }
    before_r += __shfl(r, 63, 64);
    before_t += __shfl(ts, 63, 64);
  }
  s.total = before_t;
  return s;
}

}  // namespace mx

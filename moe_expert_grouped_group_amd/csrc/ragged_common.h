// Shared pieces of the products grouped by expert with ragged row counts
// (ragged.hip): element types, the expert lookup from the device splits, and
// the output conversion.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kernels.h"

namespace mx {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRaggedMaxGroups = 1024;

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
};

// Forward products of experts with few rows (ragged_few.hip).
hipError_t launch_ragged_few(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_few_int8(int out, const RaggedArgs& p, hipStream_t st);
// The large-tile form (ragged_tile.h), by layout.
hipError_t launch_ragged_tile_nt(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_nn(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_tn(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_int8(int out, const RaggedArgs& p, hipStream_t st);

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
};
struct TypeF16 {
  typedef uint16_t elem;
  typedef f32x16 acc;
  typedef _Float16 vec __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ acc mma(u32x4_t a, u32x4_t b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(vec, a),
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

// A split as the kernels take it: negative ones count as empty, and none is
// longer than the R rows there are, so that sums cannot overflow.
__device__ __forceinline__ int64_t split_rows(const int64_t* m_splits, int g, int64_t R) {
  const int64_t m = m_splits[g];
  return m < 0 ? 0 : (m < R ? m : R);
}

}  // namespace mx

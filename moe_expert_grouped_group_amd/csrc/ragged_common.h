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
                        // fp8: scales of blocks of 128, sa [S, K / 128], sb [G, N / 128, K / 128] (rounded up)
  int32_t G;
  // for the large tiles
  int64_t con;          // NT, NN: contraction with its zero padding
  int64_t ccols;        // columns that a row of C has room for
  void* ws;             // partial sums of split tiles (large tiles), or NULL
  // gated products (Epilogue): both projections [R, 2F], contiguous
  void* h;              // kGated: written unless NULL; kGatedBwd: read
  void* act;            // kGatedBwd: the activation [R, F], contiguous, or NULL
};

// A copy, member by member: of an assignment the compiler makes private arrays that it then puts into LDS,
// and for their addresses every wave reads the launch's packet in the host's memory, one XCD after the
// other: up to 12 us before the last one's workgroups began.
__device__ __forceinline__ void copy_args(RaggedArgs& to, const RaggedArgs& p) {
  to.a = p.a, to.b = p.b, to.c = p.c;
  to.lda = p.lda, to.ldb = p.ldb, to.ldc = p.ldc;
  to.R = p.R, to.S = p.S, to.N = p.N, to.K = p.K;
  to.m_splits = p.m_splits, to.row_index = p.row_index;
  to.sa = p.sa, to.sb = p.sb;
  to.G = p.G;
  to.con = p.con, to.ccols = p.ccols;
  to.ws = p.ws, to.h = p.h, to.act = p.act;
}

// What becomes of a product's sums.
//  kGated (NT, W [G, 2F, K] gate rows then up rows): C[r, f] = silu(z[r, f]) z[r, F + f], z the
//    sums; kGatedKeep writes h = z too.
//  kGatedBwd (NN, K = F; h given): the sums are da; C [R, 2F] = da up silu'(gate) | da silu(gate),
//    act = silu(gate) up.
// Everything from the fp32 sums, each result rounded once.
enum Epilogue { kPlain = 0, kGated = 1, kGatedKeep = 2, kGatedBwd = 3 };

// Forward products of experts with few rows (ragged_few.hip).
hipError_t launch_ragged_few(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_few_int8(int out, const RaggedArgs& p, hipStream_t st);
// The large-tile form (ragged_tile.h), by layout.
hipError_t launch_ragged_tile_nt(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_nn(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_tn(bool f16, int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_int8(int out, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_few_gated(bool f16, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_gated(bool f16, const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_gated_f16(const RaggedArgs& p, hipStream_t st);
hipError_t launch_ragged_tile_gated_bwd(bool f16, const RaggedArgs& p, hipStream_t st);
// 8-bit floating point (ragged_fp8.hip has the formula, ragged_fp8_tile.hip the large tiles).
hipError_t launch_ragged_fp8_tile(int out, bool fast, const RaggedArgs& p, hipStream_t st);
// Rows of a tile, whether tiles may be split, about how long it takes (us; fp32 sums only).
struct Fp8Plan {
  int rows;
  bool split;
  double us;
};
Fp8Plan ragged_fp8_plan(bool fast, bool can_split, const RaggedArgs& p);
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

// The value of 16 stored bits.
template <typename T>
__device__ __forceinline__ float widen(uint16_t v) {
  if constexpr (std::is_same<T, TypeF16>::value) return (float)__builtin_bit_cast(_Float16, v);
  else return __uint_as_float((uint32_t)v << 16);
}

// 8 codes of 8-bit floating point (e4m3) as bf16 values: exact, e4m3 has 3 bits behind the leading one.
__device__ __forceinline__ u32x4_t widen_codes8(uint32_t lo, uint32_t hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return u32x4_t{__builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
                 __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
                 __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
                 __builtin_bit_cast(uint32_t, (bf16x2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true))};
}

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

// 16 bytes at any address, from the dwords that hold them (each holds one of the bytes, so it may be
// read): a load that is not on 4 bytes takes two to three times as long as one that is.
__device__ __forceinline__ u32x4_t load16_odd(const uint8_t* p) {
  const uint32_t off = (uint32_t)(uintptr_t)p & 3u;
  const uint32_t* w = (const uint32_t*)(p - off);
  u32x4_t v;
  __builtin_memcpy(&v, __builtin_assume_aligned(w, 4), 16);
  const uint32_t last = w[off != 0 ? 4 : 3];
  return u32x4_t{__builtin_amdgcn_alignbyte(v[1], v[0], off), __builtin_amdgcn_alignbyte(v[2], v[1], off),
                 __builtin_amdgcn_alignbyte(v[3], v[2], off), __builtin_amdgcn_alignbyte(last, v[3], off)};
}

// silu(g) = g sigmoid(g) with the hardware's exponential and reciprocal, 1 ulp each, ahead
// of a rounding to 16 bits.  exp2 gives infinity for g below -88: sigmoid 0.
__device__ __forceinline__ float sigmoid_of(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}
__device__ __forceinline__ float gated(float gate, float up) { return gate * sigmoid_of(gate) * up; }
struct GatedGrad {
  float gate, up, act;
};
// silu'(g) = s (1 + g (1 - s)), s = sigmoid(g)
__device__ __forceinline__ GatedGrad gated_grad(float da, float gate, float up) {
  const float s = sigmoid_of(gate), silu = gate * s;
  GatedGrad r;
  r.gate = da * up * (s + silu * (1.f - s));
  r.up = da * silu;
  r.act = silu * up;
  return r;
}

// A split as the kernels take it: negative ones count as empty, and none is
// longer than the R rows there are, so that sums cannot overflow.
__device__ __forceinline__ int64_t split_rows(const int64_t* m_splits, int g, int64_t R) {
  const int64_t m = m_splits[g];
  return m < 0 ? 0 : (m < R ? m : R);
}

// Inclusive sums over the wave's lanes, all of them active; MOST: none past `most` (below 2^31).
template <bool MOST>
__device__ __forceinline__ uint32_t wave_sums(uint32_t v, uint32_t most) {
  auto add = [&](uint32_t u) { v = MOST ? min(v + u, most) : v + u; };
  add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));   // row_shr: 1, 2, 4, 8
  add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
  add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
  add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
  add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // row_bcast: 15, 31
  add((uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
  return v;
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
  const uint32_t most = (uint32_t)R;
  RowSpan s;
  s.g = -1;
  s.rows = 0;
  s.row0 = 0;
  uint32_t before_r = 0;
  int64_t before_t = 0;
  for (int base = 0; base < G; base += 64) {
    const int e = base + lane;
    // rows, then tiles, of the experts up to this one, cut at R
    const uint32_t r = wave_sums<true>(e < G ? (uint32_t)split_rows(m_splits, e, R) : 0u, most);
    const uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)r, 0x138, 0xF, 0xF, false);   // wave_shr: 1
    const uint32_t hi = min(before_r + r, most), lo = min(before_r + before, most);
    const uint32_t t = (hi - lo + (uint32_t)tile - 1) / (uint32_t)tile;
    const uint32_t ts = wave_sums<false>(t, 0);
    const int64_t first = before_t + ts - t;
    const uint64_t who = __ballot(rt >= first && rt < first + t);
    if (who != 0) {
      const int src = __builtin_ctzll(who);
      s.g = base + src;
      const int64_t tiles = __builtin_amdgcn_readlane((int)(uint32_t)(rt - first), src);
      s.row0 = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)lo, src) + tiles * tile;
      s.rows = (int)min((int64_t)tile, (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, src) - s.row0);
      if (!want_total) break;
    }
    before_r = min(before_r + (uint32_t)__builtin_amdgcn_readlane((int)r, 63), most);
    before_t += (uint32_t)__builtin_amdgcn_readlane((int)ts, 63);
  }
  s.total = before_t;
  return s;
}

}  // namespace mx

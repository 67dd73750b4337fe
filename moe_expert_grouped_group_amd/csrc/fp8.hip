// Tensors quantized to 8-bit floating point (e4m3) with a scale for each block of 128.
//
//   scale = max|x| / 448 over the block, in fp32 (nearest)
//   q     = the e4m3 value nearest to x / scale, ties to even, at most 448 in size
//
// Tokens have blocks of 1 x 128, weights of 128 x 128; a row's (and a weight's) last block may
// be short.  A block of zeros has scale 0, one with an infinity or NaN has scale NaN, codes 0.
// Bound by memory: x is read once, held in registers between the maximum and the codes.
#include <algorithm>

#include "fp8_quotient.h"
#include "ragged_common.h"

namespace mx {

constexpr float kE4m3Max = 448.f;

// Maximum over the 16 lanes of a row, in all of them.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  // row_ror: 8, 4, 2, 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false));
  return v;
}

// Largest sizes of 8 values by halves of words, as bits of their type without the sign: bits order
// like sizes, infinities and NaN above all.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2 max_bits(u32x4_t v, u16x2 m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
  return m;
}
__device__ __forceinline__ uint32_t larger(u16x2 m) { return m[0] > m[1] ? m[0] : m[1]; }

struct BlockScale {
  float scale, low, high;   // the inverse, less and more 2^-21 of it
  bool zero;    // codes are 0 (no values, or no number among them)
  bool small;   // scales near the smallest numbers: every code by the exact way
};
template <typename T>
__device__ __forceinline__ BlockScale block_scale(uint32_t bits) {
  constexpr uint32_t kInf = std::is_same<T, TypeF16>::value ? 0x7C00u : 0x7F80u;
  BlockScale b;
  const float top = widen<T>((uint16_t)bits);
  b.zero = bits == 0 || bits >= kInf;
  b.small = top < 0x1p-90f;
  // top / 448: the product with the inverse and one correction are correctly rounded, but not
  // where numbers lose bits
  constexpr float kInverse = 1.f / kE4m3Max;
  const float near = top * kInverse;
  b.scale = __builtin_fmaf(__builtin_fmaf(-near, kE4m3Max, top), kInverse, near);
  if (b.small) b.scale = top / kE4m3Max;
  if (b.zero) b.scale = bits == 0 ? 0.f : __builtin_nanf("");
  const float inverse = __builtin_amdgcn_rcpf(b.scale);
  b.low = inverse * (1.f - 0x1p-21f);
  b.high = inverse * (1.f + 0x1p-21f);
  return b;
}

__device__ __forceinline__ uint2 convert(const float (&y)[8]) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// 8 values to codes.  The quotient lies between the products with the two inverses (the hardware's
// is off by 2^-23 of it, each product by 2^-24): where both give the same code, it is the quotient's.
// The rest goes the exact way, one wave in 20 on normal values.
template <typename T>
__device__ __forceinline__ uint2 codes_of(u32x4_t v, const BlockScale& b) {
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = widen<T>((uint16_t)(v[i / 2] >> (16 * (i & 1))));
    y[i] = x[i] * b.low;
  }
  const uint2 one = convert(y);
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i] * b.high;
  uint2 codes = convert(y);
  const bool differ = (one.x != codes.x) | (one.y != codes.y) | b.small;
  if (differ & !b.zero) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = __builtin_amdgcn_fmed3f(exact_quotient(x[i], b.scale), -kE4m3Max, kE4m3Max);
    codes = convert(y);
  }
  return b.zero ? make_uint2(0u, 0u) : codes;
}

// 8 codes at any alignment, the first n of them.
__device__ __forceinline__ void store_codes(uint8_t* q, uint2 c, int64_t n) {
  if (n >= 8) {
    __builtin_memcpy(q, &c, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// n / d for n below 2^31, by the division by invariant integers of Granlund and Montgomery (1994):
// (n + the high half of n magic) >> shift.
struct Divide {
  uint32_t magic, shift;
  static Divide by(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return Divide{(uint32_t)(((((1ull << l) - d) << 32) / d) + 1), l};
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, magic) + n) >> shift; }
};

// 8 values of a row from `left` before its end; WHOLE: all or none.
template <bool WHOLE>
__device__ __forceinline__ u32x4_t load_values(const uint16_t* p, int64_t left) {
  if constexpr (WHOLE) {
    u32x4_t v = {0, 0, 0, 0};
    if (left > 0) __builtin_memcpy(&v, p, 16);
    return v;
  } else {
    return chunk_end<uint16_t>((const uint8_t*)p, left * 2);
  }
}
template <bool WHOLE>
__device__ __forceinline__ void store_values(uint8_t* q, uint2 c, int64_t left) {
  if constexpr (!WHOLE) store_codes(q, c, left);
  else if (left > 0) __builtin_memcpy(q, &c, 8);
}

// Tokens: 16 lanes a block, two blocks of a lane's in flight (8192 x 4096: 29.9 us, with four 31.8).  WHOLE: K is a multiple of 8.  LONG:
// block numbers past 31 bits.
constexpr int kFp8Unroll = 2;
template <typename T, bool WHOLE, bool LONG>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(const uint16_t* x, int64_t ldx, int64_t K, int64_t nb,
                                                           Divide by_nb, int64_t blocks, uint8_t* q, float* scale) {
  const int sub = threadIdx.x & 15;
  const int64_t step = (int64_t)gridDim.x * 16;
  for (int64_t first = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); first < blocks; first += step * kFp8Unroll) {
    u32x4_t v[kFp8Unroll];
    int64_t row[kFp8Unroll], at[kFp8Unroll];
#pragma unroll
    for (int u = 0; u < kFp8Unroll; ++u) {
      const int64_t b = first + step * u;
      if constexpr (LONG) row[u] = b / nb;
      else row[u] = by_nb((uint32_t)b);
      at[u] = b < blocks ? (b - row[u] * nb) * 128 + sub * 8 : K;
      if (b >= blocks) row[u] = 0;
      v[u] = load_values<WHOLE>(x + row[u] * ldx + at[u], K - at[u]);
    }
#pragma unroll
    for (int u = 0; u < kFp8Unroll; ++u) {
      if (first + step * u >= blocks) break;   // the same for the 16 lanes of a block
      const BlockScale b = block_scale<T>(row_max(larger(max_bits(v[u], u16x2{0, 0}))));
      store_values<WHOLE>(q + row[u] * K + at[u], codes_of<T>(v[u], b), K - at[u]);
      if (sub == 0) scale[first + step * u] = b.scale;
    }
  }
}

// Weights: a workgroup a block, 16 rows at a time, the block in registers.
template <typename T, bool WHOLE>
__global__ __launch_bounds__(256) void quantize_fp8_weight_kernel(const uint16_t* w, int64_t N, int64_t K,
                                                                  uint32_t nb, uint32_t kb, uint8_t* q,
                                                                  float* scale, uint32_t first) {
  __shared__ uint32_t top[4];
  const uint32_t block = first + blockIdx.x;
  const uint32_t k0 = block % kb, rest = block / kb, n0 = rest % nb, g = rest / nb;
  const int64_t k = (int64_t)k0 * 128 + (threadIdx.x & 15) * 8;
  const int64_t row0 = (int64_t)n0 * 128 + (threadIdx.x >> 4);
  u32x4_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    v[i] = load_values<WHOLE>(w + ((int64_t)g * N + n) * K + k, n < N ? K - k : 0);
  }
  u16x2 halves = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) halves = max_bits(v[i], halves);
  uint32_t m = row_max(larger(halves));
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
  const BlockScale b = block_scale<T>(max(max(top[0], top[1]), max(top[2], top[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    if (n < N) store_values<WHOLE>(q + ((int64_t)g * N + n) * K + k, codes_of<T>(v[i], b), K - k);
  }
  if (threadIdx.x == 0) scale[((int64_t)g * nb + n0) * kb + k0] = b.scale;
}

hipError_t launch_quantize_fp8(const void* x, bool f16, int64_t T, int64_t K, int64_t ldx, uint8_t* q,
                               float* scale, hipStream_t st) {
  const int64_t nb = (K + 127) / 128, blocks = T * nb;
  const dim3 grid((uint32_t)std::min<int64_t>((blocks + 16 * kFp8Unroll - 1) / (16 * kFp8Unroll), 65536));
  const bool whole = K % 8 == 0, is_long = blocks + 16 * 65536ll * kFp8Unroll >= (1ll << 31);
  const Divide by = is_long ? Divide{} : Divide::by((uint32_t)nb);
#define MX_QUANTIZE(T, WHOLE, LONG) \
  quantize_fp8_kernel<T, WHOLE, LONG><<<grid, dim3(256), 0, st>>>((const uint16_t*)x, ldx, K, nb, by, blocks, q, scale)
  if (is_long) {
    if (f16) MX_QUANTIZE(TypeF16, false, true);
    else MX_QUANTIZE(TypeBf16, false, true);
  } else if (whole) {
    if (f16) MX_QUANTIZE(TypeF16, true, false);
    else MX_QUANTIZE(TypeBf16, true, false);
  } else {
    if (f16) MX_QUANTIZE(TypeF16, false, false);
    else MX_QUANTIZE(TypeBf16, false, false);
  }
#undef MX_QUANTIZE
  return hipGetLastError();
}

hipError_t launch_quantize_fp8_weight(const void* w, bool f16, int64_t G, int64_t N, int64_t K, uint8_t* q,
                                      float* scale, hipStream_t st) {
  const uint32_t nb = (uint32_t)((N + 127) / 128), kb = (uint32_t)((K + 127) / 128);
  return launch_in_parts(G * nb * (int64_t)kb, 256, [&](uint32_t first, uint32_t n) {
    const uint16_t* in = (const uint16_t*)w;
    const bool whole = K % 8 == 0;
    if (f16 && whole) quantize_fp8_weight_kernel<TypeF16, true><<<dim3(n), dim3(256), 0, st>>>(in, N, K, nb, kb, q, scale, first);
    else if (f16) quantize_fp8_weight_kernel<TypeF16, false><<<dim3(n), dim3(256), 0, st>>>(in, N, K, nb, kb, q, scale, first);
    else if (whole) quantize_fp8_weight_kernel<TypeBf16, true><<<dim3(n), dim3(256), 0, st>>>(in, N, K, nb, kb, q, scale, first);
    else quantize_fp8_weight_kernel<TypeBf16, false><<<dim3(n), dim3(256), 0, st>>>(in, N, K, nb, kb, q, scale, first);
  });
}

}  // namespace mx

// Tensors quantized to 8-bit floating point (e4m3) with a scale for each block of 128.
//
//   scale = max|x| / 448 over the block, in fp32 (nearest)
//   q     = the e4m3 value nearest to x / scale, ties to even, at most 448 in size
//
// Tokens have blocks of 1 x 128, weights of 128 x 128; a row's (and a weight's) last block may
// be short.  A block of zeros has scale 0, one with an infinity or NaN has scale NaN, codes 0.
// Bound by memory: x is read once, held in registers between the maximum and the codes.
#include <algorithm>

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

// Largest size of 8 values, as bits of their type without the sign: bits order like sizes,
// infinities and NaN above all.
__device__ __forceinline__ uint32_t max_bits(u32x4_t v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
  return m;
}

struct BlockScale {
  float scale, inverse;
  bool zero;    // codes are 0 (no values, or no number among them)
  bool small;   // scales near the smallest numbers: every code by the exact way
};
template <typename T>
__device__ __forceinline__ BlockScale block_scale(uint32_t bits) {
  constexpr uint32_t kInf = std::is_same<T, TypeF16>::value ? 0x7C00u : 0x7F80u;
  BlockScale b;
  b.scale = bits < kInf ? widen<T>((uint16_t)bits) / kE4m3Max : __builtin_nanf("");
  b.zero = bits == 0 || bits >= kInf;
  b.small = b.scale < 0x1p-100f;
  b.inverse = b.zero ? 0.f : __builtin_amdgcn_rcpf(b.scale);
  return b;
}

// x / scale for the conversion, decided exactly: the quotient rounded to fp32 and, where it is
// even (a border between two codes is) and not exact, one step towards the exact one, so that
// it lies on the exact quotient's side of every border.
__device__ __forceinline__ float exact_quotient(float x, float scale) {
  if (scale < 0x1p-100f) x *= 0x1p100f, scale *= 0x1p100f;   // the remainder below stays a number
  const float v = x / scale;
  const float rest = __builtin_fmaf(-v, scale, x);
  uint32_t bits = __float_as_uint(v);
  if (rest != 0.f && (bits & 1) == 0) bits += (rest > 0.f) == (v > 0.f) ? 1u : ~0u;
  return __uint_as_float(bits);
}

// 8 values to codes.  x * (1 / scale) is within 2 steps of fp32 of the quotient.  Codes of 2^-6
// and more have 3 bits behind the leading one: where the other 20 are not within 4 steps of a
// half, the product rounds as the quotient does.  The rest, and what is smaller, goes the exact
// way (8 in 2^20 of the values, and those 28672 times smaller than their block's largest).
template <typename T>
__device__ __forceinline__ uint2 codes_of(u32x4_t v, const BlockScale& b) {
  if (b.zero) return make_uint2(0u, 0u);
  float x[8], y[8];
  bool near = b.small;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = widen<T>((uint16_t)(v[i / 2] >> (16 * (i & 1))));
    y[i] = x[i] * b.inverse;
    const uint32_t bits = __float_as_uint(y[i]) & 0x7FFFFFFFu;
    near |= (((bits + 4u - 0x80000u) & 0xFFFFFu) <= 8u) | (bits - 1u < 0x3C800000u - 1u);
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = exact_quotient(x[i], b.scale);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __builtin_amdgcn_fmed3f(y[i], -kE4m3Max, kE4m3Max);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
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

// Tokens: 16 lanes a block, four blocks of a lane's in flight.
constexpr int kFp8Unroll = 4;
template <typename T, typename I>
__global__ __launch_bounds__(256) void quantize_fp8_kernel(const uint16_t* x, int64_t ldx, int64_t K, I nb,
                                                           I blocks, uint8_t* q, float* scale) {
  const int sub = threadIdx.x & 15;
  const I step = (I)gridDim.x * 16;
  for (I first = (I)blockIdx.x * 16 + (threadIdx.x >> 4); first < blocks;
       first = blocks - first > step * kFp8Unroll ? first + step * kFp8Unroll : blocks) {
    u32x4_t v[kFp8Unroll];
    int64_t row[kFp8Unroll], at[kFp8Unroll];
#pragma unroll
    for (int u = 0; u < kFp8Unroll; ++u) {
      const I b = first + step * u;
      const bool in = u == 0 || blocks - first > step * u;
      row[u] = in ? (int64_t)(b / nb) : -1;
      at[u] = in ? (int64_t)(b % nb) * 128 + sub * 8 : K;
      v[u] = chunk_end<uint16_t>((const uint8_t*)(x + (in ? row[u] : 0) * ldx + at[u]), (K - at[u]) * 2);
    }
#pragma unroll
    for (int u = 0; u < kFp8Unroll; ++u) {
      if (row[u] < 0) break;   // the same for the 16 lanes of a block
      const BlockScale b = block_scale<T>(row_max(max_bits(v[u], 0)));
      store_codes(q + row[u] * K + at[u], codes_of<T>(v[u], b), K - at[u]);
      if (sub == 0) scale[row[u] * (int64_t)nb + at[u] / 128] = b.scale;
    }
  }
}

// Weights: a workgroup a block, 16 rows at a time, the block in registers.
template <typename T>
__global__ __launch_bounds__(256) void quantize_fp8_weight_kernel(const uint16_t* w, int64_t N, int64_t K,
                                                                  uint32_t nb, uint32_t kb, uint8_t* q,
                                                                  float* scale, uint32_t first) {
  __shared__ uint32_t top[4];
  const uint32_t block = first + blockIdx.x;
  const uint32_t k0 = block % kb, rest = block / kb, n0 = rest % nb, g = rest / nb;
  const int64_t k = (int64_t)k0 * 128 + (threadIdx.x & 15) * 8;
  const int64_t row0 = (int64_t)n0 * 128 + (threadIdx.x >> 4);
  u32x4_t v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    v[i] = chunk_end<uint16_t>((const uint8_t*)(w + ((int64_t)g * N + n) * K + k), n < N ? (K - k) * 2 : 0);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_bits(v[i], m);
  m = row_max(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
  const BlockScale b = block_scale<T>(max(max(top[0], top[1]), max(top[2], top[3])));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    if (n < N) store_codes(q + ((int64_t)g * N + n) * K + k, codes_of<T>(v[i], b), K - k);
  }
  if (threadIdx.x == 0) scale[((int64_t)g * nb + n0) * kb + k0] = b.scale;
}

hipError_t launch_quantize_fp8(const void* x, bool f16, int64_t T, int64_t K, int64_t ldx, uint8_t* q,
                               float* scale, hipStream_t st) {
  const int64_t nb = (K + 127) / 128, blocks = T * nb;
  const dim3 grid((uint32_t)std::min<int64_t>((blocks + 16 * kFp8Unroll - 1) / (16 * kFp8Unroll), 8192));
  const uint16_t* in = (const uint16_t*)x;
  // block numbers in 32 bits where they fit: the division by nb is three times shorter
  if (blocks < (1ll << 31)) {
    const uint32_t n = (uint32_t)nb, all = (uint32_t)blocks;
    if (f16) quantize_fp8_kernel<TypeF16, uint32_t><<<grid, dim3(256), 0, st>>>(in, ldx, K, n, all, q, scale);
    else quantize_fp8_kernel<TypeBf16, uint32_t><<<grid, dim3(256), 0, st>>>(in, ldx, K, n, all, q, scale);
  } else {
    const uint64_t n = (uint64_t)nb, all = (uint64_t)blocks;
    if (f16) quantize_fp8_kernel<TypeF16, uint64_t><<<grid, dim3(256), 0, st>>>(in, ldx, K, n, all, q, scale);
    else quantize_fp8_kernel<TypeBf16, uint64_t><<<grid, dim3(256), 0, st>>>(in, ldx, K, n, all, q, scale);
  }
  return hipGetLastError();
}

hipError_t launch_quantize_fp8_weight(const void* w, bool f16, int64_t G, int64_t N, int64_t K, uint8_t* q,
                                      float* scale, hipStream_t st) {
  const uint32_t nb = (uint32_t)((N + 127) / 128), kb = (uint32_t)((K + 127) / 128);
  return launch_in_parts(G * nb * (int64_t)kb, 256, [&](uint32_t first, uint32_t n) {
    if (f16)
      quantize_fp8_weight_kernel<TypeF16><<<dim3(n), dim3(256), 0, st>>>((const uint16_t*)w, N, K, nb, kb, q, scale, first);
    else
      quantize_fp8_weight_kernel<TypeBf16><<<dim3(n), dim3(256), 0, st>>>((const uint16_t*)w, N, K, nb, kb, q, scale, first);
  });
}

}  // namespace mx

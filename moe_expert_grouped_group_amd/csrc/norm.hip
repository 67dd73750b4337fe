// What follows a block: its output normalized, gated and added to the scaled residual, and the sum
// normalized for the next block; and the gradients of that.
//
//   n(v) = v / sqrt(mean(v^2) + eps) over a row
//   b = n(f) post (or f),  r = residual_scale x + gate b,  y = n(r) pre     r as it is stored
//
//   total = dr + d n(r) for (dy pre),  d n(v) for u: rs (u - (rs mean(u v)) n(v)),  rs = 1 / sqrt(mean(v^2) + eps)
//     (rs^3 itself would leave the fp32 range for rows of 2^43 and of 2^-43)
//   dx = residual_scale total,  db = gate total,  df = d n(f) for (db post) (or db),  dgate = <total, b>
//   dpre = sum over rows of dy n(r),  dpost = sum over rows of db n(f)
//
// Bound by memory: every tensor passes once.  A row lies in the registers of a wave, of 4, 8 or 16
// waves, or 16 or 32 lanes (8 values a lane and chunk), so the second norm and the gradients need no second read.  The
// statistics are fp32.  Column sums stay in registers over the rows that a workgroup takes, one after
// the other, and are joined by a second launch in a fixed order.
#include <algorithm>

#include "ragged_common.h"

namespace mx {

struct NormArgs {
  const void *x, *f;            // forward; backward: x is r
  const void *dy, *dr;          // backward
  const float* gate;
  const void *post, *pre;
  bool w_f32;                   // type of the weights: fp32, else that of f
  float scale, eps;
  int64_t T;
  int32_t H;
  void *r, *y;                  // forward
  void *dx, *df;                // backward
  float* dgate;
  float *dpre, *dpost;          // partial sums [slots, H], or NULL
};

// 8 values of a row as they lie in memory; the type is an output type.
template <typename X>
struct Eight {
  static constexpr int kRegs = sizeof(typename X::elem) / 2;
  u32x4_t v[kRegs];
  // n: values that the row has from here on (zeros behind)
  __device__ __forceinline__ void load(const void* base, int64_t at, int n) {
    const uint8_t* p = (const uint8_t*)base + at * (int64_t)sizeof(typename X::elem);
#pragma unroll
    for (int i = 0; i < kRegs; ++i)
      v[i] = chunk_end<typename X::elem>(p + 16 * i, (int64_t)n * (int64_t)sizeof(typename X::elem) - 16 * i);
  }
  __device__ __forceinline__ void store(void* base, int64_t at, int n) const {
    uint8_t* p = (uint8_t*)base + at * (int64_t)sizeof(typename X::elem);
    if (n >= 8) {
      __builtin_memcpy(p, v, sizeof(v));
    } else {
      typename X::elem e[8];
      __builtin_memcpy(e, v, sizeof(v));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) ((typename X::elem*)p)[i] = e[i];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (std::is_same<X, OutF32>::value) return __uint_as_float(v[i / 4][i % 4]);
    else if constexpr (std::is_same<X, OutF16>::value) return widen<TypeF16>((uint16_t)(v[0][i / 2] >> (16 * (i & 1))));
    else return widen<TypeBf16>((uint16_t)(v[0][i / 2] >> (16 * (i & 1))));
  }
  __device__ __forceinline__ void set(const float (&e)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (std::is_same<X, OutF32>::value) v[i / 4][i % 4] = __float_as_uint(e[i]);
      else if (i % 2 == 0) v[0][i / 2] = (uint32_t)X::cvt(e[i]) | ((uint32_t)X::cvt(e[i + 1]) << 16);
    }
  }
};

// 8 weights; 1 where there are none.
template <typename F>
__device__ __forceinline__ void weights8(const void* w, bool f32, int at, int n, float (&out)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = 1.f;
  } else if (f32) {
    Eight<OutF32> e;
    e.load(w, at, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = e.get(i);
  } else {
    Eight<F> e;
    e.load(w, at, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = e.get(i);
  }
}

// Sums over the W threads of a row, in all of them, in a fixed order.  `side` alternates from call
// to call, so that one barrier does: between two uses of a side lies the other's barrier.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[N], int& side) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int d = W < 64 ? W / 2 : 32; d > 0; d >>= 1) v[i] += __shfl_xor(v[i], d, 64);
  if constexpr (W > 64) {
    constexpr int kWaves = W / 64;
    float(*at)[N] = lds + side * kWaves;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) at[threadIdx.x >> 6][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = at[0][i];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v[i] += at[w][i];
    }
    side ^= 1;
  }
}

// W threads a row, NC chunks of 8 values a thread; workgroups of max(W, 256) threads.
template <typename F, typename X, int W, int NC>
__global__ __launch_bounds__(W < 256 ? 256 : W) void residual_norm_kernel(NormArgs p) {
  constexpr int kPer = W < 256 ? 256 / W : 1;
  __shared__ float lds[W < 64 ? 1 : 2 * (W / 64)][1];
  const int t = threadIdx.x % W;
  int side = 0;
  const float each = 1.f / (float)p.H;
  for (int64_t row = (int64_t)blockIdx.x * kPer + threadIdx.x / W; row < p.T; row += (int64_t)gridDim.x * kPer) {
    Eight<X> x[NC];
    Eight<F> f[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * W + t) * 8, n = p.H - at;
      x[c].load(p.x, row * p.H + at, n);
      if (p.f != nullptr) f[c].load(p.f, row * p.H + at, n);
    }
    if (p.f != nullptr) {
      float rs = p.gate != nullptr ? p.gate[row] : 1.f;
      if (p.post != nullptr) {
        float sum[1] = {0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(f[c].get(i), f[c].get(i), sum[0]);
        row_sums<W>(sum, lds, side);
        rs *= __builtin_amdgcn_rsqf(sum[0] * each + p.eps);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * W + t) * 8, n = p.H - at;
        float w[8], e[8];
        weights8<F>(p.post, p.w_f32, at, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_fmaf(p.scale, x[c].get(i), f[c].get(i) * w[i] * rs);
          // (an fp32 number before it is rounded to the stored type, in every type: the compiler would round
          // once to fp16, another value next to a tie)
          asm("" : "+v"(e[i]));
        }
        x[c].set(e);
        x[c].store(p.r, row * p.H + at, n);
      }
    }
    if (p.pre != nullptr) {
      float sum[1] = {0.f};
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0] = __builtin_fmaf(x[c].get(i), x[c].get(i), sum[0]);
      row_sums<W>(sum, lds, side);
      const float rs = __builtin_amdgcn_rsqf(sum[0] * each + p.eps);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int at = (c * W + t) * 8, n = p.H - at;
        float w[8], e[8];
        weights8<F>(p.pre, p.w_f32, at, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = x[c].get(i) * rs * w[i];
        Eight<F> y;
        y.set(e);
        y.store(p.y, row * p.H + at, n);
      }
    }
  }
}

// ALL: every input and output but the gate's is there, as in a training step; then the next row is
// read while one is worked on, and rows of up to 512 threads keep the weights in registers.  Rows of
// 1024 threads keep their column sums in LDS, for want of registers.
template <typename F, typename X, int W, int NC, bool ALL>
__global__ __launch_bounds__(W < 256 ? 256 : W) void residual_norm_bwd_kernel(NormArgs p) {
  constexpr int kPer = W < 256 ? 256 / W : 1;
  constexpr bool kAhead = ALL && W <= 512;
  __shared__ float lds3[2 * (W / 64)][3], lds1[2 * (W / 64)][1];
  const int t = threadIdx.x % W;
  const int64_t slot = (int64_t)blockIdx.x * kPer + threadIdx.x / W, step = (int64_t)gridDim.x * kPer;
  int side3 = 0, side1 = 0;
  const float each = 1.f / (float)p.H;
  const bool has_dr = ALL || p.dr != nullptr, has_dy = ALL || p.dy != nullptr, has_f = ALL || p.f != nullptr;
  const bool has_post = ALL || p.post != nullptr;
  // without its norm, f itself is in the gate's gradient only
  const bool uses_f = has_post || p.dgate != nullptr;
  constexpr bool kLdsSums = W > 512;
  __shared__ f32x4 lds_sums[kLdsSums ? 2 * NC * 2 * W : 1];
  float kept_sums[2][kLdsSums ? 1 : NC][8];   // of dpre, dpost
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (kLdsSums) {
        lds_sums[(2 * (2 * c + k)) * W + t] = f32x4{0, 0, 0, 0};
        lds_sums[(2 * (2 * c + k) + 1) * W + t] = f32x4{0, 0, 0, 0};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) kept_sums[k][c][i] = 0.f;
      }
    }
  // sums k of chunk c: passed to fn and kept
  auto sums = [&](int k, int c, auto fn) {
    if constexpr (kLdsSums) {
      float v[8];
      f32x4* at = lds_sums + (2 * (2 * c + k)) * W + t;
      const f32x4 lo = at[0], hi = at[W];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
      fn(v);
      at[0] = f32x4{v[0], v[1], v[2], v[3]};
      at[W] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
      fn(kept_sums[k][c]);
    }
  };
  struct Row {
    Eight<X> r[NC], dr[NC];
    Eight<F> f[NC], dy[NC];
  };
  auto load = [&](Row& v, int64_t row) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * W + t) * 8, n = p.H - at;
      if (has_dr) v.dr[c].load(p.dr, row * p.H + at, n);
      if (has_dy) {
        v.r[c].load(p.x, row * p.H + at, n);
        v.dy[c].load(p.dy, row * p.H + at, n);
      }
      if (uses_f) v.f[c].load(p.f, row * p.H + at, n);
    }
  };
  float kept_pre[kAhead ? NC : 1][8], kept_post[kAhead ? NC : 1][8];
  Row ahead;
  if constexpr (kAhead) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * W + t) * 8;
      weights8<F>(p.pre, p.w_f32, at, p.H - at, kept_pre[c]);
      weights8<F>(p.post, p.w_f32, at, p.H - at, kept_post[c]);
    }
    if (slot < p.T) load(ahead, slot);
  }
  auto weights = [&](const void* w, const float (&kept)[8], int at, float (&out)[8]) {
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i] = kept[i];
    } else {
      weights8<F>(w, p.w_f32, at, p.H - at, out);
    }
  };
  for (int64_t row = slot; row < p.T; row += step) {
    Row v;
    if constexpr (kAhead) {
      v = ahead;
      if (row + step < p.T) load(ahead, row + step);
    } else {
      load(v, row);
    }
    const float gate = p.gate != nullptr ? p.gate[row] : 1.f;
    // r^2, dy pre r, f^2
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (has_dy) {
        float w[8];
        weights(p.pre, kept_pre[kAhead ? c : 0], (c * W + t) * 8, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] = __builtin_fmaf(v.r[c].get(i), v.r[c].get(i), sum[0]);
          sum[1] = __builtin_fmaf(v.dy[c].get(i) * w[i], v.r[c].get(i), sum[1]);
        }
      }
      if (has_post) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[2] = __builtin_fmaf(v.f[c].get(i), v.f[c].get(i), sum[2]);
      }
    }
    row_sums<W>(sum, lds3, side3);
    const float rs = __builtin_amdgcn_rsqf(sum[0] * each + p.eps);
    const float pull = rs * (rs * (sum[1] * each));
    const float rf = has_post ? __builtin_amdgcn_rsqf(sum[2] * each + p.eps) : 1.f;
    float total[NC][8];
    float dot[1] = {0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * W + t) * 8, n = p.H - at;
#pragma unroll
      for (int i = 0; i < 8; ++i) total[c][i] = has_dr ? v.dr[c].get(i) : 0.f;
      if (has_dy) {
        float w[8];
        weights(p.pre, kept_pre[kAhead ? c : 0], at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) total[c][i] += v.dy[c].get(i) * w[i] * rs - pull * (v.r[c].get(i) * rs);
        sums(0, c, [&](float (&d)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = __builtin_fmaf(v.dy[c].get(i), v.r[c].get(i) * rs, d[i]);
        });
      }
      if (ALL || p.dx != nullptr) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = p.scale * total[c][i];
        Eight<X> o;
        o.set(e);
        o.store(p.dx, row * p.H + at, n);
      }
      if (uses_f) {
        float w[8];
        weights(p.post, kept_post[kAhead ? c : 0], at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[0] = __builtin_fmaf(total[c][i] * w[i], v.f[c].get(i), dot[0]);
      }
    }
    if (!has_f) continue;
    if (uses_f) row_sums<W>(dot, lds1, side1);
    if (p.dgate != nullptr && t == 0) p.dgate[row] = rf * dot[0];
    const float back = has_post ? rf * (rf * (gate * dot[0] * each)) : 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int at = (c * W + t) * 8, n = p.H - at;
      float w[8], e[8];
      weights(p.post, kept_post[kAhead ? c : 0], at, w);
      if (has_post)
        sums(1, c, [&](float (&d)[8]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = __builtin_fmaf(gate * total[c][i], v.f[c].get(i) * rf, d[i]);
        });
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = gate * total[c][i] * w[i] * rf;
        if (has_post) e[i] -= back * (v.f[c].get(i) * rf);
      }
      if (ALL || p.df != nullptr) {
        Eight<F> o;
        o.set(e);
        o.store(p.df, row * p.H + at, n);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int at = (c * W + t) * 8, n = p.H - at;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float* to = k == 0 ? p.dpre : p.dpost;
      if (to == nullptr || n <= 0) continue;
      Eight<OutF32> o;
      sums(k, c, [&](float (&d)[8]) { o.set(d); });
      o.store(to, slot * p.H + at, n);
    }
  }
}

// Sums of the slots' rows: 64 columns a workgroup, 16 waves take every 16th slot.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const float* pre, const float* post, int32_t slots,
                                                            int32_t H, float* dpre, float* dpost) {
  __shared__ float part[16][64];
  const float* in = blockIdx.y == 0 ? pre : post;
  float* out = blockIdx.y == 0 ? dpre : dpost;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float sum = 0.f;
  if (out != nullptr && col < H) {
    int s = wave;
    for (; s + 16 * 7 < slots; s += 16 * 8) {   // 8 loads in flight
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = in[(int64_t)(s + 16 * i) * H + col];
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
    for (; s < slots; s += 16) sum += in[(int64_t)s * H + col];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || out == nullptr || col >= H) return;
#pragma unroll
  for (int w = 1; w < 16; ++w) sum += part[w][lane];
  out[col] = sum;
}

namespace {

constexpr int kNormMaxH = 16384;

// Threads of a row and chunks of a thread.
template <bool FORWARD, typename G>
hipError_t with_shape(int64_t H, G launch) {
  using std::integral_constant;
#define MX_SHAPE(w, c) return launch(integral_constant<int, w>{}, integral_constant<int, c>{})
  if constexpr (FORWARD) {   // (70674 x 88, fp32 stream: 16 us, with 64 threads 31; the gradients would have more partial sums)
    if (H <= 128) MX_SHAPE(16, 1);
    if (H <= 256) MX_SHAPE(32, 1);
  }
  if (H <= 512) MX_SHAPE(64, 1);
  if (H <= 1024) MX_SHAPE(64, 2);
  if (H <= 2048) MX_SHAPE(256, 1);
  if (H <= 4096) MX_SHAPE(256, 2);
  if constexpr (FORWARD) {   // (8192 x 4104: 65 us, with 512 threads 76; the gradients have no registers for it)
    if (H <= 6144) MX_SHAPE(256, 3);
  }
  if (H <= 8192) MX_SHAPE(512, 2);
  MX_SHAPE(1024, 2);
#undef MX_SHAPE
}

int rows_at_once(int64_t H) { return H <= 1024 ? 4 : 1; }   // of a workgroup

// Workgroups of the backward launch, each with a row of partial sums for each row at once.
int64_t bwd_blocks(int64_t T, int64_t H) {
  // as many as the registers leave room for on 256 CUs
  const int64_t per = rows_at_once(H), most = H <= 512 || (H > 1024 && H <= 2048) ? 768 : H <= 4096 ? 512 : 256;
  return std::min((T + per - 1) / per, most);
}

template <typename G>
hipError_t with_types(bool f16, bool x_f32, G go) {
  if (f16) return x_f32 ? go(OutF16{}, OutF32{}) : go(OutF16{}, OutF16{});
  return x_f32 ? go(OutBf16{}, OutF32{}) : go(OutBf16{}, OutBf16{});
}

}  // namespace

int64_t norm_max_hidden() { return kNormMaxH; }

size_t norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  return (size_t)bwd_blocks(T, H) * rows_at_once(H) * H * 2 * sizeof(float);
}

hipError_t launch_residual_norm(const void* x, bool x_f32, const void* f, bool f16, int64_t T, int64_t H,
                                float scale, const float* gate, const void* post, const void* pre, bool w_f32,
                                float eps, void* r, void* y, hipStream_t st) {
  NormArgs p{};
  p.x = x;
  p.f = f;
  p.T = T;
  p.H = (int32_t)H;
  p.scale = scale;
  p.gate = gate;
  p.post = post;
  p.pre = pre;
  p.w_f32 = w_f32;
  p.eps = eps;
  p.r = r;
  p.y = y;
  return with_types(f16, x_f32, [&](auto F, auto X) {
    return with_shape<true>(H, [&](auto W, auto C) {
      constexpr int w = decltype(W)::value, per = w < 256 ? 256 / w : 1;
      const int64_t blocks = std::min<int64_t>((T + per - 1) / per, 1 << 20);
      residual_norm_kernel<decltype(F), decltype(X), w, decltype(C)::value>
          <<<dim3((uint32_t)blocks), dim3(w < 256 ? 256 : w), 0, st>>>(p);
      return hipGetLastError();
    });
  });
}

hipError_t launch_residual_norm_bwd(const void* dy, const void* dr, const void* r, bool x_f32, const void* f,
                                    bool f16, int64_t T, int64_t H, float scale, const float* gate,
                                    const void* post, const void* pre, bool w_f32, float eps, void* dx, void* df,
                                    float* dgate, float* dpost, float* dpre, void* ws, hipStream_t st) {
  NormArgs p{};
  p.x = r;
  p.f = f;
  p.dy = dy;
  p.dr = dr;
  p.T = T;
  p.H = (int32_t)H;
  p.scale = scale;
  p.gate = gate;
  p.post = post;
  p.pre = pre;
  p.w_f32 = w_f32;
  p.eps = eps;
  p.dx = dx;
  p.df = df;
  p.dgate = dgate;
  const int64_t blocks = bwd_blocks(T, H), slots = blocks * rows_at_once(H);
  if (dpre != nullptr) p.dpre = (float*)ws;
  if (dpost != nullptr) p.dpost = (float*)ws + slots * H;
  if (T > 0) {
    const bool all = dy && dr && f && post && dx && df && dpre && dpost;
    const hipError_t e = with_types(f16, x_f32, [&](auto F, auto X) {
      return with_shape<false>(H, [&](auto W, auto C) {
        constexpr int w = decltype(W)::value, c = decltype(C)::value;
        const dim3 grid((uint32_t)blocks), threads(w < 256 ? 256 : w);
        if (all) residual_norm_bwd_kernel<decltype(F), decltype(X), w, c, true><<<grid, threads, 0, st>>>(p);
        else residual_norm_bwd_kernel<decltype(F), decltype(X), w, c, false><<<grid, threads, 0, st>>>(p);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (dpre == nullptr && dpost == nullptr) return hipSuccess;
  norm_columns_kernel<<<dim3((uint32_t)((H + 63) / 64), 2), dim3(1024), 0, st>>>(p.dpre, p.dpost, (int32_t)slots,
                                                                               (int32_t)H, dpre, dpost);
  return hipGetLastError();
}

}  // namespace mx

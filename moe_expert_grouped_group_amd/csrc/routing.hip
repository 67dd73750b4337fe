// Routing around the experts' products: the k best experts of each token and
// their weights, the order of the rows by expert, the weighted sum of the
// experts' rows, and the gradients of both.
//
//   choice   the top_k largest logits of a token, equal ones by lowest index;
//            -inf and NaN are never chosen, masked tokens choose nothing
//   weights  w_j = exp(l_j - max) / Z, Z over the chosen experts (renormalize)
//            or over all of them
//   order    rows of expert 0, then expert 1, ...; by token within an expert
//   gradient renormalize: dl_j = w_j (dw_j - sum_i w_i dw_i) at the chosen
//            experts, 0 elsewhere; otherwise dl_e = p_e (d_e - sum_i w_i dw_i)
//            with d_e = dw_j where e is choice j, else 0
//   join     out[t] = sum_j w[t, j] y[pos[t, j]]; dy[pos[t, j]] = w[t, j] dout[t];
//            dw[t, j] = <y[pos[t, j]], dout[t]>
//
// Nothing here depends on the order in which workgroups or atomics run: the
// only atomics set bits.
#include <algorithm>

#include "ragged_common.h"

namespace mx {

constexpr int kRouteThreads = 1024;
constexpr int kMaxTopK = 16;
constexpr int kMaxChunk = 512;      // tokens of a workgroup at most, twice that above 2^30

// Element i of a 16- or 32-bit floating tensor as fp32.  type: 0 fp32, 1 bf16, 2 fp16.
template <int TYPE>
__device__ __forceinline__ float load_float(const void* p, int64_t i) {
  if (TYPE == 0) return ((const float*)p)[i];
  if (TYPE == 1) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return (float)((const _Float16*)p)[i];
}
template <int TYPE>
__device__ __forceinline__ void store_float(void* p, int64_t i, float v) {
  if (TYPE == 0) ((float*)p)[i] = v;
  else if (TYPE == 1) ((__bf16*)p)[i] = (__bf16)v;
  else ((_Float16*)p)[i] = (_Float16)v;
}

// Reductions over the L = 16 or 64 lanes that share a token, every lane getting
// the result: rotations within rows of 16 lanes (DPP, no LDS), then the
// gfx950 swaps of rows and halves.
template <int CTRL>
__device__ __forceinline__ float rotate(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int L, typename F>
__device__ __forceinline__ float lanes_all(float v, F f) {
  v = f(v, rotate<0x128>(v));   // row_ror:8, 4, 2, 1
  v = f(v, rotate<0x124>(v));
  v = f(v, rotate<0x122>(v));
  v = f(v, rotate<0x121>(v));
  if (L == 64) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = f(__uint_as_float((uint32_t)r[0]), __uint_as_float((uint32_t)r[1]));
    const uint32_t w = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    v = f(__uint_as_float((uint32_t)h[0]), __uint_as_float((uint32_t)h[1]));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_all<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_all<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ int lanes_min(int v) {
  return __float_as_int(lanes_all<L>(__int_as_float(v), [](float a, float b) {
    return __int_as_float(min(__float_as_int(a), __float_as_int(b)));
  }));
}

struct RouteArgs {
  const void* logits;       // [T, E]
  const uint8_t* mask;      // [T] or NULL; 0: the token is not routed
  int64_t T;
  int32_t E, k, renorm;
  int32_t chunk;            // tokens of a workgroup, a multiple of 32
  int32_t blocks;
  int32_t* ids;             // [T, k]
  float* weights;           // [T, k]
  int64_t* m_splits;        // [E]
  int32_t* row_token;       // [T k]
  int32_t* row_pos;         // [T, k]
  uint16_t* hist;           // workspace [blocks, E rounded up to 2]: rows of each expert in a chunk
  int32_t vec;              // logits rows lie on 4 values
};

// A token's logits in its L lanes: lane s holds experts 4 s .. 4 s + 3, then
// 4 (L + s) ..., V of them (expert_of).  NaN and what lies past E become -inf.
template <int L>
__device__ __forceinline__ int expert_of(int sub, int i) {
  return ((i >> 2) * L + sub) * 4 + (i & 3);
}
template <int TYPE, int L, int V>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, int sub,
                                            bool on, bool vec, float* v) {
  constexpr int kSize = TYPE == 0 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    const int e = expert_of<L>(sub, i);
    char raw[4 * kSize];
    if (vec) {   // E is a multiple of 4: all four or none
      if (on && e < E)
        __builtin_memcpy(raw, __builtin_assume_aligned((const char*)logits + (t * E + e) * kSize, 4 * kSize),
                         sizeof(raw));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (on && e + c < E)
          __builtin_memcpy(raw + c * kSize, (const char*)logits + (t * E + e + c) * kSize, kSize);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float x = load_float<TYPE>(raw, c);
      v[i + c] = on && e + c < E && x == x ? x : -INFINITY;
    }
  }
}

// Choice and weights of one workgroup's tokens, and which tokens of the chunk
// each expert got (bits[e * words + t / 32]).  U tokens for each group of L lanes
// at a time: their loads and reductions overlap.
template <int TYPE, int L, int V, int U>
__device__ __forceinline__ void choose_some(const RouteArgs& p, int64_t t0, int n, int base,
                                            uint32_t* bits) {
  constexpr int kTokens = kRouteThreads / L;
  const int sub = threadIdx.x % L, words = p.chunk / 32;
  float v[U][V], top[U], all[U], mine[U];
  int at[U], mine_id[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = base + u * kTokens + (int)threadIdx.x / L;
    const int64_t t = t0 + at[u];
    const bool on = at[u] < n && (p.mask == nullptr || p.mask[t] != 0);
    load_logits<TYPE, L, V>(p.logits, t, p.E, sub, on, p.vec != 0, v[u]);
    top[u] = 0.f;
    all[u] = 0.f;
    mine[u] = -INFINITY;
    mine_id[u] = -1;
  }
  for (int j = 0; j < p.k; ++j) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float best = v[u][0];
#pragma unroll
      for (int i = 1; i < V; ++i) best = fmaxf(best, v[u][i]);
      best = lanes_max<L>(best);
      int id = INT32_MAX;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (v[u][i] == best) id = expert_of<L>(sub, i);
      id = lanes_min<L>(id);
      const bool live = best > -INFINITY;
      if (j == 0) {
        top[u] = live ? best : 0.f;
        if (!p.renorm) {
#pragma unroll
          for (int i = 0; i < V; ++i) all[u] += expf(v[u][i] - top[u]);
          all[u] = lanes_sum<L>(all[u]);
        }
      }
      // the chosen one leaves; lane j keeps choice j (k <= 16 <= L)
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (live && id == expert_of<L>(sub, i)) v[u][i] = -INFINITY;
      if (sub == j && live) {
        mine[u] = best;
        mine_id[u] = id;
        atomicOr(&bits[id * words + at[u] / 32], 1u << (at[u] & 31));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float w = mine_id[u] >= 0 ? expf(mine[u] - top[u]) : 0.f;
    const float z = p.renorm ? lanes_sum<L>(w) : all[u];
    if (at[u] < n && sub < p.k) {
      const int64_t c = (t0 + at[u]) * p.k + sub;
      p.ids[c] = mine_id[u];
      p.weights[c] = mine_id[u] >= 0 ? w / z : 0.f;
    }
  }
}
template <int TYPE, int L, int V>
__device__ __forceinline__ void choose(const RouteArgs& p, int64_t t0, int n, uint32_t* bits) {
  constexpr int kTokens = kRouteThreads / L;
  int base = 0;
  if (V <= 8)
    for (; base + kTokens < n; base += 2 * kTokens) choose_some<TYPE, L, V, 2>(p, t0, n, base, bits);
  for (; base < n; base += kTokens) choose_some<TYPE, L, V, 1>(p, t0, n, base, bits);
}

// Exclusive prefix over the experts of total[0..E), by the whole workgroup
// (E <= 1024 threads); returns the total of all.  scan: 1024 words of LDS.
__device__ int prefix_experts(int mine, int* scan) {
  const int tid = threadIdx.x, lane = tid & 63;
  int v = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  if (lane == 63) scan[tid >> 6] = v;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < (tid >> 6); ++w) before += scan[w];
  return before + v - mine;
}

// The rank of choice i of the chunk: earlier tokens of the chunk with the same expert.
__device__ __forceinline__ int rank_of(const uint32_t* bits, int words, int id, int at) {
  const uint32_t* b = bits + id * words;
  int rank = __popc(b[at / 32] & ((1u << (at & 31)) - 1u));
  for (int w = 0; w < at / 32; ++w) rank += __popc(b[w]);
  return rank;
}

// LDS: bits [E * words] (and base [E] in the one-launch form).
extern __shared__ uint32_t route_lds[];

// One workgroup for all tokens (T <= chunk): everything in one launch.
template <int TYPE, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_one_kernel(RouteArgs p) {
  __shared__ int scan[16], routed;
  const int tid = threadIdx.x, words = p.chunk / 32;
  uint32_t* bits = route_lds;
  int* base = (int*)(route_lds + p.E * words);
  for (int i = tid; i < p.E * words; i += kRouteThreads) bits[i] = 0;
  __syncthreads();
  choose<TYPE, L, V>(p, 0, (int)p.T, bits);
  __syncthreads();
  int mine = 0;
  if (tid < p.E)
    for (int w = 0; w < words; ++w) mine += __popc(bits[tid * words + w]);
  const int at = prefix_experts(mine, scan);
  if (tid < p.E) {
    base[tid] = at;
    p.m_splits[tid] = mine;
  }
  if (tid == p.E - 1) routed = at + mine;
  __syncthreads();
  const int n = (int)p.T * p.k;
  for (int i = tid; i < n; i += kRouteThreads) {
    const int t = i / p.k, id = p.ids[i];
    int pos = -1;
    if (id >= 0) {
      pos = base[id] + rank_of(bits, words, id, t);
      p.row_token[pos] = t;
    }
    p.row_pos[i] = pos;
  }
  for (int i = routed + tid; i < n; i += kRouteThreads) p.row_token[i] = -1;
}

// Several workgroups: choice, the chunk's counts, and each choice's rank within
// its chunk (left in row_pos); then, in a second launch that sees all counts,
// the positions.
template <int TYPE, int L, int V>
__global__ __launch_bounds__(kRouteThreads) void route_choose_kernel(RouteArgs p) {
  const int tid = threadIdx.x, words = p.chunk / 32;
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
  const int n = (int)min((int64_t)p.chunk, p.T - t0);
  for (int i = tid; i < p.E * words; i += kRouteThreads) route_lds[i] = 0;
  __syncthreads();
  choose<TYPE, L, V>(p, t0, n, route_lds);
  __syncthreads();
  if (tid < p.E) {
    int mine = 0;
    for (int w = 0; w < words; ++w) mine += __popc(route_lds[tid * words + w]);
    p.hist[(int64_t)blockIdx.x * ((p.E + 1) & ~1) + tid] = (uint16_t)mine;
  }
  for (int i = tid; i < n * p.k; i += kRouteThreads) {
    const int id = p.ids[t0 * p.k + i];
    p.row_pos[t0 * p.k + i] = id >= 0 ? rank_of(route_lds, words, id, i / p.k) : -1;
  }
}

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs p) {
  __shared__ int scan[16], routed, base[kRouteThreads];
  __shared__ uint32_t part[2][kRouteThreads][2];
  const int tid = threadIdx.x, pairs = (p.E + 1) / 2;
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
  const int n = (int)min((int64_t)p.chunk, p.T - t0);
  // counts of every chunk: slice s of the workgroup sums chunks s, s + slices, ...
  // for a pair of experts, apart for all chunks and for those before this one
  const int slices = kRouteThreads / pairs, s = tid / pairs, e2 = tid % pairs;
  uint32_t all0 = 0, all1 = 0, bef0 = 0, bef1 = 0;
  if (s < slices) {
    const uint32_t* h = (const uint32_t*)p.hist + e2;
#pragma unroll 4
    for (int b = s; b < p.blocks; b += slices) {
      const uint32_t x = h[(int64_t)b * pairs];
      all0 += x & 0xFFFFu;
      all1 += x >> 16;
      if (b < (int)blockIdx.x) {
        bef0 += x & 0xFFFFu;
        bef1 += x >> 16;
      }
    }
  }
  part[0][tid][0] = all0;
  part[0][tid][1] = all1;
  part[1][tid][0] = bef0;
  part[1][tid][1] = bef1;
  __syncthreads();
  int all = 0, before = 0;
  if (tid < p.E)
    for (int i = 0; i < slices; ++i) {
      all += (int)part[0][i * pairs + tid / 2][tid & 1];
      before += (int)part[1][i * pairs + tid / 2][tid & 1];
    }
  const int at = prefix_experts(all, scan);
  if (tid < p.E) {
    base[tid] = at + before;
    if (blockIdx.x == 0) p.m_splits[tid] = all;
  }
  if (tid == p.E - 1) routed = at + all;
  __syncthreads();
  for (int i = tid; i < n * p.k; i += kRouteThreads) {
    const int64_t c = t0 * p.k + i;
    const int id = p.ids[c];
    if (id < 0) continue;   // row_pos is -1 already
    const int pos = base[id] + p.row_pos[c];
    p.row_token[pos] = (int32_t)(t0 + i / p.k);
    p.row_pos[c] = pos;
  }
  for (int64_t i = routed + (int64_t)blockIdx.x * kRouteThreads + tid; i < p.T * p.k;
       i += (int64_t)gridDim.x * kRouteThreads)
    p.row_token[i] = -1;
}

struct RouteBwdArgs {
  const void* logits;
  const int32_t* ids;
  const float* weights;
  const float* dweights;
  void* dlogits;
  int64_t T;
  int32_t E, k, renorm, vec;
};

template <int TYPE, int L, int V>
__global__ __launch_bounds__(256) void route_bwd_kernel(RouteBwdArgs p, uint32_t first) {
  const int sub = threadIdx.x % L;
  const int64_t t = (int64_t)(first + blockIdx.x) * (256 / L) + threadIdx.x / L;
  const bool on = t < p.T;
  // lane j holds choice j
  int id = -1;
  float w = 0.f, d = 0.f;
  if (on && sub < p.k) {
    id = p.ids[t * p.k + sub];
    if (id >= 0) {
      w = p.weights[t * p.k + sub];
      d = p.dweights[t * p.k + sub];
    }
  }
  const float inner = lanes_sum<L>(w * d);
  float g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = 0.f;
  const int best = __shfl(id, (threadIdx.x & 63) / L * L, 64);
  if (!p.renorm) {
    float v[V];
    load_logits<TYPE, L, V>(p.logits, t, p.E, sub, on && best >= 0, p.vec != 0, v);
    float top = v[0], sum = 0.f;
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, v[i]);
    top = lanes_max<L>(top);
    if (!(top > -INFINITY)) top = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) sum += v[i] = expf(v[i] - top);
    sum = lanes_sum<L>(sum);
    if (best >= 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = -inner * (v[i] / sum);
    }
  }
  const float add = p.renorm ? w * (d - inner) : w * d;
  for (int j = 0; j < p.k; ++j) {
    const int src = (threadIdx.x & 63) / L * L + j;
    const int ej = __shfl(id, src, 64);
    const float aj = __shfl(add, src, 64);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (ej == expert_of<L>(sub, i)) g[i] += aj;
  }
  if (!on) return;
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    constexpr int kSize = TYPE == 0 ? 4 : 2;
    const int e = expert_of<L>(sub, i);
    char raw[4 * kSize];
#pragma unroll
    for (int c = 0; c < 4; ++c) store_float<TYPE>(raw, c, g[i + c]);
    char* to = (char*)p.dlogits + (t * p.E + e) * kSize;
    if (p.vec) {
      if (e < p.E) __builtin_memcpy(__builtin_assume_aligned(to, 4 * kSize), raw, sizeof(raw));
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (e + c < p.E) __builtin_memcpy(to + c * kSize, raw + c * kSize, kSize);
    }
  }
}

// ---------------------------------------------------------------------------
// The experts' rows joined for each token.
// ---------------------------------------------------------------------------
constexpr int kJoinWidth = 8;   // values of a thread at a time (16 bytes)

struct JoinArgs {
  const void* y;            // [R, H]
  const void* dout;         // [T, H]
  const int32_t* pos;       // [T, k]
  const float* weights;     // [T, k] or NULL (all 1)
  void* out;                // [T, H]; backward: dy [R, H] or NULL
  float* dweights;          // [T, k] or NULL
  int64_t T, R, H;
  int32_t k;
};

// n (up to 8) values of 16 bits as they lie, zeros behind; and as fp32.  Apart, so
// that several loads can be in flight before the first conversion waits.
__device__ __forceinline__ u32x4_t load_raw(const uint16_t* p, int n) {
  u32x4_t raw = {0, 0, 0, 0};
  if (n == kJoinWidth) {
    __builtin_memcpy(&raw, p, 16);
  } else {
    uint16_t e[kJoinWidth];
#pragma unroll
    for (int i = 0; i < kJoinWidth; ++i) e[i] = i < n ? p[i] : (uint16_t)0;
    __builtin_memcpy(&raw, e, 16);
  }
  return raw;
}
template <int TYPE>
__device__ __forceinline__ void to_floats(u32x4_t raw, float* v) {
  uint16_t e[kJoinWidth];
  __builtin_memcpy(e, &raw, 16);
#pragma unroll
  for (int i = 0; i < kJoinWidth; ++i) v[i] = load_float<TYPE>(e, i);
}
template <int TYPE>
__device__ __forceinline__ void load8(const uint16_t* p, int n, float* v) {
  to_floats<TYPE>(load_raw(p, n), v);
}
template <int TYPE>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float* v) {
  uint16_t e[kJoinWidth];
#pragma unroll
  for (int i = 0; i < kJoinWidth; ++i) store_float<TYPE>(e, i, v[i]);
  if (n == kJoinWidth) {
    __builtin_memcpy(p, e, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kJoinWidth; ++i)
      if (i < n) p[i] = e[i];
  }
}

// K rows a token at most (p.k of them): a thread has the chunks of all of them
// in flight before it adds the first.  Workgroups are rows of `lanes` threads
// for each of 256 / lanes tokens.
template <int TYPE, int K>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs p, int lanes, uint32_t first) {
  const int64_t t = (int64_t)(first + blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
  if (t >= p.T) return;
  int64_t row[K];
  float w[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t r = j < p.k ? p.pos[t * p.k + j] : -1;
    row[j] = r >= 0 && r < p.R ? r : -1;
    w[j] = j < p.k && p.weights != nullptr ? p.weights[t * p.k + j] : 1.f;
  }
  for (int64_t h = (int64_t)(threadIdx.x % lanes) * kJoinWidth; h < p.H; h += lanes * kJoinWidth) {
    const int n = (int)min((int64_t)kJoinWidth, p.H - h);
    u32x4_t raw[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      raw[j] = u32x4_t{0, 0, 0, 0};
      if (row[j] >= 0) raw[j] = load_raw((const uint16_t*)p.y + row[j] * p.H + h, n);
    }
    float sum[kJoinWidth] = {};
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (row[j] >= 0) {
        float v[kJoinWidth];
        to_floats<TYPE>(raw[j], v);
#pragma unroll
        for (int e = 0; e < kJoinWidth; ++e) sum[e] += w[j] * v[e];
      }
    store8<TYPE>((uint16_t*)p.out + t * p.H + h, n, sum);
  }
}

// dy and dweights: tokens as above; a token's dot products are joined over its
// lanes (lanes is 64 or 256).
template <int TYPE, int K>
__global__ __launch_bounds__(256) void join_bwd_kernel(JoinArgs p, int lanes, uint32_t first) {
  __shared__ float part[4][K];
  const int64_t t = (int64_t)(first + blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
  const bool on = t < p.T;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t row[K];
  float w[K], dot[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int64_t r = on && j < p.k ? p.pos[t * p.k + j] : -1;
    row[j] = r >= 0 && r < p.R ? r : -1;
    w[j] = on && j < p.k && p.weights != nullptr ? p.weights[t * p.k + j] : 1.f;
    dot[j] = 0.f;
  }
  for (int64_t h = (int64_t)(threadIdx.x % lanes) * kJoinWidth; on && h < p.H; h += lanes * kJoinWidth) {
    const int n = (int)min((int64_t)kJoinWidth, p.H - h);
    float d[kJoinWidth];
    load8<TYPE>((const uint16_t*)p.dout + t * p.H + h, n, d);
    if (p.dweights != nullptr) {
      u32x4_t raw[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        raw[j] = u32x4_t{0, 0, 0, 0};
        if (row[j] >= 0) raw[j] = load_raw((const uint16_t*)p.y + row[j] * p.H + h, n);
      }
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (row[j] >= 0) {
          float v[kJoinWidth];
          to_floats<TYPE>(raw[j], v);
#pragma unroll
          for (int e = 0; e < kJoinWidth; ++e) dot[j] += v[e] * d[e];
        }
    }
    if (p.out != nullptr) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (row[j] >= 0) {
          float v[kJoinWidth];
#pragma unroll
          for (int e = 0; e < kJoinWidth; ++e) v[e] = w[j] * d[e];
          store8<TYPE>((uint16_t*)p.out + row[j] * p.H + h, n, v);
        }
    }
  }
  if (p.dweights == nullptr) return;
#pragma unroll
  for (int j = 0; j < K; ++j) dot[j] = lanes_sum<64>(dot[j]);
  if (lanes == 64) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (on && lane == j && j < p.k) p.dweights[t * p.k + j] = dot[j];
    return;
  }
#pragma unroll
  for (int j = 0; j < K; ++j)
    if (lane == 0) part[wave][j] = dot[j];
  __syncthreads();
  const int j = (int)threadIdx.x;
  if (on && j < p.k) p.dweights[t * p.k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
}

// ---------------------------------------------------------------------------
// Tokens to 8-bit integers: scale = amax / 127 (fp32, nearest), code = the
// integer nearest to x / scale (ties to even) in exact arithmetic.  A row of
// zeros has scale 0 and codes 0; a row with an infinity or NaN scale NaN.
// ---------------------------------------------------------------------------
constexpr int kQuantThreads = 1024;   // at most
constexpr int kQuantHeld = 4;          // chunks of 8 values a thread keeps: rows up to 8192 (32768
                                       // where they are few) are read once

__device__ __forceinline__ int code_int8(float x, float scale, float inv) {
  // The product with the reciprocal is within 3 units in the last place of the
  // quotient, so 2.3e-5 of it for |q| <= 127: its nearest integer is the right one
  // unless it lies that near to a border between two.  There x - q scale, exact in
  // one fused multiply-add (both are multiples of the last place of scale, the
  // difference is at most about scale), tells the side of the border, or that x
  // lies on it.
  const float t = x * inv;
  float q = rintf(t);
  if (fabsf(fabsf(t - q) - 0.5f) < 1e-4f) {
    const float r = __builtin_fmaf(-q, scale, x);
    const float half = 0.5f * scale;
    const bool odd = ((int)q & 1) != 0;
    if (r > half || (r == half && odd)) q += 1.f;
    else if (r < -half || (r == -half && odd)) q -= 1.f;
  }
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

template <int TYPE>
__global__ __launch_bounds__(kQuantThreads) void quantize_int8_kernel(const void* x, int64_t ldx,
                                                                      int64_t K, int8_t* q,
                                                                      float* scale, uint32_t first) {
  __shared__ uint32_t part[kQuantThreads / 64];
  const int64_t row = first + blockIdx.x;
  const uint16_t* src = (const uint16_t*)x + row * ldx;
  int8_t* dst = q + row * K;
  const int64_t step = (int64_t)blockDim.x * 8;
  // the largest magnitude, compared as bits: infinities and NaN lie above all
  uint32_t top = 0;
  float held[kQuantHeld][8];
  int64_t h = (int64_t)threadIdx.x * 8;
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c, h += step) {
    if (h >= K) break;
    load8<TYPE>(src + h, (int)min((int64_t)8, K - h), held[c]);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(held[c][e]) & 0x7FFFFFFFu);
  }
  for (; h < K; h += step) {
    float v[8];
    load8<TYPE>(src + h, (int)min((int64_t)8, K - h), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x / 64; ++w) top = max(top, part[w]);
  const float s = top >= 0x7F800000u ? NAN : __fdiv_rn(__uint_as_float(top), 127.f);
  const bool none = !(s > 0.f);
  // tiny scales are worked with 2^64 larger, values and all: the reciprocal
  // of a subnormal overflows
  const float up = s < 0x1p-90f ? 0x1p64f : 1.f;
  const float su = s * up;
  const float inv = none ? 0.f : 1.f / su;
  if (threadIdx.x == 0) scale[row] = s;
  auto put = [&](int64_t at, const float* v) {
    const int n = (int)min((int64_t)8, K - at);
    int8_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = none ? 0 : (int8_t)code_int8(v[e] * up, su, inv);
    if (n == 8) {
      __builtin_memcpy(dst + at, c, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) dst[at + e] = c[e];
    }
  };
  h = (int64_t)threadIdx.x * 8;
#pragma unroll
  for (int c = 0; c < kQuantHeld; ++c, h += step) {
    if (h >= K) break;
    put(h, held[c]);
  }
  for (; h < K; h += step) {
    float v[8];
    load8<TYPE>(src + h, (int)min((int64_t)8, K - h), v);
    put(h, v);
  }
}

namespace {

// Tokens of a workgroup: about 256 workgroups, 64 to 512 tokens each
// at most, and at most 32 KiB of bits (chunk * E / 8 bytes).  Above 2^30 tokens (of 256
// experts at most: more would be 512 GiB of logits) 1024, as a launch holds fewer than
// 2^32 threads.
int route_chunk(int64_t T, int32_t E) {
  const int64_t per = (T + 255) / 256, cap = T > (1 << 30) ? 2 * kMaxChunk : kMaxChunk;
  const int64_t most = std::min<int64_t>(cap, (1 << 18) / E / 32 * 32);
  return (int)std::min<int64_t>(std::max<int64_t>((per + 63) / 64 * 64, 64), most);
}
// Tokens that one workgroup alone takes: the second launch of the other form
// costs about as much as these.
constexpr int64_t kOneLaunch = 256;

template <int TYPE, int L, int V>
hipError_t launch_route_lv(RouteArgs p, hipStream_t st) {
  const bool one = p.T <= kOneLaunch;
  p.chunk = one ? (int)std::max<int64_t>((p.T + 31) / 32 * 32, 32) : route_chunk(p.T, p.E);
  p.blocks = (int)((p.T + p.chunk - 1) / p.chunk);
  p.vec = p.E % 4 == 0 && (uintptr_t)p.logits % (TYPE == 0 ? 16 : 8) == 0;
  const size_t bits = (size_t)p.E * (p.chunk / 32) * 4;
  if (one) {
    route_one_kernel<TYPE, L, V><<<1, kRouteThreads, bits + (size_t)p.E * 4, st>>>(p);
  } else {
    route_choose_kernel<TYPE, L, V><<<p.blocks, kRouteThreads, bits, st>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    route_place_kernel<<<p.blocks, kRouteThreads, 0, st>>>(p);
  }
  return hipGetLastError();
}

template <int TYPE, int L, int V>
hipError_t launch_bwd_lv(RouteBwdArgs p, hipStream_t st) {
  const uintptr_t on = (uintptr_t)p.logits | (uintptr_t)p.dlogits;
  p.vec = p.E % 4 == 0 && on % (TYPE == 0 ? 16 : 8) == 0;
  const int64_t per = 256 / L;
  return launch_in_parts((p.T + per - 1) / per, 256, [&](uint32_t first, uint32_t n) {
    route_bwd_kernel<TYPE, L, V><<<n, 256, 0, st>>>(p, first);
  });
}

// 16 lanes for a token up to 256 experts (4 tokens a wave, short reductions),
// a whole wave above, and for few tokens, whose latency counts: fewer logits
// a lane.
#define MX_ROUTE_PICK(FN, TYPE, P)                                     \
  (P).T <= 64 && (P).E <= 256 ? FN<TYPE, 64, 4>(P, st)                 \
  : (P).E <= 64  ? FN<TYPE, 16, 4>(P, st)                              \
  : (P).E <= 128 ? FN<TYPE, 16, 8>(P, st)                              \
  : (P).E <= 256 ? FN<TYPE, 16, 16>(P, st)                             \
  : (P).E <= 512 ? FN<TYPE, 64, 8>(P, st)                              \
                 : FN<TYPE, 64, 16>(P, st)

template <int TYPE, int K>
hipError_t launch_join_k(const JoinArgs& p, bool bwd, hipStream_t st) {
  // threads for a token: one wave for rows up to 1024 values, else the workgroup
  const int lanes = p.H <= 64 * kJoinWidth * 2 ? 64 : 256;
  const int64_t per = 256 / lanes;
  return launch_in_parts((p.T + per - 1) / per, 256, [&](uint32_t first, uint32_t n) {
    if (bwd) join_bwd_kernel<TYPE, K><<<n, 256, 0, st>>>(p, lanes, first);
    else join_kernel<TYPE, K><<<n, 256, 0, st>>>(p, lanes, first);
  });
}
template <int TYPE>
hipError_t launch_join_type(const JoinArgs& p, bool bwd, hipStream_t st) {
  if (p.k == 1) return launch_join_k<TYPE, 1>(p, bwd, st);
  if (p.k == 2) return launch_join_k<TYPE, 2>(p, bwd, st);
  if (p.k <= 4) return launch_join_k<TYPE, 4>(p, bwd, st);
  if (p.k <= 8) return launch_join_k<TYPE, 8>(p, bwd, st);
  return launch_join_k<TYPE, kMaxTopK>(p, bwd, st);
}

}  // namespace

// T and E as launch_route takes them.
size_t route_workspace_bytes(int64_t T, int32_t E) {
  if (T <= kOneLaunch) return 0;
  const int64_t c = route_chunk(T, E);
  return (size_t)((T + c - 1) / c) * (size_t)((E + 1) & ~1) * sizeof(uint16_t);
}

hipError_t launch_route(const void* logits, int type, int64_t T, int32_t E, int32_t k, bool renorm,
                        const uint8_t* mask, int32_t* ids, float* weights, int64_t* m_splits,
                        int32_t* row_token, int32_t* row_pos, void* ws, hipStream_t st) {
  RouteArgs p{};
  p.logits = logits;
  p.mask = mask;
  p.T = T;
  p.E = E;
  p.k = k;
  p.renorm = renorm;
  p.ids = ids;
  p.weights = weights;
  p.m_splits = m_splits;
  p.row_token = row_token;
  p.row_pos = row_pos;
  p.hist = (uint16_t*)ws;
  if (type == 0) return MX_ROUTE_PICK(launch_route_lv, 0, p);
  if (type == 1) return MX_ROUTE_PICK(launch_route_lv, 1, p);
  return MX_ROUTE_PICK(launch_route_lv, 2, p);
}

hipError_t launch_route_bwd(const void* logits, int type, int64_t T, int32_t E, int32_t k,
                            bool renorm, const int32_t* ids, const float* weights,
                            const float* dweights, void* dlogits, hipStream_t st) {
  RouteBwdArgs p{logits, ids, weights, dweights, dlogits, T, E, k, renorm, 0};
  if (type == 0) return MX_ROUTE_PICK(launch_bwd_lv, 0, p);
  if (type == 1) return MX_ROUTE_PICK(launch_bwd_lv, 1, p);
  return MX_ROUTE_PICK(launch_bwd_lv, 2, p);
}

hipError_t launch_join(const void* y, bool f16, int64_t T, int64_t R, int64_t H, int32_t k,
                       const int32_t* pos, const float* weights, void* out, hipStream_t st) {
  JoinArgs p{};
  p.y = y;
  p.pos = pos;
  p.weights = weights;
  p.out = out;
  p.T = T;
  p.R = R;
  p.H = H;
  p.k = k;
  return f16 ? launch_join_type<2>(p, false, st) : launch_join_type<1>(p, false, st);
}

hipError_t launch_join_bwd(const void* dout, const void* y, bool f16, int64_t T, int64_t R,
                           int64_t H, int32_t k, const int32_t* pos, const float* weights,
                           void* dy, float* dweights, hipStream_t st) {
  JoinArgs p{};
  p.y = y;
  p.dout = dout;
  p.pos = pos;
  p.weights = weights;
  p.out = dy;
  p.dweights = dweights;
  p.T = T;
  p.R = R;
  p.H = H;
  p.k = k;
  return f16 ? launch_join_type<2>(p, true, st) : launch_join_type<1>(p, true, st);
}

hipError_t launch_quantize_int8(const void* x, bool f16, int64_t T, int64_t K, int64_t ldx,
                                int8_t* q, float* scale, hipStream_t st) {
  // One workgroup a row.  Where rows are few, a thread for every 8 values: 8 rows of
  // 7168 took 7.9 us with 256 threads each and 5.0 with 896.
  const int64_t most = T >= 1024 ? 256 : kQuantThreads;
  const uint32_t threads = (uint32_t)std::min<int64_t>(((K + 7) / 8 + 63) / 64 * 64, most);
  return launch_in_parts(T, (int)threads, [&](uint32_t first, uint32_t n) {
    if (f16) quantize_int8_kernel<2><<<n, threads, 0, st>>>(x, ldx, K, q, scale, first);
    else quantize_int8_kernel<1><<<n, threads, 0, st>>>(x, ldx, K, q, scale, first);
  });
}

}  // namespace mx

// Products grouped by expert with any number of rows per expert.
//
//   forward (NT): C[r, n]    = sum_k X[i(r), k] W[g, n, k]     r a row of expert g
//   dgrad   (NN): C[r, k]    = sum_n dY[r, n]   W[g, n, k]
//   wgrad   (TN): C[g, n, k] = sum over rows r of g of dY[r, n] X[i(r), k]
//
// i(r) is row_index[r] or r.  Experts own consecutive rows, m_splits[g] of
// them, read on the device; rows after the last expert's are not touched.
#include <algorithm>
#include <cmath>

#include "ragged_common.h"

namespace mx {

// ---------------------------------------------------------------------------
// Any size, stride and alignment.
//
// 128 x 128 output tile, 4 waves of 64 x 64, contraction in steps of 64 bytes.
// Chunks go through registers: a 16-byte load at element alignment where the
// whole chunk lies inside the operand, single elements at its edge, zeros
// outside.  Both operands lie in LDS with the contraction contiguous; an operand whose
// contraction runs over its rows (W in NN, both in TN) is transposed by the
// store to LDS.
// ---------------------------------------------------------------------------
constexpr int kAnyT = 128;         // tile edge
constexpr int kAnyBytes = 64;      // contraction bytes per step
constexpr int kAnyPitch = 80;      // LDS row: 64 bytes + 16, so that 16-byte reads of
                                   // consecutive rows start in different banks

// Up to 16 bytes from p, the first n elements of them valid (n <= 0: none).
template <typename E>
__device__ __forceinline__ u32x4_t load_chunk(const E* p, int64_t n) {
  constexpr int kN = 16 / sizeof(E);
  u32x4_t v = {0, 0, 0, 0};
  if (n >= kN) {
    __builtin_memcpy(&v, p, 16);
  } else if (n > 0) {
    E e[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) e[i] = i < n ? p[i] : (E)0;
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// The row tile `t` (of `tile` rows) among all experts: its expert, first row
// and row count, from the splits, by the whole workgroup.  Returns false past
// the last tile.  G <= 1024, 256 threads.
struct RowTile {
  int g;
  int64_t row0;
  int rows;
};
__device__ bool find_row_tile(const int64_t* m_splits, int G, int64_t R, int tile, int64_t t,
                              RowTile* out, int64_t* lds /* 2 * 256 + 3 */) {
  const int tid = threadIdx.x;
  constexpr int per = kRaggedMaxGroups / 256;
  int64_t rows[per], r_sum = 0, t_sum = 0;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int g = tid * per + i;
    rows[i] = g < G ? split_rows(m_splits, g, R) : 0;
    r_sum += rows[i];
    t_sum += (rows[i] + tile - 1) / tile;
  }
  int64_t* sr = lds;
  int64_t* st = lds + 256;
  int64_t* found = lds + 512;
  sr[tid] = r_sum;
  st[tid] = t_sum;
  if (tid == 0) found[0] = -1;
  __syncthreads();
  for (int d = 1; d < 256; d <<= 1) {
    const int64_t r = tid >= d ? sr[tid - d] : 0, u = tid >= d ? st[tid - d] : 0;
    __syncthreads();
    sr[tid] += r;
    st[tid] += u;
    __syncthreads();
  }
  int64_t r0 = sr[tid] - r_sum, t0 = st[tid] - t_sum;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int64_t nt = (rows[i] + tile - 1) / tile;
    if (t >= t0 && t < t0 + nt) {
      const int64_t lo = r0 + (t - t0) * tile;
      const int64_t hi = r0 + rows[i] < R ? r0 + rows[i] : R;   // never past the rows there are
      found[0] = tid * per + i;
      found[1] = lo;
      found[2] = hi - lo < tile ? hi - lo : tile;
    }
    r0 += rows[i];
    t0 += nt;
  }
  __syncthreads();
  out->g = (int)found[0];
  out->row0 = found[1];
  out->rows = (int)found[2];
  return found[0] >= 0 && found[2] > 0;
}

// Rows [lo, lo + len) of expert g (TN), clipped to the R rows there are.
__device__ void expert_rows(const int64_t* m_splits, int g, int64_t R, int64_t* lo, int64_t* len,
                            int64_t* lds /* 256 */) {
  const int tid = threadIdx.x;
  int64_t s = 0;
  for (int i = tid; i < g; i += 256) s += split_rows(m_splits, i, R);
  lds[tid] = s;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if (tid < d) lds[tid] += lds[tid + d];
    __syncthreads();
  }
  const int64_t at = lds[0] < R ? lds[0] : R;
  const int64_t m = split_rows(m_splits, g, R);
  *lo = at;
  *len = m < R - at ? m : R - at;
  __syncthreads();
}

template <typename T, typename O, int LAYOUT>
__global__ __launch_bounds__(256, 2) void ragged_any_kernel(RaggedArgs p, uint32_t first) {
  typedef typename T::elem E;
  constexpr int kPer = 16 / sizeof(E);             // elements of a chunk
  constexpr int kStep = kAnyBytes / sizeof(E);     // contraction elements per step
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * kAnyT * kAnyPitch];
  __shared__ int64_t scan[2 * 256 + 3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;

  // the tile: rows [m0, m0 + rows) of A's output dimension, columns from n0
  const int64_t cols = LAYOUT == 0 ? p.N : p.K;
  const int64_t nt = (cols + kAnyT - 1) / kAnyT;
  const int64_t at = first + blockIdx.x, ct = at % nt, rt = at / nt;
  const int64_t n0 = ct * kAnyT;
  int g;
  int64_t m0, rows, con, lo = 0;   // con: contraction length; lo: its first row (TN)
  if (LAYOUT != 2) {
    RowTile t;
    if (!find_row_tile(p.m_splits, p.G, p.R, kAnyT, rt, &t, scan)) return;
    g = t.g;
    m0 = t.row0;
    rows = t.rows;
    con = LAYOUT == 0 ? p.K : p.N;
  } else {
    const int64_t mt = (p.N + kAnyT - 1) / kAnyT;
    g = (int)(rt / mt);
    m0 = (rt % mt) * kAnyT;
    rows = p.N - m0 < kAnyT ? p.N - m0 : kAnyT;
    expert_rows(p.m_splits, g, p.R, &lo, &con, scan);
  }

  // this thread's chunks: two of each operand.  Contraction contiguous: row
  // (tid >> 2) + 64 i, chunk tid & 3.  Contraction over rows: contraction
  // row (tid >> 4) + 16 i, 8 columns from 8 (tid & 15).
  const E* a = (const E*)p.a;
  const E* b = (const E*)p.b;
  if (LAYOUT != 2) b += (int64_t)g * p.N * p.K;
  u32x4_t ra[2], rb[2];
  auto fetch = [&](int64_t k0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (LAYOUT != 2) {
        const int r = (tid >> 2) + 64 * i;
        const int64_t k = k0 + (tid & 3) * kPer;
        int64_t n = r < rows ? con - k : 0;
        int64_t row = m0 + r;
        if (LAYOUT == 0 && p.row_index != nullptr) {
          row = n > 0 ? p.row_index[row] : 0;
          if (row < 0 || row >= p.S) n = 0, row = 0;
        }
        ra[i] = load_chunk<E>(a + row * p.lda + k, n);
      } else {
        const int64_t k = k0 + (tid >> 4) + 16 * i;
        const int64_t c = (tid & 15) * 8;
        ra[i] = load_chunk<E>(a + (lo + k) * p.lda + m0 + c, k < con ? p.N - m0 - c : 0);
      }
      if (LAYOUT == 0) {
        const int64_t r = n0 + (tid >> 2) + 64 * i;
        const int64_t k = k0 + (tid & 3) * kPer;
        rb[i] = load_chunk<E>(b + r * p.K + k, r < p.N ? con - k : 0);
      } else {
        const int64_t k = k0 + (tid >> 4) + 16 * i;
        const int64_t c = n0 + (tid & 15) * 8;
        int64_t n = k < con ? p.K - c : 0;
        int64_t row = lo + k;
        if (LAYOUT == 2 && p.row_index != nullptr) {
          row = n > 0 ? p.row_index[row] : 0;
          if (row < 0 || row >= p.S) n = 0, row = 0;
        }
        rb[i] = load_chunk<E>(b + row * (LAYOUT == 2 ? p.ldb : p.K) + c, n);
      }
    }
  };
  uint8_t* la = smem;
  uint8_t* lb = smem + kAnyT * kAnyPitch;
  auto put = [&](uint8_t* at, u32x4_t v, int i, bool over_rows) {
    if (!over_rows) {
      *(u32x4_t*)(at + ((tid >> 2) + 64 * i) * kAnyPitch + (tid & 3) * 16) = v;
    } else {
      E e[kPer];
      __builtin_memcpy(e, &v, 16);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        *(E*)(at + ((tid & 15) * 8 + j) * kAnyPitch + ((tid >> 4) + 16 * i) * sizeof(E)) = e[j];
    }
  };

  typename T::acc acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i >> 1][i & 1][r] = 0;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const uint8_t* fa = la + (wm + (lane & 31)) * kAnyPitch + (lane >> 5) * 16;
  const uint8_t* fb = lb + (wn + (lane & 31)) * kAnyPitch + (lane >> 5) * 16;

  if (con > 0) fetch(0);
  for (int64_t k0 = 0; k0 < con; k0 += kStep) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      put(la, ra[i], i, LAYOUT == 2);
      put(lb, rb[i], i, LAYOUT != 0);
    }
    __syncthreads();
    if (k0 + kStep < con) fetch(k0 + kStep);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4_t va[2], vb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        va[i] = *(const u32x4_t*)(fa + i * 32 * kAnyPitch + s * 32);
        vb[i] = *(const u32x4_t*)(fb + i * 32 * kAnyPitch + s * 32);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = T::mma(va[i], vb[j], acc[i][j]);
    }
    __syncthreads();
  }

  // accumulator r of a 32 x 32 block in lane l: row 8 (r / 4) + 4 (l / 32) + r % 4,
  // column l % 32
  typename O::elem* c = (typename O::elem*)p.c;
  const int64_t ldc = LAYOUT == 2 ? p.K : p.ldc;
  c += LAYOUT == 2 ? ((int64_t)g * p.N + m0) * p.K : m0 * ldc;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t n = n0 + wn + 32 * j + (lane & 31);
      float sb = 1.f;
      if (sizeof(E) == 1 && n < cols) sb = p.sb[(int64_t)g * p.N + n];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int m = wm + 32 * i + 8 * (r / 4) + 4 * (lane >> 5) + (r & 3);
        if (m < rows && n < cols) {
          float v = (float)acc[i][j][r];
          if constexpr (sizeof(E) == 1) {
            int64_t row = m0 + m;
            if (p.row_index != nullptr) row = p.row_index[row];
            v = scaled<O>(acc[i][j][r], row >= 0 && row < p.S ? p.sa[row] : 0.f, sb);
          }
          c[m * ldc + n] = O::cvt(v);
        }
      }
    }
}

namespace {

// Tiles of ragged_any_kernel.  An expert's last one may be partial: at most one more
// for each expert that has rows.
int64_t ragged_any_blocks(int layout, int64_t R, int64_t N, int64_t K, int32_t G) {
  const int64_t cols = ((layout == 0 ? N : K) + kAnyT - 1) / kAnyT;
  return cols * (layout == 2 ? (int64_t)G * ((N + kAnyT - 1) / kAnyT)
                             : R / kAnyT + std::min<int64_t>(G, R));
}

template <typename T, typename O, int LAYOUT>
hipError_t launch_any(const RaggedArgs& p, hipStream_t st) {
  const int64_t blocks = ragged_any_blocks(LAYOUT, p.R, p.N, p.K, p.G);
  return launch_in_parts(blocks, 256, [&](uint32_t first, uint32_t n) {
    ragged_any_kernel<T, O, LAYOUT><<<dim3(n), dim3(256), 0, st>>>(p, first);
  });
}

template <typename T, typename O>
hipError_t launch_layout(int layout, const RaggedArgs& p, hipStream_t st) {
  if (layout == 0) return launch_any<T, O, 0>(p, st);
  if (layout == 1) return launch_any<T, O, 1>(p, st);
  return launch_any<T, O, 2>(p, st);
}

bool on16(const void* p, int64_t stride_bytes) {
  return (uintptr_t)p % 16 == 0 && stride_bytes % 16 == 0;
}
int64_t pad16(int64_t n, int64_t size) { return (n * size + 15) / 16 * 16 / size; }

// Whether experts have few rows, so that the forward product is bound by reading
// the weights and ragged_few.hip takes it.  Measured with equal experts (us; here, in
// the large tiles), by MB of weights (experts x N x K) and m rows an expert:
//    34 (1 x 4096 x 4096)     m 16:  11,  30   64:  22,  34    96:  35,  35   192:  58,  44
//    67 (8 x 2048 x 2048)     m 16:  18,  41   64:  41,  45    96:  70,  45
//   134 (4 x 4096 x 4096)     m 16:  31,  43   20:  38,  44    32:  46,  44
//   235 (4 x 7168 x 4096)     m 12:  48,  53   16:  53,  53    24:  67,  55
//   268 (64 x 2048 x 1024)    m  8:  54,  56   12:  62,  57    16:  71,  58
//   940 (8 x 14336 x 4096)    m  4: 165, 177    6: 177, 178     8: 195, 179
//   8-bit, 470 (the same)     m  8: 103, 115   12: 115, 115    16: 129, 116
// About W (0.16 + 0.0075 m) here; the tiles take some 25 us at least and 0.19 W or
// 0.24 W (8-bit) where W is large.  Off by most with many experts of short rows (537,
// 128 x 2048 x 1024: 116, 108 at m 4 already).  Up to 256 rows, though small weights
// would stay ahead beyond (1 x 1024 x 1024 at 384: 14, 32), because 22 experts of 808 x 151
// with 760 rows each took 130 us here.
bool few_rows(const RaggedArgs& p, int esize) {
  const int64_t groups = std::min<int64_t>(p.G, p.R), mean = p.R / groups;
  const double mb = 1e-6 * (double)groups * (double)p.N * (double)p.K * esize;
  const double most = mb < 100.0 ? 4200.0 : 3000.0;
  return p.R < (1 << 20) && mean <= 256 && (mean <= 4 || (double)(mean - 4) * mb <= most);
}

// What the large tiles want and an operand may lack: rows on 16 bytes, the
// contiguous contraction and the result's rows multiples of 16 bytes.  Such an
// operand is laid out anew in the workspace first (zeros behind its rows), a
// result is copied from there.
struct Repack {
  bool a, b, c;
  int64_t lda, ldb, ldc;      // of the copies
  int64_t rows_b, rows_c;
  size_t bytes_a, bytes_b, bytes_c;
  size_t bytes() const { return bytes_a + bytes_b + bytes_c; }
};
Repack repack_of(int layout, int esize, int osize, const RaggedArgs& p) {
  Repack r{};
  const int64_t cols = layout == 0 ? p.N : p.K, ca = layout == 0 ? p.K : p.N;
  const bool odd = layout != 2 && ca * esize % 16 != 0;
  r.a = odd || !on16(p.a, p.lda * esize);
  r.b = (layout == 0 && odd) || !on16(p.b, p.ldb * esize);
  r.c = !on16(p.c, p.ldc * osize) || cols * osize % 16 != 0;
  r.rows_b = layout == 2 ? p.S : (int64_t)p.G * p.N;
  r.rows_c = layout == 2 ? (int64_t)p.G * p.N : p.R;
  r.lda = pad16(ca, esize);
  r.ldb = pad16(p.K, esize);
  r.ldc = pad16(cols, osize);
  r.bytes_a = r.a ? (size_t)(layout == 0 ? p.S : p.R) * r.lda * esize : 0;
  r.bytes_b = r.b ? (size_t)r.rows_b * r.ldb * esize : 0;
  r.bytes_c = r.c ? (size_t)r.rows_c * r.ldc * osize : 0;
  return r;
}
// Copying pays where the arithmetic is long enough.  Measured (us: ragged_any_kernel, the
// copies and the large tiles; rows, N x K, experts):
//   NT  3000, 2011 x 1031, 3:  40,  68   4000, 1003 x 4011, 4: 118, 102   16384, 14331 x 4091, 8: 3830, 2011
//       9000,  777 x 2051, 8:  82, 103   20000, 1021 x 515, 64: 70, 106   8-bit 4000, 1003 x 4011: 75, 89
//   NN  1777,  517 x 1031, 5:  40,  52   3000, 2011 x 1031, 3: 132,  85   9000, 777 x 2051, 8: 154, 101
//   TN  1777,  517 x 1031, 5:  43,  49   600, 4099 x 1003, 1:   94,  55   9000, 777 x 2051, 8: 291, 111
// There a step of 64 contraction bytes takes 1.1 us (NT), 2.1 (NN) and 4.0 (TN) for each
// round of two workgroups a CU, of 256; here 48 us, 1350 TFLOP/s and every byte twice at 4.5 TB/s.
bool repack_pays(int layout, int esize, const RaggedArgs& p, size_t bytes) {
  const double us = layout == 0 ? 1.1 : layout == 1 ? 2.1 : 4.0;
  const double con = layout == 0 ? (double)p.K : layout == 1 ? (double)p.N : (double)p.R / p.G;
  const double rounds = std::max(1.0, (double)ragged_any_blocks(layout, p.R, p.N, p.K, p.G) / 512);
  const double any = 1e-6 * us * std::ceil(con * esize / kAnyBytes) * rounds;
  const double tflop = 2e-12 * (double)p.R * (double)p.N * (double)p.K;
  return bytes <= ((size_t)8 << 30) && any > tflop / 1350.0 + 2.0 * (double)bytes / 4.5e12 + 48e-6;
}
size_t split_bytes() { return ragged_split_bytes(); }

// Lane offsets (256 rows, 64 contraction rows, any gathered row) within 32 bits.
bool tile_spans(int layout, int esize, int osize, const RaggedArgs& p) {
  const int64_t ea = p.lda * esize, eb = p.ldb * esize, ec = p.ldc * osize;
  const int64_t span = (int64_t)kSpan;
  if (256 * ea > span || 256 * eb > span || 256 * ec > span) return false;
  return p.row_index == nullptr || (p.S > 0 && p.S * (layout == 2 ? eb : ea) <= span);
}

// Rows of `bytes` bytes from one pitch to another, 16 bytes a lane, zeros up to
// `fill` bytes.  splits: only the experts' rows.
template <typename E>
__global__ __launch_bounds__(256) void repack_kernel(const uint8_t* src, int64_t src_pitch, uint8_t* dst,
                                                     int64_t dst_pitch, int64_t rows, int64_t bytes,
                                                     int64_t fill, const int64_t* m_splits, int G) {
  if (m_splits != nullptr) rows = wave_row_tile(m_splits, G, rows, 1, -1, true).total;
  const int lane = threadIdx.x & 63;
  for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < rows; r += (int64_t)gridDim.x * 4)
    for (int64_t at = lane * 16; at < fill; at += 64 * 16) {
      const u32x4_t v = load_chunk<E>((const E*)(src + r * src_pitch + at), (bytes - at) / (int64_t)sizeof(E));
      uint8_t* to = dst + r * dst_pitch + at;
      if (at + 16 <= fill) {
        __builtin_memcpy(to, &v, 16);
      } else {
        E e[16 / sizeof(E)];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < (int)(16 / sizeof(E)); ++i)
          if (at + (int64_t)((i + 1) * sizeof(E)) <= fill) ((E*)to)[i] = e[i];
      }
    }
}
template <typename E>
hipError_t repack(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int64_t rows, int64_t n,
                  int64_t fill, const int64_t* m_splits, int G, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  const int64_t size = sizeof(E);
  repack_kernel<E><<<dim3((uint32_t)std::min<int64_t>((rows + 3) / 4, 4096)), dim3(256), 0, st>>>(
      (const uint8_t*)src, ld_src * size, (uint8_t*)dst, ld_dst * size, rows, n * size, fill * size, m_splits, G);
  return hipGetLastError();
}

// Runs `launch` with operands that the large tiles take; *done is false where
// they cannot (no room in the workspace, too large, or not worth it).
template <typename E, typename F>
hipError_t with_tiles(int layout, int osize, RaggedArgs p, size_t ws_bytes, hipStream_t st, bool* done,
                      F launch) {
  const int esize = sizeof(E);
  const int64_t cols = layout == 0 ? p.N : p.K, ca = layout == 0 ? p.K : p.N;
  const Repack r = repack_of(layout, esize, osize, p);
  *done = false;
  uint8_t* ws = (uint8_t*)p.ws;
  if (r.bytes() > 0 && (ws == nullptr || ws_bytes < split_bytes() + r.bytes() ||
                        !repack_pays(layout, esize, p, r.bytes())))
    return hipSuccess;
  RaggedArgs q = p;
  if (ws_bytes < split_bytes()) q.ws = nullptr;
  uint8_t* at = ws + split_bytes();
  if (r.a) q.a = at, q.lda = r.lda, at += r.bytes_a;
  if (r.b) q.b = at, q.ldb = r.ldb, at += r.bytes_b;
  if (r.c) q.c = at, q.ldc = r.ldc;
  q.con = layout == 2 ? 0 : (r.a ? r.lda : ca);
  q.ccols = r.c ? r.ldc : cols;
  if (!tile_spans(layout, esize, osize, q)) return hipSuccess;
  *done = true;
  hipError_t e = hipSuccess;
  if (r.a)
    e = repack<E>(p.a, p.lda, (void*)q.a, r.lda, layout == 0 ? p.S : p.R, ca, r.lda, nullptr, 0, st);
  if (e == hipSuccess && r.b) e = repack<E>(p.b, p.ldb, (void*)q.b, r.ldb, r.rows_b, p.K, r.ldb, nullptr, 0, st);
  if (e == hipSuccess) e = launch(q);
  if (e == hipSuccess && r.c) {
    const int64_t* rows = layout == 2 ? nullptr : p.m_splits;
    if (osize == 4) e = repack<uint32_t>(q.c, r.ldc, p.c, p.ldc, r.rows_c, cols, cols, rows, p.G, st);
    else e = repack<uint16_t>(q.c, r.ldc, p.c, p.ldc, r.rows_c, cols, cols, rows, p.G, st);
  }
  return e;
}

}  // namespace

// Workspace that a product of these sizes uses (0: none), operands contiguous.
size_t ragged_workspace_bytes(int layout, int esize, int64_t R, int64_t S, int64_t N, int64_t K, int32_t G) {
  if (R == 0) return 0;
  RaggedArgs p{};
  p.R = R;
  p.S = S;
  p.N = N;
  p.K = K;
  p.G = G;
  p.lda = layout == 0 ? K : N;
  p.ldb = K;
  p.ldc = layout == 0 ? N : K;
  if (layout == 0 && few_rows(p, esize)) return 0;
  size_t most = 0;
  for (int osize = 2; osize <= 4; osize += 2) {
    const size_t n = repack_of(layout, esize, osize, p).bytes();
    if (n > 0 && repack_pays(layout, esize, p, n)) most = std::max(most, n);
  }
  return split_bytes() + most;
}

hipError_t launch_ragged_gemm(int layout, bool f16, int out, const RaggedArgs& p, size_t ws_bytes,
                              hipStream_t st) {
  if (layout == 0 && few_rows(p, 2)) return launch_ragged_few(f16, out, p, st);
  if (p.R > 0) {
    bool done = false;
    const hipError_t e = with_tiles<uint16_t>(
        layout, out == 0 ? 4 : 2, p, ws_bytes, st, &done, [&](const RaggedArgs& q) {
          return layout == 0   ? launch_ragged_tile_nt(f16, out, q, st)
                 : layout == 1 ? launch_ragged_tile_nn(f16, out, q, st)
                               : launch_ragged_tile_tn(f16, out, q, st);
        });
    if (done || e != hipSuccess) return e;
  }
  if (f16) {
    if (out == 0) return launch_layout<TypeF16, OutF32>(layout, p, st);
    return launch_layout<TypeF16, OutF16>(layout, p, st);
  }
  if (out == 0) return launch_layout<TypeBf16, OutF32>(layout, p, st);
  return launch_layout<TypeBf16, OutBf16>(layout, p, st);
}

hipError_t launch_ragged_gemm_int8(int out, const RaggedArgs& p, size_t ws_bytes, hipStream_t st) {
  if (few_rows(p, 1)) return launch_ragged_few_int8(out, p, st);
  bool done = false;
  const hipError_t e = with_tiles<uint8_t>(
      0, out == 0 ? 4 : 2, p, ws_bytes, st, &done,
      [&](const RaggedArgs& q) { return launch_ragged_tile_int8(out, q, st); });
  if (done || e != hipSuccess) return e;
  if (out == 0) return launch_any<TypeI8, OutF32, 0>(p, st);
  if (out == 1) return launch_any<TypeI8, OutBf16, 0>(p, st);
  return launch_any<TypeI8, OutF16, 0>(p, st);
}

// Workgroups that any call may need at most.
int64_t ragged_blocks(int layout, int64_t R, int64_t N, int64_t K, int32_t G) {
  const int64_t any = ragged_any_blocks(layout, R, N, K, G);
  // the smallest tiles: 16 rows by 16 columns, where rows are few
  if (layout != 0 || R >= (1 << 20)) return any;
  return std::max(any, ((N + 15) / 16) * (R / 16 + std::min<int64_t>(G, R)));
}

}  // namespace mx

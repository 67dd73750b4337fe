// The launch of one large-tile product (ragged_tile.h).  Each layout's kernels
// are compiled in a file of their own.
#pragma once

#include <algorithm>

#include "ragged_tile.h"

namespace mx {

inline int compute_units() {
  int dev = 0, cus = 256;
  if (hipGetDevice(&dev) == hipSuccess)
    (void)hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
  return cus;
}

template <typename T, typename O, int LAYOUT, int FA, bool GATHER>
hipError_t launch_tile(const RaggedArgs& p, hipStream_t st) {
  const int64_t m = 64 * FA, cols = ((LAYOUT == 0 ? p.N : p.K) + kTileN - 1) / kTileN;
  // one workgroup per CU; fewer where there are fewer tiles than CUs and no
  // workspace to split them
  const int64_t most = p.ws != nullptr ? INT32_MAX : cols * (LAYOUT == 2 ? p.G * ((p.N + m - 1) / m)
                                           : p.R / m + std::min<int64_t>(p.G, p.R));
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, compute_units()));
  ragged_tile_kernel<T, O, LAYOUT, FA, GATHER><<<dim3(grid), dim3(256), 0, st>>>(p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.ws == nullptr) return e;
  // half the tiles of a round at most are split, 8 FA strips each
  const unsigned strips = std::max(1u, grid / 2) * 8 * FA;
  ragged_join_kernel<T, O, LAYOUT, FA><<<dim3(std::min(strips, 1024u)), dim3(256), 0, st>>>(p, grid);
  return hipGetLastError();
}

template <typename T, typename O, int LAYOUT, int FA>
hipError_t launch_tile_gather(const RaggedArgs& p, hipStream_t st) {
  return p.row_index != nullptr ? launch_tile<T, O, LAYOUT, FA, true>(p, st)
                                : launch_tile<T, O, LAYOUT, FA, false>(p, st);
}

// Rows of a forward tile.  Experts of few rows want low tiles: what the copies
// bring of other experts' rows is wasted.  Measured, 8 x 4096 x 14336 bf16, for
// 64, 128 and 256 rows a tile: 210, 216 and 237 us at 32 rows an expert; 283, 224
// and 249 at 96; 371, 310 and 261 at 192.  The bounds lie lower than the tile
// heights because experts differ from the mean, which is over all of them, those without
// rows too: only the device knows the splits.
template <typename T, typename O>
hipError_t launch_tile_rows(const RaggedArgs& p, hipStream_t st) {
  const int64_t mean = p.R / std::min<int64_t>(p.G, p.R);
  if (mean <= 32) return launch_tile_gather<T, O, 0, 1>(p, st);
  if (mean <= 96) return launch_tile_gather<T, O, 0, 2>(p, st);
  return launch_tile_gather<T, O, 0, 4>(p, st);
}

}  // namespace mx

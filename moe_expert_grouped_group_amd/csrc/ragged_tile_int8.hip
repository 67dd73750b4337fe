// Large tiles of the forward product in 8-bit integers.
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_int8(int out, const RaggedArgs& p, hipStream_t st) {
  if (out == 0) return launch_tile_rows<TypeI8, OutF32>(p, st);
  if (out == 1) return launch_tile_rows<TypeI8, OutBf16>(p, st);
  return launch_tile_rows<TypeI8, OutF16>(p, st);
}

size_t ragged_split_bytes() { return (size_t)compute_units() * 256 * 256 * 4; }

}  // namespace mx

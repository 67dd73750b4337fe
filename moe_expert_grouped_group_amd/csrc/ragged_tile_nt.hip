// Large tiles of the forward product (NT).
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_nt(bool f16, int out, const RaggedArgs& p, hipStream_t st) {
  if (f16)
    return out == 0 ? launch_tile_rows<TypeF16, OutF32>(p, st)
                    : launch_tile_rows<TypeF16, OutF16>(p, st);
  return out == 0 ? launch_tile_rows<TypeBf16, OutF32>(p, st)
                  : launch_tile_rows<TypeBf16, OutBf16>(p, st);
}

}  // namespace mx

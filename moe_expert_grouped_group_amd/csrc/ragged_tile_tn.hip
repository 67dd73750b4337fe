// Large tiles of the weight's gradient (TN).
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_tn(bool f16, int out, const RaggedArgs& p, hipStream_t st) {
  if (f16)
    return out == 0 ? launch_tile_gather<TypeF16, OutF32, 2, 4>(p, st)
                    : launch_tile_gather<TypeF16, OutF16, 2, 4>(p, st);
  return out == 0 ? launch_tile_gather<TypeBf16, OutF32, 2, 4>(p, st)
                  : launch_tile_gather<TypeBf16, OutBf16, 2, 4>(p, st);
}

}  // namespace mx

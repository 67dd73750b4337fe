// Large tiles of the gated block's backward product (NN).
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_gated_bwd(bool f16, const RaggedArgs& p, hipStream_t st) {
  return f16 ? launch_tile<TypeF16, OutF16, 1, 4, false, kGatedBwd>(p, st)
             : launch_tile<TypeBf16, OutBf16, 1, 4, false, kGatedBwd>(p, st);
}

}  // namespace mx

// Large tiles of the input's gradient (NN).
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_nn(bool f16, int out, const RaggedArgs& p, hipStream_t st) {
  if (f16)
    return out == 0 ? launch_tile<TypeF16, OutF32, 1, 4, false>(p, st)
                    : launch_tile<TypeF16, OutF16, 1, 4, false>(p, st);
  return out == 0 ? launch_tile<TypeBf16, OutF32, 1, 4, false>(p, st)
                  : launch_tile<TypeBf16, OutBf16, 1, 4, false>(p, st);
}

}  // namespace mx

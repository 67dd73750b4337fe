// Large tiles of the gated forward product (NT) in fp16.
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_gated_f16(const RaggedArgs& p, hipStream_t st) {
  return p.h != nullptr ? launch_tile_rows<TypeF16, OutF16, kGatedKeep>(p, st)
                        : launch_tile_rows<TypeF16, OutF16, kGated>(p, st);
}

}  // namespace mx

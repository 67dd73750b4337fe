// Large tiles of the gated forward product (NT) in bf16; ragged_tile_gated_f16.hip has fp16.
#include "ragged_tile_launch.h"

namespace mx {

hipError_t launch_ragged_tile_gated(bool f16, const RaggedArgs& p, hipStream_t st) {
  if (f16) return launch_ragged_tile_gated_f16(p, st);
  return p.h != nullptr ? launch_tile_rows<TypeBf16, OutBf16, kGatedKeep>(p, st)
                        : launch_tile_rows<TypeBf16, OutBf16, kGated>(p, st);
}

}  // namespace mx

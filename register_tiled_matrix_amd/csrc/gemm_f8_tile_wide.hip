// gemm_f8_tile_wide.hip -- 256 x 128 tiles of gemm_f8_tile.h, 8 waves of 64 x 64, 2 to a SIMD: what 256 x 256 tiles
// have no registers for.
#include "gemm_f8_tile.h"

namespace regtile {
hipError_t launch_f8_tile_wide(const F8Problem &p, bool exact, hipStream_t s, int splits) {
    return exact ? f8::launch_tile_of<4, 2, 4, 4, 2, true>(p, s, splits) : f8::launch_tile_of<4, 2, 4, 4, 2, false>(p, s, splits);
}
}  // namespace regtile

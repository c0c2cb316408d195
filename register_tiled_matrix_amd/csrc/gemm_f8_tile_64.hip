// gemm_f8_tile_64.hip -- 64 x 64 tiles of gemm_f8_tile.h: 4 waves of 32 x 32, for few tiles or few rows in a group.
#include "gemm_f8_tile.h"

namespace regtile {
hipError_t launch_f8_tile_64(const F8Problem &p, bool exact, hipStream_t s, int splits) {
    return exact ? f8::launch_tile_of<2, 2, 2, 2, 3, true>(p, s, splits) : f8::launch_tile_of<2, 2, 2, 2, 3, false>(p, s, splits);
}
}  // namespace regtile

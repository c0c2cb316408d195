// gemm_f8_tile_128.hip -- 128 x 128 tiles of gemm_f8_tile.h: 4 waves of 64 x 64, two workgroups to a CU.
#include "gemm_f8_tile.h"

namespace regtile {
hipError_t launch_f8_tile_128(const F8Problem &p, bool exact, hipStream_t s, int splits) {
    return exact ? f8::launch_tile_of<2, 2, 4, 4, 2, true>(p, s, splits) : f8::launch_tile_of<2, 2, 4, 4, 2, false>(p, s, splits);
}
}  // namespace regtile

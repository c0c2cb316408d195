// gemm_f8_tile_deep.hip -- 128 x 128 tiles of gemm_f8_tile.h with four stages, one workgroup to a CU: for few tiles.
#include "gemm_f8_tile.h"

namespace regtile {
hipError_t launch_f8_tile_deep(const F8Problem &p, bool exact, hipStream_t s, int splits) {
    return exact ? f8::launch_tile_of<2, 2, 4, 4, 4, true>(p, s, splits) : f8::launch_tile_of<2, 2, 4, 4, 4, false>(p, s, splits);
}
}  // namespace regtile

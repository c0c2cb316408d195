// gemm_f8_tile_256.hip -- 256 x 256 tiles of gemm_f8_tile.h, 8 waves of 128 x 64, 2 to a SIMD: the 8-bit matrix
// instructions with one scale of B for 128 columns.
#include "gemm_f8_tile.h"

namespace regtile {
hipError_t launch_f8_tile_256(const F8Problem &p, hipStream_t s) {
    if (p.b.step != 1) return p.a.type ? f8::launch_tile<2, 4, 8, 4, 2, false, 1, true, false>(p, s, 1) : f8::launch_tile<2, 4, 8, 4, 2, false, 0, true, false>(p, s, 1);
    return p.a.type ? f8::launch_tile<2, 4, 8, 4, 2, false, 1, false, false>(p, s, 1) : f8::launch_tile<2, 4, 8, 4, 2, false, 0, false, false>(p, s, 1);
}
}  // namespace regtile

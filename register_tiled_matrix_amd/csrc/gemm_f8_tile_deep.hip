// gemm_f8_tile_deep.hip -- 128 x 128 tiles of gemm_f8_tile.h with four stages, one workgroup to a CU: for few tiles on the
// 8-bit matrix instructions (bf16 ones take twice as long for a block, and gain nothing).
#include "gemm_f8_tile.h"

namespace regtile {
hipError_t launch_f8_tile_deep(const F8Problem &p, hipStream_t s) {
    return f8::launch_tile_of<2, 2, 4, 4, 4, false>(p, s, 1);
}
}  // namespace regtile

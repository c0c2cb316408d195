// gemm_f8.hip -- which kernel takes a product of 8-bit float matrices, in how many parts of k, and the sum of
// the parts.
#include "f8_common.h"
#include "regtile.h"

namespace regtile {
namespace {
using namespace f8;
using mfma::f32x4;

constexpr int JOIN_NT = 256;

// C = alpha (sum of the parts, in order) + beta C: 4 columns a thread
__global__ __launch_bounds__(JOIN_NT) void f8_join_kernel(F8Problem p, int splits, int units, bool wide, bool wide_parts) {
    const int64_t n = (int64_t)p.M * units, part = (int64_t)p.M * p.N;
    for (int64_t u = (int64_t)blockIdx.x * JOIN_NT + threadIdx.x; u < n; u += (int64_t)gridDim.x * JOIN_NT) {
        const int64_t row = u / units;
        const int col = (int)(u - row * units) * 4, count = min(p.N - col, 4);
        const float *at = static_cast<const float *>(p.work) + row * p.N + col;
        f32x4 sum = {};
        for (int i = 0; i < splits; ++i, at += part) {
            if (wide_parts && count == 4) {
                sum += *reinterpret_cast<const f32x4 *>(at);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (v < count) sum[v] += at[v];
            }
        }
        c_store4(p.out, row, col, count, p.alpha, p.beta, sum, wide);
    }
}

constexpr int64_t SPAN = int64_t(1) << 31;  // bytes that a descriptor's offsets may reach

// What the DMA-fed tiles take: K-contiguous A, e4m3 B, aligned rows, and operands within the reach of a tile's
// descriptors
bool tile_takes(const F8Problem &p) {
    const F8Operand &a = p.a, &b = p.b;
    const bool nn = b.step != 1;
    const int64_t ldb = nn ? b.step : b.row, kb = ((int64_t)p.K + BLOCK - 1) / BLOCK;
    if (a.step != 1 || b.type != REGTILE_F8_E4M3) return false;
    if (!aligned16(a.q) || !aligned16(b.q) || a.row % 16 != 0 || ldb % 16 != 0 || p.b_stack % 16 != 0) return false;
    const int64_t rows_a = p.slots != nullptr ? p.a_rows : 256;
    if (rows_a * a.row + p.K + BLOCK >= SPAN || (nn ? ((int64_t)p.K + BLOCK) * ldb + 256 : 256 * ldb + p.K + BLOCK) >= SPAN) return false;
    const int64_t all_a = p.slots != nullptr ? p.a_rows : p.M;
    return ((all_a >> a.shift) * a.s_row + kb * a.s_col) * 4 < SPAN && (((int64_t)p.N >> b.shift) * b.s_row + kb * b.s_col) * 4 < SPAN;
}

struct Plan {
    enum { ANY, TILE_128, TILE_WIDE, TILE_256 } kernel;
    bool exact;
    int parts;  // of k, through the workspace
};

Plan plan_of(const F8Problem &p) {
    Plan plan = {Plan::ANY, p.out.dtype == 0, 1};
    if (!tile_takes(p)) return plan;
    const int64_t tiles256 = most_row_tiles(p, 256) * (((int64_t)p.N + 255) / 256);
    const int64_t tiles128 = most_row_tiles(p, 128) * (((int64_t)p.N + 127) / 128) * (p.mode == F8Problem::DEPTH ? p.experts : 1);
    // 256 x 256 tiles run one to a CU: with fewer than 192 too many of the 256 CUs are idle (2048^3, 64 tiles: 35.3 us
    // against 20.9; 4096 x 4096 x 8192, 256 tiles: 130 against 161)
    if (!plan.exact && p.b.shift != 0 && tiles256 >= 192 && p.mode != F8Problem::ROWS) {
        plan.kernel = Plan::TILE_256;
        return plan;
    }
    plan.kernel = Plan::TILE_128;
    // two 128 x 128 tiles run on a CU: fewer than 512 of them go in parts of at least 1024 k (1024 x 1024 x 8192, 64
    // tiles: 63.9 us whole, 27.4 in 4 parts, 27.2 in 8; 2048 x 2048 x 2048: 20.9 whole, 28.7 in 2)
    if (p.mode == F8Problem::DENSE) {
        const int64_t blocks = ((int64_t)p.K + BLOCK - 1) / BLOCK, fill = 512 / tiles128;
        plan.parts = (int)(fill < blocks / 8 ? fill : blocks / 8);
        if (plan.parts < 1 || (tiles128 >= 256 && blocks < 32)) plan.parts = 1;
    }
    return plan;  // tuned
}

}  // namespace

int64_t f8_work_bytes(const F8Problem &p) {
    const int parts = plan_of(p).parts;
    return parts > 1 ? (int64_t)parts * p.M * p.N * 4 : 0;
}

hipError_t launch_f8(const F8Problem &p, hipStream_t s, const char **name) {
    Plan plan = plan_of(p);
    while (plan.parts > 1 && (int64_t)plan.parts * p.M * p.N * 4 > p.work_bytes) --plan.parts;
    static const char *const wide[2] = {"f8_tile_256x128", "f8_tile_256x128_exact"};
    static const char *const small[2] = {"f8_tile_128x128", "f8_tile_128x128_exact"};
    switch (plan.kernel) {
        case Plan::TILE_256: *name = "f8_tile_256x256"; return launch_f8_tile_256(p, s);
        case Plan::TILE_WIDE: *name = wide[plan.exact]; return launch_f8_tile_wide(p, plan.exact, s, plan.parts);
        case Plan::TILE_128: *name = small[plan.exact]; return launch_f8_tile_128(p, plan.exact, s, plan.parts);
        default: return launch_f8_any(p, s, name);
    }
}

hipError_t launch_f8_join(const F8Problem &p, hipStream_t s, int splits) {
    const int units = (int)(((int64_t)p.N + 3) / 4);
    const int64_t groups = ((int64_t)p.M * units + JOIN_NT - 1) / JOIN_NT;
    hipLaunchKernelGGL(f8_join_kernel, dim3((unsigned)(groups < 4096 ? groups : 4096)), dim3(JOIN_NT), 0, s, p, splits, units, c_wide(p),
                       p.N % 4 == 0);
    return hipGetLastError();
}

}  // namespace regtile

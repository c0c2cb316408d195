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

// Rows that DMA reads begin at multiples of 16 bytes; operands that lie otherwise are copied into a workspace first.
bool a_aligned(const F8Problem &p) { return aligned16(p.a.q) && p.a.row % 16 == 0; }
bool b_aligned(const F8Problem &p) { return aligned16(p.b.q) && (p.b.step != 1 ? p.b.step : p.b.row) % 16 == 0 && p.b_stack % 16 == 0; }

// A's and B's stored matrices: rows, columns, how many
struct Stored {
    int64_t rows, cols, count;
    int64_t ld() const { return (cols + 15) / 16 * 16; }
    int64_t bytes() const { return rows * ld() * count; }
};
Stored stored_a(const F8Problem &p) { return {p.slots != nullptr ? p.a_rows : p.M, p.K, 1}; }
Stored stored_b(const F8Problem &p) {
    const int64_t count = p.mode == F8Problem::ROWS ? p.experts : 1;
    return p.b.step != 1 ? Stored{p.K, p.N, count} : Stored{p.N, p.K, count};
}

// One matrix (or stack) to aligned rows: 16 bytes a thread, a row of threads along each row; what lies behind a
// row's end up to a multiple of 16 becomes 0.
struct Copy {
    const uint8_t *from;
    uint8_t *to;
    int64_t ld, stack, to_ld;
    int64_t rows, cols, count;
    int across;  // threads to a row
};
constexpr int COPY_NT = 256;
__global__ __launch_bounds__(COPY_NT) void f8_align_kernel(Copy c0, Copy c1, int z1) {
    const bool second = (int)blockIdx.z >= z1;
    const Copy c = second ? c1 : c0;
    const int z = second ? blockIdx.z - z1 : blockIdx.z, nz = second ? gridDim.z - z1 : z1;
    const int across = c.across, tx = threadIdx.x % across, ty = threadIdx.x / across;
    for (int64_t e = z; e < c.count; e += nz)
        for (int64_t r = (int64_t)blockIdx.x * (COPY_NT / across) + ty; r < c.rows; r += (int64_t)gridDim.x * (COPY_NT / across)) {
            const uint8_t *from = c.from + e * c.stack + r * c.ld;
            uint8_t *to = c.to + (e * c.rows + r) * c.to_ld;
            for (int64_t k = ((int64_t)blockIdx.y * across + tx) * 16; k < c.cols; k += (int64_t)gridDim.y * across * 16)
                *reinterpret_cast<mfma::u32x4 *>(to + k) = load16(from + k, (int)min(c.cols - k, (int64_t)16), (int)min(k, (int64_t)16));
        }
}
// Copies of one or two operands (count 0: none), in one launch
hipError_t align_rows(Copy a, Copy b, hipStream_t s) {
    int64_t gx = 1, gy = 1;
    for (Copy *c : {&a, &b}) {
        const int64_t units = (c->cols + 15) / 16;
        c->across = COPY_NT;
        while (c->across > 8 && c->across / 2 >= units) c->across /= 2;
        const int64_t x = (c->rows * c->across + COPY_NT - 1) / COPY_NT, y = (units + c->across - 1) / c->across;
        if (c->count > 0 && x > gx) gx = x;
        if (c->count > 0 && y > gy) gy = y;
    }
    const int za = (int)(a.count < 1024 ? a.count : 1024), zb = (int)(b.count < 1024 ? b.count : 1024);
    hipLaunchKernelGGL(f8_align_kernel, dim3((unsigned)(gx < (1 << 16) ? gx : 1 << 16), (unsigned)(gy < 64 ? gy : 64), (unsigned)(za + zb)),
                       dim3(COPY_NT), 0, s, a, b, za);
    return hipGetLastError();
}

// Scales of 1 x 128 blocks whose rows are apart: a block's load by DMA then touches a line for each row, as many as the
// codes' loads together. Products of 2^37 operations or more have them turned in the workspace first (8192^3: 497 us
// against 449 with turned scales, 4096^3 with both operands' so 94 against 83; turning takes about 5).
bool scales_apart(const F8Problem &p, const F8Operand &o, int64_t rows) {
    const double work = 2.0 * p.M * p.N * p.K;
    const int64_t turned = rows * (((int64_t)p.K + BLOCK - 1) / BLOCK) * 4;
    return o.shift == 0 && o.s_row != 1 && work >= (double)(int64_t(1) << 37) && turned < int64_t(1) << 31;
}
struct Turn {
    const float *from;
    float *to;
    int64_t s_row, s_col, rows, blocks;
};
int64_t turned_bytes(int64_t rows, int64_t blocks) { return (rows * blocks * 4 + 15) / 16 * 16; }
// 64 rows x 64 blocks at a time, through LDS
__global__ __launch_bounds__(256) void f8_turn_scales_kernel(Turn a, Turn b, int ya) {
    __shared__ float tile[64][65];
    const bool second = (int)blockIdx.y >= ya;
    const Turn t = second ? b : a;
    const int y = second ? blockIdx.y - ya : blockIdx.y, ny = second ? gridDim.y - ya : ya;
    const int x = threadIdx.x & 63, z = threadIdx.x >> 6;
    for (int64_t k0 = (int64_t)y * 64; k0 < t.blocks; k0 += (int64_t)ny * 64)
        for (int64_t r0 = (int64_t)blockIdx.x * 64; r0 < t.rows; r0 += (int64_t)gridDim.x * 64) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int64_t r = min(r0 + z * 16 + i, t.rows - 1), k = min(k0 + x, t.blocks - 1);
                tile[z * 16 + i][x] = t.from[r * t.s_row + k * t.s_col];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k0 + z * 16 + i < t.blocks && r0 + x < t.rows) t.to[(k0 + z * 16 + i) * t.rows + r0 + x] = tile[x][z * 16 + i];
            __syncthreads();
        }
}

// What the tiles take: K-contiguous A, e4m3 B, and operands within the reach of a tile's 32-bit offsets
bool tile_takes(const F8Problem &p) {
    const F8Operand &a = p.a, &b = p.b;
    const bool nn = b.step != 1;
    auto whole = [](int64_t ld) { return (ld + 15) / 16 * 16; };  // (a copy's rows may be that far apart)
    const int64_t lda = whole(a.row), ldb = whole(nn ? b.step : b.row), kb = ((int64_t)p.K + BLOCK - 1) / BLOCK;
    if (a.step != 1 || b.type != REGTILE_F8_E4M3) return false;
    if (!addr::f8_reach(false, p.slots != nullptr ? p.a_rows : 256, p.K, lda) || !addr::f8_reach(nn, 256, p.K, ldb)) return false;
    const int64_t all_a = p.slots != nullptr ? p.a_rows : p.M;
    return addr::f8_scales_reach(all_a >> a.shift, a.s_row, kb, a.s_col) && addr::f8_scales_reach((int64_t)p.N >> b.shift, b.s_row, kb, b.s_col);
}

struct Plan {
    enum { ANY, TILE_128, TILE_256, TOKEN, TILE_DEEP, TILE_64 } kernel;
    int shape;
    bool exact;
    int parts;     // of k, through the workspace
    bool copy_a, copy_b;  // operands that it needs copies of,
    bool turn_a, turn_b;  // and whose scales it wants turned
    int64_t copy_bytes, turn_bytes;
};

Plan plan_of(const F8Problem &p) {
    Plan plan = {Plan::ANY, 0, p.out.dtype == 0, 1, false, false, false, false, 0, 0};
    if (p.K == 0 || !tile_takes(p)) return plan;
    const bool dense = p.mode == F8Problem::DENSE, rows = p.mode == F8Problem::ROWS;
    // Few rows: codes straight to registers. us on 128 x 128 tiles: 16x4096x4096 13.0, here 6.8. Of rows in groups that pays up to
    // 16 in all, and where B's rows would have to be copied first (50 us for 32 x 2048 x 4096, and 70.6 here). 64 x 64 tiles,
    // here: 1 token x 2 of 8 experts (4096 x 4096) 13.0, 9.3; x 6 of 64 (4096 x 2048) 12.7, 12.2; 4 x 6 of 64 27.7, 32.0;
    // 8 x 2 of 8 21.1, 30.4; 32 x 6 of 64 96.6, 106.
    const int64_t weights = (int64_t)p.N * p.K, group = rows ? p.mean_rows : p.M;
    // (a launch counts 2^23 of its workgroups, which take 16 rows and 16 columns or more)
    const int64_t most_token = most_row_tiles(p, 16) * (((int64_t)p.N + 15) / 16);
    if (p.b.step == 1 && (dense || rows) && most_token < 1 << 23) {
        plan.kernel = Plan::TOKEN;
        if (dense && p.M <= 16) return plan.shape = 11, plan;
        // (32x4096x4096 9.0, on 64 x 64 tiles 10.0; 32x4096x8192 14.4, 11.7; 48x1024x4096 8.4, 9.3; 64x4096x4096 12.0, 11.1,
        // and 10 more to copy unaligned rows)
        const bool aligned = a_aligned(p) && b_aligned(p);
        if (dense && p.M <= 32 && weights <= 1 << (aligned ? 24 : 27)) return plan.shape = 21, plan;
        if (dense && p.M <= 64 && weights <= 1 << 22) return plan.shape = 21, plan;
        if (dense && p.M <= 64 && !aligned && weights <= 1 << 27) return plan.shape = 22, plan;
        if (rows && (p.n_slots <= 16 || (!b_aligned(p) && group <= 48))) return plan.shape = 12, plan;
    }
    plan.copy_a = !a_aligned(p);
    plan.copy_b = !b_aligned(p);
    plan.turn_a = scales_apart(p, p.a, stored_a(p).rows);
    plan.turn_b = !rows && scales_apart(p, p.b, p.N);
    const int64_t blocks = ((int64_t)p.K + BLOCK - 1) / BLOCK;
    plan.copy_bytes = (plan.copy_a ? stored_a(p).bytes() : 0) + (plan.copy_b ? stored_b(p).bytes() : 0);
    plan.turn_bytes = (plan.turn_a ? turned_bytes(stored_a(p).rows, blocks) : 0) + (plan.turn_b ? turned_bytes(p.N, blocks) : 0);
    auto tiles = [&](int64_t side) {
        return most_row_tiles(p, (int)side) * (((int64_t)p.N + side - 1) / side) * (p.mode == F8Problem::DEPTH ? p.experts : 1);
    };
    // 64 x 64 tiles while there are at most 512 of them, or few rows in a group. us on 128 x 128 (best of two and four stages
    // and parts of k), here: 1024^3 10.5, 5.5 (fp32 C 14.2, 7.1); 1024x1024x4096 21.6, 12.3 (25.6, 19.7); 296x2984x1056 11.2,
    // 7.5; 2048^3, 1024 tiles, 16.5, 18.8 (25.3, 27.7); 32 tokens x 6 of 64 experts 107, 97.7; 256 x 8 of 128 190, 160;
    // 256 x 6 of 64 114, 117; 1024 x 6 of 64 145, 210.
    // They go in parts of at least 1024 k, one workgroup to a CU (K x N B, whole, 2 and 4 parts: 1216x176x4720 16.3, 13.2, 11.5,
    // 256x1024x4096 13.6, 11.8, 10.7; two to a CU cost more in the join: 1024x1024x4096 12.3 whole, 16.7 in 2). Two parts
    // of the 8-bit instructions take at least 2048 (64x2048x2048 7.5 whole, 8.7 in 2; 64x8192x8192 27.0, 20.5).
    const int64_t tiles64 = tiles(64);
    if (rows ? group <= 48 : tiles64 <= 512) {
        plan.kernel = Plan::TILE_64;
        if (dense) {
            const int64_t fill = 256 / tiles64, most = blocks / 8;
            plan.parts = (int)(fill < most ? fill : most);
            if (plan.parts < 1 || (plan.parts == 2 && !plan.exact && blocks < 32)) plan.parts = 1;
        }
        return plan;
    }
    // 256 x 256 tiles run one to a CU: with fewer than 192 too many of the 256 CUs are idle (2048^3, 64 tiles: 31.7
    // us against 16.5; 4096 x 4096 x 8192, 256 tiles: 107 against 128). Groups of fewer than 128 rows leave them too empty (64
    // experts of 4096 x 2048 with 96 rows on the average: 171 us against 145; 141 rows: 176 against 182)
    if (!plan.exact && p.b.shift != 0 && p.mode != F8Problem::DEPTH && tiles(256) >= 192 && (!rows || group >= 128)) {
        plan.kernel = Plan::TILE_256;
        return plan;
    }
    // 128 x 128 tiles (129 or more of them: else there are at most 512 of 64 x 64). The bf16 instructions' go in parts of at
    // least 1024 k while they are fewer than the chip holds, two to a CU with two stages (2048 x 1504 x 8096: 80 us whole, 70 in
    // 2 parts; with four stages 78). The 8-bit instructions' run one to a CU with four stages while there is one for each (2048^3,
    // 256 tiles: 16.5, with two stages 17.5).
    plan.kernel = Plan::TILE_128;
    if (dense) {
        const int64_t tiles128 = tiles(128), fill = 512 / tiles128;
        if (plan.exact) plan.parts = (int)(fill < blocks / 8 ? fill : blocks / 8);
        if (plan.parts < 1) plan.parts = 1;
        if (!plan.exact && tiles128 <= 256) plan.kernel = Plan::TILE_DEEP;
    }
    return plan;
}

}  // namespace

int64_t f8_work_bytes(const F8Problem &p) {
    const Plan plan = plan_of(p);
    return plan.copy_bytes + plan.turn_bytes + (plan.parts > 1 ? (int64_t)plan.parts * p.M * p.N * 4 : 0);
}

hipError_t launch_f8(const F8Problem &given, hipStream_t s, const char **name) {
    Plan plan = plan_of(given);
    F8Problem p = given;
    // what there is no room for: scales can stay as they are, rows cannot
    if (plan.copy_bytes > p.work_bytes) return launch_f8_any(p, s, name);
    if (plan.copy_bytes + plan.turn_bytes > p.work_bytes) {
        plan.turn_a = plan.turn_b = false;
        plan.turn_bytes = 0;
    }
    uint8_t *work = static_cast<uint8_t *>(p.work);
    Copy copies[2] = {};
    if (plan.copy_a) {
        const Stored m = stored_a(p);
        copies[0] = {p.a.q, work, p.a.row, 0, m.ld(), m.rows, m.cols, 1, 0};
        p.a.q = work;
        p.a.row = m.ld();
        work += m.bytes();
    }
    if (plan.copy_b) {
        const Stored m = stored_b(p);
        int64_t &ld = p.b.step != 1 ? p.b.step : p.b.row;
        copies[1] = {p.b.q, work, ld, p.b_stack, m.ld(), m.rows, m.cols, m.count, 0};
        p.b.q = work;
        p.b_stack = m.rows * m.ld();
        ld = m.ld();
        work += m.bytes();
    }
    if (plan.copy_a || plan.copy_b) {
        const hipError_t e = align_rows(copies[0], copies[1], s);
        if (e != hipSuccess) return e;
    }
    Turn turns[2] = {};
    if (plan.turn_a) {
        const int64_t rows = stored_a(p).rows, blocks = ((int64_t)p.K + BLOCK - 1) / BLOCK;
        turns[0] = {p.a.s, reinterpret_cast<float *>(work), p.a.s_row, p.a.s_col, rows, blocks};
        p.a.s = turns[0].to;
        p.a.s_row = 1;
        p.a.s_col = rows;
        work += turned_bytes(rows, blocks);
    }
    if (plan.turn_b) {
        const int64_t rows = p.N, blocks = ((int64_t)p.K + BLOCK - 1) / BLOCK;
        turns[1] = {p.b.s, reinterpret_cast<float *>(work), p.b.s_row, p.b.s_col, rows, blocks};
        p.b.s = turns[1].to;
        p.b.s_row = 1;
        p.b.s_col = rows;
        work += turned_bytes(rows, blocks);
    }
    if (plan.turn_a || plan.turn_b) {
        const int64_t rows = turns[0].rows > turns[1].rows ? turns[0].rows : turns[1].rows, gx = (rows + 63) / 64;
        auto tiles = [](const Turn &t) { return (int)((t.blocks + 63) / 64 < 1024 ? (t.blocks + 63) / 64 : 1024); };
        const int ya = tiles(turns[0]), yb = tiles(turns[1]);
        hipLaunchKernelGGL(f8_turn_scales_kernel, dim3((unsigned)(gx < (1 << 16) ? gx : 1 << 16), (unsigned)(ya + yb)), dim3(256), 0, s,
                           turns[0], turns[1], ya);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    p.work = work;
    p.work_bytes -= plan.copy_bytes + plan.turn_bytes;
    while (plan.parts > 1 && (int64_t)plan.parts * p.M * p.N * 4 > p.work_bytes) --plan.parts;
    static const char *const small[2] = {"f8_tile_128x128", "f8_tile_128x128_exact"};
    static const char *const tiny[2] = {"f8_tile_64x64", "f8_tile_64x64_exact"};
    switch (plan.kernel) {
        case Plan::TILE_256: *name = "f8_tile_256x256"; return launch_f8_tile_256(p, s);
        case Plan::TILE_128: *name = small[plan.exact]; return launch_f8_tile_128(p, plan.exact, s, plan.parts);
        case Plan::TILE_64: *name = tiny[plan.exact]; return launch_f8_tile_64(p, plan.exact, s, plan.parts);
        case Plan::TILE_DEEP: *name = "f8_tile_128x128_deep"; return launch_f8_tile_deep(p, s);
        case Plan::TOKEN: *name = "f8_token"; return launch_f8_token(p, plan.shape, s);
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

// gemm_f8_token.hip -- C = alpha A B + beta C for block-scaled 8-bit floats with a few rows of A (or a few in each
// group) and B stored N x K: the weights' bytes are what counts.
//
// Codes go from memory to registers at any alignment, without LDS. A workgroup of 8 waves takes 16 NF columns and
// 16 MF rows; wave w takes the blocks w, w + 8, ... of 128 k, U of them under way, so that a workgroup reads
// 1 KB of each column at a time. Codes are expanded and summed exactly, whatever C's type (the matrix pipes have time).
// The waves' sums are added through LDS in their order. Bound by the latency of its loads, and by the weights' bytes where
// they come from memory: 1x4096x4096 5.9 us (16.8 MB, 2.8 TB/s), 16x8192x8192 18.8 from the cache and
// 23.7 from memory (67 MB, 2.8 TB/s), each wave's loads and products in turn.
#include "f8_common.h"

namespace regtile {
namespace {
using namespace f8;
using namespace mfma;

constexpr int WAVES = 8, NT = 64 * WAVES;

template <int MF, int NF, int U, int TA, bool SB>
__global__ __launch_bounds__(NT) void f8_token_kernel(F8Problem p, int tiles_n, bool wide) {
    __shared__ f32x4 part[WAVES][MF * NF][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int fr = lane & 15, fg = lane >> 4;
    const int tile = blockIdx.x / tiles_n, n0 = (blockIdx.x - tile * tiles_n) * 16 * NF;
    Work w;
    if (!work_of(p, 16 * MF, tile, 0, w)) return;
    const int K = w.used > 0 ? w.K : 0, all = (K + BLOCK - 1) / BLOCK, whole = K / BLOCK;
    f32x4 acc[MF][NF] = {};
    if (wave < all) {
        const uint8_t *ap[MF], *bp[NF];
        const float *sa[MF], *sb[NF][SB ? 4 : 1];
#pragma unroll
        for (int i = 0; i < MF; ++i) {
            const int64_t row = a_row(p, w, min(i * 16 + fr, w.used - 1));
            ap[i] = w.a.q + row * w.a.row + fg * 16;
            sa[i] = w.a.s + (row >> w.a.shift) * w.a.s_row;
        }
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            bp[j] = w.b.q + (int64_t)min(n0 + j * 16 + fr, p.N - 1) * w.b.row + fg * 16;
#pragma unroll
            for (int v = 0; v < (SB ? 4 : 1); ++v)
                sb[j][v] = w.b.s + (int64_t)(min(n0 + j * 16 + (SB ? fg * 4 + v : 0), p.N - 1) >> w.b.shift) * w.b.s_row;
        }
        u32x4 qa[U][MF][2], qb[U][NF][2];
        float fa[U][MF], fb[U][NF][SB ? 4 : 1];
        auto scales = [&](int u, int kb) {
#pragma unroll
            for (int i = 0; i < MF; ++i) fa[u][i] = sa[i][kb * w.a.s_col];
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
                for (int v = 0; v < (SB ? 4 : 1); ++v) fb[u][j][v] = sb[j][v][kb * w.b.s_col];
        };
        auto load = [&](int u, int kb) {
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                __builtin_memcpy(&qb[u][j][0], bp[j] + (int64_t)kb * BLOCK, 16);
                __builtin_memcpy(&qb[u][j][1], bp[j] + (int64_t)kb * BLOCK + 64, 16);
            }
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                __builtin_memcpy(&qa[u][i][0], ap[i] + (int64_t)kb * BLOCK, 16);
                __builtin_memcpy(&qa[u][i][1], ap[i] + (int64_t)kb * BLOCK + 64, 16);
            }
            scales(u, kb);
        };
        auto multiply = [&](int u) {
            bf16x8 b[NF][4];
#pragma unroll
            for (int j = 0; j < NF; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) b[j][q] = bf16_of8<0>(qb[u][j][q >> 1][2 * (q & 1)], qb[u][j][q >> 1][2 * (q & 1) + 1]);
#pragma unroll
            for (int i = 0; i < MF; ++i) {
                bf16x8 a[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) a[q] = bf16_of8<TA>(qa[u][i][q >> 1][2 * (q & 1)], qa[u][i][q >> 1][2 * (q & 1) + 1]);
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    f32x4 d = {};
#pragma unroll
                    for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][q], a[q], d, 0, 0, 0);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[v], fa[u][i] * fb[u][j][SB ? v : 0], acc[i][j][v]);
                }
            }
        };
        int kb = wave;
        for (; kb + (U - 1) * WAVES < whole; kb += U * WAVES) {
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, kb + u * WAVES);
#pragma unroll
            for (int u = 0; u < U; ++u) multiply(u);
        }
        for (; kb < whole; kb += WAVES) {
            load(0, kb);
            multiply(0);
        }
        if (kb < all) {  // the short block
            const int k0 = kb * BLOCK;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = k0 + h * 64 + fg * 16;
#pragma unroll
                for (int j = 0; j < NF; ++j) qb[0][j][h] = load16(bp[j] + k0 + h * 64, K - at, at);
#pragma unroll
                for (int i = 0; i < MF; ++i) qa[0][i][h] = load16(ap[i] + k0 + h * 64, K - at, at);
            }
            scales(0, kb);
            multiply(0);
        }
    }
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) part[wave][i * NF + j][lane] = acc[i][j];
    __syncthreads();
    for (int f = wave; f < MF * NF; f += WAVES) {
        f32x4 sum = part[0][f][lane];
#pragma unroll
        for (int v = 1; v < WAVES; ++v) sum += part[v][f][lane];
        const int r = f / NF * 16 + fr, c = n0 + f % NF * 16 + fg * 4;
        if (r < w.rows) {
            const bool used = r < w.used;
            const f32x4 zero = {};
            c_store4(w.out, w.row0 + r, c, min(p.N - c, 4), p.alpha, used ? p.beta : 0.0f, used ? sum : zero, wide);
        }
    }
}

template <int MF, int NF, int U>
hipError_t launch(const F8Problem &p, hipStream_t s) {
    const int64_t tiles_n = ((int64_t)p.N + 16 * NF - 1) / (16 * NF), tiles = most_row_tiles(p, 16 * MF) * tiles_n;
    if (tiles * NT > 0xFFFFFFFFll) return hipErrorInvalidConfiguration;
    auto go = [&](auto f) {
        note_launch(reinterpret_cast<const void *>(f), NT);
        hipLaunchKernelGGL(f, dim3((unsigned)tiles), dim3(NT), 0, s, p, (int)tiles_n, c_wide(p));
        return hipGetLastError();
    };
    if (p.b.shift == 0) return p.a.type ? go(f8_token_kernel<MF, NF, U, 1, true>) : go(f8_token_kernel<MF, NF, U, 0, true>);
    return p.a.type ? go(f8_token_kernel<MF, NF, U, 1, false>) : go(f8_token_kernel<MF, NF, U, 0, false>);
}

}  // namespace

hipError_t launch_f8_token(const F8Problem &p, int shape, hipStream_t s) {
    switch (shape) {
        case 12: return launch<1, 2, 4>(p, s);
        case 22: return launch<2, 2, 2>(p, s);
        case 21: return launch<2, 1, 4>(p, s);
        default: return launch<1, 1, 4>(p, s);
    }
}

}  // namespace regtile

// gemm_f8_any.hip -- C = alpha A B + beta C for block-scaled 8-bit float operands in any storage order and
// alignment: the kernel for what the DMA-fed kernels do not take.
//
// 64 x 64 tiles, 4 waves of 32 x 32, blocks of 128 k through registers into LDS as [row][k] bytes. A block's
// products are summed by four 16x16x32 bf16 MFMAs from zero (codes are exact in bf16), and the sum enters the
// accumulator times the two scales: c += (sa sb) sum. B's fragment is the first operand, so that a lane holds
// 4 consecutive columns of one row of C, and one scale of A.
//
// Bound by the latency of a block's loads, which nothing overlaps: 8192^3 takes 3.3 ms, where tiles take 0.43. What comes here
// is an e5m2 B, a transposed A, rows too far apart for 32-bit offsets, unaligned rows without a workspace, and K = 0.
//
// A K-contiguous chunk of 16 codes is one load at any address; a chunk across K's end, and operands contiguous
// the other way (16 rows at one k, scattered into LDS), take bytes.
#include "f8_common.h"

namespace regtile {
namespace {
using namespace f8;
using namespace mfma;

constexpr int T = 64, NT = 256, LD = BLOCK + 16;

// Chunk c (0 .. 511) of an operand's 64 x 128 block from `k0` on; src[0]: a K-contiguous chunk's row
__device__ __forceinline__ void stage(uint8_t *lds, const F8Operand &o, const uint8_t *row_of_chunk, int c, int row0, int rows, int64_t k0,
                                      int K) {
    if (o.step == 1) {
        const int r = c >> 3, kk = (c & 7) * 16, left = r < rows ? (int)(K - k0) - kk : 0;
        uint32_t d[4] = {0, 0, 0, 0};
        const uint8_t *p = row_of_chunk + k0 + kk;
        if (left >= 16) {
            __builtin_memcpy(d, p, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left) d[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
        }
        const u32x4 v = {d[0], d[1], d[2], d[3]};
        *reinterpret_cast<u32x4 *>(lds + r * LD + kk) = v;
    } else {
        const int kk = c >> 2, r = (c & 3) * 16;
        const uint8_t *p = o.q + (k0 + kk) * o.step + row0 + r;
        const int left = k0 + kk < K ? rows - r : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) lds[(r + i) * LD + kk] = i < left ? p[i] : (uint8_t)0;
    }
}

template <int TA, int TB>
__global__ __launch_bounds__(NT) void f8_any_kernel(F8Problem p, int tiles_n, bool wide) {
    __shared__ __align__(16) uint8_t la[T * LD];
    __shared__ __align__(16) uint8_t lb[T * LD];
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, wm = wave >> 1, wn = wave & 1;
    const int tile = blockIdx.x / tiles_n, n0 = (blockIdx.x - tile * tiles_n) * T;
    Work w;
    if (!work_of(p, T, tile, blockIdx.y, w)) return;
    const int cols = min(T, p.N - n0);
    const uint8_t *arow[2], *brow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = (tid + NT * j) >> 3;
        arow[j] = w.a.q + (r < w.used ? a_row(p, w, r) : 0) * w.a.row;
        brow[j] = w.b.q + (int64_t)(n0 + min(r, cols - 1)) * w.b.row;
    }
    const int fr = lane & 15, fg = lane >> 4;
    const float *sa[2], *sb[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = wm * 32 + i * 16 + fr;
        sa[i] = w.a.s + (w.used > 0 ? a_row(p, w, min(r, w.used - 1)) >> w.a.shift : 0) * w.a.s_row;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            sb[i][v] = w.b.s + (int64_t)((n0 + min(wn * 32 + i * 16 + fg * 4 + v, cols - 1)) >> w.b.shift) * w.b.s_row;
    }
    f32x4 acc[2][2] = {};
    const int K = w.used > 0 ? w.K : 0;
    for (int64_t k0 = 0; k0 < K; k0 += BLOCK) {  // (K may be the largest int)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            stage(la, w.a, arow[j], tid + NT * j, w.row0, w.used, k0, K);
            stage(lb, w.b, brow[j], tid + NT * j, n0, cols, k0, K);
        }
        __syncthreads();
        const int64_t kb = k0 / BLOCK;
        bf16x8 b[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint8_t *s = lb + (wn * 32 + j * 16 + fr) * LD + fg * 32;
            const u32x4 lo = lds_read16(s), hi = lds_read16(s + 16);
            b[j][0] = bf16_of8<TB>(lo[0], lo[1]);
            b[j][1] = bf16_of8<TB>(lo[2], lo[3]);
            b[j][2] = bf16_of8<TB>(hi[0], hi[1]);
            b[j][3] = bf16_of8<TB>(hi[2], hi[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t *s = la + (wm * 32 + i * 16 + fr) * LD + fg * 32;
            const u32x4 lo = lds_read16(s), hi = lds_read16(s + 16);
            const bf16x8 a[4] = {bf16_of8<TA>(lo[0], lo[1]), bf16_of8<TA>(lo[2], lo[3]), bf16_of8<TA>(hi[0], hi[1]),
                                 bf16_of8<TA>(hi[2], hi[3])};
            const float fa = sa[i][kb * w.a.s_col];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f32x4 d = {};
#pragma unroll
                for (int q = 0; q < 4; ++q) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][q], a[q], d, 0, 0, 0);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(d[v], fa * sb[j][v][kb * w.b.s_col], acc[i][j][v]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = wm * 32 + i * 16 + fr;
        if (r >= w.rows) continue;
        const bool used = r < w.used;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = wn * 32 + j * 16 + fg * 4;
            const f32x4 zero = {};
            c_store4(w.out, w.row0 + r, n0 + c, min(cols - c, 4), p.alpha, used ? p.beta : 0.0f, used ? acc[i][j] : zero, wide);
        }
    }
}

}  // namespace

hipError_t launch_f8_any(const F8Problem &p, hipStream_t s, const char **name) {
    static const char *const names[2][2] = {{"f8_any_64x64x128_e4m3_e4m3", "f8_any_64x64x128_e4m3_e5m2"},
                                            {"f8_any_64x64x128_e5m2_e4m3", "f8_any_64x64x128_e5m2_e5m2"}};
    *name = names[p.a.type][p.b.type];
    const int64_t tiles_n = ((int64_t)p.N + T - 1) / T, tiles = most_row_tiles(p, T) * tiles_n;
    if (tiles * NT > 0xFFFFFFFFll || (p.mode == F8Problem::DEPTH && p.experts > 65535)) return hipErrorInvalidConfiguration;
    static void (*const kernels[2][2])(F8Problem, int, bool) = {{f8_any_kernel<0, 0>, f8_any_kernel<0, 1>},
                                                                {f8_any_kernel<1, 0>, f8_any_kernel<1, 1>}};
    const auto f = kernels[p.a.type][p.b.type];
    note_launch(reinterpret_cast<const void *>(f), NT);
    hipLaunchKernelGGL(f, dim3((unsigned)tiles, p.mode == F8Problem::DEPTH ? p.experts : 1), dim3(NT), 0, s, p, (int)tiles_n,
                       c_wide(p));
    return hipGetLastError();
}

}  // namespace regtile

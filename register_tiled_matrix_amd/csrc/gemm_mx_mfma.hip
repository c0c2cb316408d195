// gemm_mx_mfma.hip -- C = alpha op(A) op(B) + beta C for a bf16 / fp16 A and a block-scaled (MX) B,
// any storage order, any size and any alignment.
//
// A workgroup of 4 waves owns a T x T tile of C (T = 128, or 64 for few tiles) and walks K in slabs
// of 64. Both operands go through registers: A as 16-byte chunks, B as 16 codes of one group with
// their scale byte, expanded to the 16-bit type (mx_common.h; exact) before they are written to LDS.
// The next slab is loaded while the current one is multiplied, on two LDS stages with one barrier
// per slab.
//
// LDS holds each operand in its own storage order, in the layouts of tile_addressing.h: K-contiguous
// slabs (rows of 64 k) feed the 32x32x16 MFMAs with 16-byte reads, M/N-contiguous ones (64 rows of T
// elements) with transposing reads. Groups run along the stored rows and tiles and slabs start at
// multiples of 32, so no run of 16 codes has two scales.
#include "mfma_common.h"
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {
using namespace mfma;

constexpr int MXT_BK = 64;   // slab depth
constexpr int MXT_NT = 256;  // threads: 2 x 2 waves

// slot (16-byte units) of chunk c of slab row r
template <bool MAJOR_K, int T>
__device__ __forceinline__ int slab_slot(int r, int c) {
    if constexpr (MAJOR_K) return r * 8 + (c ^ slab_key<8, 32>(r));
    constexpr int MCH = T / 8;
    return r * MCH + (c ^ (MCH == 8 ? addr::sk_mn_key(r) : addr::mn_key(r)));
}

// The stored operand as rows x cols: K-contiguous, rows are the tile's M (or N) index and columns k;
// otherwise rows are k and columns the tile's.
template <int T, bool FP4, bool F16, bool TA, bool TB>
__global__ __launch_bounds__(MXT_NT) void mx_mfma_kernel(int M, int N, int K, float alpha,
                                                         const uint16_t *__restrict__ A, int64_t lda,
                                                         const uint8_t *__restrict__ Q, int64_t ldq,
                                                         const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                         float *__restrict__ C, int64_t ldc, int tiles_m, int tiles_n) {
    typedef Frag<32, F16> F;
    constexpr bool A_K = !TA, B_K = TB;  // K-contiguous storage
    constexpr int MI = T / 64, NI = T / 64;
    constexpr int SLOTS = T * 8;               // 16-byte slots of one operand's slab
    constexpr int JA = SLOTS / MXT_NT;         // chunks of A per thread and slab
    constexpr int JB = SLOTS / 2 / MXT_NT;     // half groups (16 codes) of B per thread and slab
    constexpr int HB = FP4 ? 8 : 16;           // bytes of a half group
    __shared__ uint4 smem[2][2][SLOTS];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    grouped_tile<8>(xcd_contiguous_id(blockIdx.x, gridDim.x), tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * T, n0 = (int64_t)tn * T;
    const int64_t nslabs = ((int64_t)K + MXT_BK - 1) / MXT_BK;

    // slab row and first column of this thread's j-th run of `run` elements, in slabs of 64 columns
    // (K-contiguous) or T columns
    auto place = [&](bool major_k, int run, int j, int &r, int &c) {
        const int per_row = (major_k ? MXT_BK : T) / run, p = tid + MXT_NT * j;
        r = p / per_row;
        c = p % per_row * run;
    };

    uint4 ra[JA];
    uint32_t rq[JB][HB / 4], rs[JB];
    auto load = [&](int64_t slab) {
        const int64_t k0 = slab * MXT_BK;
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            int r, c;
            place(A_K, 8, j, r, c);
            const int64_t row = (A_K ? m0 : k0) + r, col = (A_K ? k0 : m0) + c;
            const int64_t left = (A_K ? K : M) - col;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < (A_K ? M : K) && left > 0) {
                const uint16_t *p = A + row * lda + col;
                if (left >= 8) {
                    __builtin_memcpy(&v, p, 16);
                } else {
                    uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (i < left) d[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
                    v = make_uint4(d[0], d[1], d[2], d[3]);
                }
            }
            ra[j] = v;
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            int r, c;
            place(B_K, 16, j, r, c);
            const int64_t row = (B_K ? n0 : k0) + r, col = (B_K ? k0 : n0) + c;
            const int64_t left = (B_K ? K : N) - col;
#pragma unroll
            for (int i = 0; i < HB / 4; ++i) rq[j][i] = 0;
            rs[j] = 0;
            if (row < (B_K ? N : K) && left > 0) {
                const uint8_t *p = Q + row * ldq + (FP4 ? col / 2 : col);
                rs[j] = S[row * lds + col / mx::GROUP];
                if (left >= 16)
                    mx::load_bytes<HB>(p, rq[j]);
                else
                    mx::load_codes_tail<FP4, HB>(p, (int)left, rq[j]);
            }
        }
    };
    auto write = [&](int st) {
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            int r, c;
            place(A_K, 8, j, r, c);
            smem[st][0][slab_slot<A_K, T>(r, c / 8)] = ra[j];
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            int r, c;
            place(B_K, 16, j, r, c);
            const float s = mx::scale_value<FP4>(rs[j]);
            smem[st][1][slab_slot<B_K, T>(r, c / 8)] = mx::expand8<FP4, F16>(rq[j], 0, s);
            smem[st][1][slab_slot<B_K, T>(r, c / 8 + 1)] = mx::expand8<FP4, F16>(rq[j], 1, s);
        }
    };

    // fragment of 32 rows (columns of C for B) from `base`, k step kk: 8 k of each lane's row
    const int tr_t = lane & 15;
    auto frag = [&](auto k_tag, const uint4 *slab, int base, int kk) {
        constexpr bool MK = decltype(k_tag)::value;
        if constexpr (MK) {
            return __builtin_bit_cast(bf16x8, slab[slab_slot<true, T>(base + (lane & 31), 2 * kk + (lane >> 5))]);
        } else {
            // the transposing read's mapping (mfma_common.h): lane t of 16 addresses row t / 4 at
            // columns 4 (t % 4) and receives its own column of four rows
            const int row = 16 * kk + 8 * (lane >> 5) + (tr_t >> 2);
            const int col = base + 16 * ((lane >> 4) & 1) + 4 * (tr_t & 3);
            const char *b = reinterpret_cast<const char *>(slab) + (col & 7) * 2;
            const uint2 lo = lds_read_tr16(b + slab_slot<false, T>(row, col >> 3) * 16);
            const uint2 hi = lds_read_tr16(b + slab_slot<false, T>(row + 4, col >> 3) * 16);
            return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
    };

    typename F::acc_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int v = 0; v < F::NACC; ++v) acc[i][j][v] = 0.0f;

    load(0);
    write(0);
    __syncthreads();
    for (int64_t s = 0; s < nslabs; ++s) {
        const int st = (int)(s & 1);
        if (s + 1 < nslabs) load(s + 1);
#pragma unroll
        for (int kk = 0; kk < MXT_BK / F::KSTEP; ++kk) {
            bf16x8 fa[MI], fb[NI];
#pragma unroll
            for (int i = 0; i < MI; ++i)
                fa[i] = frag(std::integral_constant<bool, A_K>{}, smem[st][0], wm * (T / 2) + 32 * i, kk);
#pragma unroll
            for (int j = 0; j < NI; ++j)
                fb[j] = frag(std::integral_constant<bool, B_K>{}, smem[st][1], wn * (T / 2) + 32 * j, kk);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j) acc[i][j] = F::mfma(fa[i], fb[j], acc[i][j]);
        }
        if (s + 1 < nslabs) write(st ^ 1);
        __syncthreads();
    }

    const int rl = F::row_lane(lane);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int64_t col = n0 + wn * (T / 2) + 32 * j + (lane & 31);
#pragma unroll
            for (int v = 0; v < F::NACC; ++v) {
                const int64_t row = m0 + wm * (T / 2) + 32 * i + rl + F::row_acc(v);
                if (row < M && col < N) {
                    float *c = C + row * ldc + col;
                    *c = epilogue_value(acc[i][j][v], alpha, beta, c);
                }
            }
        }
}

template <int T, bool FP4, bool F16, bool TA, bool TB>
hipError_t launch_mxt(const MxProblem &p, hipStream_t s) {
    const int tiles_m = (int)(((int64_t)p.M + T - 1) / T), tiles_n = (int)(((int64_t)p.N + T - 1) / T);
    note_launch(reinterpret_cast<const void *>(&mx_mfma_kernel<T, FP4, F16, TA, TB>), MXT_NT);
    hipLaunchKernelGGL((mx_mfma_kernel<T, FP4, F16, TA, TB>), dim3((unsigned)((int64_t)tiles_m * tiles_n)), dim3(MXT_NT),
                       0, s, p.M, p.N, p.K, p.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S, p.lds, p.beta, p.C,
                       p.ldc, tiles_m, tiles_n);
    return hipGetLastError();
}
template <int T, bool FP4, bool F16>
hipError_t launch_mxt_order(const MxProblem &p, hipStream_t s) {
    if (p.ta) return p.tb ? launch_mxt<T, FP4, F16, true, true>(p, s) : launch_mxt<T, FP4, F16, true, false>(p, s);
    return p.tb ? launch_mxt<T, FP4, F16, false, true>(p, s) : launch_mxt<T, FP4, F16, false, false>(p, s);
}
template <int T>
hipError_t launch_mxt_types(const MxProblem &p, hipStream_t s) {
    if (p.fp4) return p.f16 ? launch_mxt_order<T, true, true>(p, s) : launch_mxt_order<T, true, false>(p, s);
    return p.f16 ? launch_mxt_order<T, false, true>(p, s) : launch_mxt_order<T, false, false>(p, s);
}

}  // namespace

hipError_t launch_mx_mfma(const MxProblem &p, hipStream_t s, const char **name) {
    const int64_t tiles128 = (((int64_t)p.M + 127) / 128) * (((int64_t)p.N + 127) / 128);
    const bool small = tiles128 < 256;  // fewer than one 128 x 128 tile per CU
#define REGTILE_MX_NAMES(elt, fmt, t) \
    {{elt "_" fmt "_mfma_" t "_nn", elt "_" fmt "_mfma_" t "_nt"}, {elt "_" fmt "_mfma_" t "_tn", elt "_" fmt "_mfma_" t "_tt"}}
#define REGTILE_MX_SIZES(elt, fmt) {REGTILE_MX_NAMES(elt, fmt, "128x128x64"), REGTILE_MX_NAMES(elt, fmt, "64x64x64")}
    static const char *const names[2][2][2][2][2] = {{REGTILE_MX_SIZES("bf16", "int8"), REGTILE_MX_SIZES("bf16", "fp4")},
                                                     {REGTILE_MX_SIZES("f16", "int8"), REGTILE_MX_SIZES("f16", "fp4")}};
#undef REGTILE_MX_SIZES
#undef REGTILE_MX_NAMES
    *name = names[p.f16][p.fp4][small][p.ta][p.tb];
    return small ? launch_mxt_types<64>(p, s) : launch_mxt_types<128>(p, s);
}

}  // namespace regtile

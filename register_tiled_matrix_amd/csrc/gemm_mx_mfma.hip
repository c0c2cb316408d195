// gemm_mx_mfma.hip -- C = alpha op(A) op(B) + beta C for a bf16 / fp16 A and a block-scaled (MX) B,
// any storage order, any size and any alignment.
//
// Four waves own a T x T tile of C and walk K in slabs of 64. Both operands go through registers: A as
// 16-byte chunks, B as 16 codes of one group with their scale byte, expanded to the 16-bit type
// (mx_common.h; exact) before they are written to LDS. 64-wide tiles load two slabs ahead of the
// one that is multiplied (a load takes longer than a slab), into two sets of registers; 128-wide ones,
// whose slabs take longer, one. Slabs pass through two LDS stages with one barrier per slab that
// waits for LDS only.
//
// Few tiles leave most of the chip idle and their slabs are a chain of memory latencies. There KS = 4
// groups of four waves share a 64 x 64 tile, each with its own slabs (every fourth) and its own
// stages, and the four sums are added through LDS in order.
//
// LDS holds each operand in its own storage order, in the layouts of tile_addressing.h: K-contiguous
// slabs (rows of 64 k) feed the 32x32x16 MFMAs with 16-byte reads, M/N-contiguous ones (64 rows of T
// elements) with transposing reads. Groups run along the stored rows and tiles and slabs start at
// multiples of 32, so no run of 16 codes has two scales.
#include <type_traits>

#include "mfma_common.h"
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {
using namespace mfma;

constexpr int MXT_BK = 64;   // slab depth
constexpr int MXT_NT = 256;  // threads of a group: 2 x 2 waves

// slot (16-byte units) of chunk c of slab row r
template <bool MAJOR_K, int T>
__device__ __forceinline__ int slab_slot(int r, int c) {
    if constexpr (MAJOR_K) return r * 8 + (c ^ slab_key<8, 32>(r));
    constexpr int MCH = T / 8;
    return r * MCH + (c ^ (MCH == 8 ? addr::sk_mn_key(r) : addr::mn_key(r)));
}

// The stored operand as rows x cols: K-contiguous, rows are the tile's M (or N) index and columns k;
// otherwise rows are k and columns the tile's.
template <int T, int KS, bool FP4, bool F16, bool TA, bool TB>
__global__ __launch_bounds__(MXT_NT *KS, KS == 1 ? 2 : 4) void mx_mfma_kernel(int M, int N, int K, float alpha,
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
    constexpr int PSTRIDE = T + 4;             // row stride (floats) of a group's sums in LDS
    constexpr int STAGES = KS * 2 * 2 * SLOTS, SUMS = KS * T * PSTRIDE / 4;
    __shared__ uint4 lds_all[KS > 1 && SUMS > STAGES ? SUMS : STAGES];
    const int group = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / MXT_NT);
    uint4(*const smem)[2][SLOTS] = reinterpret_cast<uint4(*)[2][SLOTS]>(lds_all + group * (4 * SLOTS));

    const int tid = threadIdx.x % MXT_NT;
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

    // Runs that pass their row's end (in K-contiguous storage only the last slab has them, in
    // M/N-contiguous storage every slab of the last tiles) are loaded as the whole run that ends
    // there and moved down when they are written to LDS, so that every load has the same time to
    // land; rows shorter than a run are read by element.
    constexpr int PF = T == 128 ? 1 : 2;  // register sets: slabs loaded ahead
    uint32_t ra[PF][JA][4], rq[PF][JB][HB / 4], rs[PF][JB];
    const int a_cols = A_K ? K : M, b_cols = B_K ? K : N;
    const int b_bytes = (int)mx::row_bytes(FP4, b_cols);
    auto load_edge = [&](int64_t slab, int set) {
        const int64_t k0 = slab * MXT_BK;
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            int r, c;
            place(A_K, 8, j, r, c);
            const int64_t row = (A_K ? m0 : k0) + r, col = (A_K ? k0 : m0) + c;
#pragma unroll
            for (int i = 0; i < 4; ++i) ra[set][j][i] = 0;
            if (row < (A_K ? M : K) && col < a_cols) {
                const uint16_t *p = A + row * lda;
                if (a_cols >= 8) {
                    __builtin_memcpy(ra[set][j], p + min(col, (int64_t)a_cols - 8), 16);
                } else {
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (i < a_cols) ra[set][j][i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            int r, c;
            place(B_K, 16, j, r, c);
            const int64_t row = (B_K ? n0 : k0) + r, col = (B_K ? k0 : n0) + c;
#pragma unroll
            for (int i = 0; i < HB / 4; ++i) rq[set][j][i] = 0;
            rs[set][j] = 0;
            if (row < (B_K ? N : K) && col < b_cols) {
                const uint8_t *p = Q + row * ldq;
                rs[set][j] = S[row * lds + col / mx::GROUP];
                if (b_bytes >= HB)
                    mx::load_bytes<HB>(p + min(FP4 ? col / 2 : col, (int64_t)b_bytes - HB), rq[set][j]);
                else
                    mx::load_codes_tail<FP4, HB>(p, b_cols, rq[set][j]);
            }
        }
    };
    // Slabs that end before K need no checks: rows (columns) past M or N are loaded from the last
    // ones and feed outputs that are not stored.
    const uint16_t *pa[JA];
    const uint8_t *pq[JB], *ps[JB];
    const bool a_runs = a_cols >= 8, b_runs = b_bytes >= HB;  // rows as long as a run
#pragma unroll
    for (int j = 0; j < JA; ++j) {
        int r, c;
        place(A_K, 8, j, r, c);
        pa[j] = A + (A_K ? min(m0 + r, (int64_t)M - 1) * lda + c : r * lda + min(m0 + c, (int64_t)M - 8));
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) {
        int r, c;
        place(B_K, 16, j, r, c);
        const int64_t row = B_K ? min(n0 + r, (int64_t)N - 1) : r, col = B_K ? c : n0 + c;
        pq[j] = Q + row * ldq + (B_K ? (FP4 ? col / 2 : col) : min(FP4 ? col / 2 : col, (int64_t)b_bytes - HB));
        ps[j] = S + row * lds + (B_K ? col / mx::GROUP : min(col / mx::GROUP, ((int64_t)N - 1) / mx::GROUP));
    }
    auto load = [&](int64_t slab, int set) {
        if (!a_runs || !b_runs || (slab + 1) * MXT_BK > K) {
            load_edge(slab, set);
            return;
        }
        const int64_t k0 = slab * MXT_BK, ao = A_K ? k0 : k0 * lda;
        const int64_t qo = B_K ? (FP4 ? k0 / 2 : k0) : k0 * ldq, so = B_K ? k0 / mx::GROUP : k0 * lds;
#pragma unroll
        for (int j = 0; j < JA; ++j) __builtin_memcpy(ra[set][j], pa[j] + ao, 16);
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            mx::load_bytes<HB>(pq[j] + qo, rq[set][j]);
            rs[set][j] = ps[j][so];
        }
    };
    auto write = [&](int64_t slab, int st, int set) {
        const int64_t k0 = slab * MXT_BK;
        // does this slab of this tile hold runs that pass the end of their rows?
        if (a_runs && (A_K ? k0 + MXT_BK > K : m0 + T > M)) {
#pragma unroll
            for (int j = 0; j < JA; ++j) {
                int r, c;
                place(A_K, 8, j, r, c);
                const int64_t early = (A_K ? k0 : m0) + c - (a_cols - 8);  // elements
                if (early > 0 && early < 8) mx::move_down(ra[set][j], 2 * (int)early);
            }
        }
        if (b_runs && (B_K ? k0 + MXT_BK > K : n0 + T > N)) {
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                int r, c;
                place(B_K, 16, j, r, c);
                const int64_t col = (B_K ? k0 : n0) + c, early = (FP4 ? col / 2 : col) - (b_bytes - HB);  // bytes
                if (early >= 0 && early < HB) {
                    mx::move_down(rq[set][j], (int)early);
                    const int at = HB - 1 - (int)early;  // the half byte behind an odd row
#pragma unroll
                    for (int i = 0; i < HB / 4; ++i)
                        if (FP4 && (b_cols & 1) && at / 4 == i) rq[set][j][i] &= ~(0xF0u << (8 * (at % 4)));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            int r, c;
            place(A_K, 8, j, r, c);
            smem[st][0][slab_slot<A_K, T>(r, c / 8)] = make_uint4(ra[set][j][0], ra[set][j][1], ra[set][j][2], ra[set][j][3]);
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            int r, c;
            place(B_K, 16, j, r, c);
            const float s = mx::scale_value<FP4>(rs[set][j]);
            smem[st][1][slab_slot<B_K, T>(r, c / 8)] = mx::expand8<FP4, F16>(rq[set][j], 0, s);
            smem[st][1][slab_slot<B_K, T>(r, c / 8 + 1)] = mx::expand8<FP4, F16>(rq[set][j], 1, s);
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

    // This group's slabs are group, group + KS, ...; every group walks `steps` of them, those past
    // the end (past K) all zeros. Step i uses stage i % 2 (and, with two sets, registers i % 2).
    const int64_t steps = (nslabs + KS - 1) / KS;
    auto slab_of = [&](int64_t i) { return group + i * KS; };
    auto step = [&](int64_t i, auto parity) {
        constexpr int P = decltype(parity)::value;
        if (i + PF < steps) load(slab_of(i + PF), PF == 2 ? P : 0);
#pragma unroll
        for (int kk = 0; kk < MXT_BK / F::KSTEP; ++kk) {
            bf16x8 fa[MI], fb[NI];
#pragma unroll
            for (int a = 0; a < MI; ++a)
                fa[a] = frag(std::integral_constant<bool, A_K>{}, smem[P][0], wm * (T / 2) + 32 * a, kk);
#pragma unroll
            for (int b = 0; b < NI; ++b)
                fb[b] = frag(std::integral_constant<bool, B_K>{}, smem[P][1], wn * (T / 2) + 32 * b, kk);
#pragma unroll
            for (int a = 0; a < MI; ++a)
#pragma unroll
                for (int b = 0; b < NI; ++b) acc[a][b] = F::mfma(fa[a], fb[b], acc[a][b]);
        }
        if (i + 1 < steps) write(slab_of(i + 1), P ^ 1, PF == 2 ? P ^ 1 : 0);
        wait_lgkmcnt0();
        lds_barrier();  // the next stage is written, this one has been read
    };
    load(slab_of(0), 0);
    if (PF == 2 && steps > 1) load(slab_of(1), PF - 1);
    write(slab_of(0), 0, 0);
    wait_lgkmcnt0();
    lds_barrier();
    for (int64_t i = 0; i < steps; i += 2) {
        step(i, std::integral_constant<int, 0>{});
        if (i + 1 < steps) step(i + 1, std::integral_constant<int, 1>{});
    }

    const int rl = F::row_lane(lane);
    if constexpr (KS == 1) {
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
    } else {
        // (the last step's barrier has freed the stages)
        float *const sums = reinterpret_cast<float *>(lds_all);
        float *const mine = sums + group * (T * PSTRIDE);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < F::NACC; ++v)
                    mine[(wm * (T / 2) + 32 * i + rl + F::row_acc(v)) * PSTRIDE + wn * (T / 2) + 32 * j + (lane & 31)] =
                        acc[i][j][v];
        __syncthreads();
        for (int e = threadIdx.x; e < T * T; e += MXT_NT * KS) {
            const int r = e / T, c = e % T;
            if (m0 + r < M && n0 + c < N) {
                float v = sums[r * PSTRIDE + c];
#pragma unroll
                for (int g = 1; g < KS; ++g) v += sums[g * (T * PSTRIDE) + r * PSTRIDE + c];
                float *cp = C + (m0 + r) * ldc + n0 + c;
                *cp = epilogue_value(v, alpha, beta, cp);
            }
        }
    }
}

template <int T, int KS, bool FP4, bool F16, bool TA, bool TB>
hipError_t launch_mxt(const MxProblem &p, hipStream_t s) {
    const int tiles_m = (int)(((int64_t)p.M + T - 1) / T), tiles_n = (int)(((int64_t)p.N + T - 1) / T);
    note_launch(reinterpret_cast<const void *>(&mx_mfma_kernel<T, KS, FP4, F16, TA, TB>), MXT_NT * KS);
    hipLaunchKernelGGL((mx_mfma_kernel<T, KS, FP4, F16, TA, TB>), dim3((unsigned)((int64_t)tiles_m * tiles_n)),
                       dim3(MXT_NT * KS), 0, s, p.M, p.N, p.K, p.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S,
                       p.lds, p.beta, p.C, p.ldc, tiles_m, tiles_n);
    return hipGetLastError();
}
template <int T, int KS, bool FP4, bool F16>
hipError_t launch_mxt_order(const MxProblem &p, hipStream_t s) {
    if (p.ta) return p.tb ? launch_mxt<T, KS, FP4, F16, true, true>(p, s) : launch_mxt<T, KS, FP4, F16, true, false>(p, s);
    return p.tb ? launch_mxt<T, KS, FP4, F16, false, true>(p, s) : launch_mxt<T, KS, FP4, F16, false, false>(p, s);
}
template <int T, int KS>
hipError_t launch_mxt_types(const MxProblem &p, hipStream_t s) {
    if (p.fp4) return p.f16 ? launch_mxt_order<T, KS, true, true>(p, s) : launch_mxt_order<T, KS, true, false>(p, s);
    return p.f16 ? launch_mxt_order<T, KS, false, true>(p, s) : launch_mxt_order<T, KS, false, false>(p, s);
}

}  // namespace

hipError_t launch_mx_mfma(const MxProblem &p, hipStream_t s, const char **name) {
    const int64_t tiles128 = (((int64_t)p.M + 127) / 128) * (((int64_t)p.N + 127) / 128);
    const int64_t tiles64 = (((int64_t)p.M + 63) / 64) * (((int64_t)p.N + 63) / 64);
    // 128-wide tiles from one per CU (3001x2003x1001 fp4 nt, 384 of them: 31 us against 37 on 64-wide
    // ones; 1500x2200x1001 nn, 216: 28 against 26); four groups to a 64-wide tile up to one of those
    // per CU (1000x777x1500 nn, 208: 13.7 us against 32; 1000x1500x777 nt, 384: 17.9 against 14.8)
    const int kind = tiles128 >= 256 ? 0 : tiles64 > 256 ? 1 : 2;
#define REGTILE_MX_NAMES(elt, fmt, t) \
    {{elt "_" fmt "_mfma_" t "_nn", elt "_" fmt "_mfma_" t "_nt"}, {elt "_" fmt "_mfma_" t "_tn", elt "_" fmt "_mfma_" t "_tt"}}
#define REGTILE_MX_SIZES(elt, fmt)                                                                              \
    {REGTILE_MX_NAMES(elt, fmt, "128x128x64"), REGTILE_MX_NAMES(elt, fmt, "64x64x64"),                           \
     REGTILE_MX_NAMES(elt, fmt, "64x64x64_k4")}
    static const char *const names[2][2][3][2][2] = {{REGTILE_MX_SIZES("bf16", "int8"), REGTILE_MX_SIZES("bf16", "fp4")},
                                                     {REGTILE_MX_SIZES("f16", "int8"), REGTILE_MX_SIZES("f16", "fp4")}};
#undef REGTILE_MX_SIZES
#undef REGTILE_MX_NAMES
    *name = names[p.f16][p.fp4][kind][p.ta][p.tb];
    return kind == 0   ? launch_mxt_types<128, 1>(p, s)
           : kind == 1 ? launch_mxt_types<64, 1>(p, s)
                       : launch_mxt_types<64, 4>(p, s);
}

}  // namespace regtile

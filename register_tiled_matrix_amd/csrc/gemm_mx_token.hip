// gemm_mx_token.hip -- C = alpha A op(B) + beta C for a few rows of A (the tokens of a decoding step)
// and a block-scaled B stored N x K: a product bound by reading B's codes once.
//
// The MFMA is 16x16x32 with B's values as its rows and A's as its columns, so that codes go from
// memory to registers and are expanded there (mx_common.h): no LDS, no barrier in the loop. Which 32
// of k a step takes is free as long as both operands agree, so every lane loads a whole group, 32
// consecutive codes (16 bytes of fp4) with their one scale byte, and feeds four MFMAs with 8 codes
// each.
//
// Few tokens leave columns of the MFMA unused. H = 1 uses its 16 rows for 16 rows of B. With H = 2 or
// 4, row r stands for row r / H of B at part r % H of k, and column c for token c / H at part c % H:
// the products on the diagonal (equal parts) are wanted and the rest is not looked at. That gives up
// matrix throughput, of which there is plenty, for consecutive lanes that read consecutive memory and
// for 16 / H rows of B a wave, so that a small N still fills the chip.
//
// The NW waves of a workgroup take chunks of k in turn and their sums are added through LDS in wave
// order: a fixed order, deterministic.
#include "mfma_common.h"
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {
using namespace mfma;

template <int NF, int MC>
using Acc = f32x4[NF][MC];

// acc += the products of one chunk: each lane's group of 32 codes of NF rows of B (q, scale bytes s)
// with the same 32 of k of MC tokens (x, 8 to a uint4)
template <bool FP4, bool F16, int NF, int MC>
__device__ __forceinline__ void multiply_group(const uint32_t (&q)[NF][FP4 ? 4 : 8], const uint32_t (&s)[NF],
                                               const uint4 (&x)[MC][4], Acc<NF, MC> &acc) {
    float sc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) sc[f] = mx::scale_value<FP4>(s[f]);
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const bf16x8 w = __builtin_bit_cast(bf16x8, mx::expand8<FP4, F16>(q[f], t, sc[f]));
#pragma unroll
            for (int i = 0; i < MC; ++i) acc[f][i] = Frag<16, F16>::mfma(w, __builtin_bit_cast(bf16x8, x[i][t]), acc[f][i]);
        }
}

// The last, short chunk: `left` of this lane's 32 of k remain (none below 1), read without touching
// what lies behind them; qp, sp and xp point at the lane's group.
template <bool FP4, bool F16, int NF, int MC>
__device__ __forceinline__ void short_chunk(int left, const uint8_t *const (&qp)[NF], const uint8_t *const (&sp)[NF],
                                            const uint16_t *const (&xp)[MC], Acc<NF, MC> &acc) {
    constexpr int GB = FP4 ? 16 : 32;
    uint32_t q[NF][GB / 4], s[NF];
    uint4 x[MC][4];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
#pragma unroll
        for (int i = 0; i < GB / 4; ++i) q[f][i] = 0;
        s[f] = 0;
        if (left > 0) {
            s[f] = *sp[f];
            if (left >= 32)
                mx::load_bytes<GB>(qp[f], q[f]);
            else
                mx::load_codes_tail<FP4, GB>(qp[f], left, q[f]);
        }
    }
#pragma unroll
    for (int i = 0; i < MC; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint16_t *p = xp[i] + 8 * t;
            uint32_t d[4] = {0, 0, 0, 0};
            if (left >= 8 * t + 8) {
                __builtin_memcpy(d, p, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (8 * t + e < left) d[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
            }
            x[i][t] = make_uint4(d[0], d[1], d[2], d[3]);
        }
    multiply_group<FP4, F16, NF, MC>(q, s, x, acc);
}

// The sum of the waves' accumulators (part[wave][fragment][lane]) in wave order, and the epilogue.
// Accumulator v of lane l: row 4 (l / 16) + v of B's fragment, column l % 16 of A's.
template <int H, int NF, int MC, int NW>
__device__ __forceinline__ void join_and_store(const float4 (&part)[NW][NF * MC][64], int M, int N, int64_t n0,
                                               float alpha, float beta, float *__restrict__ C, int64_t ldc, int vec_c) {
    constexpr int R = 16 / H;
    const int lane = threadIdx.x & 63, r = lane & 15, j = lane >> 4;
    for (int o = threadIdx.x; o < NF * MC * 64; o += NW * 64) {
        const int fi = o >> 6, f = fi / MC, i = fi % MC;
        float4 v = part[0][fi][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
            const float4 p = part[w][fi][lane];
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
        }
        if constexpr (H == 1) {  // four neighbouring columns of C
            const int64_t n = n0 + f * 16 + 4 * j;
            const int m = i * 16 + r;
            if (m >= M || n >= N) continue;
            float *cp = C + (int64_t)m * ldc + n;
            if (vec_c && n + 3 < N) {
                float4 o4 = make_float4(alpha * v.x, alpha * v.y, alpha * v.z, alpha * v.w);
                if (beta != 0.0f) {
                    const float4 old = *reinterpret_cast<const float4 *>(cp);
                    o4 = make_float4(fmaf(alpha, v.x, beta * old.x), fmaf(alpha, v.y, beta * old.y),
                                     fmaf(alpha, v.z, beta * old.z), fmaf(alpha, v.w, beta * old.w));
                }
                *reinterpret_cast<float4 *>(cp) = o4;
            } else {
                const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (n + k < N) cp[k] = epilogue_value(e[k], alpha, beta, cp + k);
            }
        } else {
            // rows 4 j + v are parts v % H of rows (4 j + v) / H of B; the wanted part is the column's,
            // r % H, and the H parts of a token are summed over its H neighbouring lanes
            const int h = r % H;
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int b = 0; b < 4 / H; ++b) {  // rows of B among this lane's four
                float d = e[b * H];
#pragma unroll
                for (int k = 1; k < H; ++k) d = h == k ? e[b * H + k] : d;
#pragma unroll
                for (int k = 1; k < H; k *= 2) d += __shfl_xor(d, k);
                const int64_t n = n0 + f * R + (4 / H) * j + b;
                const int m = i * R + r / H;
                if (h == 0 && m < M && n < N) {
                    float *cp = C + (int64_t)m * ldc + n;
                    *cp = epilogue_value(d, alpha, beta, cp);
                }
            }
        }
    }
}

// NF fragments of 16 / H rows of B and MC fragments of 16 / H tokens a wave; U chunks in flight
template <bool FP4, bool F16, int H, int NF, int MC, int NW, int U>
__global__ __launch_bounds__(NW * 64) void mx_token_kernel(int M, int N, int K, float alpha,
                                                           const uint16_t *__restrict__ A, int64_t lda,
                                                           const uint8_t *__restrict__ Q, int64_t ldq,
                                                           const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                           float *__restrict__ C, int64_t ldc, int vec_c) {
    constexpr int R = 16 / H;            // rows of B (tokens) per fragment
    constexpr int CHUNK = 128 * H;       // k per step of a wave
    constexpr int GB = FP4 ? 16 : 32;    // bytes of a group's codes
    __shared__ float4 part[NW][NF * MC][64];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = lane & 15, j = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (R * NF);
    const int koff = (j * H + r % H) * 32;  // this lane's group within a chunk
    // rows past the end repeat the last one: their outputs are not stored
    const uint8_t *qp[NF], *sp[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        const int64_t n = min(n0 + f * R + r / H, (int64_t)N - 1);
        qp[f] = Q + n * ldq + koff / 32 * GB;
        sp[f] = S + n * lds + koff / 32;
    }
    const uint16_t *xp[MC];
#pragma unroll
    for (int i = 0; i < MC; ++i) xp[i] = A + (int64_t)min(i * R + r / H, M - 1) * lda + koff;

    Acc<NF, MC> acc;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MC; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    uint32_t q[U][NF][GB / 4], s[U][NF];
    uint4 x[U][MC][4];
    const int nfull = K / CHUNK;
    for (int c0 = wave; c0 < nfull; c0 += NW * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = min(c0 + u * NW, nfull - 1);  // past the end: loaded again, not used
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                mx::load_bytes<GB>(qp[f] + c * (CHUNK / 32 * GB), q[u][f]);
                s[u][f] = sp[f][c * (CHUNK / 32)];
            }
#pragma unroll
            for (int i = 0; i < MC; ++i) __builtin_memcpy(x[u][i], xp[i] + c * CHUNK, 64);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * NW < nfull) multiply_group<FP4, F16, NF, MC>(q[u], s[u], x[u], acc);
    }
    if (K % CHUNK != 0 && wave == nfull % NW) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            qp[f] += (int64_t)nfull * (CHUNK / 32 * GB);
            sp[f] += (int64_t)nfull * (CHUNK / 32);
        }
#pragma unroll
        for (int i = 0; i < MC; ++i) xp[i] += (int64_t)nfull * CHUNK;
        short_chunk<FP4, F16, NF, MC>(K - nfull * CHUNK - koff, qp, sp, xp, acc);
    }

#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MC; ++i) part[wave][f * MC + i][lane] = __builtin_bit_cast(float4, acc[f][i]);
    __syncthreads();
    join_and_store<H, NF, MC, NW>(part, M, N, n0, alpha, beta, C, ldc, vec_c);
}

// The same product (H = 1) for more tokens and 16-byte aligned rows, through LDS. Reading fragments
// straight from memory, 16 neighbouring lanes touch 16 rows, 16 bytes of each, and the loads of A (four
// for one of fp4 codes) spend more of the CU's address unit than the codes do. Here each wave
// brings its chunk (128 of k: 16 NF rows of codes, their scales, 16 MC rows of A) to its own part of LDS by
// DMA, 256 consecutive bytes of a row of A and 64 (128) of a row of codes at a time, in a ring of D
// chunks, and reads the fragments from there. Waves share nothing until their sums are joined, so the
// loop has no barrier.
//
// A's rows are 16 chunks of 16 bytes, chunk c of row r at slot c ^ r; rows of codes are 4 (8) chunks, at
// c ^ (r >> 2 & 3) (c ^ (r >> 1 & 7)): 16 lanes that read one chunk of 16 rows reach all banks.
template <bool FP4, bool F16, int NF, int MC, int NW, int D>
__global__ __launch_bounds__(NW * 64) void mx_batch_kernel(int M, int N, int K, float alpha,
                                                           const uint16_t *__restrict__ A, int64_t lda,
                                                           const uint8_t *__restrict__ Q, int64_t ldq,
                                                           const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                           float *__restrict__ C, int64_t ldc, int vec_c) {
    constexpr int QCH = FP4 ? 4 : 8;                 // 16-byte chunks of a row of codes
    constexpr int XS = MC * 256, QS = NF * 16 * QCH;  // 16-byte slots of A and of the codes
    constexpr int STAGE = XS + QS + 16;              // and of the scales (16 NF <= 64 dwords)
    constexpr int PER = MC * 4 + NF * QCH / 4 + 1;   // DMA instructions of a chunk
    static_assert(NF * 16 <= 64 && PER * (D - 1) < 64 && D >= 2, "scales of a chunk in one DMA; vmcnt range");
    constexpr int SLOTS = NW * D * STAGE, SLOTS_PART = NW * NF * MC * 64;
    static_assert(SLOTS * 16 <= 160 * 1024 && SLOTS_PART <= SLOTS, "LDS");
    __shared__ uint4 smem[SLOTS];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int r = lane & 15, j = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NF);
    uint4 *const mine = smem + wave * (D * STAGE);
    auto row_n = [&](int i) { return min(n0 + i, (int64_t)N - 1); };  // rows past the end repeat the last

    // this lane's part of each DMA instruction
    const uint16_t *xsrc[MC * 4];
    const uint8_t *qsrc[NF * QCH / 4], *ssrc;
#pragma unroll
    for (int i = 0; i < MC * 4; ++i) {
        const int row = 4 * i + (lane >> 4);
        xsrc[i] = A + (int64_t)min(row, M - 1) * lda + ((lane & 15) ^ (row & 15)) * 8;
    }
#pragma unroll
    for (int i = 0; i < NF * QCH / 4; ++i) {
        const int slot = i * 64 + lane, row = slot / QCH, ch = slot % QCH;
        qsrc[i] = Q + row_n(row) * ldq + (ch ^ (FP4 ? (row >> 2) & 3 : (row >> 1) & 7)) * 16;
    }
    ssrc = S + row_n(lane % (16 * NF)) * lds;
    auto issue = [&](int64_t c, int st) {
        uint4 *d = mine + st * STAGE;
#pragma unroll
        for (int i = 0; i < NF * QCH / 4; ++i) dma16(qsrc[i] + c * (QCH * 16), d + XS + i * 64);
        dma4(ssrc + c * 4, d + XS + QS);
#pragma unroll
        for (int i = 0; i < MC * 4; ++i) dma16(xsrc[i] + c * 128, d + i * 64);
    };

    Acc<NF, MC> acc;
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MC; ++i) acc[f][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int nfull = K / 128;
    const int mychunks = nfull > wave ? (nfull - wave + NW - 1) / NW : 0;
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        if (i < mychunks) issue(wave + i * NW, i);
    int st = 0;
    for (int i = 0; i < mychunks; ++i) {
        if (i + D - 1 < mychunks) {
            issue(wave + (int64_t)(i + D - 1) * NW, st == 0 ? D - 1 : st - 1);  // the chunk before's slot
            wait_vmcnt<PER *(D - 1)>();
        } else {
            wait_vmcnt<0>();
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const uint4 *d = mine + st * STAGE;
        uint32_t q[NF][QCH], s[NF];
        uint4 x[MC][4];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const uint4 *row = d + XS + (f * 16 + r) * QCH;
#pragma unroll
            for (int e = 0; e < QCH / 4; ++e) {
                const u32x4 v = lds_read16(&row[FP4 ? j ^ ((r >> 2) & 3) : (2 * j + e) ^ ((r >> 1) & 7)]);
#pragma unroll
                for (int u = 0; u < 4; ++u) q[f][4 * e + u] = v[u];
            }
            s[f] = reinterpret_cast<const uint8_t *>(d + XS + QS)[(f * 16 + r) * 4 + j];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int m = 0; m < MC; ++m) x[m][t] = __builtin_bit_cast(uint4, lds_read16(&d[(m * 16 + r) * 16 + ((4 * j + t) ^ r)]));
        multiply_group<FP4, F16, NF, MC>(q, s, x, acc);
        wait_lgkmcnt0();  // the chunk is in registers before its slot is filled again
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        st = st + 1 == D ? 0 : st + 1;
    }
    if (K % 128 != 0 && wave == nfull % NW) {
        const uint8_t *qp[NF], *sp[NF];
        const uint16_t *xp[MC];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            qp[f] = Q + row_n(f * 16 + r) * ldq + ((int64_t)nfull * 4 + j) * (QCH * 4);
            sp[f] = S + row_n(f * 16 + r) * lds + (int64_t)nfull * 4 + j;
        }
#pragma unroll
        for (int m = 0; m < MC; ++m) xp[m] = A + (int64_t)min(m * 16 + r, M - 1) * lda + (int64_t)nfull * 128 + 32 * j;
        short_chunk<FP4, F16, NF, MC>(K - nfull * 128 - 32 * j, qp, sp, xp, acc);
    }

    __syncthreads();  // the sums take the rings' place
    auto &part = *reinterpret_cast<float4(*)[NW][NF * MC][64]>(smem);
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int m = 0; m < MC; ++m) part[wave][f * MC + m][lane] = __builtin_bit_cast(float4, acc[f][m]);
    __syncthreads();
    join_and_store<1, NF, MC, NW>(part, M, N, n0, alpha, beta, C, ldc, vec_c);
}

template <bool FP4, bool F16, int NF, int MC, int NW, int D>
hipError_t launch_batch(const MxProblem &p, hipStream_t s) {
    const int vec_c = p.ldc % 4 == 0 && aligned16(p.C);
    note_launch(reinterpret_cast<const void *>(&mx_batch_kernel<FP4, F16, NF, MC, NW, D>), NW * 64);
    hipLaunchKernelGGL((mx_batch_kernel<FP4, F16, NF, MC, NW, D>), dim3((unsigned)(((int64_t)p.N + 16 * NF - 1) / (16 * NF))),
                       dim3(NW * 64), 0, s, p.M, p.N, p.K, p.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S, p.lds,
                       p.beta, p.C, p.ldc, vec_c);
    return hipGetLastError();
}

template <bool FP4, bool F16, int H, int NF, int MC, int NW, int U>
hipError_t launch_token(const MxProblem &p, hipStream_t s) {
    constexpr int ROWS = 16 / H * NF;
    const int vec_c = p.ldc % 4 == 0 && aligned16(p.C);
    note_launch(reinterpret_cast<const void *>(&mx_token_kernel<FP4, F16, H, NF, MC, NW, U>), NW * 64);
    hipLaunchKernelGGL((mx_token_kernel<FP4, F16, H, NF, MC, NW, U>), dim3((unsigned)(((int64_t)p.N + ROWS - 1) / ROWS)),
                       dim3(NW * 64), 0, s, p.M, p.N, p.K, p.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S, p.lds,
                       p.beta, p.C, p.ldc, vec_c);
    return hipGetLastError();
}

// Shapes <NF, MC, NW, U or D>, times in us at N x K = 8192 x 8192 unless stated. Register kernel: more
// rows of B a wave reuse A's fragments (the loads of A bound it: at one token fp4 13.1, 10.6, 10.0 with NF
// = 1, 2, 4), fewer fill more of the chip (2048 x 2048: 3.3, 3.1, 3.4), so NF = 4 waits for N = 8192;
// int8 codes take twice the registers and stay at NF = 2 (17.3; NF = 4: 19.9). Eight waves: four lose
// 0-12%, sixteen 10-40%.
template <bool FP4, bool F16>
hipError_t launch_token_rows(const MxProblem &p, hipStream_t s) {
    if (p.M <= 4) {
        if constexpr (FP4) {
            if (p.N >= 8192) return launch_token<FP4, F16, 4, 4, 1, 8, 1>(p, s);
            return launch_token<FP4, F16, 4, 2, 1, 8, 2>(p, s);
        } else {
            return launch_token<FP4, F16, 4, 2, 1, 8, 1>(p, s);
        }
    }
    if (p.M <= 8) return launch_token<FP4, F16, 2, 2, 1, 8, 2>(p, s);
    if (p.M <= 16) return launch_token<FP4, F16, 1, 2, 1, 8, 4>(p, s);
    return launch_token<FP4, F16, 1, 2, 2, 4, 2>(p, s);
}
// LDS kernel: 16 NF rows of B a workgroup. One fragment while that gives at most one workgroup per CU
// (N <= 4096; 16 tokens at 4096 x 4096 fp4: 5.6 against 6.7 with two), then two, which read A half as
// often (14.5 against 19.0 at 8192 x 8192). LDS is split into as many waves as leave two chunks each
// (three where that is no fewer waves than eight): more waves hide more latency than deeper rings (32
// tokens fp4 7 waves x 2 chunks 18.7, 5 x 3 19.3, 3 x 5 25.2).
template <bool F16>
hipError_t launch_batch_rows(const MxProblem &p, hipStream_t s) {
    if (p.N <= 4096) {
        if (p.M <= 16) return p.fp4 ? launch_batch<true, F16, 1, 1, 12, 2>(p, s) : launch_batch<false, F16, 1, 1, 12, 2>(p, s);
        if (p.M <= 32) return p.fp4 ? launch_batch<true, F16, 1, 2, 8, 2>(p, s) : launch_batch<false, F16, 1, 2, 7, 2>(p, s);
        if (p.M <= 48) return p.fp4 ? launch_batch<true, F16, 1, 3, 6, 2>(p, s) : launch_batch<false, F16, 1, 3, 5, 2>(p, s);
        return p.fp4 ? launch_batch<true, F16, 1, 4, 4, 2>(p, s) : launch_batch<false, F16, 1, 4, 4, 2>(p, s);
    }
    if (p.M <= 16) return p.fp4 ? launch_batch<true, F16, 2, 1, 8, 3>(p, s) : launch_batch<false, F16, 2, 1, 9, 2>(p, s);
    if (p.M <= 32) return p.fp4 ? launch_batch<true, F16, 2, 2, 7, 2>(p, s) : launch_batch<false, F16, 2, 2, 6, 2>(p, s);
    if (p.M <= 48) return p.fp4 ? launch_batch<true, F16, 2, 3, 5, 2>(p, s) : launch_batch<false, F16, 2, 3, 4, 2>(p, s);
    return p.fp4 ? launch_batch<true, F16, 2, 4, 4, 2>(p, s) : launch_batch<false, F16, 2, 4, 3, 2>(p, s);
}

}  // namespace

// Products of at most 64 rows of A, row-major, with B stored N x K: the register kernel up to 8 rows
// and, up to 32, where rows are not aligned for the LDS kernel, which takes the others.
bool mx_token_takes(const MxProblem &p) {
    // (a launch's threads are counted in 32 bits: at most 512 for 4 rows of B here)
    if (p.ta || !p.tb || p.N >= (1 << 24)) return false;
    return p.M <= 32 || (p.M <= 64 && mx_rows_aligned(p));
}

hipError_t launch_mx_token(const MxProblem &p, hipStream_t s, const char **name) {
    const bool lds = p.M > 8 && mx_rows_aligned(p);
#define REGTILE_TOKEN_SET(elt, fmt)                                                                            \
    {{elt "_" fmt "_token4", elt "_" fmt "_token8", elt "_" fmt "_token16", elt "_" fmt "_token32"},          \
     {elt "_" fmt "_batch16", elt "_" fmt "_batch32", elt "_" fmt "_batch48", elt "_" fmt "_batch64"}}
    static const char *const names[2][2][2][4] = {{REGTILE_TOKEN_SET("bf16", "int8"), REGTILE_TOKEN_SET("bf16", "fp4")},
                                                  {REGTILE_TOKEN_SET("f16", "int8"), REGTILE_TOKEN_SET("f16", "fp4")}};
#undef REGTILE_TOKEN_SET
    if (lds) {
        *name = names[p.f16][p.fp4][1][(p.M - 1) / 16];
        return p.f16 ? launch_batch_rows<true>(p, s) : launch_batch_rows<false>(p, s);
    }
    *name = names[p.f16][p.fp4][0][p.M <= 4 ? 0 : p.M <= 8 ? 1 : p.M <= 16 ? 2 : 3];
    if (p.fp4) return p.f16 ? launch_token_rows<true, true>(p, s) : launch_token_rows<true, false>(p, s);
    return p.f16 ? launch_token_rows<false, true>(p, s) : launch_token_rows<false, false>(p, s);
}

}  // namespace regtile

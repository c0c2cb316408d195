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

// NF fragments of 16 / H rows of B and MC fragments of 16 / H tokens a wave; U chunks in flight
template <bool FP4, bool F16, int H, int NF, int MC, int NW, int U>
__global__ __launch_bounds__(NW * 64) void mx_token_kernel(int M, int N, int K, float alpha,
                                                           const uint16_t *__restrict__ A, int64_t lda,
                                                           const uint8_t *__restrict__ Q, int64_t ldq,
                                                           const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                           float *__restrict__ C, int64_t ldc, int vec_c) {
    typedef Frag<16, F16> F;
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

    typename F::acc_t acc[NF][MC];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MC; ++i) acc[f][i] = typename F::acc_t{0.f, 0.f, 0.f, 0.f};

    uint32_t q[U][NF][GB / 4], s[U][NF];
    uint4 x[U][MC][4];
    auto compute = [&](int u) {
        float sc[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) sc[f] = mx::scale_value<FP4>(s[u][f]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                const bf16x8 w = __builtin_bit_cast(bf16x8, mx::expand8<FP4, F16>(q[u][f], t, sc[f]));
#pragma unroll
                for (int i = 0; i < MC; ++i) acc[f][i] = F::mfma(w, __builtin_bit_cast(bf16x8, x[u][i][t]), acc[f][i]);
            }
    };

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
            if (c0 + u * NW < nfull) compute(u);
    }
    if (K % CHUNK != 0 && wave == nfull % NW) {  // the last, short chunk
        const int64_t c = nfull;
        const int left = K - nfull * CHUNK - koff;  // of this lane's group
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            const uint8_t *p = qp[f] + c * (CHUNK / 32 * GB);
#pragma unroll
            for (int i = 0; i < GB / 4; ++i) q[0][f][i] = 0;
            s[0][f] = 0;
            if (left > 0) {
                s[0][f] = sp[f][c * (CHUNK / 32)];
                if (left >= 32)
                    mx::load_bytes<GB>(p, q[0][f]);
                else
                    mx::load_codes_tail<FP4, GB>(p, left, q[0][f]);
            }
        }
#pragma unroll
        for (int i = 0; i < MC; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint16_t *p = xp[i] + c * CHUNK + 8 * t;
                uint32_t d[4] = {0, 0, 0, 0};
                if (left >= 8 * t + 8) {
                    __builtin_memcpy(d, p, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (8 * t + e < left) d[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
                }
                x[0][i][t] = make_uint4(d[0], d[1], d[2], d[3]);
            }
        compute(0);
    }

    // accumulator v of lane l: row 4 (l / 16) + v of B's fragment, column l % 16 of A's
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int i = 0; i < MC; ++i) part[wave][f * MC + i][lane] = __builtin_bit_cast(float4, acc[f][i]);
    __syncthreads();
    for (int o = tid; o < NF * MC * 64; o += NW * 64) {
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

#ifndef TK_CFG4
#define TK_CFG4 1, 1, 8, 2
#define TK_CFG2 1, 1, 8, 4
#define TK_CFG1 1, 1, 8, 4
#define TK_CFGM 1, 2, 8, 4
#endif

template <bool FP4, bool F16>
hipError_t launch_token_rows(const MxProblem &p, hipStream_t s) {
    if (p.M <= 4) return launch_token<FP4, F16, 4, TK_CFG4>(p, s);
    if (p.M <= 8) return launch_token<FP4, F16, 2, TK_CFG2>(p, s);
    if (p.M <= 16) return launch_token<FP4, F16, 1, TK_CFG1>(p, s);
    return launch_token<FP4, F16, 1, TK_CFGM>(p, s);
}

}  // namespace

// Takes (and launches, status in *err) products of at most 32 rows of A, row-major, with B stored
// N x K; returns false, launching nothing, for any other.
bool launch_mx_token(const MxProblem &p, hipStream_t s, const char **name, hipError_t *err) {
    if (p.ta || !p.tb || p.M > 32) return false;
#define REGTILE_TOKEN_SET(elt, fmt) {elt "_" fmt "_token4", elt "_" fmt "_token8", elt "_" fmt "_token16", elt "_" fmt "_token32"}
    static const char *const names[2][2][4] = {{REGTILE_TOKEN_SET("bf16", "int8"), REGTILE_TOKEN_SET("bf16", "fp4")},
                                               {REGTILE_TOKEN_SET("f16", "int8"), REGTILE_TOKEN_SET("f16", "fp4")}};
#undef REGTILE_TOKEN_SET
    *name = names[p.f16][p.fp4][p.M <= 4 ? 0 : p.M <= 8 ? 1 : p.M <= 16 ? 2 : 3];
    if (p.fp4)
        *err = p.f16 ? launch_token_rows<true, true>(p, s) : launch_token_rows<true, false>(p, s);
    else
        *err = p.f16 ? launch_token_rows<false, true>(p, s) : launch_token_rows<false, false>(p, s);
    return true;
}

}  // namespace regtile

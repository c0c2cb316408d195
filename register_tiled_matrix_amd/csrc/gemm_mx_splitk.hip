// gemm_mx_splitk.hip -- C = alpha A op(B) + beta C for products of few tiles with a row-major A and a
// block-scaled (MX) B stored N x K: K split over the waves of a workgroup (and over workgroups).
//
// The 16-bit split-K kernel (gemm_bf16_mfma_splitk.hip) with B left in its codes until the last
// moment: a workgroup owns a 64x64 tile and walks K in slabs of 128, whose A rows, codes and scale bytes
// all come to LDS by DMA, into a ring of R slabs. Wave w takes the slab's k 32 w .. 32 w + 31, one group of
// every row of B, and accumulates the whole tile over its share, so each code is expanded by one wave
// only, in registers (mx_common.h; exact). Per slab and CU LDS moves 2 x 21 KB for fp4 (2 x 26 int8)
// where 16-bit operands move 2 x 32, and L1 fills 21 KB against 32: the two rates that bound the
// 16-bit kernel.
//
// The k order inside a group is free as long as both operands agree: lanes 0-31 take k 0 .. 15 of the
// group and lanes 32-63 k 16 .. 31, 8 of them in each of two MFMAs, so that a lane's codes are one LDS
// read of 8 bytes (fp4) or 16 (int8) for both.
//
// LDS, in 16-byte chunks: A's rows are 16 of them, chunk c of row r at slot c ^ (r & 15); fp4 rows 4, at
// c ^ (r >> 2 & 3); int8 rows 8, at c ^ (r >> 1 & 7); then one dword of scale bytes a row, a copy for each
// wave. Rows past M or N repeat the last (their outputs are not stored); the K tail of less than a slab
// goes from memory to registers with checks.
#include <type_traits>

#include "mfma_common.h"
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {
using namespace mfma;

constexpr int MXS_T = 64, MXS_BK = 128, MXS_NW = 4, MXS_NT = MXS_NW * 64;
constexpr int MXS_PSTRIDE = MXS_T + 8;  // row stride (floats) of a partial tile in LDS

template <bool FP4, bool F16, int R>
__global__ __launch_bounds__(MXS_NT) void mx_splitk_kernel(int M, int N, int K, float alpha,
                                                           const uint16_t *__restrict__ A, int64_t lda,
                                                           const uint8_t *__restrict__ Q, int64_t ldq,
                                                           const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                           float *__restrict__ C, int64_t ldc, int tiles_m, int tiles_n,
                                                           int per_split, int64_t split_stride, int vec_c) {
    typedef Frag<32, F16> F;
    constexpr int QCH = FP4 ? 4 : 8;                 // chunks of a row of codes
    constexpr int A_SLOTS = MXS_T * 16, Q_SLOTS = MXS_T * QCH;
    constexpr int SLAB = A_SLOTS + Q_SLOTS + MXS_NW * 16;
    constexpr int JA = A_SLOTS / MXS_NT, JQ = Q_SLOTS / MXS_NT, PER = JA + JQ + 1;  // DMA instructions a wave and slab
    constexpr int PART = MXS_NW * MXS_T * MXS_PSTRIDE / 4;
    static_assert(R >= 4 && PER * (R - 2) < 64 && R * SLAB * 16 <= 160 * 1024 && PART <= R * SLAB, "ring");
    __shared__ uint4 smem[R * SLAB];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n;
    const int split = id / tiles;  // part of k: per_split slabs
    int tm, tn;
    grouped_tile<8>(id - split * tiles, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * MXS_T, n0 = (int64_t)tn * MXS_T;
    C += split * split_stride;
    const int nfull = K / MXS_BK, all = (K + MXS_BK - 1) / MXS_BK;
    const int first = split * per_split, last = min(first + per_split, all);
    const int nslabs = min(last, nfull) - first;  // whole slabs of this part (none below 1)
    auto row_m = [&](int r) { return min(m0 + r, (int64_t)M - 1); };
    auto row_n = [&](int r) { return min(n0 + r, (int64_t)N - 1); };

    // ---- DMA: this lane's source of each instruction, at this part's first slab ----
    const uint16_t *asrc[JA];
    const uint8_t *qsrc[JQ], *ssrc;
#pragma unroll
    for (int j = 0; j < JA; ++j) {
        const int p = (wave * JA + j) * 64 + lane, r = p / 16, c = (p % 16) ^ (r & 15);
        asrc[j] = A + row_m(r) * lda + (int64_t)first * MXS_BK + c * 8;
    }
#pragma unroll
    for (int j = 0; j < JQ; ++j) {
        const int p = (wave * JQ + j) * 64 + lane, r = p / QCH, c = (p % QCH) ^ (FP4 ? (r >> 2) & 3 : (r >> 1) & 7);
        qsrc[j] = Q + row_n(r) * ldq + (int64_t)first * (QCH * 16) + c * 16;
    }
    ssrc = S + row_n(lane) * lds + (int64_t)first * 4;
    // slab `slab` of the part into ring slot `slot`; past the last the last is loaded again, into a
    // slot that is not read any more, so that every wait has the same count
    auto issue = [&](int slab, int slot) {
        const int64_t s = min(slab, nslabs - 1);
        uint4 *d = smem + slot * SLAB;
#pragma unroll
        for (int j = 0; j < JA; ++j) dma16(asrc[j] + s * MXS_BK, d + (wave * JA + j) * 64);
#pragma unroll
        for (int j = 0; j < JQ; ++j) dma16(qsrc[j] + s * (QCH * 16), d + A_SLOTS + (wave * JQ + j) * 64);
        dma4(ssrc + s * 4, d + A_SLOTS + Q_SLOTS + wave * 16);
    };

    typename F::acc_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < F::NACC; ++v) acc[i][j][v] = 0.0f;

    // ---- one slab's operands of this wave: A fragments, codes and scales of two columns of C ----
    const int fr = lane & 31, half = lane >> 5;
    bf16x8 fa[2][2][2];               // [buffer][k step][i]
    uint32_t q[2][2][FP4 ? 2 : 4], sc[2][2];  // [buffer][j]
    auto read_slab = [&](int slot, int buf) {
        const uint4 *d = smem + slot * SLAB;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 32 * i + fr;
                fa[buf][t][i] = __builtin_bit_cast(bf16x8, lds_read16(&d[r * 16 + ((4 * wave + 2 * half + t) ^ (r & 15))]));
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 32 * j + fr;
            const uint4 *row = d + A_SLOTS + r * QCH;
            if constexpr (FP4) {
                const u32x2 v = lds_read8(reinterpret_cast<const char *>(row + (wave ^ ((r >> 2) & 3))) + 8 * half);
                q[buf][j][0] = v[0];
                q[buf][j][1] = v[1];
            } else {
                const u32x4 v = lds_read16(&row[(2 * wave + half) ^ ((r >> 1) & 7)]);
#pragma unroll
                for (int e = 0; e < 4; ++e) q[buf][j][e] = v[e];
            }
            sc[buf][j] = reinterpret_cast<const uint8_t *>(d + A_SLOTS + Q_SLOTS + wave * 16)[r * 4 + wave];
        }
    };
    auto multiply = [&](int buf) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float s = mx::scale_value<FP4>(sc[buf][j]);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bf16x8 b = __builtin_bit_cast(bf16x8, mx::expand8<FP4, F16>(q[buf][j], t, s));
#pragma unroll
                for (int i = 0; i < 2; ++i) acc[i][j] = F::mfma(fa[buf][t][i], b, acc[i][j]);
            }
        }
    };

    if (nslabs > 0) {
        auto wrap = [](int x) { return x >= R ? x - R : x; };
        // slab s, in register buffer BUF: its operands were read while slab s - 1 was multiplied
        auto iteration = [&](int s, int slot, auto buf_tag) {
            constexpr int BUF = decltype(buf_tag)::value;
            wait_lgkmcnt0();
            __builtin_amdgcn_sched_barrier(0);
            read_slab(wrap(slot + 1), BUF ^ 1);     // slab s + 1, published a barrier ago
            issue(s + R - 1, wrap(slot + R - 1));   // into slab s - 1's slot
            multiply(BUF);
            __builtin_amdgcn_sched_barrier(0);
            wait_vmcnt<PER *(R - 3)>();  // own loads of slab s + 2 have landed
            lds_barrier();               // slab s + 2 published; slab s's slot read by nobody any more
        };
#pragma unroll
        for (int s = 0; s + 1 < R; ++s) issue(s, s);
        wait_vmcnt<PER *(R - 2)>();  // own loads of slab 0
        lds_barrier();
        read_slab(0, 0);
        wait_vmcnt<PER *(R - 3)>();  // own loads of slab 1
        lds_barrier();
        int slot = 0;
        for (int s = 0; s < nslabs; s += 2) {
            iteration(s, slot, std::integral_constant<int, 0>{});
            slot = wrap(slot + 1);
            if (s + 1 < nslabs) {
                iteration(s + 1, slot, std::integral_constant<int, 1>{});
                slot = wrap(slot + 1);
            }
        }
        wait_vmcnt<0>();  // no DMA may still be writing the ring when it turns into partial tiles
        wait_lgkmcnt0();
    }
    // ---- the K tail: less than a slab, this wave's group of it, with checks ----
    if (last > nfull && K % MXS_BK != 0) {
        const int64_t k0 = (int64_t)nfull * MXS_BK + 32 * wave + 16 * half;
        const int left = (int)min((int64_t)16, K - k0);  // of this lane's 16
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint16_t *p = A + row_m(32 * i + fr) * lda + k0 + 8 * t;
                uint32_t d[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (8 * t + e < left) d[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
                fa[0][t][i] = __builtin_bit_cast(bf16x8, make_uint4(d[0], d[1], d[2], d[3]));
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t r = row_n(32 * j + fr);
#pragma unroll
            for (int e = 0; e < (FP4 ? 2 : 4); ++e) q[0][j][e] = 0;
            sc[0][j] = 0;
            if (left > 0) {
                sc[0][j] = S[r * lds + k0 / mx::GROUP];
                mx::load_codes_tail<FP4, FP4 ? 8 : 16>(Q + r * ldq + (FP4 ? k0 / 2 : k0), left, q[0][j]);
            }
        }
        multiply(0);
    }
    __syncthreads();  // every wave is done with the ring

    // ---- partial tiles, their sum in wave order, the epilogue ----
    float *part = reinterpret_cast<float *>(smem);
    {
        float *mine = part + wave * MXS_T * MXS_PSTRIDE;
        const int rl = F::row_lane(lane);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < F::NACC; ++v)
                    mine[(i * 32 + rl + F::row_acc(v)) * MXS_PSTRIDE + j * 32 + fr] = acc[i][j][v];
    }
    __syncthreads();
    // thread t: four columns 4 (t % 16) .. of rows t / 16, t / 16 + 16, ...
    const int ecol = 4 * (tid % 16);
    const int64_t gcol = n0 + ecol;
#pragma unroll
    for (int e = 0; e < MXS_T / 16; ++e) {
        const int r = tid / 16 + 16 * e;
        if (m0 + r >= M || gcol >= N) continue;
        float4 v = *reinterpret_cast<const float4 *>(&part[r * MXS_PSTRIDE + ecol]);
#pragma unroll
        for (int w = 1; w < MXS_NW; ++w) {
            const float4 p = *reinterpret_cast<const float4 *>(&part[(w * MXS_T + r) * MXS_PSTRIDE + ecol]);
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
        }
        float *cp = C + (m0 + r) * ldc + gcol;
        if (vec_c && gcol + 3 < N) {
            float4 o = make_float4(alpha * v.x, alpha * v.y, alpha * v.z, alpha * v.w);
            if (beta != 0.0f) {
                const float4 old = *reinterpret_cast<const float4 *>(cp);
                o = make_float4(fmaf(alpha, v.x, beta * old.x), fmaf(alpha, v.y, beta * old.y),
                                fmaf(alpha, v.z, beta * old.z), fmaf(alpha, v.w, beta * old.w));
            }
            *reinterpret_cast<float4 *>(cp) = o;
        } else {
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (gcol + u < N) cp[u] = epilogue_value(x[u], alpha, beta, cp + u);
        }
    }
}

// slabs in the ring, as many as LDS holds
constexpr int MXS_RF = 7, MXS_RI = 6;

template <bool FP4, bool F16>
hipError_t launch_mxs(const MxProblem &p, hipStream_t s, int splits) {
    constexpr int R = FP4 ? MXS_RF : MXS_RI;
    const int tiles_m = (p.M + MXS_T - 1) / MXS_T, tiles_n = (p.N + MXS_T - 1) / MXS_T;
    const int slabs = (p.K + MXS_BK - 1) / MXS_BK, per = (slabs + splits - 1) / splits;
    const MxParts o = mx_parts(p, splits);
    note_launch(reinterpret_cast<const void *>(&mx_splitk_kernel<FP4, F16, R>), MXS_NT);
    hipLaunchKernelGGL((mx_splitk_kernel<FP4, F16, R>), dim3((unsigned)((int64_t)tiles_m * tiles_n * splits)), dim3(MXS_NT),
                       0, s, p.M, p.N, p.K, o.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S, p.lds, o.beta, o.C,
                       o.ldc, tiles_m, tiles_n, per, o.stride, o.ldc % 4 == 0 && aligned16(o.C) && o.stride % 4 == 0);
    hipError_t e = hipGetLastError();
    return e == hipSuccess && splits > 1 ? launch_mx_join(p, s, splits) : e;
}

}  // namespace

// Two rounds of tiles at most, and few tiles where K is long: past tiles x K = 2^21 the tiles re-read
// A and B from L2 more than 128-wide ones, split over workgroups, lose. us, this kernel against that one
// (fp4): 1024 x 2048 x 1024 14.9, 21.2; 256 x 4096 x 4096 19.0, 27.1; 1024 x 1024 x 8192 34.0, 33.8;
// 512 x 8192 x 4096 47.5, 46.6; past it 1024 x 1024 x 16384 62.9, 56.6; 256 x 8192 x 8192 60.9, 53.2.
bool mx_splitk_takes(const MxProblem &p) {
    if (p.ta || !p.tb || !mx_rows_aligned(p)) return false;
    const int64_t tiles = (((int64_t)p.M + MXS_T - 1) / MXS_T) * (((int64_t)p.N + MXS_T - 1) / MXS_T);
    return p.M > 64 && p.K >= 512 && tiles <= 512 && tiles * p.K <= (int64_t(1) << 21);
}

hipError_t launch_mx_splitk(const MxProblem &p, const MxPlan &plan, hipStream_t s, const char **name) {
    static const char *const names[2][2] = {{"bf16_int8_splitk4_64x64x128", "bf16_fp4_splitk4_64x64x128"},
                                            {"f16_int8_splitk4_64x64x128", "f16_fp4_splitk4_64x64x128"}};
    *name = names[p.f16][p.fp4];
    const int splits = mx_fit_parts(p, plan);
    if (p.fp4) return p.f16 ? launch_mxs<true, true>(p, s, splits) : launch_mxs<true, false>(p, s, splits);
    return p.f16 ? launch_mxs<false, true>(p, s, splits) : launch_mxs<false, false>(p, s, splits);
}

}  // namespace regtile

// gemm_mx_codes.hip -- C = alpha A op(B) + beta C for large products with a row-major A and a 4-bit
// block-scaled (MX fp4) B stored N x K: B stays in codes in LDS and is expanded as fragments are read.
//
// The T x T tile of 4 waves (T = 256, or 128 for few tiles), the LDS DMA and the schedule are those of
// gemm_mx_dma.hip; what differs is B. There, codes pass through registers into 16-bit LDS slabs: at T =
// 256, 32 KB are written and 64 KB read back (each column by two waves) a slab. Here they go to LDS by
// DMA and each wave expands its own fragments: 8 KB in and 16 KB out. The expansion is done twice (in
// the two waves that share a column), but it is 4 conversions for a fragment that feeds 4 (2) MFMAs,
// and they fit between those. Against that kernel: 8192^3 809 us, 887.
//
// Units of K are 128 deep: two slabs of A (a ring of three, 32 KB each) and 64 bytes of codes and one
// dword of scale bytes for each column (a ring of two units, 17 KB each; half of all that at T = 128). The k order inside a group
// of 32 is free as long as both operands agree: lanes 0-31 take k 0 .. 15 and lanes 32-63 k 16 .. 31, 8 of
// them in each of two k steps, so that a lane's codes for both are one 8-byte read.
//
// Edges: rows of A past M load zeros through the descriptor, columns past N repeat the last; K is whole
// units.
#include <type_traits>

#include "mfma_common.h"
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {
using namespace mfma;

constexpr int MXC_NT = 256;
typedef uint32_t __attribute__((may_alias)) u32_any;  // as lds_read16 and lds_read8: no wait for DMA

template <int T, bool F16>
__global__ __launch_bounds__(MXC_NT) void mx_codes_kernel(int M, int N, int K, float alpha,
                                                          const uint16_t *__restrict__ A, int64_t lda,
                                                          const uint8_t *__restrict__ Q, int64_t ldq,
                                                          const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                          float *__restrict__ C, int64_t ldc, int tiles_m, int tiles_n,
                                                          int per_split, int64_t split_stride) {
    constexpr int MF = 32, KCH = 8;
    typedef Frag<MF, F16> F;
    constexpr int WT = T / 2, MI = WT / MF, NI = WT / MF, NMFMA = MI * NI;
    constexpr int SLAB = T * KCH, CODES = T * 4, UNIT = CODES + MXC_NT / 4;  // 16-byte slots
    constexpr int JA = SLAB / MXC_NT, JQ = CODES / MXC_NT, PER_UNIT = JQ + 1;
    __shared__ uint4 smem[3 * SLAB + 2 * UNIT];
    uint4 *const units = smem + 3 * SLAB;

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n;
    const int split = id / tiles;  // part of k, per_split units
    grouped_tile<8>(id - split * tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * T, n0 = tn * T;
    const int first = split * per_split, nunits = min(per_split, K / 128 - first), nslabs = 2 * nunits;
    C += split * split_stride;

    // ---- DMA ----
    const rsrc_t a_rsrc = make_rsrc(A + (int64_t)m0 * lda, addr::desc_bytes(min(T, M - m0), lda, K, 2));
    uint32_t a_voff[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int ka;
        a_voff[j] = addr::kc_dma_lane<KCH, MF>(wave, JA, j, lane, lda, &ka);
    }
    auto dma_a = [&](int slab, int slot) {  // past the last slab the last again, into a free slot
        const int k0 = (2 * first + min(slab, nslabs - 1)) * 64;
#pragma unroll
        for (int q = 0; q < JA; ++q)
            dma16_buf(a_rsrc, a_voff[q & 1], addr::kc_dma_instr<KCH>(q, k0, lda), smem + slot * SLAB + (wave * JA + q) * 64);
    };
    const uint8_t *qsrc[JQ], *ssrc;
    auto row_n = [&](int r) { return min(n0 + r, N - 1); };
#pragma unroll
    for (int j = 0; j < JQ; ++j) {
        const int p = (wave * JQ + j) * 64 + lane, r = p / 4, c = (p % 4) ^ ((r >> 2) & 3);
        qsrc[j] = Q + (int64_t)row_n(r) * ldq + c * 16;
    }
    ssrc = S + (int64_t)row_n((wave * 64 + lane) % T) * lds;  // (T = 128: twice, to keep the waves' counts alike)
    auto dma_codes = [&](int unit, int slot) {
        const int64_t u = first + min(unit, nunits - 1);
        uint4 *d = units + slot * UNIT;
#pragma unroll
        for (int j = 0; j < JQ; ++j) dma16(qsrc[j] + u * 64, d + (wave * JQ + j) * 64);
        dma4(ssrc + u * 4, d + CODES + wave * 16);
    };

    // ---- fragments ----
    typename F::acc_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int v = 0; v < F::NACC; ++v) acc[i][j][v] = 0.0f;
    const int fr = lane & 31, half = lane >> 5;
    bf16x8 fa[2][MI];
    u32x2 codes[2][NI];    // [group parity]: this lane's 16 codes of each column of C
    uint32_t scale4[NI];   // a unit's four scale bytes of each
    // A's fragments of k step kk (0 .. 3) of the slab in `slot`: k 16 half + 8 (kk % 2) of group kk / 2
    auto read_a = [&](int slot, int kk, int buf) {
        const uint4 *s = smem + slot * SLAB;
        const int c = 4 * (kk >> 1) + 2 * half + (kk & 1);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = wm * WT + i * MF + fr;
            fa[buf][i] = __builtin_bit_cast(bf16x8, lds_read16(&s[r * KCH + (c ^ slab_key<KCH, MF>(r))]));
        }
    };
    auto read_codes = [&](int slot, int g, int buf) {
        const uint4 *u = units + slot * UNIT;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int r = wn * WT + j * MF + fr;
            codes[buf][j] = lds_read8(reinterpret_cast<const char *>(u + r * 4 + (g ^ ((r >> 2) & 3))) + 8 * half);
        }
    };
    auto read_scales = [&](int slot) {
        const u32_any *s = reinterpret_cast<const u32_any *>(units + slot * UNIT + CODES);
#pragma unroll
        for (int j = 0; j < NI; ++j) scale4[j] = s[wn * WT + j * MF + fr];
    };
    // the MFMAs of unit k step k (0 .. 7), column by column of fragments: each column is expanded
    // while the one before it is multiplied
    auto multiply = [&](int k, int vmem, int reads) {
        const int g = k >> 1;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const float s = mx::scale_value<true>((scale4[j] >> (8 * g)) & 255u);
            const uint32_t q[1] = {codes[g & 1][j][k & 1]};
            const bf16x8 b = __builtin_bit_cast(bf16x8, mx::expand8<true, F16>(q, 0, s));
#pragma unroll
            for (int ii = 0; ii < MI; ++ii) {
                const int i = (j & 1) ? MI - 1 - ii : ii;
                acc[i][j] = F::mfma(fa[k & 1][i], b, acc[i][j]);
            }
        }
        auto share = [](int n, int g_) { return ((g_ + 1) * n) / NMFMA - (g_ * n) / NMFMA; };
        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
#pragma unroll
        for (int m = 0; m < NMFMA; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t < share(vmem, m)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t < share(reads, m)) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            if (m < NMFMA - MI) {  // the next column's 4 conversions and its scale
                __builtin_amdgcn_sched_group_barrier(0x002, 4 / MI, 0);
                if (m % MI == MI - 1) __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    auto wrap3 = [](int x) { return x >= 3 ? x - 3 : x; };
    // SH: the second half of the waves issues its DMA a k step later, so that on each pair of waves one
    // keeps the matrix pipes busy
    auto loop = [&](auto shift_tag) {
        constexpr int SH = decltype(shift_tag)::value;
        dma_codes(0, 0);
        dma_a(0, 0);
        dma_a(1, 1);
        if (SH == 0) {
            dma_codes(1, 1);
            dma_a(2, 2);
        }
        wait_vmcnt<JA + (SH == 0 ? PER_UNIT + JA : 0)>();  // A of slab 0 and unit 0 have landed
        lds_barrier();
        read_a(0, 0, 0);
        read_codes(0, 0, 0);
        read_scales(0);
        int a0 = 0;  // ring slot of the unit's first slab
        for (int u = 0; u < nunits; ++u) {
            const int a1 = wrap3(a0 + 1), a2 = wrap3(a0 + 2), slot = u & 1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                wait_lgkmcnt0();  // this step's operands
                __builtin_amdgcn_sched_barrier(0);
                int vmem = 0, reads = MI;
                if (k == 3) {
                    // the other slab of this unit has landed: unit u + 1's codes and A of slab
                    // 2 u + 2 are younger
                    wait_vmcnt<PER_UNIT + JA>();
                    lds_barrier();
                } else if (k == 7) {
                    // A of slab 2 u + 2 and the codes of unit u + 1 have landed: A of slab 2 u + 3 is younger
                    wait_vmcnt<JA>();
                    lds_barrier();
                }
                if (k == 7) {
                    read_a(a2, 0, 0);
                    read_codes(slot ^ 1, 0, 0);
                } else {
                    read_a(k < 3 ? a0 : a1, (k + 1) & 3, (k + 1) & 1);
                    if (k & 1) read_codes(slot, (k + 1) >> 1, ((k + 1) >> 1) & 1);
                }
                if (k & 1) reads += NI;
                // freed by the barrier of step 7 of unit u - 1: the codes' other unit and the slot of
                // slab 2 u - 1; by that of step 3: slab 2 u's
                if (k == (SH ? 0 : 7)) {
                    const int v = SH ? u : u + 1;  // the unit that begins after that barrier
                    dma_codes(v + 1, (v + 1) & 1);
                    dma_a(2 * v + 2, SH ? a2 : a1);
                    vmem = PER_UNIT + JA;
                }
                if (k == (SH ? 4 : 3)) {
                    dma_a(2 * u + 3, a0);
                    vmem = JA;
                }
                multiply(k, vmem, reads);
                if (k == 7) read_scales(slot ^ 1);
            }
            a0 = a2;
        }
    };
    if (wave >= 2)
        loop(std::integral_constant<int, 1>{});
    else
        loop(std::integral_constant<int, 0>{});
    wait_vmcnt<0>();  // no LDS DMA may still be in flight when the workgroup retires

    // ---- epilogue: buffer stores through a descriptor that ends at C's last element ----
    const rsrc_t c_rsrc = make_rsrc(C + (int64_t)m0 * ldc + n0, addr::desc_bytes(min(T, M - m0), ldc, N - n0, 4));
    const int elane = __lane_id();
    const uint32_t lane_off = addr::c_lane_off<MF>(wm * WT, wn * WT, elane, ldc);
    uint32_t off_j[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) off_j[j] = n0 + wn * WT + j * MF + elane % MF < N ? lane_off : addr::kPastEnd;
    if (beta != 0.0f) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            float c[NI][F::NACC];
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < F::NACC; ++v) c[j][v] = load_f32_buf(c_rsrc, off_j[j], addr::c_acc_off<MF>(i, j, v, ldc));
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < F::NACC; ++v)
                    store_f32_buf(c_rsrc, off_j[j], addr::c_acc_off<MF>(i, j, v, ldc),
                                  fmaf(alpha, acc[i][j][v], beta * c[j][v]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < F::NACC; ++v)
                    store_f32_buf(c_rsrc, off_j[j], addr::c_acc_off<MF>(i, j, v, ldc), alpha * acc[i][j][v]);
    }
}

template <int T, bool F16>
hipError_t launch_codes(const MxProblem &p, hipStream_t s, int splits) {
    const int tiles_m = (p.M + T - 1) / T, tiles_n = (p.N + T - 1) / T;
    const int per = (p.K / 128 + splits - 1) / splits;
    const MxParts o = mx_parts(p, splits);
    note_launch(reinterpret_cast<const void *>(&mx_codes_kernel<T, F16>), MXC_NT);
    hipLaunchKernelGGL((mx_codes_kernel<T, F16>), dim3((unsigned)((int64_t)tiles_m * tiles_n * splits)), dim3(MXC_NT), 0, s,
                       p.M, p.N, p.K, o.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S, p.lds, o.beta, o.C, o.ldc,
                       tiles_m, tiles_n, per, o.stride);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && splits > 1 ? launch_mx_join(p, s, splits) : e;
}

}  // namespace

// fp4 products that the DMA kernel would run, with B stored N x K, rows aligned for the DMA and K in
// whole units
bool mx_codes_takes(const MxProblem &p) {
    return p.fp4 && !p.ta && p.tb && p.K % 128 == 0 && mx_rows_aligned(p) && mx_dma_takes(p);
}

hipError_t launch_mx_codes(const MxProblem &p, const MxPlan &plan, hipStream_t s, const char **name) {
    const int splits = mx_fit_parts(p, plan);
    const bool small = (splits == plan.parts ? plan.tile : plan.narrow) == 128;
    static const char *const names[2][2] = {{"bf16_fp4_codes_256x256x128_nt", "bf16_fp4_codes_128x128x128_nt"},
                                            {"f16_fp4_codes_256x256x128_nt", "f16_fp4_codes_128x128x128_nt"}};
    *name = names[p.f16][small];
    if (small) return p.f16 ? launch_codes<128, true>(p, s, splits) : launch_codes<128, false>(p, s, splits);
    return p.f16 ? launch_codes<256, true>(p, s, splits) : launch_codes<256, false>(p, s, splits);
}

}  // namespace regtile

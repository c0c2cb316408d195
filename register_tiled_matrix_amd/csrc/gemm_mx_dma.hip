// gemm_mx_dma.hip -- C = alpha op(A) op(B) + beta C with a block-scaled (MX) B for large products:
// A from HBM to LDS by DMA, B's codes through registers.
//
// The tile, ring and schedule are those of the 16-bit kernel (gemm_bf16_mfma_dma.hip): 4 waves on a
// T x T tile (T = 256, or 128 for few tiles), slabs of 64 k in a ring of five LDS halves, fragments of
// the next k step read and DMA issued between the MFMAs of this one, one barrier a slab. Slab t's A
// part sits in half (2 t) % 5 and its B part in half (2 t + 1) % 5.
//
// B: a thread owns T / 128 groups of 32 codes of each slab. Codes and scale bytes are loaded two slabs
// ahead, and while slab s is multiplied those of slab s + 1 are expanded to the 16-bit type (exact;
// mx_common.h) and written to their half, a group in a k step, between MFMAs. Expanding costs 0.5
// (fp4) or 2.5 (int8) vector instructions a value and happens once a workgroup; keeping the codes in
// LDS and expanding fragments would repeat it in the two waves that share each column.
//
// LDS holds each operand in its own storage order: K-contiguous rows (64 k, slab_key), M/N-contiguous
// ones (64 rows of T elements) read with transposing reads. B's N-contiguous slab has a swizzle of its
// own, for its writes: the 16 lanes of a write hold the same chunk of 8 groups of 2 rows (T = 256) or
// 4 groups of 4 rows (T = 128), which the key spreads over all 16 slots of a 256-byte line.
//
// Edges: A as in the 16-bit kernel (descriptors that end at the matrix's last element; zeros past K).
// B's groups past N or K are loaded from the last one before the edge. Past N they feed outputs that
// are not stored; past K their scale is replaced by 2^-127, so that they are finite and meet zeros of
// A. The launcher admits only whole groups (B's columns a multiple of 32), so that no load passes the
// end of a row.
#include <type_traits>

#include "mfma_common.h"
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {
using namespace mfma;

constexpr int MXD_BK = 64, MXD_NT = 256;

// f on four parts of LDS that do not overlap
template <class F>
__device__ __forceinline__ void apart(const uint4 *__restrict__ ra, const uint4 *__restrict__ rb, uint4 *__restrict__ wa,
                                      uint4 *__restrict__ wb, F f) {
    f(ra, rb, wa, wb);
}

template <int T, bool FP4, bool F16, bool A_MN, bool B_MN, bool KTAIL, int NWIN, int STAGGER>
__global__ __launch_bounds__(MXD_NT) void mx_dma_kernel(int M, int N, int K, float alpha,
                                                        const uint16_t *__restrict__ A, int64_t lda,
                                                        const uint8_t *__restrict__ Q, int64_t ldq,
                                                        const uint8_t *__restrict__ S, int64_t lds, float beta,
                                                        float *__restrict__ C, int64_t ldc, int tiles_m, int tiles_n,
                                                        int per_split, int64_t split_stride) {
    constexpr int MF = 32, KCH = MXD_BK / 8, MCH = T / 8;
    typedef Frag<MF, F16> F;
    constexpr int WT = T / 2, MI = WT / MF, NI = WT / MF;
    constexpr int HALF = T * KCH;              // 16-byte slots
    constexpr int JA = HALF / MXD_NT;          // DMA instructions per wave and slab
    constexpr int NG = T * 2 / MXD_NT;         // groups of B per thread and slab
    constexpr int GB = FP4 ? 16 : 32;          // bytes of a group
    constexpr int LG = GB / 16 + 1;            // loads of a group
    constexpr int KSTEPS = MXD_BK / F::KSTEP, NMFMA = MI * NI;
    constexpr int NREAD = MI * (A_MN ? 2 : 1) + NI * (B_MN ? 2 : 1);
    constexpr int PER_WIN = JA / NWIN;
    static_assert(KSTEPS == 4 && JA % NWIN == 0 && NWIN + STAGGER <= 2, "windows at the last and the first k step");
    static_assert(NG == 1 || NG == 2, "groups go in k steps 1 and 2");
    __shared__ uint4 smem[5 * HALF];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave >> 1, wn = wave & 1;
    const int id = xcd_contiguous_id(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n;
    const int split = id / tiles;  // part of k, per_split slabs
    int tm, tn;
    grouped_tile<8>(id - split * tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * T, n0 = tn * T;
    const int all_slabs = (K + MXD_BK - 1) / MXD_BK, k_last = (all_slabs - 1) * MXD_BK;
    const int first_slab = split * per_split, nslabs = min(per_split, all_slabs - first_slab);
    C += split * split_stride;

    // ---- A ----
    const rsrc_t a_rsrc = A_MN ? make_rsrc(A + m0, addr::desc_bytes(K, lda, M - m0, 2))
                               : make_rsrc(A + (int64_t)m0 * lda, addr::desc_bytes(min(T, M - m0), lda, K, 2));
    uint32_t a_voff[2], a_voff_last[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        int ka;
        a_voff[j] = addr::kc_dma_lane<KCH, MF>(wave, JA, j, lane, lda, &ka);
        a_voff_last[j] = k_last + ka < K ? a_voff[j] : a_voff[j] | addr::kPastEnd;
        if (A_MN) a_voff[j] = addr::mn_dma_lane(lane, j, lda, MCH);
    }
    auto dma_a = [&](int q, int slab, uint4 *half) {
        const int k0 = (first_slab + min(slab, nslabs - 1)) * MXD_BK;
        const uint32_t voff = KTAIL && !A_MN && k0 == k_last ? a_voff_last[q & 1] : a_voff[q & 1];
        const uint32_t soff = A_MN ? addr::mn_dma_instr(wave, JA, q, k0, lda, MCH) : addr::kc_dma_instr<KCH>(q, k0, lda);
        dma16_buf(a_rsrc, voff, soff, half + (wave * JA + q) * 64);
    };
    auto window = [&](int win, int slab, uint4 *half) {
#pragma unroll
        for (int d = 0; d < PER_WIN; ++d) dma_a(win * PER_WIN + d, slab, half);
    };

    // ---- B ----
    // group i of this thread: slab row b_row and group b_g along it
    int b_row[NG], b_g[NG];
    const uint8_t *qbase[NG], *sbase[NG];
    constexpr int GPR = B_MN ? T / 32 : 2;  // groups of a slab row
    const int last_g = (B_MN ? N : K) / 32 - 1;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const int p = tid + MXD_NT * i;
        b_row[i] = p / GPR;
        b_g[i] = p % GPR;
        const int64_t row = B_MN ? 0 : min(n0 + b_row[i], N - 1), g = B_MN ? min(n0 / 32 + b_g[i], last_g) : 0;
        qbase[i] = Q + row * ldq + g * GB;
        sbase[i] = S + row * lds + g;
    }
    uint32_t q[NG][GB / 4];
    uint8_t sc[NG];  // (as bytes: widened where they are loaded, they are waited for there)
    auto load_group = [&](int i, int s) {
        const int slab = first_slab + s;
        int64_t qo, so;
        if constexpr (B_MN) {
            const int64_t k = min((int64_t)slab * MXD_BK + b_row[i], (int64_t)K - 1);
            qo = k * ldq;
            so = k * lds;
        } else {
            so = min(2 * slab + b_g[i], last_g);
            qo = so * GB;
        }
        mx::load_bytes<GB>(qbase[i] + qo, q[i]);
        sc[i] = sbase[i][so];
    };
    auto b_slot = [](int r, int c) {
        if constexpr (!B_MN) return r * KCH + (c ^ slab_key<KCH, MF>(r));
        const int low = T == 256 ? ((r & 1) << 1) | ((c >> 4) & 1) : r & 3;
        return r * MCH + (c ^ (4 * (r & 3)) ^ low);
    };
    auto write_group = [&](int i, int s_, uint4 *half) {
        const int slab = first_slab + s_;
        const bool past = B_MN ? slab * MXD_BK + b_row[i] >= K : 2 * slab + b_g[i] > last_g;
        const float s = mx::scale_value<FP4>(past ? 0u : sc[i]);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            lds_write16(half + b_slot(b_row[i], 4 * b_g[i] + t), mx::expand8<FP4, F16>(q[i], t, s));
    };

    // ---- fragments ----
    typename F::acc_t acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int v = 0; v < F::NACC; ++v) acc[i][j][v] = 0.0f;
    const int tr_t = lane & 15;
    const int tr_row = 8 * (lane >> 5) + (tr_t >> 2);             // row within the k step
    const int tr_col = 16 * ((lane >> 4) & 1) + 4 * (tr_t & 3);  // column within the fragment
    auto kc_frag = [&](const uint4 *slab, int row0, int kk) {
        const int row = row0 + (lane & 31), chunk = 2 * kk + (lane >> 5);
        return __builtin_bit_cast(bf16x8, lds_read16(&slab[row * KCH + (chunk ^ slab_key<KCH, MF>(row))]));
    };
    auto pair = [](const char *lo_at, const char *hi_at) {
        const uint2 lo = lds_read_tr16(lo_at), hi = lds_read_tr16(hi_at);
        return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
    };
    bf16x8 fa[2][MI], fb[2][NI];
    auto read_frags = [&](const uint4 *sa, const uint4 *sb, int kk, int buf) {
        const int row = 16 * kk + tr_row;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int col = wm * WT + i * MF + tr_col;
            const char *base = reinterpret_cast<const char *>(sa) + (col & 7) * 2;
            if constexpr (A_MN)
                fa[buf][i] = pair(base + (row * MCH + ((col >> 3) ^ addr::mn_key(row))) * 16,
                                  base + ((row + 4) * MCH + ((col >> 3) ^ addr::mn_key(row))) * 16);
            else
                fa[buf][i] = kc_frag(sa, wm * WT + i * MF, kk);
        }
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int col = wn * WT + j * MF + tr_col;
            const char *base = reinterpret_cast<const char *>(sb) + (col & 7) * 2;
            if constexpr (B_MN)
                fb[buf][j] = pair(base + b_slot(row, col >> 3) * 16, base + b_slot(row + 4, col >> 3) * 16);
            else
                fb[buf][j] = kc_frag(sb, wn * WT + j * MF, kk);
        }
    };

    // The MFMAs of register buffer cb with the other instructions of the k step spread evenly over
    // them: LDS reads, vector-memory loads, VALU and LDS writes.
    auto mfmas = [&](int cb, int vmem, int valu, int dsw) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int jj = 0; jj < NI; ++jj) {
                const int j = (i & 1) ? NI - 1 - jj : jj;
                acc[i][j] = F::mfma(fa[cb][i], fb[cb][j], acc[i][j]);
            }
        auto share = [](int n, int g) { return ((g + 1) * n) / NMFMA - (g * n) / NMFMA; };
#pragma unroll
        for (int g = 0; g < NMFMA; ++g) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t < share(vmem, g)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t < share(NREAD, g)) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
            for (int t = 0; t < 24; ++t)
                if (t < share(valu, g)) __builtin_amdgcn_sched_group_barrier(0x002, 1, 0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t < share(dsw, g)) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int NVALU = FP4 ? 18 : 84;  // of a group's expansion

    // One barrier to the next: the last k step of slab s - 1 (its fragments are in registers), then the
    // first three of slab s, whose parts are `ra` and `rb`. Freed by the barrier: `wa`, which takes the
    // A part of slab s + 2, and `wb`, which takes the B part of slab s + 1. The four halves differ; the
    // restrict qualifiers say so, without which the compiler waits for all DMA under way before each
    // transposing read.
    auto period = [&](int s, const uint4 *ra, const uint4 *rb, uint4 *wa, uint4 *wb, auto first_tag, auto shift_tag) {
        constexpr bool FIRST = decltype(first_tag)::value;  // slab 0: nothing precedes it
        constexpr int SH = decltype(shift_tag)::value;
        if constexpr (!FIRST) {
            read_frags(ra, rb, 0, 0);
            if (SH == 0) window(0, s + 2, wa);
            mfmas(1, SH == 0 ? PER_WIN : 0, 0, 0);
        }
#pragma unroll
        for (int kk = 0; kk + 1 < KSTEPS; ++kk) {
            const int cb = kk & 1;
            wait_lgkmcnt0();  // this step's fragments
            __builtin_amdgcn_sched_barrier(0);
            read_frags(ra, rb, kk + 1, cb ^ 1);
            int vmem = 0, valu = 0, dsw = 0;
            if (kk == 0 && 1 - SH < NWIN) {
                window(1 - SH, s + 2, wa);
                vmem += PER_WIN;
            }
            const int i = kk - (3 - NG);  // the group of this k step
            if (i >= 0 && kk > 0 && i < NG) {
                // younger than the group: A's windows and the slab's other group. (So A of slab
                // s + 1, older than all of them, has landed too.)
                wait_vmcnt<JA + (NG - 1) * LG>();
                __builtin_amdgcn_sched_barrier(0);
                write_group(i, s + 1, wb);
                load_group(i, s + 2);
                vmem += LG;
                valu = NVALU;
                dsw = 4;
            }
            mfmas(cb, vmem, valu, dsw);
        }
        wait_lgkmcnt0();  // the last step's fragments and the writes of slab s + 1
    };

    auto wrap5 = [](int h) { return h >= 5 ? h - 5 : h; };
    // SH: with STAGGER the second half of the waves issues its DMA a k step later
    auto loop = [&](auto shift_tag) {
        constexpr int SH = decltype(shift_tag)::value;
#pragma unroll
        for (int i = 0; i < NG; ++i) load_group(i, 0);
#pragma unroll
        for (int d = 0; d < JA; ++d) dma_a(d, 0, smem);
#pragma unroll
        for (int d = 0; d < JA; ++d) dma_a(d, 1, smem + 2 * HALF);
#pragma unroll
        for (int i = 0; i < NG; ++i) write_group(i, 0, smem + HALF);
#pragma unroll
        for (int i = 0; i < NG; ++i) load_group(i, 1);
        if (SH == 0) window(0, 2, smem + 4 * HALF);
        __builtin_amdgcn_sched_barrier(0);
        // A of slab 0 has landed: only A of slab 1, B's loads after it and the window are younger
        wait_vmcnt<JA + NG * LG + (SH == 0 ? PER_WIN : 0)>();
        wait_lgkmcnt0();
        lds_barrier();
        read_frags(smem, smem + HALF, 0, 0);
        apart(smem, smem + HALF, smem + 4 * HALF, smem + 3 * HALF,
              [&](const uint4 *ra, const uint4 *rb, uint4 *wa, uint4 *wb) { period(0, ra, rb, wa, wb, std::true_type{}, shift_tag); });
        int ha = 0;  // the half of slab s - 1's A part
        for (int s = 1; s < nslabs; ++s) {
            lds_barrier();  // slab s published; slab s - 1's halves read by nobody any more
            ha = wrap5(ha + 2);
            apart(smem + ha * HALF, smem + wrap5(ha + 1) * HALF, smem + wrap5(ha + 4) * HALF, smem + wrap5(ha + 3) * HALF,
                  [&](const uint4 *ra, const uint4 *rb, uint4 *wa, uint4 *wb) { period(s, ra, rb, wa, wb, std::false_type{}, shift_tag); });
        }
        mfmas(1, 0, 0, 0);  // the last k step
    };
    if (STAGGER && wave >= 2)
        loop(std::integral_constant<int, STAGGER ? 1 : 0>{});
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

// C = alpha (sum of the splits' parts, in their order) + beta C; bound by reading the parts
__global__ __launch_bounds__(256) void mx_join_kernel(int splits, int M, int N, float alpha,
                                                      const float *__restrict__ work, float beta,
                                                      float *__restrict__ C, int64_t ldc, int vec) {
    const int64_t n = (int64_t)M * N, per_row = vec ? N / 4 : N, total = vec ? n / 4 : n;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < total; u += (int64_t)gridDim.x * 256) {
        int64_t row, unit;
        if (total < (int64_t(1) << 32)) {
            row = (uint32_t)u / (uint32_t)per_row;
            unit = (uint32_t)u - (uint32_t)row * (uint32_t)per_row;
        } else {
            row = u / per_row;
            unit = u - row * per_row;
        }
        if (vec) {
            const float4 *w = reinterpret_cast<const float4 *>(work) + u;
            float4 v = w[0];
            for (int z = 1; z < splits; ++z) {
                const float4 p = w[z * (n / 4)];
                v.x += p.x;
                v.y += p.y;
                v.z += p.z;
                v.w += p.w;
            }
            float4 *c = reinterpret_cast<float4 *>(C + row * ldc) + unit;
            if (beta == 0.0f) {
                *c = make_float4(alpha * v.x, alpha * v.y, alpha * v.z, alpha * v.w);
            } else {
                const float4 o = *c;
                *c = make_float4(fmaf(alpha, v.x, beta * o.x), fmaf(alpha, v.y, beta * o.y), fmaf(alpha, v.z, beta * o.z),
                                 fmaf(alpha, v.w, beta * o.w));
            }
        } else {
            float v = work[u];
            for (int z = 1; z < splits; ++z) v += work[z * n + u];
            float *c = C + row * ldc + unit;
            *c = epilogue_value(v, alpha, beta, c);
        }
    }
}

// DMA windows a slab and stagger, as in the 16-bit kernel (two windows and no stagger on 256-wide tiles:
// 939 against 912 us at 8192^3 fp4 nt, 287 against 252 at 4096 x 4096 x 8192 nn)
constexpr int MXD_WIN = 1, MXD_STAG = 1, MXD_SWIN = 2, MXD_SSTAG = 0;

template <bool FP4, bool F16, bool A_MN, bool B_MN, bool KTAIL>
hipError_t launch_mxd(const MxProblem &p, hipStream_t s, int t, int splits) {
    const int tiles_m = (p.M + t - 1) / t, tiles_n = (p.N + t - 1) / t;
    const dim3 grid((unsigned)((int64_t)tiles_m * tiles_n * splits));
    const int slabs = (p.K + MXD_BK - 1) / MXD_BK, per = (slabs + splits - 1) / splits;
    const MxParts o = mx_parts(p, splits);
#define REGTILE_MXD(T_, W_, S_)                                                                                    \
    do {                                                                                                           \
        note_launch(reinterpret_cast<const void *>(&mx_dma_kernel<T_, FP4, F16, A_MN, B_MN, KTAIL, W_, S_>), MXD_NT); \
        hipLaunchKernelGGL((mx_dma_kernel<T_, FP4, F16, A_MN, B_MN, KTAIL, W_, S_>), grid, dim3(MXD_NT), 0, s, p.M,   \
                           p.N, p.K, o.alpha, (const uint16_t *)p.A, p.lda, p.Q, p.ldq, p.S, p.lds, o.beta, o.C,    \
                           o.ldc, tiles_m, tiles_n, per, o.stride);                                                \
    } while (0)
    if (t == 256) REGTILE_MXD(256, MXD_WIN, MXD_STAG);
    else REGTILE_MXD(128, MXD_SWIN, MXD_SSTAG);
#undef REGTILE_MXD
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && splits > 1 ? launch_mx_join(p, s, splits) : e;
}
template <bool FP4, bool F16>
hipError_t launch_mxd_order(const MxProblem &p, hipStream_t s, int t, int splits) {
    const bool ktail = p.K % MXD_BK != 0;  // (an M-contiguous A ends with its descriptor)
    if (p.ta) return p.tb ? launch_mxd<FP4, F16, true, false, false>(p, s, t, splits) : launch_mxd<FP4, F16, true, true, false>(p, s, t, splits);
    if (p.tb) return ktail ? launch_mxd<FP4, F16, false, false, true>(p, s, t, splits) : launch_mxd<FP4, F16, false, false, false>(p, s, t, splits);
    return ktail ? launch_mxd<FP4, F16, false, true, true>(p, s, t, splits) : launch_mxd<FP4, F16, false, true, false>(p, s, t, splits);
}

}  // namespace

hipError_t launch_mx_join(const MxProblem &p, hipStream_t s, int splits) {
    const int64_t n = (int64_t)p.M * p.N;
    const int vec = p.N % 4 == 0 && p.ldc % 4 == 0 && aligned16(p.C) && aligned16(p.work);
    const int64_t units = vec ? n / 4 : n, blocks = (units + 255) / 256;
    hipLaunchKernelGGL(mx_join_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, splits, p.M, p.N,
                       p.alpha, (const float *)p.work, p.beta, p.C, p.ldc, vec);
    return hipGetLastError();
}

// How many parts of k: enough to fill the chip (two 128-wide workgroups, or one of the split-K kernel's,
// to a CU), each of at least 512 k, and none where the tiles do that. us by number of parts, fp4 / int8, 128-wide:
// tn 1024 x 1024 x 16384: 1 315, 2 163, 4 88, 8 57, 16 66; nn 1024 x 1024 x 4096: 1 68, 2 40, 4 30, 6 27,
// 8 29, 16 35; nt 1024 x 1024 x 1024: 1 15.7, 2 16.8, 4 18.8.
// Between 33 and 128 tiles of 256x256 with K from 8192 on, those tiles in parts that fill the chip
// (addr::mx_wide_parts) rather than whole 128-wide ones: tn int8 2048 x 4096 x 8192 157 us, 181; 2048 x 2048 x
// 8192 89, 98; tn fp4 1024 x 4096 x 16384 136, 164; nt fp4 1024 x 8192 x 8192 130, 135. (K = 4096: 92, 89 at
// tn int8 2048 x 4096; 32 tiles: 57.6, 55.3 at 1024 x 2048 x 8192.)
static int parts_of(int64_t tiles, int64_t workgroups, int K) {
    const int64_t want = workgroups / tiles, most = K / 512, n = want < most ? want : most;
    return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}

MxPlan mx_plan(const MxProblem &p) {
    if (mx_token_takes(p)) return {MxPlan::TOKEN, 0, 0, 1, 1};
    auto tiles = [&](int64_t t) { return ((p.M + t - 1) / t) * ((p.N + t - 1) / t); };
    MxPlan plan = {MxPlan::MFMA, 0, 0, 1, 1};
    if (mx_splitk_takes(p)) {
        plan = {MxPlan::SPLITK, 64, 64, parts_of(tiles(64), 256, p.K), (p.K + 127) / 128};
    } else if (mx_dma_takes(p)) {
        const bool codes = mx_codes_takes(p);
        plan.kernel = codes ? MxPlan::CODES : MxPlan::DMA;
        plan.slabs = codes ? p.K / 128 : (p.K + MXD_BK - 1) / MXD_BK;
        plan.tile = plan.narrow = addr::dma_tile(p.M, p.N);
        const int wide = addr::mx_wide_parts(p.ta, p.M, p.N, p.K, p.lda);
        if (wide > 1) {
            plan.tile = 256;
            plan.parts = wide;
        } else if (plan.tile == 128 && tiles(128) <= 128) {
            plan.parts = parts_of(tiles(128), 512, p.K);
        }
    }
    // as many as there are when each takes the same number of slabs
    const int per = (plan.slabs + plan.parts - 1) / plan.parts;
    plan.parts = (plan.slabs + per - 1) / per;
    return plan;
}

int mx_fit_parts(const MxProblem &p, const MxPlan &plan) {
    if (plan.parts == 1) return 1;
    const int64_t room = p.work_bytes / ((int64_t)p.M * p.N * 4);
    if (room >= plan.parts) return plan.parts;
    if (room < 2 || plan.tile != plan.narrow) return 1;
    const int per = (plan.slabs + (int)room - 1) / (int)room;
    return (plan.slabs + per - 1) / per;
}

// A meets the 16-bit kernels' DMA conditions in its storage order with 16-byte aligned rows, and B has
// whole groups
bool mx_dma_takes(const MxProblem &p) {
    return addr::mx_dma_takes(p.ta, p.tb, p.M, p.N, p.K, p.lda, p.ldc) && aligned16(p.A);
}

hipError_t launch_mx_dma(const MxProblem &p, const MxPlan &plan, hipStream_t s, const char **name) {
    const int splits = mx_fit_parts(p, plan);
    const int t = splits == plan.parts ? plan.tile : plan.narrow;
#define REGTILE_MXD_NAMES(elt, fmt, t) \
    {{elt "_" fmt "_dma_" t "_nn", elt "_" fmt "_dma_" t "_nt"}, {elt "_" fmt "_dma_" t "_tn", elt "_" fmt "_dma_" t "_tt"}}
#define REGTILE_MXD_SIZES(elt, fmt) {REGTILE_MXD_NAMES(elt, fmt, "256x256x64"), REGTILE_MXD_NAMES(elt, fmt, "128x128x64")}
    static const char *const names[2][2][2][2][2] = {{REGTILE_MXD_SIZES("bf16", "int8"), REGTILE_MXD_SIZES("bf16", "fp4")},
                                                     {REGTILE_MXD_SIZES("f16", "int8"), REGTILE_MXD_SIZES("f16", "fp4")}};
#undef REGTILE_MXD_SIZES
#undef REGTILE_MXD_NAMES
    *name = names[p.f16][p.fp4][t == 128][p.ta][p.tb];
    if (p.fp4) return p.f16 ? launch_mxd_order<true, true>(p, s, t, splits) : launch_mxd_order<true, false>(p, s, t, splits);
    return p.f16 ? launch_mxd_order<false, true>(p, s, t, splits) : launch_mxd_order<false, false>(p, s, t, splits);
}

}  // namespace regtile

// gemm_f8_tile.h -- C = alpha A B + beta C for block-scaled 8-bit floats on LDS tiles fed by DMA: a row-major A
// (rows may be gathered), B stored N x K or K x N, dense or in groups.
//
// A stage in LDS is one block of 128 k: BM + BN rows of 128 codes and as many scales. While one is
// multiplied the next STAGES - 1 are on their way, and one barrier a block hands over. Two stages let two workgroups of
// 128 x 128 share a CU; with too few tiles for that, three and four hide the latency of memory better. A block's products are summed from
// zero by the matrix instructions and enter the fp32 accumulators as c += (sa sb) sum, so the scales cost a
// vector instruction for each of a lane's sums (two where B has a scale for each column), and the other wave
// of the SIMD keeps the matrix pipe busy meanwhile. B's fragment is the first operand: a lane holds 4
// consecutive columns of one row of C, and needs one scale of A.
//
// EXACT: sums of exact products, four 16x16x32 bf16 MFMAs on codes expanded in registers; else one
// 16x16x128 8-bit MFMA at twice the rate (f8_common.h has what that loses).
//
// LDS (tile_addressing.h has the layouts): K-contiguous rows of 128 codes, of which a lane reads chunks g and 4 + g (g =
// lane / 16), for both operands the same k. A K x N operand keeps its storage: rows of BN codes at one k, read by
// transposing reads (8 k of 16 columns for 16 lanes).
//
// What bounds it: 8192^3 of e4m3 into bf16 takes 418-429 us (2560-2630 TFLOP/s; the library's product with one scale a matrix
// 377): the matrix pipes are busy 62% of the time, at 1.85 GHz, and the rest is the sums' 4 vector instructions a tile, LDS reads
// of fragments and the last store of each round of tiles. With an fp32 C 880-955 us: expanding codes takes as many issue
// slots as the bf16 MFMAs. Few columns of k a tile (2048) add what a tile costs at its ends, 7 us.
//
// Edges: rows past the last are not loaded and are zeros, chunks past N come from the last one that holds an element. What
// lies past K in the last block (bytes between rows, or zeros from behind the descriptor) is overwritten with
// zeros in LDS, in both operands: a code there may be a NaN.
#pragma once

#include <type_traits>

#include "f8_common.h"

namespace regtile {
namespace f8 {
using namespace mfma;
typedef float __attribute__((may_alias)) f32_any;  // as lds_read16: no wait for DMA
typedef uint32_t __attribute__((ext_vector_type(2), may_alias)) u32x2_any;

// Transposing LDS read of 8-bit elements (ds_read_b64_tr_b8): in each group of 16 lanes, lane 2 j + h gives the
// address of 8 bytes at columns 8 h .. 8 h + 7 of row j, and lane i receives column i of rows 0 .. 7 (measured).
__device__ __forceinline__ u32x2 lds_read_tr8(const void *lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef int v2i32 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) v2i32 *)lds));
#else
    (void)lds;
    return u32x2{};
#endif
}

// Two stages that the compiler knows to be apart: without it, it waits for all DMA under way before each
// transposing read.
template <typename F>
__device__ __forceinline__ void apart(const uint8_t *__restrict__ cur, uint8_t *__restrict__ next, F f) {
    f(cur, next);
}

// WM x WN waves of MI x NI fragments of 16 x 16. TA: A's type (B is e4m3). NN: B stored K x N. SB: B has a scale
// for each column, else one for 128.
template <int WM, int WN, int MI, int NI, int STAGES, bool EXACT, int TA, bool NN, bool SB>
__global__ __launch_bounds__(64 * WM * WN, 2) void f8_tile_kernel(F8Problem p, int tiles_m, int tiles_n, int group_m,
                                                                      int per_split, bool wide, bool lines) {
    constexpr int WAVES = WM * WN, NT = 64 * WAVES, BM = WM * MI * 16, BN = WN * NI * 16;
    constexpr int JA = BM / 8 / WAVES, JB = BN / 8 / WAVES;       // DMA instructions of a wave
    constexpr int SC = (BM + BN) / 64;                            // waves' worth of scales
    constexpr int STAGE = (BM + BN) * BLOCK + (SC > WAVES ? SC : WAVES) * 256;
    static_assert(JA * 8 * WAVES == BM && JB * 8 * WAVES == BN && SC <= WAVES && NI * 16 <= BLOCK, "whole instructions");
    __shared__ __align__(16) uint8_t smem[STAGES * STAGE];

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave / WN, wn = wave % WN;
    int tm, tn;
    // (of rows in groups only the device knows how many tiles there are; without the count the last XCDs would get all
    // the workgroups that have none)
    if (p.mode == F8Problem::ROWS) tiles_m = min(tiles_m, row_tiles(p.offsets, p.counts, p.experts, p.M, BM));
    const int tiles = tiles_m * tiles_n, count = p.mode == F8Problem::ROWS ? tiles : gridDim.x;
    if ((int)blockIdx.x >= count) return;
    const int id = contiguous_id(blockIdx.x, count);
    const int split = id / tiles;  // part of k, per_split blocks
    {  // group_m tile rows at a time, column by column
        const int at = id - split * tiles, group = at / (group_m * tiles_n), row = group * group_m;
        const int rows = min(tiles_m - row, group_m), in_group = at - group * group_m * tiles_n;
        tm = row + in_group % rows;
        tn = in_group / rows;
    }
    Work w;
    if (!work_of(p, BM, tm, blockIdx.y, w)) return;
    // (the same in every lane; where it comes from memory or a division it would stay in vector registers, and an offset
    // in one costs a loop at each DMA)
    auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
    w.used = uniform(w.used);
    w.row0 = uniform(w.row0);
    const int n0 = uniform(tn * BN);
    const int K = uniform(w.used > 0 ? w.K : 0), all = (K + BLOCK - 1) / BLOCK;
    const int first = uniform(split * per_split), blocks = min(per_split, all - first);
    if (count > tiles) w.out.C = static_cast<float *>(w.out.C) + (int64_t)split * p.M * p.N;

    f32x4 acc[MI][NI] = {};
    if (blocks > 0) {
        // ---- DMA ----
        // Descriptors begin at the tile's first row (where rows are gathered: at A) and end behind the last chunk
        // that holds an element; chunks past it arrive as zeros. Lanes hold offsets, the block's is uniform.
        const bool gather = p.slots != nullptr;
        const int n_rows = min(BN, p.N - n0);
        const rsrc_t a_rsrc = make_rsrc(gather ? w.a.q : w.a.q + (int64_t)w.row0 * w.a.row,
                                        addr::f8_span(gather ? p.a_rows : w.used, w.a.row, K));
        const rsrc_t b_rsrc = NN ? make_rsrc(w.b.q + n0, addr::f8_span(K, w.b.step, p.N - n0))
                                 : make_rsrc(w.b.q + (int64_t)n0 * w.b.row, addr::f8_span(n_rows, w.b.row, K));
        uint32_t av[JA], bv[JB];
#pragma unroll
        for (int j = 0; j < JA; ++j) {
            const int q = wave * JA + j, at = min(addr::f8_row(q, lane), w.used - 1);
            av[j] = addr::f8_row_lane(q, lane, w.used, gather ? a_row(p, w, at) : at, w.a.row);
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int q = wave * JB + j;
            if constexpr (NN)
                bv[j] = addr::f8_nn_lane<BN>(q, lane, n_rows, w.b.step);
            else
                bv[j] = addr::f8_row_lane(q, lane, n_rows, addr::f8_row(q, lane), w.b.row);
        }
        // scales: a wave brings 64 rows' of A or 64 columns' of B
        static_assert(BM % 64 == 0, "a wave's scales are all of one operand");
        const bool sa_wave = wave * 64 < BM || wave >= SC;
        const int si = sa_wave ? min((wave < SC ? wave * 64 : 0) + lane, w.used - 1) : min(n0 + wave * 64 - BM + lane, p.N - 1);
        const uint32_t sv = sa_wave ? addr::f8_scale_lane(a_row(p, w, si) >> w.a.shift, w.a.s_row)
                                    : addr::f8_scale_lane(si >> w.b.shift, w.b.s_row);
        const int s_step = uniform(addr::f8_scale_step(sa_wave ? w.a.s_col : w.b.s_col));
        const rsrc_t s_rsrc = make_rsrc(sa_wave ? w.a.s : w.b.s, 0x7FFFFFFFu);

        constexpr int PIECES = JA + JB + 1;
        // A block's DMA goes out over the first half of the time that a block takes: what leaves last still has half of it to
        // arrive (over the whole of it 8192^3 took 429 us and 4096 tokens x 6 of 64 experts, whose weights come from memory, 358;
        // over half 418 and 350; over a quarter 442 and 353).
        constexpr int SPREAD = 2;
        // instruction n of a block's DMA; past the last block the last again, into the stage that is free then
        auto dma = [&](int n, int block, uint8_t *to) {
            const int kb = first + min(block, blocks - 1);
            if (n < JA)
                dma16_buf(a_rsrc, av[n], addr::f8_block(false, kb, 0), to + (wave * JA + n) * 1024);
            else if (n < JA + JB)
                dma16_buf(b_rsrc, bv[n - JA], addr::f8_block(NN, kb, w.b.step), to + BM * BLOCK + (wave * JB + n - JA) * 1024);
            else
                dma4_buf(s_rsrc, sv, addr::f8_scale_block(kb, s_step), to + (BM + BN) * BLOCK + wave * 256);
        };

        // ---- one block ----
        const int fr = lane & 15, fg = lane >> 4;
        // A lane's place in the first fragment of its wave's rows (columns, factors); the others are at constant distances
        const int key = addr::slab_key<8, 16>(fr), lo = (fg ^ key) * 16, hi = ((fg + 4) ^ key) * 16;
        const int a_at = (wm * MI * 16 + fr) * BLOCK, b_at = BM * BLOCK + (wn * NI * 16 + fr) * BLOCK;
        const int sa_at = (BM + BN) * BLOCK + (wm * MI * 16 + fr) * 4, sb_at = (BM + BN) * BLOCK + (BM + wn * NI * 16) * 4;
        const int tr_row = fg * 16 + (fr >> 1), tr_at = BM * BLOCK + tr_row * BN + (fr & 1) * 8, tr_key = addr::f8_nn_key<BN>(tr_row);
        auto whole = [](u32x4 l, u32x4 h) {
            return i32x8{(int)l[0], (int)l[1], (int)l[2], (int)l[3], (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
        };
        auto column_frag = [&](const uint8_t *s, int j) {
            const uint8_t *at = s + tr_at + ((wn * NI + j) ^ tr_key) * 16;
            u32x2 v[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) v[h] = lds_read_tr8(at + ((h >> 1) * 64 + (h & 1) * 8) * BN);
            return i32x8{(int)v[0][0], (int)v[0][1], (int)v[1][0], (int)v[1][1], (int)v[2][0], (int)v[2][1], (int)v[3][0], (int)v[3][1]};
        };
        // A fragment as the matrix instructions take it: the codes, or expanded
        struct Wide {
            bf16x8 v[4];
        };
        typedef typename std::conditional<EXACT, Wide, i32x8>::type Frag;
        auto frag = [](i32x8 q, auto type) -> Frag {
            if constexpr (EXACT) {
                constexpr int T = decltype(type)::value;
                return Wide{{bf16_of8<T>(q[0], q[1]), bf16_of8<T>(q[2], q[3]), bf16_of8<T>(q[4], q[5]), bf16_of8<T>(q[6], q[7])}};
            } else {
                return q;
            }
        };
        const std::integral_constant<int, TA> type_a{};
        const std::integral_constant<int, 0> type_b{};

        // Tiles are multiplied in the order of rows and columns of fragments, and each is added to its
        // accumulator LAG tiles later, when its sum has left the matrix pipe. The sums of the last tiles of a
        // block are added in the next one's time, with that block's factors.
        constexpr int LAG = EXACT ? 1 : 2, RING = EXACT ? 2 : 4, TILES = MI * NI;
        static_assert(TILES % RING == 0 && MI % 2 == 0 && NI >= LAG, "a tile has one slot of the ring, a row one of two factors");
        f32x4 d[RING] = {};
        i32x8 qa[2], qb[NI];  // codes that have been read: of the next two rows (row i in qa[i % 2]), of the next block's columns
        Frag a, b[NI];
        float fa[2] = {0.0f, 0.0f}, sb_all;  // row i's factor in fa[i % 2]; sb_all: of the block that is read, sb: of the one that is added
        // (with two rows of fragments a block's rows are all multiplied in the next one's time, when its stage is gone: its
        // columns' factors wait in sb_in)
        constexpr bool TWO = MI == 2;
        f32x4 sb[SB ? NI : 1] = {}, sb_in[SB && TWO ? NI : 1];
        float sa_next[2];
        auto read_a = [&](const uint8_t *s, int i) {
            qa[i & 1] = whole(lds_read16(s + a_at + lo + i * 16 * BLOCK), lds_read16(s + a_at + hi + i * 16 * BLOCK));
            sa_next[i & 1] = *reinterpret_cast<const f32_any *>(s + sa_at + i * 64);
        };
        auto read_b = [&](const uint8_t *s, int j) {
            if constexpr (NN)
                qb[j] = column_frag(s, j);
            else
                qb[j] = whole(lds_read16(s + b_at + lo + j * 16 * BLOCK), lds_read16(s + b_at + hi + j * 16 * BLOCK));
            if (!SB && j == 0) sb_all = *reinterpret_cast<const f32_any *>(s + sb_at);
        };
        auto read_sb = [&](const uint8_t *s) {
#pragma unroll
            for (int j = 0; j < (SB ? NI : 0); ++j)
                (TWO ? sb_in : sb)[j] = __builtin_bit_cast(f32x4, lds_read16(s + sb_at + fg * 16 + j * 64));
        };
        // Tile t of a block is multiplied: its column's fragment and factor are the block's from the first row on
        auto next_columns = [&](int t) {
            if (t < NI) b[t] = frag(qb[t], type_b);
        };
        auto next_factors = [&](int t, const uint8_t *s) {  // behind the last sum of the block before
            if constexpr (SB) {
                if (t != LAG - 1) return;
                if constexpr (TWO) {
#pragma unroll
                    for (int j = 0; j < NI; ++j) sb[j] = sb_in[j];
                } else {
                    read_sb(s);
                }
            }
        };
        auto add = [&](int t) {  // tile t of a block's
            const int i = t / NI, j = t % NI;
            const f32x4 &v = d[t % RING];
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(v[e], SB ? fa[i & 1] * sb[j][e] : fa[i & 1], acc[i][j][e]);
        };
        auto tile = [&](int t) {
            const int j = t % NI;
            f32x4 &v = d[t % RING];
            v = f32x4{};
            if constexpr (EXACT) {
#pragma unroll
                for (int q = 0; q < 4; ++q) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j].v[q], a.v[q], v, 0, 0, 0);
            } else {
                v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a, v, 0, TA, 0, 0, 0, 0);
            }
        };
        // Row `id / NI` begins: its fragment and its factor have been read
        auto begin_row = [&](int i) {
            a = frag(qa[i & 1], type_a);
            fa[i & 1] = SB ? sa_next[i & 1] : sa_next[i & 1] * sb_all;
        };
        // Between two barriers: the last two rows of fragments of block t - 1 (they are in registers), while block t's
        // first are read from `cur`, then all rows of block t but the last two. Rows are read two ahead. The other
        // stage, `next`, takes block t + STAGES - 1.
        auto period = [&](int t, const uint8_t *cur, uint8_t *next, auto first_tag) {
            constexpr bool FIRST = decltype(first_tag)::value;
            constexpr int START = FIRST ? 2 * NI : 0;
            if constexpr (FIRST) {
#pragma unroll
                for (int j = 0; j < NI; ++j) read_b(cur, j);
                read_a(cur, 0);
                read_a(cur, 1);
                if constexpr (SB && TWO) read_sb(cur);
                if constexpr (START == TILES) {
#pragma unroll
                    for (int m = 0; m < PIECES; ++m) dma(m, t + STAGES - 1, next);
                }
            }
#pragma unroll
            for (int n = START; n < TILES; ++n) {
                const int i = n / NI - 2, j = n % NI;  // rows -2 and -1: the last of block t - 1
                const int id = ((i + MI) % MI) * NI + j;
                if (j == 0) begin_row(id / NI);
                next_columns(id);
                tile(id);
                if constexpr (!EXACT) __builtin_amdgcn_sched_barrier(0);  // (the sum that is added next needs time)
                if (!FIRST || n - LAG >= START) add((id + TILES - LAG) % TILES);
                next_factors(id, cur);
                if (j == 0) read_a(cur, i + 2);
                if (i == -1) read_b(cur, j);
                if (SB && TWO && i == -1 && j == NI - 1) read_sb(cur);
#pragma unroll
                for (int m = 0; m < PIECES; ++m)
                    if (m * (TILES - START) / (SPREAD * PIECES) + START == n) dma(m, t + STAGES - 1, next);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        // zeros past K in the stage of the last block
        auto clear = [&](uint8_t *s, int left) {
            for (int c = tid; c < (NN ? BM : BM + BN) * 8; c += NT) {
                const int r = c >> 3, kk = (c & 7) * 16;
                if (kk + 16 <= left) continue;
                u32x4 *at = reinterpret_cast<u32x4 *>(s + r * BLOCK + ((c & 7) ^ addr::slab_key<8, 16>(r)) * 16);
                u32x4 v = *at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int bytes = min(max(left - kk - 4 * i, 0), 4);
                    v[i] &= bytes == 4 ? ~0u : (1u << 8 * bytes) - 1;
                }
                *at = v;
            }
            wait_lgkmcnt0();
            lds_barrier();
        };

#pragma unroll
        for (int t = 0; t < STAGES - 1; ++t)
#pragma unroll
            for (int n = 0; n < PIECES; ++n) dma(n, t, smem + t * STAGE);
        auto arrive = [&](int t, uint8_t *cur) {
            wait_vmcnt<(STAGES - 2) * PIECES>();  // block t's DMA (of this wave) has landed, STAGES - 2 blocks are younger,
            wait_lgkmcnt0();                      // and the last rows of the block before have been read:
            lds_barrier();                        // of every wave
            const int left = K - (first + t) * BLOCK;
            if (left < BLOCK) clear(cur, left);
        };
        // A wave whose rows or columns are all past the tile's last only brings its part of each block: its SIMD's matrix
        // pipe is then the other wave's alone, and a half-filled tile takes little more than half the time.
        const bool idle = uniform(wm * MI * 16 >= w.used || n0 + wn * NI * 16 >= p.N);
        if (idle) {
            for (int t = 0; t < blocks; ++t) {
                arrive(t, smem + (t % STAGES) * STAGE);
#pragma unroll
                for (int n = 0; n < PIECES; ++n) dma(n, t + STAGES - 1, smem + ((t + STAGES - 1) % STAGES) * STAGE);
            }
        } else {
            arrive(0, smem);
            apart(smem, smem + (STAGES - 1) * STAGE, [&](const uint8_t *c, uint8_t *n) { period(0, c, n, std::true_type{}); });
            for (int t = 1; t < blocks; ++t) {
                uint8_t *cur = smem + (t % STAGES) * STAGE, *next = smem + ((t - 1) % STAGES) * STAGE;
                arrive(t, cur);
                apart(cur, next, [&](const uint8_t *c, uint8_t *n) { period(t, c, n, std::false_type{}); });
            }
            // the last two rows of the last block
#pragma unroll
            for (int n = 0; n < 2 * NI + LAG; ++n) {
                const int id = (MI - 2) * NI + n;
                if (n < 2 * NI && n % NI == 0) begin_row(id / NI);
                if (n < 2 * NI) {
                    if (TWO) next_columns(id);
                    tile(id);
                }
                add((id + TILES - LAG) % TILES);
                if (TWO && n < 2 * NI) next_factors(id, smem);
            }
        }
        wait_vmcnt<0>();  // no LDS DMA may still be in flight when the workgroup retires
    }

    // ---- epilogue ----
    // `lines`: each wave turns its part of C through LDS and stores 128 bytes of a row at a time, at any alignment (from the
    // accumulators 32 bytes of an aligned row leave in one instruction, 2 of another, and 8192^3 took 450 us instead of 429,
    // 8191 x 8190 x 8192 490 instead of 426)
    if constexpr (!EXACT && NI == 4) {
        if (lines) {
            lds_barrier();  // every wave's DMA has landed and every wave has read its last fragments
            uint8_t *mine = smem + wave * (MI * 16 * 128);
            const bool bf = w.out.dtype == 1;
            auto bits = [&](float x) { return bf ? __builtin_bit_cast(uint16_t, (__bf16)x) : __builtin_bit_cast(uint16_t, (_Float16)x); };
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int r = i * 16 + (lane & 15);
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    f32x4 v = acc[i][j] * p.alpha;
                    if (wm * MI * 16 + r >= w.used) v = f32x4{};
                    *reinterpret_cast<u32x2_any *>(mine + r * 128 + ((j * 2 + (lane >> 5)) ^ (r & 7)) * 16 + (lane >> 4 & 1) * 8) =
                        u32x2_any{bits(v[0]) | (uint32_t)bits(v[1]) << 16, bits(v[2]) | (uint32_t)bits(v[3]) << 16};
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int chunk = lane & 7, c = n0 + wn * 64 + chunk * 8;
#pragma unroll
            for (int i = 0; i < MI * 2; ++i) {
                const int at = i * 8 + (lane >> 3), r = wm * MI * 16 + at;
                const u32x4 v = lds_read16(mine + at * 128 + (chunk ^ (at & 7)) * 16);
                if (r >= w.rows) continue;
                uint16_t *to = static_cast<uint16_t *>(w.out.C) + (w.row0 + r) * w.out.ldc + c;
                if (c + 8 <= p.N) {
                    __builtin_memcpy(to, &v, 16);  // (at any address)
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < p.N) to[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                }
            }
            return;
        }
    }
    const int row0 = wm * MI * 16 + (lane & 15), col0 = wn * NI * 16 + (lane >> 4) * 4;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int r = row0 + i * 16;
        if (r >= w.rows) continue;
        const bool used = r < w.used;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
            const int c = n0 + col0 + j * 16;
            const f32x4 zero = {};
            c_store4(w.out, w.row0 + r, c, min(p.N - c, 4), p.alpha, used ? p.beta : 0.0f, used ? acc[i][j] : zero, wide);
        }
    }
}

template <int WM, int WN, int MI, int NI, int STAGES, bool EXACT, int TA, bool NN, bool SB>
hipError_t launch_tile(const F8Problem &p, hipStream_t s, int splits) {
    constexpr int BM = WM * MI * 16, BN = WN * NI * 16, NT = 64 * WM * WN;
    const int64_t tiles_m = most_row_tiles(p, BM), tiles_n = ((int64_t)p.N + BN - 1) / BN, grid = tiles_m * tiles_n * splits;
    if (grid * NT > 0xFFFFFFFFll || (p.mode == F8Problem::DEPTH && p.experts > 65535)) return hipErrorInvalidConfiguration;
    const int blocks = (p.K + BLOCK - 1) / BLOCK, per = blocks > 0 ? (blocks + splits - 1) / splits : 1;
    // tile rows that share B's panels: 8, in groups as many as a group has on the average (the others have another B)
    int group_m = 8;
    if (p.mode == F8Problem::ROWS) {
        const int64_t mean = ((int64_t)p.mean_rows + BM - 1) / BM;
        group_m = (int)(mean < 1 ? 1 : mean < 8 ? mean : 8);
    }
    F8Problem q = p;
    if (splits > 1) {  // parts of M x N fp32, joined by f8_join
        q.out.C = p.work;
        q.out.ldc = p.N;
        q.out.dtype = 0;
        q.alpha = 1.0f;
        q.beta = 0.0f;
    }
    const bool lines = q.out.dtype != 0 && q.beta == 0.0f;
    auto f = f8_tile_kernel<WM, WN, MI, NI, STAGES, EXACT, TA, NN, SB>;
    note_launch(reinterpret_cast<const void *>(f), NT);
    hipLaunchKernelGGL(f, dim3((unsigned)grid, p.mode == F8Problem::DEPTH ? p.experts : 1), dim3(NT), 0, s, q, (int)tiles_m, (int)tiles_n,
                       group_m, per, c_wide(q), lines);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && splits > 1 ? launch_f8_join(p, s, splits) : e;
}

// A's type, B's storage and B's scales, from a problem that these tiles take
template <int WM, int WN, int MI, int NI, int STAGES, bool EXACT>
hipError_t launch_tile_of(const F8Problem &p, hipStream_t s, int splits) {
    const bool nn = p.b.step != 1, sb = p.b.shift == 0;
    auto go = [&](auto ta) {
        constexpr int TA = decltype(ta)::value;
        if (nn) return launch_tile<WM, WN, MI, NI, STAGES, EXACT, TA, true, false>(p, s, splits);
        if (sb) return launch_tile<WM, WN, MI, NI, STAGES, EXACT, TA, false, true>(p, s, splits);
        return launch_tile<WM, WN, MI, NI, STAGES, EXACT, TA, false, false>(p, s, splits);
    };
    return p.a.type ? go(std::integral_constant<int, 1>{}) : go(std::integral_constant<int, 0>{});
}

}  // namespace f8
}  // namespace regtile

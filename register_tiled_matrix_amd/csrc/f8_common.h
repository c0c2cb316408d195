// f8_common.h -- block-scaled 8-bit float matrices of include/regtile.h on the device: one validated
// problem, conversions of codes, the lookup of a group's tile, and the epilogue that the GEMM kernels
// share.
//
// Codes are OCP e4m3 (S.1111.111 is NaN, no infinities) or e5m2 floats. Every code is exact in bf16, so
// products of bf16 fragments are exact and the sum of a block of 128 is as exact as gemm_bf16's. The
// 8-bit matrix instructions run at twice that rate but align the products of a group of 32 to the largest and
// cut off what falls more than 17 bits below its leading one: 31 2^-17 = 2.4e-4 of the sum of magnitudes at most, and
// sums of positive products come out low. Against 64 bits one block measured (rms, worst) 2.0e-6 and 1.2e-5 for normally distributed codes,
// 3.3e-6 and 1.6e-5 for positive ones, 7.2e-5 and 1.0e-4 for one large product among small ones, 2.4e-5 and 1.8e-4
// for random bits. bf16's half step is 2e-3 of the value and fp16's 2.4e-4: that is where these instructions are used, and a
// 32-bit C, which would lose by them, is made without. 8192^3 into bf16 takes 420 us with them, and an fp32 C 880.
//
// A block's sum enters the accumulators times the fp32 product of its two scales, one instruction. Multiplying by one
// scale after the other would keep the bits of a product below 2^-126, but lose sums past 2^128 instead, and costs an
// instruction for each sum: 8192^3 420 -> 494 us into bf16, 880 -> 962 into fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mfma_common.h"
#include "regtile_internal.h"

namespace regtile {
namespace f8 {

constexpr int BLOCK = 128;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Two codes of a dword (the low half, or the high one) as bf16 values; exact (scale 1).
template <int TYPE, bool HI>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t codes) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (TYPE == 0)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, HI));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, 1.0f, HI));
#else
    (void)codes;
    return 0;
#endif
}
// 8 codes as the bf16 operand of one lane
template <int TYPE>
__device__ __forceinline__ mfma::bf16x8 bf16_of8(uint32_t lo, uint32_t hi) {
    const mfma::u32x4 v = {bf16_pair<TYPE, false>(lo), bf16_pair<TYPE, true>(lo), bf16_pair<TYPE, false>(hi),
                           bf16_pair<TYPE, true>(hi)};
    return __builtin_bit_cast(mfma::bf16x8, v);
}
// Two codes as fp32
template <bool HI>
__device__ __forceinline__ f32x2 f32_pair(int type, uint32_t codes) {
#if defined(__HIP_DEVICE_COMPILE__)
    return type == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, HI) : __builtin_amdgcn_cvt_pk_f32_bf8((int)codes, HI);
#else
    (void)type;
    (void)codes;
    return f32x2{};
#endif
}

// 16 codes at `p`, of which the first `left` belong to the row and the rest become 0; `have` codes of the row lie before p
__device__ __forceinline__ mfma::u32x4 load16(const uint8_t *p, int left, int have) {
    mfma::u32x4 v = {};
    if (left >= 16) {
        __builtin_memcpy(&v, p, 16);
    } else if (left > 0) {
        if (have + left >= 16) {  // the 16 that end where the row ends, moved down
            uint64_t lo, hi;
            __builtin_memcpy(&lo, p + left - 16, 8);
            __builtin_memcpy(&hi, p + left - 8, 8);
            const int s = 8 * (16 - left);
            if (s >= 64) {
                lo = hi >> (s - 64);
                hi = 0;
            } else {
                lo = lo >> s | hi << (64 - s);
                hi >>= s;
            }
            v = mfma::u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (i < left) v[i / 4] |= (uint32_t)p[i] << (8 * (i & 3));
        }
    }
    return v;
}

// Where a group of `rows` begins, its used rows and its room, kept inside the matrix whatever the arrays hold.
struct Group {
    int first, count, room;
};
__device__ __forceinline__ Group group_of(const int32_t *offsets, const int32_t *counts, int e, int rows) {
    Group g;
    g.first = min(max(offsets[e], 0), rows);
    g.room = min(max(offsets[e + 1], g.first), rows) - g.first;
    g.count = min(max(counts[e], 0), g.room);
    return g;
}

// Workgroups take the XCDs in turn: each XCD's get consecutive tiles, of any `count`
__device__ __forceinline__ int contiguous_id(int block, int count) {
    const int xcd = block & 7, each = count >> 3, more = count & 7;
    return xcd * each + min(xcd, more) + (block >> 3);
}

// How many row tiles of `height` rows the groups have (each begins one)
__device__ __forceinline__ int row_tiles(const int32_t *offsets, const int32_t *counts, int experts, int rows, int height) {
    int n = 0;
    for (int e = __lane_id(); e < experts; e += 64) n += (group_of(offsets, counts, e, rows).room + height - 1) / height;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
    return __builtin_amdgcn_readfirstlane(n);
}

// The group that row tile `tile` (of `height` rows; groups begin a tile each) belongs to and the tile's
// number in it; false past the last. Every lane of the wave gets the same answer: 64 groups are loaded and counted
// at a time, and the one that is wanted comes out of its lane's registers.
__device__ __forceinline__ bool find_tile(const int32_t *offsets, const int32_t *counts, int experts, int rows, int height, int tile,
                                          int &expert, int &in_group, Group &group) {
    const int lane = __lane_id();
    int before = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        Group g = {0, 0, 0};
        if (e < experts) g = group_of(offsets, counts, e, rows);
        const int n = (g.room + height - 1) / height;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(upto, d);
            if (lane >= d) upto += v;
        }
        const uint64_t past = __ballot(before + upto > tile);
        if (past != 0) {
            const int l = __ffsll((unsigned long long)past) - 1;
            auto of = [&](int x) { return __builtin_amdgcn_readlane(x, l); };
            expert = __builtin_amdgcn_readfirstlane(e0 + l);
            in_group = __builtin_amdgcn_readfirstlane(tile - before - of(upto - n));
            group = Group{of(g.first), of(g.count), of(g.room)};
            return true;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// What one workgroup computes: rows row0 .. row0 + rows - 1 of C (the tile's), of which the first `used` come
// from A and the rest are zeros, over K values of depth.
struct Work {
    int row0, rows, used, K;
    F8Operand a, b;
    F8Out out;
};
// Row tile `tile` of `height` rows (DEPTH: of group `part`); false where there is none.
__device__ __forceinline__ bool work_of(const F8Problem &p, int height, int tile, int part, Work &w) {
    w.a = p.a;
    w.b = p.b;
    w.out = p.out;
    w.K = p.K;
    if (p.mode == F8Problem::ROWS) {
        int e, in_group;
        Group g;
        if (!find_tile(p.offsets, p.counts, p.experts, p.M, height, tile, e, in_group, g)) return false;
        const int at = in_group * height;
        w.row0 = g.first + at;
        w.rows = min(height, g.room - at);
        w.used = min(max(g.count - at, 0), height);
        w.b.q += e * p.b_stack;
        w.b.s += e * p.bs_stack;
        return true;
    }
    w.row0 = tile * height;
    w.rows = w.used = min(height, p.M - w.row0);
    if (p.mode == F8Problem::DEPTH) {
        Group g = group_of(p.offsets, p.counts, part, p.K);
        g.first &= ~(BLOCK - 1);  // (they are multiples of it)
        w.K = min(g.count, p.K - g.first);
        w.a.q += g.first;
        w.b.q += g.first;
        w.a.s += (g.first / BLOCK) * p.a.s_col;
        w.b.s += (g.first / BLOCK) * p.b.s_col;
        w.out.C = static_cast<char *>(w.out.C) + part * p.c_stack * (p.out.dtype == 0 ? 4 : 2);
    }
    return true;
}
// The row of A that row r of the work (0 .. used - 1) is made from
__device__ __forceinline__ int64_t a_row(const F8Problem &p, const Work &w, int r) {
    const int row = w.row0 + r;
    if (p.slots == nullptr) return row;
    return min(max(p.slots[row], 0) / p.top_k, p.a_rows - 1);
}
// Row tiles that ROWS can have at most: a part of one in each group, and what the rows fill
inline int64_t most_row_tiles(const F8Problem &p, int height) {
    if (p.mode != F8Problem::ROWS) return ((int64_t)p.M + height - 1) / height;
    return (int64_t)p.M / height + (p.experts < p.M ? p.experts : p.M);
}

// Whether 4 columns from a multiple of 4 on are one aligned store in every row of every C
inline bool c_wide(const F8Problem &p) {
    const int size = p.out.dtype == 0 ? 4 : 2;
    return (reinterpret_cast<uintptr_t>(p.out.C) % (4 * size)) == 0 && p.out.ldc % 4 == 0 && p.c_stack % 4 == 0;
}

// C elements: 4 consecutive columns of one row, of which the first `count` (at most 4) belong to C. `wide`:
// C's rows are aligned for one store of 4.
__device__ __forceinline__ float c_load(const F8Out &o, int64_t at) {
    if (o.dtype == 0) return static_cast<const float *>(o.C)[at];
    if (o.dtype == 1) return (float)static_cast<const __bf16 *>(o.C)[at];
    return (float)static_cast<const _Float16 *>(o.C)[at];
}
__device__ __forceinline__ void c_store4(const F8Out &o, int64_t row, int col, int count, float alpha, float beta, mfma::f32x4 v,
                                         bool wide) {
    if (count <= 0) return;
    const int64_t at = row * o.ldc + col;
    v *= alpha;
    if (beta != 0.0f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) v[i] = fmaf(beta, c_load(o, at + i), v[i]);
    }
    if (o.dtype == 0) {
        float *c = static_cast<float *>(o.C) + at;
        if (wide && count >= 4) {
            *reinterpret_cast<mfma::f32x4 *>(c) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < count) c[i] = v[i];
        }
        return;
    }
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = o.dtype == 1 ? __builtin_bit_cast(uint16_t, (__bf16)v[i]) : __builtin_bit_cast(uint16_t, (_Float16)v[i]);
    uint16_t *c = static_cast<uint16_t *>(o.C) + at;
    if (wide && count >= 4) {
        *reinterpret_cast<uint2 *>(c) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) c[i] = h[i];
    }
}

}  // namespace f8
}  // namespace regtile

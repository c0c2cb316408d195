// mx_common.h -- the block-scaled (MX) formats of include/regtile.h on the device: sizes of a
// stored row, and the expansion of codes to 16-bit values that the GEMM kernels and the
// dequantising kernel share.
//
// A row of `cols` values holds one scale byte E for each group of 32 columns (the last group may
// be short) and its elements: 4-bit floats (sign, 2 exponent bits, 1 mantissa bit; value
// e2m1 * 2^(E - 127)), two to a byte with the even column in the low half, or 8-bit integers
// (value q * 2^(E - 133), i.e. q / 64 * 2^(E - 127)). E = 255 makes the group NaN.
//
// A power-of-two scale keeps every value at 2 (fp4) or 7 (int8) significant bits, so it is exact in
// bf16 over the whole range of E that stays finite, and in fp16 wherever fp16 reaches: expanding
// rounds nothing, and the products with a 16-bit operand are as exact as in gemm_bf16 / gemm_f16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tile_addressing.h"

namespace regtile {
namespace mx {

constexpr int GROUP = 32;

__host__ __device__ inline int64_t groups(int64_t cols) { return (cols + GROUP - 1) / GROUP; }
__host__ __device__ inline int64_t row_bytes(bool fp4, int64_t cols) { return addr::mx_row_bytes(fp4, cols); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// What the expansion multiplies elements by. fp4: 2^(E - 127) as the exponent field of a float,
// which is all that v_cvt_scalef32_pk_* looks at (field 0 is 2^-127 and field 255 NaN there;
// checked for every scale byte against every code). int8: 2^(E - 133), subnormal below E = 7.
template <bool FP4>
__device__ __forceinline__ float scale_value(uint32_t E) {
    if constexpr (FP4)
        return __builtin_bit_cast(float, E << 23);
    else
        return E == 255 ? __builtin_nanf("") : __builtin_amdgcn_ldexpf(1.0f, (int)E - 133);
}

// 4 codes of one group (fp4: the low or high half of `q`, `HALF` 0 or 1; int8: all of `q`) as four
// 16-bit values. fp4: one conversion with its scale for two values. int8: sign-extending byte to
// float, scaled (both exact), then two floats to a dword: their high halves (bf16) or a
// round-to-nearest conversion (fp16).
template <bool FP4, bool F16, int HALF>
__device__ __forceinline__ uint2 expand4(uint32_t q, float s) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (FP4) {
        if constexpr (F16)
            return make_uint2(
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, 2 * HALF)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, s, 2 * HALF + 1)));
        else
            return make_uint2(
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2 * HALF)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2 * HALF + 1)));
    } else {
        const float a = (float)(int8_t)q * s, b = (float)(int8_t)(q >> 8) * s;
        const float c = (float)(int8_t)(q >> 16) * s, d = (float)(int8_t)(q >> 24) * s;
        if constexpr (F16) {
            const f32x2 ab = {a, b}, cd = {c, d};
            return make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(ab, f16x2)),
                              __builtin_bit_cast(uint32_t, __builtin_convertvector(cd, f16x2)));
        } else {
            return make_uint2(
                __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u),
                __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, d), __builtin_bit_cast(uint32_t, c), 0x07060302u));
        }
    }
#else
    (void)q;
    (void)s;
    return make_uint2(0u, 0u);
#endif
}

// 8 codes of one group as eight 16-bit values (a 16-byte chunk); `q` holds them at dword `w` of
// the group's codes: fp4 reads dword w, int8 dwords 2 w and 2 w + 1.
template <bool FP4, bool F16>
__device__ __forceinline__ uint4 expand8(const uint32_t *q, int w, float s) {
    uint2 lo, hi;
    if constexpr (FP4) {
        lo = expand4<FP4, F16, 0>(q[w], s);
        hi = expand4<FP4, F16, 1>(q[w], s);
    } else {
        lo = expand4<FP4, F16, 0>(q[2 * w], s);
        hi = expand4<FP4, F16, 0>(q[2 * w + 1], s);
    }
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

// NB bytes (a multiple of 4) at any address as dwords. Vector loads on gfx950 take any byte
// address, and the compiler emits the widest ones for this copy.
template <int NB>
__device__ __forceinline__ void load_bytes(const void *p, uint32_t (&out)[NB / 4]) {
    __builtin_memcpy(out, p, NB);
}

// `count` codes (0 .. 8 * NB / BITS) at p into NB bytes, zeros after the last: byte loads, and the
// unused half of an odd fp4 count's last byte cleared.
template <bool FP4, int NB>
__device__ __forceinline__ void load_codes_tail(const uint8_t *p, int count, uint32_t (&out)[NB / 4]) {
#pragma unroll
    for (int i = 0; i < NB / 4; ++i) {
        uint32_t d = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int byte = 4 * i + b;
            if constexpr (FP4) {
                if (2 * byte < count) {
                    uint32_t v = p[byte];
                    if (2 * byte + 1 == count) v &= 15u;
                    d |= v << (8 * b);
                }
            } else {
                if (byte < count) d |= (uint32_t)p[byte] << (8 * b);
            }
        }
        out[i] = d;
    }
}

// A short run at a row's end without byte loads: the NB bytes that end where the row ends are loaded
// instead (the row must have that many), and moved down by the bytes they start too early; zeros
// come in behind.
template <int N>
__device__ __forceinline__ void move_down(uint32_t (&d)[N], int bytes) {
    static_assert(N == 2 || N == 4, "8 or 16 bytes");
    const int s = 8 * bytes;
    uint64_t lo = d[0] | (uint64_t)d[1] << 32, hi = N == 4 ? d[N - 2] | (uint64_t)d[N - 1] << 32 : 0;
    if (s >= 64) {
        lo = hi >> (s - 64);
        hi = 0;
    } else if (s > 0) {
        lo = lo >> s | hi << (64 - s);
        hi >>= s;
    }
    d[0] = (uint32_t)lo;
    d[1] = (uint32_t)(lo >> 32);
    if constexpr (N == 4) {
        d[2] = (uint32_t)hi;
        d[3] = (uint32_t)(hi >> 32);
    }
}

}  // namespace mx
}  // namespace regtile

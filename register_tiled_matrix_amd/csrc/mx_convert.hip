// mx_convert.hip -- matrices to and from the block-scaled (MX) formats of include/regtile.h.
//
// Quantising a group of 32 values x with largest magnitude a: E = floor(log2 a) + 127 - t, with t = 2
// (fp4: its largest element is 1.5 * 2^2) or 0 (int8), clamped to 0 .. 254; elements are
// x * 2^(127 - E) rounded to the nearest e2m1 value (ties to the even code, saturating at 6), or
// x * 2^(133 - E) rounded to the nearest integer (ties to even, saturating at +-127). A group that
// holds a NaN or an infinity gets E = 255 and zero codes: it dequantises to NaN as a whole.
//
// Both directions read and write each byte once and are bound by memory: 8192 x 8192 at 4.7-5.6 TB/s
// (bf16 to int8 39.9 us, back 38.7; to fp4 34.4, back 36.0), the rate of a large copy. Four lanes share a
// group, 8 values each: a 16-bit row is read (written) as 16 bytes a lane, consecutive over the wave, and
// the group's maximum needs two exchanges inside a quad. The arithmetic has to be short to stay below
// that: comparing with the borders of fp4 one by one took 59.7 us where the conversion instruction takes 34.4.
#include "mx_common.h"
#include "regtile_internal.h"

namespace regtile {

namespace {

// element types by regtile_mx_dtype: 0 fp32, 1 bf16, 2 fp16
template <int DT>
__device__ __forceinline__ float to_f32(uint32_t bits) {
    if constexpr (DT == 0) return __builtin_bit_cast(float, bits);
    if constexpr (DT == 1) return __builtin_bit_cast(float, bits << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
}

// 8 consecutive values (count of them real, zeros after) of a row as floats
template <int DT>
__device__ __forceinline__ void load8(const char *p, int count, float (&x)[8]) {
    constexpr int ES = DT == 0 ? 4 : 2;
    if (count >= 8) {
        uint32_t d[2 * ES];
        mx::load_bytes<8 * ES>(p, d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = DT == 0 ? to_f32<0>(d[i]) : to_f32<DT>((i & 1) ? d[i >> 1] >> 16 : d[i >> 1] & 0xFFFFu);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t v = 0;
            if (i < count) {
                if constexpr (DT == 0)
                    v = reinterpret_cast<const uint32_t *>(p)[i];
                else
                    v = reinterpret_cast<const uint16_t *>(p)[i];
            }
            x[i] = to_f32<DT>(v);
        }
    }
}

// The codes of 8 values of a group with scale byte E (finite values). fp4: a conversion of two values
// with their scale, which rounds ties to the even code and saturates. int8: x 2^(133 - E) is exact (or
// far below the first border), and adding 1.5 * 2^23 rounds it to an integer in the low bits, ties to even.
template <bool FP4>
__device__ __forceinline__ void encode8(const float (&x)[8], int E, uint32_t (&q)[2]) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (FP4) {
        const float s = __builtin_bit_cast(float, (uint32_t)E << 23);
        uint32_t d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], s, 0);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, x[2], x[3], s, 1);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, x[4], x[5], s, 2);
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(d, x[6], x[7], s, 3);
        q[1] = 0;
    } else {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(x[i], 133 - E), -127.0f, 127.0f);
            r[i] = __builtin_bit_cast(uint32_t, y + 12582912.0f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the low bytes of four, together
            const uint32_t lo = __builtin_amdgcn_perm(r[4 * h + 1], r[4 * h], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(r[4 * h + 3], r[4 * h + 2], 0x04000C0Cu);
            q[h] = lo | hi;
        }
    }
#else
    (void)x;
    (void)E;
    q[0] = q[1] = 0;
#endif
}

constexpr int CV_NT = 256;

// u / d for u < 2^31 as a product: m = ceil(2^(31 + l) / d) with 2^l >= d > 2^(l - 1) fits 32 bits and
// errs by less than u / 2^31 / d < 1 / d. 64-bit unit indices divide.
struct RowOf {
    uint32_t m, l;
    template <typename IDX>
    __device__ __forceinline__ IDX operator()(IDX u, IDX per_row) const {
        if constexpr (sizeof(IDX) == 8)
            return u / per_row;
        else
            return (IDX)(((uint64_t)u * m) >> (31 + l));
    }
};
RowOf row_of(int64_t per_row) {
    uint32_t l = 0;
    while ((int64_t(1) << l) < per_row) ++l;
    return {(uint32_t)(((uint64_t(1) << (31 + l)) + (uint64_t)per_row - 1) / (uint64_t)per_row), l};
}

template <bool FP4, int DT, typename IDX>
__global__ __launch_bounds__(CV_NT) void mx_quantize_kernel(int rows, int cols, const char *__restrict__ X, int64_t ldx,
                                                            uint8_t *__restrict__ Q, int64_t ldq,
                                                            uint8_t *__restrict__ S, int64_t lds, RowOf row_of_unit) {
    constexpr int ES = DT == 0 ? 4 : 2;
    const IDX per_row = (IDX)mx::groups(cols) * 4, total = per_row * (IDX)rows;
    for (IDX u = (IDX)blockIdx.x * CV_NT + threadIdx.x; u < total; u += (IDX)gridDim.x * CV_NT) {
        const IDX row = row_of_unit(u, per_row);
        const int64_t unit = (int64_t)(u - row * per_row);  // of 8 columns
        const int64_t c0 = unit * 8;
        const int count = (int)(cols - c0 < 8 ? cols - c0 : 8);  // below 1 past the row's end
        float x[8];
        load8<DT>(X + ((int64_t)row * ldx + c0) * ES, count, x);
        // magnitudes as integers: their order is the floats', with infinity and NaN on top
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, x[i]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const int field = (int)(top >> 23);  // floor(log2 a) + 127 (0 for subnormal a)
        const bool bad = field == 255;
        const int E = bad ? 255 : max(field - (FP4 ? 2 : 0), 0);
        uint32_t q[2];
        encode8<FP4>(x, E, q);
        if (bad) q[0] = q[1] = 0;
        uint8_t *qp = Q + (int64_t)row * ldq + (FP4 ? c0 / 2 : c0);
        if (count >= 8) {
            __builtin_memcpy(qp, q, FP4 ? 4 : 8);
        } else {
#pragma unroll
            for (int b = 0; b < (FP4 ? 4 : 8); ++b)
                if ((FP4 ? 2 * b : b) < count) qp[b] = (uint8_t)(q[b >> 2] >> (8 * (b & 3)));
        }
        if ((unit & 3) == 0) S[(int64_t)row * lds + unit / 4] = (uint8_t)E;
    }
}

template <bool FP4, int DT, typename IDX>
__global__ __launch_bounds__(CV_NT) void mx_dequantize_kernel(int rows, int cols, const uint8_t *__restrict__ Q,
                                                              int64_t ldq, const uint8_t *__restrict__ S, int64_t lds,
                                                              char *__restrict__ X, int64_t ldx, RowOf row_of_unit) {
    constexpr int ES = DT == 0 ? 4 : 2;
    const IDX per_row = (IDX)addr::mx_units(cols), total = per_row * (IDX)rows;
    for (IDX u = (IDX)blockIdx.x * CV_NT + threadIdx.x; u < total; u += (IDX)gridDim.x * CV_NT) {
        const IDX row = row_of_unit(u, per_row);
        const int64_t unit = (int64_t)(u - row * per_row);
        const int64_t c0 = unit * 8;
        const int count = (int)(cols - c0 < 8 ? cols - c0 : 8);
        const uint8_t *qp = Q + (int64_t)row * ldq + (FP4 ? c0 / 2 : c0);
        const float s = mx::scale_value<FP4>(S[(int64_t)row * lds + unit / 4]);
        uint32_t q[FP4 ? 1 : 2];
        if (count >= 8)
            mx::load_bytes<FP4 ? 4 : 8>(qp, q);
        else
            mx::load_codes_tail<FP4, FP4 ? 4 : 8>(qp, count, q);
        char *xp = X + ((int64_t)row * ldx + c0) * ES;
        if constexpr (DT != 0) {
            const uint4 v = mx::expand8<FP4, DT == 2>(q, 0, s);
            if (count >= 8) {
                __builtin_memcpy(xp, &v, 16);
            } else {
                const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < count) reinterpret_cast<uint16_t *>(xp)[i] = (uint16_t)(d[i >> 1] >> (16 * (i & 1)));
            }
        } else {
            // bf16 holds every value exactly, so fp32 is its expansion with 16 zero bits
            const uint4 v = mx::expand8<FP4, false>(q, 0, s);
            const uint32_t d[4] = {v.x, v.y, v.z, v.w};
            uint32_t f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (i & 1) ? d[i >> 1] & 0xFFFF0000u : d[i >> 1] << 16;
            if (count >= 8) {
                __builtin_memcpy(xp, f, 32);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < count) reinterpret_cast<uint32_t *>(xp)[i] = f[i];
            }
        }
    }
}

unsigned cv_blocks(int64_t units) {
    const int64_t b = (units + CV_NT - 1) / CV_NT;
    return (unsigned)(b < (1 << 22) ? b : (1 << 22));  // the kernels stride over the rest
}

template <bool FP4, int DT>
hipError_t quantize_cfg(const MxConvert &p, hipStream_t s) {
    const int64_t units = mx::groups(p.cols) * 4 * p.rows;
    const RowOf r = row_of(mx::groups(p.cols) * 4);
#define REGTILE_MX_Q(IDX_)                                                                                          \
    do {                                                                                                            \
        note_launch(reinterpret_cast<const void *>(&mx_quantize_kernel<FP4, DT, IDX_>), CV_NT);                      \
        hipLaunchKernelGGL((mx_quantize_kernel<FP4, DT, IDX_>), dim3(cv_blocks(units)), dim3(CV_NT), 0, s, p.rows,   \
                           p.cols, (const char *)p.X, p.ldx, p.Q, p.ldq, p.S, p.lds, r);                            \
    } while (0)
    // 32-bit unit indices leave room for one more stride past the last
    if (units < (int64_t(1) << 31)) REGTILE_MX_Q(uint32_t);
    else REGTILE_MX_Q(uint64_t);
#undef REGTILE_MX_Q
    return hipGetLastError();
}

template <bool FP4, int DT>
hipError_t dequantize_cfg(const MxConvert &p, hipStream_t s) {
    const int64_t units = addr::mx_units(p.cols) * p.rows;
    const RowOf r = row_of(addr::mx_units(p.cols));
#define REGTILE_MX_D(IDX_)                                                                                          \
    do {                                                                                                            \
        note_launch(reinterpret_cast<const void *>(&mx_dequantize_kernel<FP4, DT, IDX_>), CV_NT);                    \
        hipLaunchKernelGGL((mx_dequantize_kernel<FP4, DT, IDX_>), dim3(cv_blocks(units)), dim3(CV_NT), 0, s, p.rows, \
                           p.cols, p.Q, p.ldq, p.S, p.lds, (char *)p.X, p.ldx, r);                                  \
    } while (0)
    if (units < (int64_t(1) << 31)) REGTILE_MX_D(uint32_t);
    else REGTILE_MX_D(uint64_t);
#undef REGTILE_MX_D
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxConvert &p, hipStream_t s, const char **name) {
    static const char *const names[2][3] = {{"mx_quantize_int8_f32", "mx_quantize_int8_bf16", "mx_quantize_int8_f16"},
                                            {"mx_quantize_fp4_f32", "mx_quantize_fp4_bf16", "mx_quantize_fp4_f16"}};
    *name = names[p.fp4][p.dtype];
    if (p.fp4)
        return p.dtype == 0 ? quantize_cfg<true, 0>(p, s) : p.dtype == 1 ? quantize_cfg<true, 1>(p, s) : quantize_cfg<true, 2>(p, s);
    return p.dtype == 0 ? quantize_cfg<false, 0>(p, s) : p.dtype == 1 ? quantize_cfg<false, 1>(p, s) : quantize_cfg<false, 2>(p, s);
}

hipError_t launch_mx_dequantize(const MxConvert &p, hipStream_t s, const char **name) {
    static const char *const names[2][3] = {{"mx_dequantize_int8_f32", "mx_dequantize_int8_bf16", "mx_dequantize_int8_f16"},
                                            {"mx_dequantize_fp4_f32", "mx_dequantize_fp4_bf16", "mx_dequantize_fp4_f16"}};
    *name = names[p.fp4][p.dtype];
    if (p.fp4)
        return p.dtype == 0 ? dequantize_cfg<true, 0>(p, s) : p.dtype == 1 ? dequantize_cfg<true, 1>(p, s) : dequantize_cfg<true, 2>(p, s);
    return p.dtype == 0 ? dequantize_cfg<false, 0>(p, s) : p.dtype == 1 ? dequantize_cfg<false, 1>(p, s) : dequantize_cfg<false, 2>(p, s);
}

}  // namespace regtile

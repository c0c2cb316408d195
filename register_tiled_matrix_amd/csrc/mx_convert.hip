// mx_convert.hip -- matrices to and from the block-scaled (MX) formats of include/regtile.h.
//
// Quantising a group of 32 values x with largest magnitude a: E = floor(log2 a) + 127 - t, with t = 2
// (fp4: its largest element is 1.5 * 2^2) or 0 (int8), clamped to 0 .. 254; elements are
// x * 2^(127 - E) rounded to the nearest e2m1 value (ties to the even code, saturating at 6), or
// x * 2^(133 - E) rounded to the nearest integer (ties to even, saturating at +-127). A group that
// holds a NaN or an infinity gets E = 255 and zero codes: it dequantises to NaN as a whole.
//
// Both directions read and write each byte once and are bound by memory. Four lanes share a group, 8
// values each: a 16-bit row is read (written) as 16 bytes a lane, consecutive over the wave, and the
// group's maximum needs two exchanges inside a quad.
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

// the e2m1 code of y (|y| < 8 in use): the borders between 0 .5 1 1.5 2 3 4 6, a tie going to the
// even code
__device__ __forceinline__ uint32_t fp4_code(float y) {
    const float a = fabsf(y);
    const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.0f);
    return c | ((__builtin_bit_cast(uint32_t, y) >> 31) << 3);
}

constexpr int CV_NT = 256;

template <bool FP4, int DT, typename IDX>
__global__ __launch_bounds__(CV_NT) void mx_quantize_kernel(int rows, int cols, const char *__restrict__ X, int64_t ldx,
                                                            uint8_t *__restrict__ Q, int64_t ldq,
                                                            uint8_t *__restrict__ S, int64_t lds) {
    constexpr int ES = DT == 0 ? 4 : 2;
    const IDX per_row = (IDX)mx::groups(cols) * 4, total = per_row * (IDX)rows;
    for (IDX u = (IDX)blockIdx.x * CV_NT + threadIdx.x; u < total; u += (IDX)gridDim.x * CV_NT) {
        const IDX row = u / per_row;
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
        uint32_t q[2] = {0, 0};
        if (!bad) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // exact: a power of two, and nothing below the first bit kept comes near a border
                // of the rounding from the subnormals that ldexp could round to
                const float y = __builtin_amdgcn_ldexpf(x[i], (FP4 ? 127 : 133) - E);
                if constexpr (FP4) {
                    q[0] |= fp4_code(y) << (4 * i);
                } else {
                    const int r = (int)fminf(fmaxf(rintf(y), -127.0f), 127.0f);
                    q[i >> 2] |= ((uint32_t)r & 255u) << (8 * (i & 3));
                }
            }
        }
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
                                                              char *__restrict__ X, int64_t ldx) {
    constexpr int ES = DT == 0 ? 4 : 2;
    const IDX per_row = (IDX)((cols + 7) / 8), total = per_row * (IDX)rows;
    for (IDX u = (IDX)blockIdx.x * CV_NT + threadIdx.x; u < total; u += (IDX)gridDim.x * CV_NT) {
        const IDX row = u / per_row;
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
#define REGTILE_MX_Q(IDX_)                                                                                          \
    do {                                                                                                            \
        note_launch(reinterpret_cast<const void *>(&mx_quantize_kernel<FP4, DT, IDX_>), CV_NT);                      \
        hipLaunchKernelGGL((mx_quantize_kernel<FP4, DT, IDX_>), dim3(cv_blocks(units)), dim3(CV_NT), 0, s, p.rows,   \
                           p.cols, (const char *)p.X, p.ldx, p.Q, p.ldq, p.S, p.lds);                               \
    } while (0)
    // 32-bit unit indices leave room for one more stride past the last
    if (units < (int64_t(1) << 31)) REGTILE_MX_Q(uint32_t);
    else REGTILE_MX_Q(uint64_t);
#undef REGTILE_MX_Q
    return hipGetLastError();
}

template <bool FP4, int DT>
hipError_t dequantize_cfg(const MxConvert &p, hipStream_t s) {
    const int64_t units = ((int64_t)p.cols + 7) / 8 * p.rows;
#define REGTILE_MX_D(IDX_)                                                                                          \
    do {                                                                                                            \
        note_launch(reinterpret_cast<const void *>(&mx_dequantize_kernel<FP4, DT, IDX_>), CV_NT);                    \
        hipLaunchKernelGGL((mx_dequantize_kernel<FP4, DT, IDX_>), dim3(cv_blocks(units)), dim3(CV_NT), 0, s, p.rows, \
                           p.cols, p.Q, p.ldq, p.S, p.lds, (char *)p.X, p.ldx);                                     \
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

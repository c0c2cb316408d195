// f8_convert.hip -- regtile_quantize_f8 and regtile_dequantize_f8: to and from 8-bit floats with one fp32
// scale for each block of 1 x 128 or 128 x 128.
//
// A block with largest magnitude a gets s = max(a * (1 / top), 2^-126), top the type's largest value (1 / top
// and the product rounded to fp32), and its codes are the nearest to x / s, ties to even. The quotient is wanted
// to be right at the borders between codes, and an IEEE division costs 10 instructions and more a value. So x is
// multiplied by two numbers just below and just above 1 / s: the quotient lies between the products, and where both
// have the same code it is the quotient's. Where they differ a border lies between them or on the quotient (of 16-bit
// values one in 500 is a tie), and the value takes the long way: q = x r, one correction, which leaves q within a unit
// of its last place, and the sign of the exact remainder x - q s: where it is not 0 and q's last bit is even, q moves one
// unit towards it. An odd q is no border (those end in zeros), and it is on the quotient's side of any.
//
// Bound by memory: rows, 16 lanes a block, 8 values a lane; columns (transpose), a tile of 128 rows x 64
// columns through LDS, so that both sides move whole lines. 8192 x 8192 bf16: 51-53 us to codes and 33-35 back, where a copy of
// the same bytes takes 38 each way (the second finds part of them in the cache); the exact way's instructions are the rest.
#include "f8_common.h"

namespace regtile {
namespace {
using namespace f8;
using mfma::u32x4;

constexpr int NT = 256;
__host__ __device__ constexpr float inv_top_of(int type) { return type == 0 ? 1.0f / 448.0f : 1.0f / 57344.0f; }

template <int DT>
struct Elem;
template <>
struct Elem<0> {
    typedef float T;
};
template <>
struct Elem<1> {
    typedef __bf16 T;
};
template <>
struct Elem<2> {
    typedef _Float16 T;
};

// 8 values from p on, of which `count` are there (the others are 0); `wide`: p is 16-byte aligned
template <int DT>
__device__ __forceinline__ void load8(const void *row, int64_t col, int count, bool wide, float (&x)[8]) {
    typedef typename Elem<DT>::T T;
    const T *p = static_cast<const T *>(row) + col;
    if (count >= 8 && wide) {
        T t[8];
        if constexpr (DT == 0) {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(p), b = *reinterpret_cast<const u32x4 *>(p + 4);
            __builtin_memcpy(t, &a, 16);
            __builtin_memcpy(reinterpret_cast<char *>(t) + 16, &b, 16);
        } else {
            const u32x4 a = *reinterpret_cast<const u32x4 *>(p);
            __builtin_memcpy(t, &a, 16);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)t[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = i < count ? (float)p[i] : 0.0f;
    }
}
template <int DT>
__device__ __forceinline__ void store8(void *row, int64_t col, int count, bool wide, const float (&x)[8]) {
    typedef typename Elem<DT>::T T;
    T *p = static_cast<T *>(row) + col;
    if (count >= 8 && wide) {
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = (T)x[i];
        u32x4 a;
        __builtin_memcpy(&a, t, 16);
        *reinterpret_cast<u32x4 *>(p) = a;
        if constexpr (DT == 0) {
            __builtin_memcpy(&a, reinterpret_cast<char *>(t) + 16, 16);
            *reinterpret_cast<u32x4 *>(p + 4) = a;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) p[i] = (T)x[i];
    }
}

// The same 8 values in two steps, so that several loads can be under way: aligned and there (a row's number is kept in
// range by the caller; `some` says whether the values count)
template <int DT>
struct Raw {
    u32x4 v[DT == 0 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw<DT> load_raw(const void *row, int64_t col) {
    const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const typename Elem<DT>::T *>(row) + col);
    Raw<DT> r;
    r.v[0] = p[0];
    if constexpr (DT == 0) r.v[1] = p[1];
    return r;
}
template <int DT>
__device__ __forceinline__ void values_of(const Raw<DT> &r, bool some, float (&x)[8]) {
    typename Elem<DT>::T t[8];
    __builtin_memcpy(t, &r, sizeof t);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = some ? (float)t[i] : 0.0f;
}

// The larger of magnitudes as bit patterns: NaN above infinity above every number
__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }

struct Block {
    float s, mul, r, d;  // the scale; what values are multiplied by first; 1 / (s mul); s mul
};
// A block's scale from its largest magnitude. Blocks of tiny values are scaled up, so that remainders stay
// normal numbers. NaN or infinity inside: s NaN, every value 0.
__device__ __forceinline__ Block block_of(uint32_t top_bits, float inv_top) {
    Block b;
    if (top_bits >= 0x7F800000u) {
        b.s = __builtin_nanf("");
        b.mul = 0.0f;
        b.d = b.r = 1.0f;
        return b;
    }
    b.s = fmaxf(__builtin_bit_cast(float, top_bits) * inv_top, 0x1p-126f);
    b.mul = b.s < 0x1p-60f ? 0x1p60f : 1.0f;
    b.d = b.s * b.mul;
    b.r = __builtin_amdgcn_rcpf(b.d);  // (off by a unit of its last place at most)
    return b;
}
__device__ __forceinline__ float quotient(float x, const Block &b) {
    x *= b.mul;
    float q = x * b.r;
    q = fmaf(fmaf(-q, b.d, x), b.r, q);
    const float e = fmaf(-q, b.d, x);
    const uint32_t bits = __builtin_bit_cast(uint32_t, q);
    const int towards = ((int32_t)(__builtin_bit_cast(uint32_t, e) ^ bits) >> 31) | 1;
    const float moved = __builtin_bit_cast(float, bits + (uint32_t)towards);
    q = e != 0.0f && (bits & 1u) == 0 ? moved : q;
    return copysignf(q, x);  // (-0 stays -0; what passes the largest value by a few units still rounds to it)
}
__device__ __forceinline__ uint32_t pack4(int type, const float *q) {
#if defined(__HIP_DEVICE_COMPILE__)
    if (type == 0) return __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false), true);
    return __builtin_amdgcn_cvt_pk_bf8_f32(q[2], q[3], __builtin_amdgcn_cvt_pk_bf8_f32(q[0], q[1], 0, false), true);
#else
    (void)type;
    (void)q;
    return 0;
#endif
}
// N values (4 or 8) of one block as codes
template <int N>
__device__ __forceinline__ void codes(const float (&x)[N], const Block &b, int type, uint32_t (&out)[N / 4]) {
    const float below = b.r * (1.0f - 0x1p-21f), above = b.r * (1.0f + 0x1p-21f);  // (r, and each product, is off by 2^-23 at most)
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = x[i + j] * below;
        uint32_t code = pack4(type, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = x[i + j] * above;
        if (code != pack4(type, q) || b.mul != 1.0f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = quotient(x[i + j], b);
            code = b.mul == 0.0f ? 0u : pack4(type, q);
        }
        out[i / 4] = code;
    }
}
__device__ __forceinline__ void store_codes8(uint8_t *p, int count, bool wide, uint32_t lo, uint32_t hi) {
    if (count >= 8 && wide) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < count) p[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

// Row i of what is converted
__device__ __forceinline__ int64_t source_row(const F8Convert &p, int64_t i) {
    if (p.index == nullptr) return i;
    const int r = p.index[i];
    return r >= 0 && r < p.rows ? r : -1;
}

// The largest magnitude of 8 values as its bits. 16-bit values are compared in pairs.
template <int DT>
__device__ __forceinline__ uint32_t largest(const Raw<DT> &r) {
    if constexpr (DT == 0) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, r.v[i / 4][i % 4] & 0x7FFFFFFFu);
        return m;
    } else {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, r.v[0][i] & 0x7FFF7FFFu));
        const unsigned short top = max(m[0], m[1]);
        return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(typename Elem<DT>::T, top));
    }
}
// The largest of each row of 16 lanes, in all of them
__device__ __forceinline__ uint32_t largest_of_16(uint32_t m) {
#if defined(__HIP_DEVICE_COMPILE__)
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, false));  // row_ror 8, 4, 2, 1
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xF, 0xF, false));
#endif
    return m;
}

// Blocks of 1 x 128: a workgroup takes 32 rows of 4 blocks, a wave 8 of the rows, 4 at a time so that their loads are
// under way together. Scales leave through LDS: those of 32 rows of one block are a line (one by one from the lanes
// that have them they cost as much as the rest of the kernel). WIDE: rows of X and of codes are aligned for whole
// accesses, and columns come in eights (a lane behind the last of a row then takes its last 8 values, which are of the
// same block or of none that is stored).
constexpr int U = 4, ROWS = 32;
template <int DT, bool WIDE>
__global__ __launch_bounds__(NT) void f8_rows_kernel(F8Convert p, bool wide_x, bool wide_q) {
    __shared__ float scales[4][ROWS];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const float inv_top = inv_top_of(p.type);
    const int64_t chunks = ((int64_t)p.q_cols + 511) / 512, row_bytes = p.ldx * (int64_t)sizeof(typename Elem<DT>::T);
    for (int64_t first = (int64_t)blockIdx.x * ROWS; first < p.q_rows; first += (int64_t)gridDim.x * ROWS)
        for (int64_t chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
            const int64_t col = chunk * 512 + lane * 8;
            const int count = (int)min((int64_t)8, p.q_cols - col);
            for (int r = wave * 8; r < wave * 8 + 8 && first + r < p.q_rows; r += U) {
                const int64_t row0 = first + r;
                int64_t from[U];
                Raw<DT> raw[WIDE ? U : 1];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    from[u] = row0 + u < p.q_rows ? source_row(p, row0 + u) : -1;
                    if constexpr (WIDE) {
                        raw[u] = Raw<DT>{};
                        if (from[u] >= 0) raw[u] = load_raw<DT>(static_cast<const char *>(p.X) + from[u] * row_bytes, min(col, (int64_t)p.q_cols - 8));
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float x[8] = {};
                    uint32_t m = 0;
                    if constexpr (WIDE) {
                        values_of<DT>(raw[u], true, x);
                        m = largest(raw[u]);
                    } else {
                        if (from[u] >= 0 && count > 0) load8<DT>(static_cast<const char *>(p.X) + from[u] * row_bytes, col, count, wide_x, x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) m = max(m, magnitude(x[i]));
                    }
                    const Block b = block_of(largest_of_16(m), inv_top);
                    uint32_t q[2];
                    codes(x, b, p.type, q);
                    const int64_t row = row0 + u;
                    if ((lane & 15) == 0) scales[lane >> 4][r + u] = b.s;
                    if (count > 0 && row < p.q_rows) store_codes8(p.Q + row * p.ldq + col, count, WIDE || wide_q, q[0], q[1]);
                }
            }
            __syncthreads();
            const int block = threadIdx.x / ROWS, r = threadIdx.x % ROWS;
            if (block < 4 && chunk * 512 + block * 128 < p.q_cols && first + r < p.q_rows)
                p.S[(first + r) * p.s_row + (chunk * 4 + block) * p.s_col] = scales[block][r];
            __syncthreads();
        }
}

// The transpose: row f of the matrix is column f of X, in blocks of 128 of X's rows. A workgroup takes 128
// rows and 64 columns; a thread 8 columns of the rows tid / 8 + 32 i. Codes are turned through LDS, whose
// rows of 128 bytes (one of the matrix) are padded by 4.
template <int DT, bool WIDE>
__global__ __launch_bounds__(NT) void f8_turn_kernel(F8Convert p, bool wide_x, bool wide_q) {
    __shared__ uint32_t part[4][64];
    __shared__ uint32_t turned[64][33];  // as bytes: [column][row]
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, at = (tid & 7) * 8, r0 = tid >> 3;
    const int64_t tiles_r = ((int64_t)p.q_cols + 127) / 128, tiles_c = ((int64_t)p.q_rows + 63) / 64;
    for (int64_t tc = blockIdx.x; tc < tiles_c; tc += gridDim.x)
        for (int64_t tr = blockIdx.y; tr < tiles_r; tr += gridDim.y) {
            const int64_t col = tc * 64 + at;
            const int count = (int)min((int64_t)8, p.q_rows - col);
            float x[4][8] = {};
            int64_t from[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = tr * 128 + r0 + 32 * i;
                from[i] = row < p.q_cols ? source_row(p, row) : -1;
            }
            if constexpr (WIDE) {
                Raw<DT> raw[4];
                if (p.rows > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        raw[i] = load_raw<DT>(static_cast<const char *>(p.X) + max(from[i], (int64_t)0) * p.ldx * (int64_t)sizeof(typename Elem<DT>::T),
                                              min(col, (int64_t)p.q_rows - 8));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) values_of<DT>(raw[i], from[i] >= 0 && count > 0, x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (from[i] >= 0 && count > 0)
                        load8<DT>(static_cast<const char *>(p.X) + from[i] * p.ldx * (int64_t)sizeof(typename Elem<DT>::T), col, count, wide_x, x[i]);
            }
            uint32_t m[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                m[c] = max(max(magnitude(x[0][c]), magnitude(x[1][c])), max(magnitude(x[2][c]), magnitude(x[3][c])));
#pragma unroll
                for (int d = 8; d < 64; d <<= 1) m[c] = max(m[c], (uint32_t)__shfl_xor((int)m[c], d));
            }
            if (lane < 8) {
#pragma unroll
                for (int c = 0; c < 8; ++c) part[wave][at + c] = m[c];
            }
            __syncthreads();
            uint8_t *bytes = reinterpret_cast<uint8_t *>(turned);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const Block b = block_of(max(max(part[0][at + c], part[1][at + c]), max(part[2][at + c], part[3][at + c])), inv_top_of(p.type));
                const float v[4] = {x[0][c], x[1][c], x[2][c], x[3][c]};
                uint32_t q[1];
                codes(v, b, p.type, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) bytes[(at + c) * 132 + r0 + 32 * i] = (uint8_t)(q[0] >> (8 * i));
                if (r0 == 0 && c < count) p.S[(col + c) * p.s_row + tr * p.s_col] = b.s;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 16 lanes to a row of 128 codes, 8 codes each
                const int f = (tid >> 4) + 16 * i, c = (tid & 15) * 8;
                const int64_t row = tc * 64 + f, first = tr * 128 + c;
                if (row < p.q_rows && first < p.q_cols)
                    store_codes8(p.Q + row * p.ldq + first, (int)min((int64_t)8, p.q_cols - first), wide_q, turned[f][c / 4],
                                 turned[f][c / 4 + 1]);
            }
            __syncthreads();
        }
}

// Blocks of 128 x 128, one to a workgroup: a thread holds 8 columns of the rows tid / 16 + 16 i.
template <int DT, bool WIDE>
__global__ __launch_bounds__(NT) void f8_square_kernel(F8Convert p, bool wide_x, bool wide_q) {
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x, lane = tid & 63, at = (tid & 15) * 8, r0 = tid >> 4;
    const int64_t tiles_r = ((int64_t)p.q_rows + 127) / 128, tiles_c = ((int64_t)p.q_cols + 127) / 128;
    for (int64_t tr = blockIdx.x; tr < tiles_r; tr += gridDim.x)
        for (int64_t tc = blockIdx.y; tc < tiles_c; tc += gridDim.y) {
            const int64_t col = tc * 128 + at;
            const int count = (int)min((int64_t)8, p.q_cols - col);
            float x[8][8] = {};
            uint32_t m = 0;
            int64_t from[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t row = tr * 128 + r0 + 16 * i;
                from[i] = row < p.q_rows ? source_row(p, row) : -1;
            }
            if constexpr (WIDE) {
                Raw<DT> raw[8];
                if (p.rows > 0) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        raw[i] = load_raw<DT>(static_cast<const char *>(p.X) + max(from[i], (int64_t)0) * p.ldx * (int64_t)sizeof(typename Elem<DT>::T),
                                              min(col, (int64_t)p.q_cols - 8));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) values_of<DT>(raw[i], from[i] >= 0 && count > 0, x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (from[i] >= 0 && count > 0)
                        load8<DT>(static_cast<const char *>(p.X) + from[i] * p.ldx * (int64_t)sizeof(typename Elem<DT>::T), col, count, wide_x, x[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) m = max(m, magnitude(x[i][c]));
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
            if (lane == 0) part[tid >> 6] = m;
            __syncthreads();
            const Block b = block_of(max(max(part[0], part[1]), max(part[2], part[3])), inv_top_of(p.type));
            if (tid == 0) p.S[tr * p.s_row + tc * p.s_col] = b.s;
            if (count > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t row = tr * 128 + r0 + 16 * i;
                    if (row < p.q_rows) {
                        uint32_t q[2];
                        codes(x[i], b, p.type, q);
                        store_codes8(p.Q + row * p.ldq + col, count, wide_q, q[0], q[1]);
                    }
                }
            }
            __syncthreads();
        }
}

// Values: 8 columns of a row to a thread, 512 to a wave.
template <int DT>
__global__ __launch_bounds__(NT) void f8_values_kernel(F8Convert p, bool wide_x, bool wide_q) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t chunks = ((int64_t)p.q_cols + 511) / 512;
    const int shift = p.block_rows == 1 ? 0 : 7;
    for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < p.q_rows; row += (int64_t)gridDim.x * 4) {
        const uint8_t *q_row = p.Q + row * p.ldq;
        char *x_row = static_cast<char *>(p.X) + row * p.ldx * (int64_t)sizeof(typename Elem<DT>::T);
        for (int64_t chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
            const int64_t col = chunk * 512 + lane * 8;
            const int count = (int)min((int64_t)8, p.q_cols - col);
            if (count <= 0) continue;
            const float s = p.S[(row >> shift) * p.s_row + (col >> 7) * p.s_col];
            uint2 q = make_uint2(0, 0);
            if (count >= 8 && wide_q) {
                q = *reinterpret_cast<const uint2 *>(q_row + col);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t c = i < count ? (uint32_t)q_row[col + i] << (8 * (i & 3)) : 0u;
                    (i < 4 ? q.x : q.y) |= c;
                }
            }
            float x[8];
            const f32x2 v[4] = {f32_pair<false>(p.type, q.x), f32_pair<true>(p.type, q.x), f32_pair<false>(p.type, q.y),
                                f32_pair<true>(p.type, q.y)};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = v[i / 2][i % 2] * s;
            store8<DT>(x_row, col, count, wide_x, x);
        }
    }
}

// Enough workgroups for `n` units, within what a launch counts
unsigned grid_of(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

bool wide(const void *p, int64_t ld_bytes, int to) { return (reinterpret_cast<uintptr_t>(p) % to) == 0 && ld_bytes % to == 0; }

template <typename F>
hipError_t launch(F pick, const F8Convert &p, dim3 grid, hipStream_t s) {
    const int size = p.dtype == 0 ? 4 : 2;
    const bool wx = wide(p.X, p.ldx * size, 16), wq = wide(p.Q, p.ldq, 8);
    const auto f = pick(wx && wq && p.cols % 8 == 0);
    note_launch(reinterpret_cast<const void *>(f), NT);
    hipLaunchKernelGGL(f, grid, dim3(NT), 0, s, p, wx, wq);
    return hipGetLastError();
}
#define REGTILE_PICK(kernel) \
    [&](bool w) { return w ? (p.dtype == 0 ? kernel<0, true> : p.dtype == 1 ? kernel<1, true> : kernel<2, true>) \
                           : (p.dtype == 0 ? kernel<0, false> : p.dtype == 1 ? kernel<1, false> : kernel<2, false>); }

}  // namespace

hipError_t launch_f8_quantize(const F8Convert &p, hipStream_t s, const char **name) {
    const int64_t rows = p.q_rows, cols = p.q_cols;
    if (p.transpose) {
        *name = "f8_quantize_transposed";
        return launch(REGTILE_PICK(f8_turn_kernel), p,
                      dim3(grid_of((rows + 63) / 64, 1 << 16), grid_of((cols + 127) / 128, 1 << 15)), s);
    }
    if (p.block_rows == 1) {
        *name = "f8_quantize_rows";
        return launch(REGTILE_PICK(f8_rows_kernel), p,
                      dim3(grid_of((rows + ROWS - 1) / ROWS, 1 << 16), grid_of((cols + 511) / 512, 64)), s);
    }
    *name = "f8_quantize_blocks";
    return launch(REGTILE_PICK(f8_square_kernel), p,
                  dim3(grid_of((rows + 127) / 128, 1 << 16), grid_of((cols + 127) / 128, 1 << 15)), s);
}

hipError_t launch_f8_dequantize(const F8Convert &p, hipStream_t s, const char **name) {
    *name = "f8_dequantize";
    return launch([&](bool) { return p.dtype == 0 ? f8_values_kernel<0> : p.dtype == 1 ? f8_values_kernel<1> : f8_values_kernel<2>; }, p,
                  dim3(grid_of(((int64_t)p.q_rows + 3) / 4, 1 << 18), grid_of(((int64_t)p.q_cols + 511) / 512, 64)), s);
}

}  // namespace regtile

// experts.hip -- what a mixture of experts needs around its products: the router's choice and weights with
// their gradient, the order of the tokens' rows by expert, and the weighted sum of each token's rows with its
// gradient.
//
// route: one wave a token, experts i * 64 + lane in registers. The choice is made of exact comparisons: of the
// logits themselves where softmax or sigmoid only grow with them (no bias, groups by their best), and otherwise
// of score + bias in 64 bits, since in 32 two experts whose values differ by less than a rounding change places
// about once in 5000 tokens. Each of the k steps takes the largest key over the wave with 6 DPP maxima of its
// high word; ties are settled by the low word, then by the lowest index. Only the chosen experts' weights are
// computed, by the lane that holds the choice, in 64 bits.
//
// order: a stable counting sort. A wave finds the lanes with its own expert by ballots over the index's bits,
// so that counts and ranks need no atomics and come out the same every time. A workgroup takes a chunk of the slots
// (from 4 million on several), finds its place by adding up the counts of those before it, and there are at most 1024.
//
// combine and its gradient move each row once: a token's columns go over a workgroup's threads with 4 rows under way, the
// gradient takes a wave to a row. 8192 tokens x 8 of 2048 bf16: 73 us forward and 123 back, where a copy of as many bytes takes 56
// and 106. The router (64 tokens of 256 experts 8.4 us, 8192 of 64 7.5, the gradient 6.5) and the order (512 slots of 256 experts
// 5.7 us, 65536 of 64 6.2 to count and 12.3 to place) are bound by their chains of latencies, not by bytes.
#include "f8_common.h"

namespace regtile {
namespace {

constexpr int NT = 256;  // 4 waves
typedef unsigned long long u64;

__device__ __forceinline__ float load_value(const void *p, int dtype, int64_t at) {
    if (dtype == 0) return static_cast<const float *>(p)[at];
    if (dtype == 1) return (float)static_cast<const __bf16 *>(p)[at];
    return (float)static_cast<const _Float16 *>(p)[at];
}
__device__ __forceinline__ void store_value(void *p, int dtype, int64_t at, float x) {
    if (dtype == 0)
        static_cast<float *>(p)[at] = x;
    else if (dtype == 1)
        static_cast<__bf16 *>(p)[at] = (__bf16)x;
    else
        static_cast<_Float16 *>(p)[at] = (_Float16)x;
}

// LDS that lanes of one wave hand to each other: what stands before is done before what stands behind. (A wave's LDS instructions
// run in order; this keeps the compiler from exchanging them, and costs none.)
__device__ __forceinline__ void lds_step() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The largest x of the wave, in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
#if defined(__HIP_DEVICE_COMPILE__)
#define REGTILE_STEP(ctrl) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, ctrl, 0xF, 0xF, false))
    REGTILE_STEP(0x111);  // row_shr 1, 2, 4, 8: lane 15 of each row of 16 has its maximum
    REGTILE_STEP(0x112);
    REGTILE_STEP(0x114);
    REGTILE_STEP(0x118);
    REGTILE_STEP(0x142);  // row_bcast 15 and 31: lane 63 has them all
    REGTILE_STEP(0x143);
#undef REGTILE_STEP
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
#else
    return x;
#endif
}
template <typename T>
__device__ __forceinline__ T wave_sum(T x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// Keys that compare as the values do; 0 for what is not to be chosen (-inf, NaN), which is below every other
__device__ __forceinline__ u64 key_of(float v) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);  // (-0 and 0 are equal)
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return v > -INFINITY ? (u64)k << 32 : 0;
}
__device__ __forceinline__ u64 key_of(double v) {
    const u64 b = __builtin_bit_cast(u64, v + 0.0);
    const u64 k = b ^ ((u64)((int64_t)b >> 63) | 0x8000000000000000ull);
    return v > -(double)INFINITY ? k : 0;
}

// A logit's score, up to softmax's total: 64 bits
__device__ __forceinline__ double score_of(bool sigmoid, float logit, float top) {
    return sigmoid ? 1.0 / (1.0 + exp(-(double)logit)) : exp((double)logit - (double)top);
}

// R: experts a lane; WIDE: choose by score + bias in 64 bits, else by the logits
template <int R, bool WIDE>
__global__ __launch_bounds__(NT) void route_kernel(RouteProblem p) {
    // values by expert, a group's experts one slot further on than the last's: the lanes that read a group each
    // then meet different banks
    __shared__ u64 by_expert[WIDE ? 4 : 1][WIDE ? 64 * R + 64 : 1];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t token = (int64_t)blockIdx.x * 4 + wave;
    if (token >= p.tokens) return;
    float x[R];
    bool poison = false;
    uint32_t top_key = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = i * 64 + lane;
        x[i] = e < p.experts ? load_value(p.logits, p.dtype, token * p.ldl + e) : -INFINITY;
        poison |= x[i] != x[i] || x[i] == INFINITY;
        top_key = max(top_key, (uint32_t)(key_of(x[i]) >> 32));
    }
    int32_t *chosen = p.chosen + token * p.k;
    float *weights = p.weights + token * p.k;
    if (__ballot(poison) != 0) {
        if (lane < p.k) {
            chosen[lane] = lane;
            weights[lane] = __builtin_nanf("");
        }
        return;
    }
    top_key = wave_max(top_key);  // the largest logit
    const float top = top_key == 0 ? 0.0f
                                   : __builtin_bit_cast(float, top_key & 0x80000000u ? top_key ^ 0x80000000u : ~top_key);
    double total = 1.0;
    u64 key[R];
    if constexpr (WIDE) {
        double s[R];
        total = 0.0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            s[i] = score_of(p.sigmoid, x[i], top);
            total += s[i];
        }
        total = p.sigmoid ? 1.0 : wave_sum(total);
        const double unit = total > 0.0 ? 1.0 / total : 0.0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = i * 64 + lane;
            const double b = p.bias != nullptr && e < p.experts ? (double)p.bias[e] : 0.0;
            key[i] = x[i] > -INFINITY ? key_of(s[i] * unit + b) : 0;
        }
    } else {
#pragma unroll
        for (int i = 0; i < R; ++i) key[i] = key_of(x[i]);
        if (!p.sigmoid && !p.renormalize) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) sum += expf(x[i] - top);
            total = wave_sum((double)sum);
        }
    }
    if (p.groups > 1) {
        const int per = p.experts / p.groups;
        u64 open;
        if constexpr (WIDE) {
            u64 *mine = by_expert[wave];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int e = i * 64 + lane;
                if (e < p.experts) mine[e + e / per] = key[i];
            }
            lds_step();
            // the two best of each group: `sub` lanes to a group, then over those
            int sub = 64;
            while (sub * p.groups > 64) sub >>= 1;
            const int group = lane / sub, part = lane & (sub - 1);
            u64 first = 0, second = 0;
            if (group < p.groups)
                for (int i = part; i < per; i += sub) {
                    const u64 k = mine[group * (per + 1) + i];
                    second = max(second, min(first, k));
                    first = max(first, k);
                }
            for (int d = 1; d < sub; d <<= 1) {
                const u64 f = __shfl_xor(first, d), n = __shfl_xor(second, d);
                second = max(max(second, n), min(first, f));
                first = max(first, f);
            }
            auto value = [](u64 k) { return __builtin_bit_cast(double, k >> 63 ? k ^ 0x8000000000000000ull : ~k); };
            u64 rank = first;
            if (p.group_best == 2 && second != 0) rank = key_of(value(first) + value(second));
            // groups before this one: better, or as good with a lower number
            int before = 0;
            for (int g = 0; g < p.groups; ++g) {
                const u64 other = (u64)(uint32_t)__builtin_amdgcn_readlane((int)(rank >> 32), g * sub) << 32 |
                                  (uint32_t)__builtin_amdgcn_readlane((int)rank, g * sub);
                before += other > rank || (other == rank && g < group);
            }
            const bool kept = group < p.groups && part == 0 && before < p.top_groups;
            open = 0;  // a bit for each group, from the lanes that begin one
            for (u64 m = __ballot(kept); m != 0; m &= m - 1) open |= 1ull << ((__ffsll((unsigned long long)m) - 1) / sub);
        } else {
            // by their best logit: the best of the groups that are left, top_groups times
            u64 left = p.groups == 64 ? ~0ull : (1ull << p.groups) - 1;
            for (int n = 0; n < p.top_groups; ++n) {
                uint32_t best = 0;
                int in = 0x7FFFFFFF;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const int e = i * 64 + lane, g = e / per;
                    if (e < p.experts && (left >> g & 1) && (uint32_t)(key[i] >> 32) > best) {
                        best = (uint32_t)(key[i] >> 32);
                        in = g;
                    }
                }
                const uint32_t m = wave_max(best);
                if (m == 0) break;  // nothing to choose in any of them
                const uint32_t low = ~wave_max(best == m ? ~(uint32_t)in : 0u);
                left &= ~(1ull << low);
            }
            open = ~left;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int e = i * 64 + lane;
            if (e < p.experts && !(open >> (e / per) & 1)) key[i] = 0;
        }
    }
    // the k best
    int my_expert = -1;
    float my_logit = -INFINITY;
    for (int j = 0; j < p.k; ++j) {
        u64 best = 0;
        int at = 0;
        float l = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
                l = x[i];
            }
        const uint32_t high = wave_max((uint32_t)(best >> 32));
        if (high == 0) break;
        u64 who = __ballot((uint32_t)(best >> 32) == high);
        if (who & (who - 1)) {
            if constexpr (WIDE) {
                const uint32_t low = wave_max((uint32_t)(best >> 32) == high ? (uint32_t)best : 0u);
                who = __ballot((uint32_t)(best >> 32) == high && (uint32_t)best == low);
            }
            if (who & (who - 1)) {
                const uint32_t first = wave_max(who >> lane & 1 ? ~(uint32_t)(at * 64 + lane) : 0u);
                who = __ballot((who >> lane & 1) && ~(uint32_t)(at * 64 + lane) == first);
            }
        }
        const int winner = __ffsll((unsigned long long)who) - 1;
        const int expert = __builtin_amdgcn_readlane(at, winner) * 64 + winner;
        const float logit = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, l), winner));
        if (lane == j) {
            my_expert = expert;
            my_logit = logit;
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (lane == winner && i == at) key[i] = 0;
    }
    const double s = my_expert >= 0 ? score_of(p.sigmoid, my_logit, top) : 0.0;
    if (p.renormalize) total = wave_sum(s);
    if (lane < p.k) {
        chosen[lane] = my_expert;
        weights[lane] = total > 0.0 ? (float)(s / total * (double)p.scale) : 0.0f;
    }
}

// x of lane j
__device__ __forceinline__ double lane_of(double x, int j) {
    const u64 b = __builtin_bit_cast(u64, x);
    return __builtin_bit_cast(double, (u64)(uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), j) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)b, j));
}

// The gradient with respect to the logits. With w the weights before `scale` and dot = sum_j dw_j w_j, expert
// c's is scale times:  softmax, renormalised: w_c (dw_c - dot), and 0 for experts that were not chosen;
// softmax: p_e (dw_e - dot), dw_e = 0 for those;  sigmoid, renormalised: w_c (1 - s_c) (dw_c - dot);
// sigmoid: s_c (1 - s_c) dw_c.
// Where one expert is nearly certain, dw_c - dot is the difference of two numbers that are nearly equal. The weights (the
// probabilities of all experts) sum to 1, so every dw may be counted from one of them: from the likeliest expert's (0 if it
// was not chosen), whose own terms, the large ones, are then 0. What was not chosen has dw = 0 too, and counts with the sum of
// its probabilities, which are fp32 exponentials added in 64 bits; all else is 64 bits. The slots of an expert that was chosen
// more than once are added before they are rounded, in a loop that other tokens do not run. 8192 tokens of 64 experts, k = 8:
// 6.2 us renormalised and 9.1 not (with fp32 sums 6.6, and a gradient off by a fifth of itself 16 ahead).
template <int R>
__global__ __launch_bounds__(NT) void route_grad_kernel(RouteProblem p) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t token = (int64_t)blockIdx.x * 4 + wave;
    if (token >= p.tokens) return;
    float x[R], d[R];
    bool poison = false;
    uint32_t top_key = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = i * 64 + lane;
        x[i] = e < p.experts ? load_value(p.logits, p.dtype, token * p.ldl + e) : -INFINITY;
        poison |= x[i] != x[i] || x[i] == INFINITY;
        top_key = max(top_key, (uint32_t)(key_of(x[i]) >> 32));
        d[i] = 0.0f;
    }
    poison = __ballot(poison) != 0;
    top_key = wave_max(top_key);
    const float top = top_key == 0 ? 0.0f
                                   : __builtin_bit_cast(float, top_key & 0x80000000u ? top_key ^ 0x80000000u : ~top_key);
    int expert = lane < p.k ? p.chosen[token * p.k + lane] : -1;
    if (expert >= p.experts || expert < 0) expert = -1;
    const double dw = expert >= 0 ? (double)p.dweights[token * p.k + lane] : 0.0;
    const float logit = expert >= 0 ? load_value(p.logits, p.dtype, token * p.ldl + expert) : -INFINITY;
    // the score, and a sigmoid's 1 - s (which is lost in an s near 1), from one exponential
    const bool some = expert >= 0 && !poison;
    const double power = exp(p.sigmoid ? -fabs((double)logit) : (double)logit - (double)top), far = p.sigmoid ? 1.0 / (1.0 + power) : 1.0;
    const double near = power * far, s = !some ? 0.0 : p.sigmoid && logit >= 0.0f ? far : near;
    const uint32_t key = expert >= 0 ? (uint32_t)(key_of(logit) >> 32) : 0u, best = wave_max(key);  // of the chosen
    const u64 likely = __ballot(key == best && best != 0);
    auto likeliest = [&](double v) { return likely != 0 ? lane_of(v, __ffsll((unsigned long long)likely) - 1) : 0.0; };
    double mine;
    if (p.renormalize) {
        const double total = wave_sum(s), w = total > 0.0 ? s / total : 0.0, from = likeliest(dw), diff = expert >= 0 ? dw - from : 0.0;
        mine = w * (diff - wave_sum(w * diff));
    } else if (p.sigmoid) {
        mine = s * dw;
    } else {
        // every expert's exponential; an expert's first slot stands for all of its slots
        double all = 0.0, left = 0.0, of_expert = 0.0;
        uint32_t chosen = 0;  // a bit for each of this lane's experts
        bool first = true;
        for (int j = 0; j < p.k; ++j) {
            const int c = __builtin_amdgcn_readlane(expert, j);
            const double v = lane_of(dw, j);
            if (c >= 0 && (c & 63) == lane) chosen |= 1u << (c >> 6);
            if (c == expert) of_expert += v;
            first &= c != expert || j >= lane;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            d[i] = expf(x[i] - top);
            all += (double)d[i];
            if (!(chosen >> i & 1)) left += (double)d[i];
        }
        const double own = first ? s : 0.0, from = best == top_key ? likeliest(of_expert) : 0.0, diff = of_expert - from;
        const double total = wave_sum(all), rest = wave_sum(left), shift = wave_sum(own * diff), sum = wave_sum(own * of_expert);
        const double unit = total > 0.0 ? 1.0 / total : 0.0, dot = sum * unit * unit * (double)p.scale;
        mine = own * unit * (diff - (shift - rest * from) * unit);
#pragma unroll
        for (int i = 0; i < R; ++i) d[i] = (float)(-dot * (double)d[i]);
    }
    if (p.sigmoid) mine *= logit >= 0.0f ? near : far;
    mine *= (double)p.scale;
    auto place = [&](double of_slot) {  // slots' values at their experts; whether an expert has several
        const float v = (float)of_slot;
        u64 twice = 0;
        for (int j = 0; j < p.k; ++j) {
            const int c = __builtin_amdgcn_readlane(expert, j);
            const u64 same_expert = __ballot(expert == c);
            if (c >= 0) twice |= same_expert & (same_expert - 1);
            const float of_j = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), j));
#pragma unroll
            for (int i = 0; i < R; ++i) d[i] = c == i * 64 + lane ? of_j : d[i];
        }
        return twice != 0;
    };
    if (place(mine)) {
        double sum = 0.0;
        for (int j = 0; j < p.k; ++j) sum += __builtin_amdgcn_readlane(expert, j) == expert ? lane_of(mine, j) : 0.0;
        place(sum);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int e = i * 64 + lane;
        if (e < p.experts) store_value(p.dlogits, p.dtype, token * p.ldd + e, poison ? __builtin_nanf("") : d[i]);
    }
}

// ---- order -------------------------------------------------------------------------------------
constexpr int ORDER_NT = 1024, ORDER_WAVES = 16, CHUNK = 4096, MOST_EXPERTS = 1024;

// The lanes of the wave whose e is this lane's
__device__ __forceinline__ u64 same(int e, int bits) {
    u64 m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const u64 set = __ballot(e >> b & 1);
        m &= e >> b & 1 ? set : ~set;
    }
    return m;
}
__device__ __forceinline__ int expert_of(const OrderProblem &p, int64_t slot, int64_t end) {
    if (slot >= end) return p.experts;
    const int e = p.chosen[slot];
    return e >= 0 && e < p.experts ? e : p.experts;
}

// counts[wave][expert] of a chunk's slots, each wave's own part of `per` slots from `first` on; e: this lane's experts
constexpr int MOST = CHUNK / ORDER_NT;
__device__ __forceinline__ void count_chunk(const OrderProblem &p, int *counts, int64_t first, int64_t end, int per, int bits,
                                            int (&e_of)[MOST]) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < MOST; ++i) e_of[i] = i * 64 < per ? expert_of(p, first + wave * per + i * 64 + lane, end) : p.experts;
    for (int i = threadIdx.x; i < ORDER_WAVES * p.experts; i += ORDER_NT) counts[i] = 0;
    __syncthreads();
    int *mine = counts + wave * p.experts;
#pragma unroll
    for (int i = 0; i < MOST; ++i) {
        if (i * 64 >= per) break;
        const int e = e_of[i];
        const u64 m = same(e, bits);
        if (e < p.experts && __ffsll((unsigned long long)m) - 1 == lane) mine[e] += __popcll(m);
        lds_step();
    }
    __syncthreads();
}

__global__ __launch_bounds__(ORDER_NT) void order_count_kernel(OrderProblem p, int bits, int chunks) {
    __shared__ int counts[ORDER_WAVES * MOST_EXPERTS];
    const int64_t n = (int64_t)p.tokens * p.k, span = (int64_t)chunks * CHUNK, end = min(n, (blockIdx.x + 1) * span);
    const int e = threadIdx.x;
    int e_of[MOST], sum = 0;
    for (int64_t first = blockIdx.x * span; first < end; first += CHUNK) {
        count_chunk(p, counts, first, min(end, first + CHUNK), CHUNK / ORDER_WAVES, bits, e_of);
        if (e < p.experts)
            for (int w = 0; w < ORDER_WAVES; ++w) sum += counts[w * p.experts + e];
        __syncthreads();
    }
    if (e < p.experts) p.work[(int64_t)blockIdx.x * p.experts + e] = sum;
}

__global__ __launch_bounds__(ORDER_NT) void order_place_kernel(OrderProblem p, int bits, int chunks) {
    __shared__ int counts[ORDER_WAVES * MOST_EXPERTS];
    __shared__ int wave_room[ORDER_WAVES];
    __shared__ int2 ends[MOST_EXPERTS];  // of a group's rows and of its room
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, groups = gridDim.x;
    const int64_t n = (int64_t)p.tokens * p.k, span = (int64_t)chunks * CHUNK;
    int64_t first = blockIdx.x * span, end = min(n, first + CHUNK);
    const int64_t last = min(n, first + span);
    // a wave's part of the chunk, in whole 64s
    int per = ((int)((end - first + ORDER_WAVES - 1) / ORDER_WAVES) + 63) / 64 * 64;
    int e_of[MOST];
    count_chunk(p, counts, first, end, per, bits, e_of);
    int before = 0, all = 0;
    if (tid < p.experts) {
        if (groups == 1) {
            for (int w = 0; w < ORDER_WAVES; ++w) all += counts[w * p.experts + tid];
        } else {
            for (int g = 0; g < groups; ++g) {
                const int c = p.work[(int64_t)g * p.experts + tid];
                before += g < (int)blockIdx.x ? c : 0;
                all += c;
            }
        }
    }
    const int room = (all + p.align - 1) / p.align * p.align;
    int upto = room;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
    }
    if (lane == 63) wave_room[wave] = upto;
    __syncthreads();
    int start = upto - room, used = 0;
    for (int w = 0; w < ORDER_WAVES; ++w) {
        if (w < wave) start += wave_room[w];
        used += wave_room[w];
    }
    int at_expert = start + before;  // the next row of this thread's expert
    auto begin_waves = [&]() {       // counts to first rows
        if (tid < p.experts)
            for (int w = 0; w < ORDER_WAVES; ++w) {
                const int c = counts[w * p.experts + tid];
                counts[w * p.experts + tid] = at_expert;
                at_expert += c;
            }
    };
    begin_waves();
    if (tid < p.experts) {
        if (blockIdx.x == 0) {
            p.offsets[tid] = start;
            p.counts[tid] = all;
            if (tid == 0) p.offsets[p.experts] = used;
        }
        ends[tid] = make_int2(start + all, start + room);
    }
    for (int64_t r = used + (int64_t)blockIdx.x * ORDER_NT + tid; r < p.rows; r += (int64_t)groups * ORDER_NT) p.slots[r] = -1;
    __syncthreads();
    // rows between the groups: a wave to a group
    for (int e = (int)blockIdx.x * ORDER_WAVES + wave; e < p.experts; e += groups * ORDER_WAVES)
        for (int r = ends[e].x + lane; r < ends[e].y; r += 64) p.slots[r] = -1;
    int *mine = counts + wave * p.experts;
    while (true) {
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            if (i * 64 >= per) break;
            const int64_t slot = first + wave * per + i * 64 + lane;
            const int e = e_of[i];
            const u64 m = same(e, bits);
            int at = -1;
            if (e < p.experts) at = mine[e] + __popcll(m & ((1ull << lane) - 1));
            lds_step();
            if (e < p.experts && 63 - __clzll((long long)m) == lane) mine[e] = at + 1;
            lds_step();
            if (slot < end) {
                p.position[slot] = at;
                if (at >= 0) p.slots[at] = (int32_t)slot;
            }
        }
        first += CHUNK;
        if (first >= last) return;
        end = min(last, first + CHUNK);
        per = CHUNK / ORDER_WAVES;
        __syncthreads();
        count_chunk(p, counts, first, end, per, bits, e_of);
        begin_waves();
        __syncthreads();
    }
}

// ---- combine -----------------------------------------------------------------------------------
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
// V consecutive values (V elements: one aligned load, or 1)
template <int DT, int V>
__device__ __forceinline__ void load_v(const void *p, int64_t at, float (&x)[V]) {
    typedef typename Elem<DT>::T T;
    const T *q = static_cast<const T *>(p) + at;
    if constexpr (V == 1) {
        x[0] = (float)q[0];
    } else {
        T t[V];
        __builtin_memcpy(t, __builtin_assume_aligned(q, V * sizeof(T)), V * sizeof(T));
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = (float)t[i];
    }
}
template <int DT, int V>
__device__ __forceinline__ void store_v(void *p, int64_t at, const float (&x)[V]) {
    typedef typename Elem<DT>::T T;
    T *q = static_cast<T *>(p) + at;
    T t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = (T)x[i];
    __builtin_memcpy(__builtin_assume_aligned(q, V * sizeof(T)), t, V * sizeof(T));
}
__device__ __forceinline__ int position_of(const CombineProblem &p, int64_t slot) {
    const int r = p.position[slot];
    return r < p.rows ? r : -1;
}

// out[t] = sum_j w[t, j] Y[position[t, j]], in the order of j: a workgroup's threads along a token's columns.
template <int DT, int V>
__global__ __launch_bounds__(NT) void combine_kernel(CombineProblem p, int threads_x) {
    const int tx = threadIdx.x % threads_x, ty = threadIdx.x / threads_x;
    for (int64_t t = (int64_t)blockIdx.x * (NT / threads_x) + ty; t < p.tokens; t += (int64_t)gridDim.x * (NT / threads_x))
        for (int64_t c = ((int64_t)blockIdx.y * threads_x + tx) * V; c < p.n; c += (int64_t)gridDim.y * threads_x * V) {
            float sum[V] = {};
            for (int j0 = 0; j0 < p.k; j0 += 4) {  // 4 rows under way
                float y[4][V], w[4];
                bool some[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t slot = t * p.k + j0 + j;
                    const int r = j0 + j < p.k ? position_of(p, slot) : -1;
                    some[j] = r >= 0;
                    w[j] = some[j] && p.weights != nullptr ? p.weights[slot] : 1.0f;
                    if (some[j]) load_v<DT, V>(p.Y, r * p.ldy + c, y[j]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (some[j]) {
#pragma unroll
                        for (int v = 0; v < V; ++v) sum[v] = fmaf(w[j], y[j][v], sum[v]);
                    }
            }
            store_v<DT, V>(p.out, t * p.ldo + c, sum);
        }
}

// A wave to a row r of Y: with t = slots[r] / k, dY[r] = w dout[t] and dw = <dout[t], Y[r]>; zeros where the row
// is nobody's. Slots without a row have dw = 0.
template <int DT, int V>
__global__ __launch_bounds__(NT) void combine_grad_kernel(CombineProblem p) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t n = (int64_t)p.tokens * p.k;
    for (int64_t r = (int64_t)blockIdx.x * 4 + wave; r < max((int64_t)p.rows, n); r += (int64_t)gridDim.x * 4) {
        if (p.dweights != nullptr && r < n && lane == 0 && position_of(p, r) < 0) p.dweights[r] = 0.0f;
        if (r >= p.rows) continue;
        const int slot = p.slots[r];
        const bool some = slot >= 0 && slot < n;
        const int64_t t = some ? slot / p.k : 0;
        const float w = !some ? 0.0f : p.weights != nullptr ? p.weights[slot] : 1.0f;
        float sum = 0.0f;
        for (int64_t c = lane * V; c < p.n; c += 64 * V) {
            float d[V] = {}, y[V];
            if (some) {
                load_v<DT, V>(p.dout, t * p.ldd + c, d);
                if (p.dweights != nullptr) {
                    load_v<DT, V>(p.Y, r * p.ldy + c, y);
#pragma unroll
                    for (int v = 0; v < V; ++v) sum = fmaf(d[v], y[v], sum);
                }
#pragma unroll
                for (int v = 0; v < V; ++v) d[v] *= w;
            }
            store_v<DT, V>(p.dY, r * p.lddy + c, d);
        }
        if (some && p.dweights != nullptr) {
            sum = wave_sum(sum);
            if (lane == 0) p.dweights[slot] = sum;
        }
    }
}

bool rows16(const void *p, int64_t ld, int size) { return aligned16(p) && ld * size % 16 == 0; }

template <typename F>
hipError_t go(F f, dim3 grid, unsigned threads, hipStream_t s, void **args) {
    note_launch(reinterpret_cast<const void *>(f), threads);
    return hipLaunchKernel(reinterpret_cast<const void *>(f), grid, dim3(threads), args, 0, s);
}

}  // namespace

// What a launch of 4 tokens to 256 threads counts in 32 bits
constexpr int MOST_TOKENS = (1 << 26) - 4;

hipError_t launch_route(const RouteProblem &p, hipStream_t s, const char **name) {
    // by the logits where the scores grow with them and nothing is added to them
    const bool wide = p.bias != nullptr || (p.groups > 1 && p.group_best == 2);
    *name = wide ? "route_scores" : "route_logits";
    RouteProblem q = p;
    void *args[] = {&q};
    if (p.tokens > MOST_TOKENS) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(((int64_t)p.tokens + 3) / 4));
    auto pick = [&](auto narrow_f, auto wide_f) { return go(wide ? wide_f : narrow_f, grid, NT, s, args); };
    if (p.experts <= 64) return pick(route_kernel<1, false>, route_kernel<1, true>);
    if (p.experts <= 128) return pick(route_kernel<2, false>, route_kernel<2, true>);
    if (p.experts <= 256) return pick(route_kernel<4, false>, route_kernel<4, true>);
    if (p.experts <= 512) return pick(route_kernel<8, false>, route_kernel<8, true>);
    return pick(route_kernel<16, false>, route_kernel<16, true>);
}

hipError_t launch_route_grad(const RouteProblem &p, hipStream_t s, const char **name) {
    *name = "route_grad";
    RouteProblem q = p;
    void *args[] = {&q};
    if (p.tokens > MOST_TOKENS) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)(((int64_t)p.tokens + 3) / 4));
    if (p.experts <= 64) return go(route_grad_kernel<1>, grid, NT, s, args);
    if (p.experts <= 128) return go(route_grad_kernel<2>, grid, NT, s, args);
    if (p.experts <= 256) return go(route_grad_kernel<4>, grid, NT, s, args);
    if (p.experts <= 512) return go(route_grad_kernel<8>, grid, NT, s, args);
    return go(route_grad_kernel<16>, grid, NT, s, args);
}

// One workgroup orders a chunk by itself; more of them count first, through the workspace.
namespace {
constexpr int64_t MOST_GROUPS = 1024;
int order_chunks(int64_t slots) { return (int)((slots + MOST_GROUPS * CHUNK - 1) / (MOST_GROUPS * CHUNK)); }  // to a workgroup
int64_t order_groups(int64_t slots) {
    const int64_t span = (int64_t)order_chunks(slots) * CHUNK;
    return slots > 0 ? (slots + span - 1) / span : 1;
}
}  // namespace
int64_t order_work_bytes(int64_t slots, int experts) {
    const int64_t groups = order_groups(slots);
    return groups > 1 ? groups * experts * 4 : 0;
}

hipError_t launch_order(const OrderProblem &p, hipStream_t s, const char **name) {
    const int64_t n = (int64_t)p.tokens * p.k;
    const unsigned groups = (unsigned)order_groups(n);
    int bits = 1, chunks = order_chunks(n);
    while ((p.experts >> bits) != 0) ++bits;  // 0 .. experts
    OrderProblem q = p;
    void *args[] = {&q, &bits, &chunks};
    *name = "order_experts";
    if (groups > 1) {
        const hipError_t e = go(order_count_kernel, dim3(groups), ORDER_NT, s, args);
        if (e != hipSuccess) return e;
    }
    return go(order_place_kernel, dim3(groups), ORDER_NT, s, args);
}

hipError_t launch_combine(const CombineProblem &p, hipStream_t s, const char **name) {
    *name = "combine_experts";
    const int size = p.dtype == 0 ? 4 : 2, v = 16 / size;
    const bool wide = p.n % v == 0 && rows16(p.Y, p.ldy, size) && rows16(p.out, p.ldo, size);
    const int64_t units = wide ? p.n / v : p.n;
    int threads_x = NT;  // 16 threads at least: the rows of 16 tokens are then under way in a workgroup
    while (threads_x > 16 && threads_x / 2 >= units) threads_x /= 2;
    const int64_t gx = ((int64_t)p.tokens * threads_x + NT - 1) / NT, gy = (units + threads_x - 1) / threads_x;
    CombineProblem q = p;
    void *args[] = {&q, &threads_x};
    const dim3 grid((unsigned)(gx < (1 << 20) ? gx : 1 << 20), (unsigned)(gy < 1024 ? gy : 1024));
    auto pick = [&](auto f, auto f1) { return go(wide ? f : f1, grid, NT, s, args); };
    if (p.dtype == 0) return pick(combine_kernel<0, 4>, combine_kernel<0, 1>);
    if (p.dtype == 1) return pick(combine_kernel<1, 8>, combine_kernel<1, 1>);
    return pick(combine_kernel<2, 8>, combine_kernel<2, 1>);
}

hipError_t launch_combine_grad(const CombineProblem &p, hipStream_t s, const char **name) {
    *name = "combine_experts_grad";
    const int size = p.dtype == 0 ? 4 : 2, v = 16 / size;
    const bool wide = p.n % v == 0 && (p.dweights == nullptr || rows16(p.Y, p.ldy, size)) && rows16(p.dout, p.ldd, size) &&
                      rows16(p.dY, p.lddy, size);
    const int64_t n = (int64_t)p.tokens * p.k, rows = p.rows > n ? p.rows : n, g = (rows + 3) / 4;
    CombineProblem q = p;
    void *args[] = {&q};
    const dim3 grid((unsigned)(g < (1 << 20) ? g : 1 << 20));
    auto pick = [&](auto f, auto f1) { return go(wide ? f : f1, grid, NT, s, args); };
    if (p.dtype == 0) return pick(combine_grad_kernel<0, 4>, combine_grad_kernel<0, 1>);
    if (p.dtype == 1) return pick(combine_grad_kernel<1, 8>, combine_grad_kernel<1, 1>);
    return pick(combine_grad_kernel<2, 8>, combine_grad_kernel<2, 1>);
}

}  // namespace regtile

// om_route_topk / om_route_topk_backward: routing of tokens to experts.
#include <cstdint>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "select_common.cuh"

namespace om {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;        // one lane per pick
constexpr int kMaxExpertGroups = 32;  // one lane per group

struct RouteArgs {
    const void* logits;
    int64_t tokens;
    int64_t row_stride;
    const float* bias;
    int32_t* ids;
    float* weights;
    int experts, score, groups, group_picks, group_best, top_k, renorm;
    float scale;
};

constexpr int kRouteWarps = 8;

// The renormalised sigmoid weights are s_i / sum s with s = 1 / (1 + e^-x).
// Dividing every s by e^low, low = min(largest picked x, 0), leaves the
// quotient as it is and keeps the numerators from vanishing together when
// every picked logit is far below zero.  (x >= 0 implies low == 0.)
__device__ __forceinline__ float shifted_sigmoid(float x, float low) {
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - low) / (1.0f + expf(x));
}

__device__ __forceinline__ float sigmoid(float x) {
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x) / (1.0f + expf(x));
}

// What experts are chosen by where that is the sigmoid score: the same bits in
// every kernel.  One exponential, of -|x|, so that the divisor lies in [1, 2],
// where the fast division is good to 2 ulps (it gives 0 for divisors above 2^126),
// and scores below the normal range stay apart.
__device__ __forceinline__ float sigmoid_choice(float x) {
    const float t = expf(-fabsf(x)), r = __fdividef(1.0f, 1.0f + t);
    return x >= 0.0f ? r : __fmul_rn(t, r);
}

// One warp per token; lane l holds the experts l, l + 32, ...
template <typename T, int R>
__global__ void __launch_bounds__(kRouteWarps * 32) route_topk_kernel(RouteArgs a) {
    wait_for_stream();
    __shared__ float s_choice[kRouteWarps][R * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* logits = static_cast<const T*>(a.logits);
    const bool by_logit = a.bias == nullptr && (a.groups == 1 || a.group_best == 1);
    const bool need_sum = a.score == OM_SCORE_SOFTMAX && (!a.renorm || !by_logit);
    const float kNone = -INFINITY;

    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        const T* row = logits + t * a.row_stride;
        float x[R];
        float top = kNone;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = r * 32 + lane;
            x[r] = e < a.experts ? to_float(row[e]) : kNone;
            top = fmaxf(top, x[r]);  // a NaN is passed over
        }
        top = warp_max(top);
        float sum = 1.0f;
        if (need_sum) {
            float part = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (x[r] > kNone) part += expf(x[r] - top);
            sum = warp_sum(part);
        }
        // what the experts are chosen by: the logit itself where its order is the score's
        uint32_t key[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = r * 32 + lane;
            float c = x[r];
            if (!by_logit && x[r] > kNone) {
                c = a.score == OM_SCORE_SOFTMAX ? expf(x[r] - top) / sum : sigmoid_choice(x[r]);
                if (a.bias != nullptr) c += a.bias[e];
            }
            const bool open = x[r] > kNone && c > kNone;  // false for NaN too
            key[r] = open ? score_image(c) : 0u;
            if (a.groups > 1) s_choice[warp][e] = open ? c : kNone;
        }
        if (a.groups > 1) {
            __syncwarp();
            const int size = a.experts / a.groups;
            uint32_t gkey = 0;
            if (lane < a.groups) {
                float b0 = kNone, b1 = kNone;
                for (int i = 0; i < size; ++i) {
                    const float c = s_choice[warp][lane * size + i];
                    b1 = fmaxf(b1, fminf(b0, c));
                    b0 = fmaxf(b0, c);
                }
                if (b0 > kNone) gkey = score_image(a.group_best == 2 && b1 > kNone ? b0 + b1 : b0);
            }
            uint32_t picked = 0;
            for (int i = 0; i < a.group_picks; ++i) {
                const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
                if (best == 0) break;
                const int g = __ffs(__ballot_sync(0xffffffffu, gkey == best)) - 1;
                picked |= 1u << g;
                if (lane == g) gkey = 0;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = r * 32 + lane;
                if (e < a.experts && !((picked >> (e / size)) & 1)) key[r] = 0;
            }
            __syncwarp();
        }
        // the picks, best first: lane j keeps the j-th
        int my_id = -1;
        float my_x = kNone;
        for (int j = 0; j < a.top_k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) best = max(best, key[r]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0) break;
            int at = kMaxExperts;
            float xv = 0.0f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r)
                if (key[r] == best) at = r * 32 + lane, xv = x[r];
            const int first = __reduce_min_sync(0xffffffffu, (unsigned)at);
            xv = __shfl_sync(0xffffffffu, xv, first & 31);
            if (lane == j) my_id = first, my_x = xv;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * 32 + lane == first) key[r] = 0;
        }
        float w = 0.0f;
        if (a.renorm) {
            const float best = warp_max(my_x);
            const float low = fminf(best, 0.0f);
            if (my_id >= 0) w = a.score == OM_SCORE_SOFTMAX ? expf(my_x - best) : shifted_sigmoid(my_x, low);
            const float total = warp_sum(w);
            if (my_id >= 0) w = w / total;
        } else if (my_id >= 0) {
            w = a.score == OM_SCORE_SOFTMAX ? expf(my_x - top) / sum : sigmoid(my_x);
        }
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = my_id;
            a.weights[t * a.top_k + lane] = w * a.scale;
        }
    }
}

// ---------------------------------------------------- sorted-list kernel --
//
// For top_k <= 16.  L lanes share a token (32 / L tokens a warp).  A lane takes
// its share of the row eight experts at a time: it sorts the eight by a fixed
// network and merges them into its sorted list of the best LIST, 8 or 16 (with
// 8, the greater of a[i] and b[7 - i] for every i are the best eight of both, and
// bitonic, so three more steps sort them).  The lanes' lists are merged the same
// way across the lanes, log2(L) times, after which each of them has the token's
// best.
// Nothing but minima and maxima of independent pairs, no turn through memory,
// and no warp reduction per pick.
//
// PACKED: where 16-bit logits are themselves the order, a key is the
// order-preserving image of the logit above the complement of its index, so the
// list holds the indices, and ties go to the lower one.
//
// Otherwise the list holds what the experts are chosen by, as floats, and the
// indices are found afterwards: the k-th of the list is the least that was
// chosen; a lane looks through those of its eights whose greatest (kept in
// shared memory) reaches it, and an expert's place is the number of listed
// values above its own.  Equal values among the chosen, or one past the last,
// leave places open; then the token's picks are settled one after the other.
//
// GROUPED: lane l's share is the contiguous part l of the row, which lies in one
// group of experts; after the lanes' own lists are made, the groups' scores are
// taken from their heads, and the lists of groups not picked are dropped.

// What bounds it is the rate of minima and maxima (half of the issue rate): a
// token of 128 bf16 logits takes about 40 warp instructions of them and 96 in
// all, 61 of them in that pipe.  Measured, 131071 tokens, top 8: 128 bf16 logits
// 17.7 us (2.4 TB/s), 128 f32 29 us, 256 f32 sigmoid scores with bias in 8 groups
// 74 us (there by issue: 3.1 of 4 a clock), where the kernel above takes 87, 87 and
// 271 us; top 16 of 160 bf16 42 us against 225.
constexpr int kListThreads = 128;
constexpr int kListPitch = kListThreads + 1;  // of the rows of choices: neighbouring rows start on other banks

__device__ __forceinline__ uint32_t greater(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ uint32_t lesser(uint32_t a, uint32_t b) { return min(a, b); }
__device__ __forceinline__ float greater(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float lesser(float a, float b) { return fminf(a, b); }

template <typename K>
__device__ __forceinline__ void order_pair(K& hi, K& lo) {
    const K a = hi, b = lo;
    hi = greater(a, b);
    lo = lesser(a, b);
}

// Greatest first; a bitonic sequence.
template <typename K, int N>
__device__ __forceinline__ void sort_bitonic(K (&k)[N]) {
#pragma unroll
    for (int d = N / 2; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if ((i & d) == 0) order_pair(k[i], k[i + d]);
}

// Greatest first: odd-even merges of 1, 2 and 4 (19 pairs).
template <typename K>
__device__ __forceinline__ void sort8(K (&k)[8]) {
    order_pair(k[0], k[1]), order_pair(k[2], k[3]), order_pair(k[4], k[5]), order_pair(k[6], k[7]);
    order_pair(k[0], k[2]), order_pair(k[1], k[3]), order_pair(k[4], k[6]), order_pair(k[5], k[7]);
    order_pair(k[1], k[2]), order_pair(k[5], k[6]);
    order_pair(k[0], k[4]), order_pair(k[1], k[5]), order_pair(k[2], k[6]), order_pair(k[3], k[7]);
    order_pair(k[2], k[4]), order_pair(k[3], k[5]);
    order_pair(k[1], k[2]), order_pair(k[3], k[4]), order_pair(k[5], k[6]);
}

// The best N of a's N and b's M, both greatest first.
template <typename K, int N, int M>
__device__ __forceinline__ void merge_best(K (&a)[N], const K (&b)[M]) {
#pragma unroll
    for (int i = 0; i < M; ++i) a[N - M + i] = greater(a[N - M + i], b[M - 1 - i]);
    sort_bitonic(a);
}

// Eight values of a row from e on; those at or past the end are -inf.
template <typename T>
struct Eight {
    uint32_t w[8 * sizeof(T) / 4];
};

__device__ __forceinline__ uint32_t no_value(float) { return 0xff800000u; }
__device__ __forceinline__ uint32_t no_value(__nv_bfloat16) { return 0xff80u; }
__device__ __forceinline__ uint32_t no_value(__half) { return 0xfc00u; }

template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* row, int e, int end, bool aligned) {
    constexpr int W = 8 * (int)sizeof(T) / 4;
    Eight<T> x;
    if (aligned && e + 8 <= end) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 v = reinterpret_cast<const uint4*>(row + e)[i / 4];
            x.w[i] = v.x, x.w[i + 1] = v.y, x.w[i + 2] = v.z, x.w[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t bits = no_value(T{});
            if (e + i < end) {
                if (sizeof(T) == 4) bits = reinterpret_cast<const uint32_t*>(row)[e + i];
                else bits = reinterpret_cast<const unsigned short*>(row)[e + i];
            }
            if (sizeof(T) == 4) x.w[i] = bits;
            else x.w[i / 2] = i & 1 ? x.w[i / 2] | bits << 16 : bits;
        }
    }
    return x;
}

// Two values as they lie in memory, the first one low.
__device__ __forceinline__ uint32_t pair_of(float x, float y, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pair_of(float x, float y, __half) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight values written from e on, those before the end.
template <typename T>
__device__ __forceinline__ void store_eight(T* row, int e, int end, bool aligned, const float (&y)[8]) {
    if (aligned && e + 8 <= end) {
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4*>(row + e)[0] = make_float4(y[0], y[1], y[2], y[3]);
            reinterpret_cast<float4*>(row + e)[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
            *reinterpret_cast<uint4*>(row + e) = make_uint4(pair_of(y[0], y[1], T{}), pair_of(y[2], y[3], T{}),
                                                            pair_of(y[4], y[5], T{}), pair_of(y[6], y[7], T{}));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < end) row[e + i] = from_float<T>(y[i]);
    }
}

__device__ __forceinline__ float value_of(const Eight<float>& x, int i) { return __uint_as_float(x.w[i]); }
__device__ __forceinline__ float value_of(const Eight<__nv_bfloat16>& x, int i) {
    return __uint_as_float(i & 1 ? x.w[i / 2] & 0xffff0000u : x.w[i / 2] << 16);
}
__device__ __forceinline__ float value_of(const Eight<__half>& x, int i) {
    return __half2float(__ushort_as_half((unsigned short)(i & 1 ? x.w[i / 2] >> 16 : x.w[i / 2])));
}

// The logit behind a packed key.
template <typename T>
__device__ __forceinline__ float logit_of(uint32_t key, T) {
    const uint32_t image = key >> 16;
    Eight<T> one;
    one.w[0] = (image & 0x8000u ? image ^ 0x8000u : ~image) & 0xffffu;
    return key == 0 ? -INFINITY : value_of(one, 0);
}

// All ones in each half of w whose top bit is set.
__device__ __forceinline__ uint32_t half_signs(uint32_t w) {
    uint32_t m;
    asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(m) : "r"(w));
    return m;
}

// Two 16-bit values with NaN made -inf and -0 made +0.
__device__ __forceinline__ uint32_t plain_pair(uint32_t w, __nv_bfloat16) {
    __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&w);
    v = __hadd2(__hmax2(v, __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80))),
                __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)));
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t plain_pair(uint32_t w, __half) {
    __half2 v = *reinterpret_cast<__half2*>(&w);
    v = __hadd2(__hmax2(v, __halves2half2(__ushort_as_half(0xfc00), __ushort_as_half(0xfc00))),
                __halves2half2(__ushort_as_half(0), __ushort_as_half(0)));
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t plain_pair(uint32_t, float) { return 0; }  // not used

// The greater of each two 16-bit values; of a NaN and another, the other.
__device__ __forceinline__ uint32_t greater_pair(uint32_t a, uint32_t b, __nv_bfloat16) {
    const __nv_bfloat162 v = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t greater_pair(uint32_t a, uint32_t b, __half) {
    const __half2 v = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// e^(x - top) for a sum: one multiplication and the hardware's 2^x, terms below
// 2^-126 as zero.  What the rounding of the argument costs a term falls with the
// term itself.  For sums alone: as gradients the terms are taken by expf.
// x = -inf gives 0; top must be finite or +inf.
__device__ __forceinline__ float exp_term(float x, float top) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((x - top) * 1.4426950408889634f));
    return y;
}

// What the list is made of.
enum ListMode {
    kListPacked,   // 16-bit logits with their indices
    kListLogit,    // logits
    kListSoftmax,  // softmax scores, with a bias or summed over groups
    kListSigmoid   // sigmoid scores, likewise
};

template <typename T, int MODE, bool GROUPED, int L, int LIST>
__global__ void __launch_bounds__(kListThreads) route_list_kernel(RouteArgs a, bool aligned) {
    wait_for_stream();
    constexpr bool PACKED = MODE == kListPacked, BY_LOGIT = MODE <= kListLogit;
    using Key = typename std::conditional<PACKED, uint32_t, float>::type;
    constexpr unsigned kAll = 0xffffffffu;
    const float kNone = -INFINITY;
    extern __shared__ float4 s_choice[];       // [steps][2][kListPitch]: a lane's eights; [steps]: their greatest
    __shared__ int s_id[kListThreads / L][LIST];  // the picks of a token
    const int l = threadIdx.x & (L - 1), slot = threadIdx.x / L;
    const int64_t t = (int64_t)blockIdx.x * (kListThreads / L) + slot;
    const bool live = t < a.tokens;
    const T* row = static_cast<const T*>(a.logits) + (live ? t : a.tokens - 1) * a.row_stride;
    const int steps = (a.experts + 8 * L - 1) / (8 * L);
    const int share = a.experts / L, end = GROUPED ? (l + 1) * share : a.experts;
    auto first_of = [&](int step) { return GROUPED ? l * share + step * 8 : (step * L + l) * 8; };
    float* s_greatest = reinterpret_cast<float*>(s_choice + 2 * steps * kListPitch);

    // softmax over the row, where it is needed
    float top = kNone, sum = 1.0f;
    auto top_of_row = [&] {
        for (int step = 0; step < steps; ++step) {
            const Eight<T> x = load_eight(row, first_of(step), end, aligned);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, value_of(x, i));
        }
#pragma unroll
        for (int d = 1; d < L; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
    };
    auto sum_of_row = [&] {
        float part = 0.0f;
        for (int step = 0; step < steps; ++step) {
            const Eight<T> x = load_eight(row, first_of(step), end, aligned);
#pragma unroll
            for (int i = 0; i < 8; ++i) part += exp_term(fmaxf(value_of(x, i), kNone), top > kNone ? top : 0.0f);
        }
#pragma unroll
        for (int d = 1; d < L; d <<= 1) part += __shfl_xor_sync(kAll, part, d);
        sum = part;
    };
    float inverse = 1.0f;
    if (MODE == kListSoftmax) {
        top_of_row();
        sum_of_row();
        inverse = 1.0f / sum;
    }

    Key best[LIST];
#pragma unroll
    for (int i = 0; i < LIST; ++i) best[i] = PACKED ? Key(0) : Key(kNone);
    // what the eight experts from e on, with logits x, are chosen by; -inf where masked, and no -0
    auto choose = [&](const Eight<T>& x, int e, int end, float (&k)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = value_of(x, i);
            // scores to a few units in the last place: ordered as 32 bits can order them (the
            // hardware's 2^x alone, whose error grows with |v|, would take 7 % off the largest calls)
            if (MODE == kListSoftmax) k[i] = expf(v - top) * inverse;
            else if (MODE == kListSigmoid) k[i] = sigmoid_choice(v);
            else k[i] = v;
        }
        if (!BY_LOGIT && a.bias != nullptr) {
            const Eight<float> bias = load_eight(a.bias, e, end, ((uintptr_t)(a.bias + e) & 15) == 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) k[i] += value_of(bias, i);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[i] = fmaxf(k[i], kNone) + 0.0f;
            if (!BY_LOGIT && !(value_of(x, i) > kNone)) k[i] = kNone;
        }
    };
    auto keep_choices = [&](int step, int thread, const float (&k)[8]) {
        s_choice[2 * step * kListPitch + thread] = make_float4(k[0], k[1], k[2], k[3]);
        s_choice[(2 * step + 1) * kListPitch + thread] = make_float4(k[4], k[5], k[6], k[7]);
    };
    auto list = [&](int step, Key (&k)[8]) {
        sort8(k);
        if constexpr (!PACKED) s_greatest[step * kListThreads + threadIdx.x] = k[0];
        if (step > 0) {
            merge_best(best, k);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = k[i];
        }
    };
    if (GROUPED && !PACKED && sizeof(T) == 4 && share >= 32 && share % 8 == 0) {
        // The lanes' shares lie a line or more apart, so the row is read across the
        // lanes, and the choices handed to the lanes whose they are through shared
        // memory.  (Loads of their own shares touched 32 lines each and filled 72 %
        // of the load path: 131071 tokens of 256 f32 took 16 us more; shares of 16
        // f32 and of 32 bf16 gain nothing.)
        if constexpr (!PACKED) {
            const int own = share / 8;  // eights of a lane
            Eight<T> x = load_eight(row, l * 8, a.experts, aligned);
#pragma unroll 1
            for (int step = 0; step < own; ++step) {
                const int eight = step * L + l;
                Eight<T> next = x;
                if (step + 1 < own) next = load_eight(row, (eight + L) * 8, a.experts, aligned);
                float k[8];
                choose(x, eight * 8, a.experts, k);
                const int owner = eight / own;
                keep_choices(eight - owner * own, (int)threadIdx.x - l + owner, k);
                x = next;
            }
            __syncwarp();
#pragma unroll 1
            for (int step = 0; step < own; ++step) {
                const float4* two = s_choice + 2 * step * kListPitch + threadIdx.x;
                const float4 lo = two[0], hi = two[kListPitch];
                Key k[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                list(step, k);
            }
        }
    } else {
        // one step's load is on its way while the one before is sorted
        Eight<T> x = load_eight(row, first_of(0), end, aligned);
#pragma unroll 1
        for (int step = 0; step < steps; ++step) {
            const int e = first_of(step);
            Eight<T> next = x;
            if (step + 1 < steps) next = load_eight(row, first_of(step + 1), end, aligned);
            Key k[8];
            if constexpr (PACKED) {
                uint32_t index = (uint32_t)(0xffff - e) | (uint32_t)(0xffff - e - 1) << 16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = plain_pair(x.w[i], T{});
                    // negative values are complemented, others get the top bit
                    const uint32_t image = w ^ (half_signs(w) | 0x80008000u);
                    k[2 * i] = __byte_perm(index, image, 0x5410);
                    k[2 * i + 1] = __byte_perm(index, image, 0x7632);
                    index -= 0x00020002u;
                }
            } else {
                choose(x, e, end, k);
                keep_choices(step, threadIdx.x, k);
            }
            list(step, k);
            x = next;
        }
    }
    bool open = true;  // this lane's share may be chosen from
    if constexpr (GROUPED) {
        // L / groups neighbouring lanes hold a group
        const int wide = L / a.groups;
        float b0, b1;
        if constexpr (PACKED) b0 = logit_of(best[0], T{}), b1 = logit_of(best[1], T{});
        else b0 = best[0], b1 = best[1];
        for (int d = 1; d < wide; d <<= 1) {
            const float o0 = __shfl_xor_sync(kAll, b0, d), o1 = __shfl_xor_sync(kAll, b1, d);
            b1 = fmaxf(fminf(b0, o0), fmaxf(b1, o1));
            b0 = fmaxf(b0, o0);
        }
        const int group = l / wide;
        // an empty group is NaN: never picked, and ahead of no other, not even of a sum that overflows to -inf
        const float score = !(b0 > kNone) ? NAN : a.group_best == 2 && b1 > kNone ? b0 + b1 : b0;
        int ahead = b0 > kNone ? 0 : a.groups;  // groups that go first
        for (int g = 0; g < a.groups; ++g) {
            const float other = __shfl_sync(kAll, score, (threadIdx.x & 31 & ~(L - 1)) + g * wide);
            ahead += other > score || (other == score && g < group);
        }
        open = ahead < a.group_picks;
#pragma unroll
        for (int i = 0; i < LIST; ++i)
            if (!open) best[i] = PACKED ? Key(0) : Key(kNone);
    }
#pragma unroll 1
    for (int d = 1; d < L; d <<= 1) {
        Key other[LIST];
#pragma unroll
        for (int i = 0; i < LIST; ++i) other[i] = __shfl_xor_sync(kAll, best[i], d);
        merge_best(best, other);
    }

    if constexpr (!PACKED) {
        // the indices behind the list
        int valid = 0, twins = 0;  // listed values that are there; neighbours that are equal
        float least = -3.402823466e38f;
#pragma unroll
        for (int i = 0; i < LIST; ++i) {
            if (i < a.top_k && best[i] > kNone) ++valid, least = best[i];
            if (i > 0 && i < a.top_k && best[i] > kNone) twins += best[i] == best[i - 1];
        }
#pragma unroll
        for (int i = 0; i < LIST; i += L)
            if (l + i < LIST) s_id[slot][l + i] = -1;
        __syncwarp();
        uint32_t eights = 0;  // of this lane, that reach the least chosen value
        for (int step = 0; step < steps; ++step)
            if (open && s_greatest[step * kListThreads + threadIdx.x] >= least) eights |= 1u << step;
        int found = 0;
        for (uint32_t left = eights; left != 0; left &= left - 1) {
            const int step = __ffs(left) - 1;
            const float4* two = s_choice + 2 * step * kListPitch + threadIdx.x;
            const float4 lo = two[0], hi = two[kListPitch];
            const float c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint32_t chosen = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) chosen |= c[i] >= least ? 1u << i : 0u;
            found += __popc(chosen);
            for (; chosen != 0; chosen &= chosen - 1) {
                const int i = __ffs(chosen) - 1;
                const float mine = reinterpret_cast<const float*>(two + (i >> 2) * kListPitch)[i & 3];
                int place = 0;
#pragma unroll
                for (int j = 0; j < LIST; ++j) place += best[j] > mine;
                s_id[slot][place & (LIST - 1)] = first_of(step) + i;
            }
        }
        __syncwarp();
#pragma unroll
        for (int d = 1; d < L; d <<= 1) found += __shfl_xor_sync(kAll, found, d);
        const bool unsettled = twins > 0 || found > valid;
        if (__any_sync(kAll, unsettled)) {
            // place by place: the lowest index of the place's value, above the one before if that had the same
            int before = -1;
            float last = INFINITY;
#pragma unroll 1
            for (int j = 0; j < LIST; ++j) {
                float v = kNone;
#pragma unroll
                for (int i = 0; i < LIST; ++i)
                    if (i == j) v = best[i];
                if (v != last) before = -1;
                int lowest = 0x7fffffff;
                if (unsettled && j < valid) {
                    for (uint32_t left = eights; left != 0; left &= left - 1) {
                        const int step = __ffs(left) - 1, e = first_of(step);
                        const float4* two = s_choice + 2 * step * kListPitch + threadIdx.x;
                        const float4 lo = two[0], hi = two[kListPitch];
                        const float c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (e + i > before && c[i] == v) lowest = min(lowest, e + i);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int d = 1; d < L; d <<= 1) lowest = min(lowest, __shfl_xor_sync(kAll, lowest, d));
                if (unsettled && j < valid && l == 0) s_id[slot][j] = lowest;
                before = lowest;
                last = v;
            }
            __syncwarp();
        }
    }

    // lane l finishes the picks l * P ..
    constexpr int P = L < LIST ? LIST / L : 1;
    int id[P];
    float px[P], w[P];
    float head = kNone;  // the picks' greatest logit
#pragma unroll
    for (int p = 0; p < P; ++p) {
        bool there = l * P + p < a.top_k;
        if constexpr (PACKED) {
            Key k = 0;
#pragma unroll
            for (int i = 0; i < LIST / P; ++i)
                if (l == i) k = best[i * P + p];
            px[p] = logit_of(k, T{});
            there = there && px[p] > kNone;
            id[p] = there ? (int)(0xffffu - (k & 0xffffu)) : -1;
        } else {
            id[p] = there ? s_id[slot][l * P + p] : -1;
            there = id[p] >= 0;
            px[p] = there ? to_float(row[id[p]]) : kNone;
        }
        if (!there) px[p] = kNone;
        head = fmaxf(head, px[p]);
        w[p] = 0.0f;
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) head = fmaxf(head, __shfl_xor_sync(kAll, head, d));
    if (a.renorm) {
        float total = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (id[p] >= 0)
                w[p] = a.score == OM_SCORE_SOFTMAX ? expf(px[p] - head) : shifted_sigmoid(px[p], fminf(head, 0.0f));
            total += w[p];
        }
#pragma unroll
        for (int d = 1; d < L; d <<= 1) total += __shfl_xor_sync(kAll, total, d);
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (id[p] >= 0) w[p] = w[p] / total;
    } else {
        if (a.score == OM_SCORE_SOFTMAX && BY_LOGIT) {
            top = head;  // without groups the first pick is the row's greatest logit
            if (GROUPED) top_of_row();
            sum_of_row();
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (id[p] >= 0) w[p] = a.score == OM_SCORE_SOFTMAX ? expf(px[p] - top) / sum : sigmoid(px[p]);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
        if (live && l * P + p < a.top_k) {
            a.ids[t * a.top_k + l * P + p] = id[p];
            a.weights[t * a.top_k + l * P + p] = w[p] * a.scale;
        }
    }
}

constexpr int kBackHeld = 4;  // steps of eight logits that a lane keeps

struct RouteBackArgs {
    const void* logits;
    int64_t tokens;
    int64_t row_stride;
    const int32_t* ids;
    const float* grad_weights;
    void* grad_logits;
    int experts, score, top_k, renorm;
    float scale;
};

// L lanes per token, at least as many as it has picks: lane l has the l-th.
// Only a softmax that is not renormalised (DENSE) reads the whole row, once,
// and keeps the terms of its sum in registers until they are written, times
// -dot / sum.  Elsewhere the row's zeros are written while the picks' logits
// arrive.  Rows go out in 16-byte vectors where they are aligned, and the picks
// over them, each by its own lane.
//
// Bound by issue for large batches of DENSE: its terms are gradients, so they
// are taken by expf, to its last places and through the subnormal range (2 us
// more than the hardware's 2^x alone, of which packed maxima and register pairs
// give half back); the picked logits cost a sector each.  Measured, cold: 65536
// tokens of 160 bf16, softmax, 13.4 us (45 MB); 4099 tokens of 256 f32,
// renormalised sigmoid, 4.4 us (4.6 MB), of which 2.2 are those of a single
// token.
template <typename T, bool DENSE, int L>
__global__ void __launch_bounds__(128) route_topk_backward_kernel(RouteBackArgs a, bool aligned_in, bool aligned_out) {
    wait_for_stream();
    constexpr unsigned kAll = 0xffffffffu;
    const float kNone = -INFINITY;
    const int l = threadIdx.x & (L - 1);
    const int64_t t = ((int64_t)blockIdx.x * 128 + threadIdx.x) / L;
    const bool live = t < a.tokens;
    const int64_t at = live ? t : a.tokens - 1;
    const T* row = static_cast<const T*>(a.logits) + at * a.row_stride;
    T* grad = static_cast<T*>(a.grad_logits) + at * a.experts;
    const int steps = (a.experts + 8 * L - 1) / (8 * L);
    auto reduce_max = [&](float x) {
#pragma unroll
        for (int d = 1; d < L; d <<= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
        return x;
    };
    auto reduce_sum = [&](float x) {
#pragma unroll
        for (int d = 1; d < L; d <<= 1) x += __shfl_xor_sync(kAll, x, d);
        return x;
    };
    // this lane's pick and its part of the row: all on their way at once
    int id = -1;
    float g = 0.0f;
    if (l < a.top_k) {
        id = a.ids[at * a.top_k + l];
        g = a.grad_weights[at * a.top_k + l] * a.scale;
    }
    constexpr int H = DENSE ? kBackHeld : 1;
    Eight<T> x[H];
    if (DENSE) {
#pragma unroll
        for (int step = 0; step < H; ++step)
            if (step < steps) x[step] = load_eight(row, (step * L + l) * 8, a.experts, aligned_in);
    } else if (live) {
        const float zero[8] = {};
        for (int step = 0; step < steps; ++step) store_eight(grad, (step * L + l) * 8, a.experts, aligned_out, zero);
    }
    float px = kNone;
    if (id >= 0 && id < a.experts) px = to_float(row[id]);
    const bool there = px > kNone;  // a masked one was no pick of the forward call
    if (!there) g = 0.0f;

    float top = kNone, inverse = 1.0f;
    uint64_t y[H][4];  // the terms e^(x - top), two to a register pair
    if (DENSE) {
        // NaN to -inf, and the greatest
        uint32_t most = 0xffffffffu;  // of 16-bit values, two at a time; a pair of NaN
#pragma unroll
        for (int step = 0; step < H; ++step)
            if (step < steps) {
#pragma unroll
                for (int i = 0; i < 8 * (int)sizeof(T) / 4; ++i) {
                    uint32_t& w = x[step].w[i];
                    if constexpr (sizeof(T) == 4) {
                        w = __float_as_uint(fmaxf(__uint_as_float(w), kNone));
                        top = fmaxf(top, __uint_as_float(w));
                    } else {
                        w = greater_pair(w, no_value(T{}) * 0x10001u, T{});
                        most = greater_pair(most, w, T{});
                    }
                }
            }
        if constexpr (sizeof(T) == 2) {
            Eight<T> two;
            two.w[0] = most;
            top = fmaxf(value_of(two, 0), value_of(two, 1));
        }
        top = reduce_max(top);
        if (!(top > kNone)) top = 0.0f;  // nothing is there
        const uint64_t less = pack2(-top, -top);
        uint64_t part = 0;
#pragma unroll
        for (int step = 0; step < H; ++step)
            if (step < steps) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint64_t d = pack2(value_of(x[step], 2 * i), value_of(x[step], 2 * i + 1));
                    add2(d, less);
                    const float2 f = unpack2(d);
                    y[step][i] = pack2(expf(f.x), expf(f.y));
                    add2(part, y[step][i]);
                }
            }
        const float2 sums = unpack2(part);
        const float sum = reduce_sum(sums.x + sums.y);
        inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
    }
    // w: the pick's weight before scale
    float w = 0.0f, dot = 0.0f;
    if (a.renorm) {
        const float best = reduce_max(px);
        if (there) w = a.score == OM_SCORE_SOFTMAX ? expf(px - best) : shifted_sigmoid(px, fminf(best, 0.0f));
        const float total = reduce_sum(w);
        if (there) w = w / total;
    } else if (there) {
        w = DENSE ? expf(px - top) * inverse : sigmoid(px);
    }
    if (DENSE || a.renorm) dot = reduce_sum(g * w);
    if (DENSE) {
        const float every = -dot * inverse;
        const uint64_t both = pack2(every, every);
#pragma unroll
        for (int step = 0; step < H; ++step)
            if (step < steps) {
                float out[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2(mul2(y[step][i], both));
                    out[2 * i] = f.x, out[2 * i + 1] = f.y;
                }
                if (live) store_eight(grad, (step * L + l) * 8, a.experts, aligned_out, out);
            }
    }
    __syncwarp();  // the picks are written over what another lane may have written
    if (live && there) {
        float v = w * (g - dot);  // dot is 0 for a plain sigmoid
        if (a.score == OM_SCORE_SIGMOID) v *= sigmoid(-px);
        grad[id] = from_float<T>(v);
    }
}

// Calls f with the number of experts per lane as a constant.
template <typename F>
static cudaError_t with_lane_experts(int experts, F&& f) {
    if (experts <= 32) return f(std::integral_constant<int, 1>{});
    if (experts <= 64) return f(std::integral_constant<int, 2>{});
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    if (experts <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

template <typename T, int MODE, bool GROUPED, int L, int LIST>
static cudaError_t launch_list_lanes(const RouteArgs& a, bool aligned, cudaStream_t st) {
    const int64_t blocks = (a.tokens + kListThreads / L - 1) / (kListThreads / L);
    const int steps = (a.experts + 8 * L - 1) / (8 * L);
    const size_t smem =
        MODE == kListPacked ? 0 : (size_t)steps * (2 * kListPitch * sizeof(float4) + kListThreads * sizeof(float));
    return counted([&] {
        launch_early(route_list_kernel<T, MODE, GROUPED, L, LIST>, (unsigned)blocks, kListThreads, smem, st, a,
                     aligned);
    });
}

// A token gets 32 lanes (PACKED: 16) while that gives an SM at most this many
// threads (2432 tokens): the shorter chain wins until the SMs are busy.  2048
// biased sigmoid tokens in 8 groups of 32 experts: 5.7 us against 6.9 with
// 8 lanes each; 4096: 7.9 against 7.8; 131071: 147 against 74.
constexpr int kListFewThreads = 512;
// The most experts that 4 (grouped: twice as many for 8) lanes take, whose
// choices then fill 37 KB of shared memory; not for PACKED, which keeps none.
constexpr int kListMaxExperts = 256;

template <typename T, int MODE>
static cudaError_t launch_list_mode(const RouteArgs& a, bool aligned, bool few, cudaStream_t st) {
    constexpr int kMore = MODE == kListPacked ? 16 : 32;
    if (a.top_k > 8)
        return a.groups == 1 ? launch_list_lanes<T, MODE, false, 8, 16>(a, aligned, st)
                             : launch_list_lanes<T, MODE, true, 8, 16>(a, aligned, st);
    if (a.groups == 1)
        return few ? launch_list_lanes<T, MODE, false, kMore, 8>(a, aligned, st)
                   : launch_list_lanes<T, MODE, false, 4, 8>(a, aligned, st);
    return few ? launch_list_lanes<T, MODE, true, 32, 8>(a, aligned, st)
               : launch_list_lanes<T, MODE, true, 8, 8>(a, aligned, st);
}

template <typename T>
static cudaError_t launch_list(const RouteArgs& a, bool aligned, bool few, cudaStream_t st) {
    const bool by_logit = a.bias == nullptr && (a.groups == 1 || a.group_best == 1);
    if constexpr (sizeof(T) == 2) {
        if (by_logit) return launch_list_mode<T, kListPacked>(a, aligned, few, st);
    } else {
        if (by_logit) return launch_list_mode<T, kListLogit>(a, aligned, few, st);
    }
    if (a.score == OM_SCORE_SOFTMAX) return launch_list_mode<T, kListSoftmax>(a, aligned, few, st);
    return launch_list_mode<T, kListSigmoid>(a, aligned, few, st);
}

template <typename T, bool DENSE, int L>
static void launch_back_lanes(const RouteBackArgs& a, bool in, bool out, cudaStream_t st) {
    const unsigned blocks = (unsigned)((a.tokens * L + 127) / 128);
    launch_early(route_topk_backward_kernel<T, DENSE, L>, blocks, 128, 0, st, a, in, out);
}

// 8 lanes a token, or 32: where there are more picks than 8, and in DENSE where
// the row fits the registers of 32 lanes only (65536 tokens of 257 f32: 49 us) or
// the tokens are few (`few`; 512 of 160 bf16: 3.2 us against 3.4, 4099: 3.8 against
// 3.7, 65536: 31 against 13.4).
template <typename T, bool DENSE>
static void launch_back(const RouteBackArgs& a, bool in, bool out, bool few, cudaStream_t st) {
    constexpr int kHeld8 = 8 * 8 * kBackHeld, kHeld32 = 8 * 32 * kBackHeld;
    static_assert(kHeld32 >= kMaxExperts, "32 lanes hold every row");
    if (a.top_k > 8 || (DENSE && (few || a.experts > kHeld8))) launch_back_lanes<T, DENSE, 32>(a, in, out, st);
    else launch_back_lanes<T, DENSE, 8>(a, in, out, st);
}

static unsigned route_grid(int64_t tokens) {
    const int64_t blocks = (tokens + kRouteWarps - 1) / kRouteWarps;
    return (unsigned)(blocks < (1 << 20) ? blocks : (1 << 20));
}

// Checks shared by both directions.
static om_status route_check(int value_type, const void* logits, int64_t tokens, int64_t experts, int64_t row_stride,
                             int score, int top_k) {
    const int vb = value_bytes(value_type);
    if (vb == 0 || (score != OM_SCORE_SOFTMAX && score != OM_SCORE_SIGMOID)) return OM_EINVAL;
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts) return OM_EINVAL;
    if (experts > kMaxExperts || top_k > kMaxTopK) return OM_ERANGE;
    if (tokens > 1 && row_stride < 0) return OM_EINVAL;
    // grids stay below 2^31 CTAs, and the rows' span below 2^60 bytes
    if (tokens > ((int64_t)1 << 32) || (row_stride > 0 && tokens > ((int64_t)1 << 58) / row_stride)) return OM_ERANGE;
    if (tokens > 0 && (logits == nullptr || misaligned(logits, vb))) return OM_EINVAL;
    return OM_OK;
}

}  // namespace om

using namespace om;

extern "C" {

om_status om_route_topk(int value_type, const void* logits, int64_t tokens, int64_t experts, int64_t row_stride,
                        const float* bias, int score, int groups, int group_picks, int group_best, int top_k,
                        int renorm, float scale, int32_t* ids, float* weights, void* stream) {
    const om_status s = route_check(value_type, logits, tokens, experts, row_stride, score, top_k);
    if (s != OM_OK) return s;
    if (groups < 1 || experts % groups != 0 || group_picks < 1 || group_picks > groups ||
        (group_best != 1 && group_best != 2) || top_k > group_picks * (experts / groups))
        return OM_EINVAL;
    if (groups > kMaxExpertGroups) return OM_ERANGE;
    if (tokens == 0) return OM_OK;
    if (ids == nullptr || weights == nullptr || misaligned4(bias) || misaligned4(ids) || misaligned4(weights))
        return OM_EINVAL;
    const int vb = value_bytes(value_type);
    const int64_t span = ((tokens - 1) * row_stride + experts) * vb, out = tokens * top_k * 4;
    if (overlaps(ids, out, weights, out, 1)) return OM_EINVAL;
    for (const void* o : {(const void*)ids, (const void*)weights})
        if (overlaps(o, out, logits, span, 1) || (bias && overlaps(o, out, bias, experts * 4, 1))) return OM_EINVAL;
    RouteArgs a{logits, tokens, row_stride, bias, ids, weights, (int)experts, score, groups, group_picks, group_best,
                top_k, renorm != 0, scale};
    cudaStream_t st = (cudaStream_t)stream;
    DeviceState* d = nullptr;
    const om_status ds = device_state(&d);
    if (ds != OM_OK) return ds;
    const bool packed = vb == 2 && bias == nullptr && (groups == 1 || group_best == 1);
    // grouped: a lane's share of a row has to lie in one group
    auto fits = [&](int lanes) { return groups == 1 || (lanes % groups == 0 && experts % lanes == 0); };
    const bool room = packed || experts <= kListMaxExperts * (groups == 1 && top_k <= 8 ? 1 : 2);  // for 4 or 8 lanes
    const bool some = tokens * 32 <= d->sm_count * (int64_t)kListFewThreads;
    bool listed, few = false;
    if (top_k <= 8) {
        few = some || !room;
        // the other number of lanes where only that one fits: still half the time of a warp reduction per pick
        if (!fits(few ? 32 : 8) && fits(few ? 8 : 32) && (!few || room)) few = !few;
        listed = fits(few ? 32 : 8);
    } else {
        // 8 lanes and lists of 16; a few tokens' f32 logits are as well off with a warp each (512 of 128, top 10:
        // 3.7 us against 4.9; of 256 with bias, top 12: 10.7 against 8.1; 131071 of 160 bf16, top 16: 225 against 42)
        listed = top_k <= 16 && room && fits(8) && !(some && vb == 4 && bias == nullptr && groups == 1);
    }
    if (listed) {
        const int lanes = few ? 32 : 8;
        bool aligned = !misaligned(logits, 16) && (tokens == 1 || row_stride * vb % 16 == 0);
        if (groups > 1) aligned = aligned && experts / lanes * vb % 16 == 0;
        const cudaError_t e = with_value_type(value_type, [&](auto v) {
            return launch_list<decltype(v)>(a, aligned, few, st);
        });
        return e == cudaSuccess ? OM_OK : cuda_fail(e);
    }
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        return with_lane_experts((int)experts, [&](auto r) {
            return counted([&] {
                launch_early(route_topk_kernel<decltype(v), decltype(r)::value>, route_grid(tokens), kRouteWarps * 32, 0, st, a);
            });
        });
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_route_topk_backward(int value_type, const void* logits, int64_t tokens, int64_t experts,
                                 int64_t row_stride, const int32_t* ids, const float* grad_weights, int score,
                                 int top_k, int renorm, float scale, void* grad_logits, void* stream) {
    const om_status s = route_check(value_type, logits, tokens, experts, row_stride, score, top_k);
    if (s != OM_OK) return s;
    if (tokens == 0) return OM_OK;
    const int vb = value_bytes(value_type);
    if (ids == nullptr || grad_weights == nullptr || grad_logits == nullptr || misaligned4(ids) ||
        misaligned4(grad_weights) || misaligned(grad_logits, vb))
        return OM_EINVAL;
    const int64_t span = ((tokens - 1) * row_stride + experts) * vb, out = tokens * experts * vb;
    if (overlaps(grad_logits, out, logits, span, 1) || overlaps(grad_logits, out, ids, tokens * top_k * 4, 1) ||
        overlaps(grad_logits, out, grad_weights, tokens * top_k * 4, 1))
        return OM_EINVAL;
    RouteBackArgs a{logits, tokens, row_stride, ids, grad_weights, grad_logits, (int)experts, score, top_k,
                    renorm != 0, scale};
    cudaStream_t st = (cudaStream_t)stream;
    const bool aligned_in = !misaligned(logits, 16) && (tokens == 1 || row_stride * vb % 16 == 0);
    const bool aligned_out = !misaligned(grad_logits, 16) && (tokens == 1 || experts * vb % 16 == 0);
    const bool dense = score == OM_SCORE_SOFTMAX && !renorm;
    DeviceState* d = nullptr;
    const om_status ds = device_state(&d);
    if (ds != OM_OK) return ds;
    const bool few = tokens * 32 <= d->sm_count * (int64_t)kListFewThreads;
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        using T = decltype(v);
        return counted([&] {
            if (dense) launch_back<T, true>(a, aligned_in, aligned_out, few, st);
            else launch_back<T, false>(a, aligned_in, aligned_out, few, st);
        });
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

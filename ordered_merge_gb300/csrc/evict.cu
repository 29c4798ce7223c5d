// om_accumulate_weights / om_evict_select / om_evict_gather: eviction from a
// cache by accumulated attention weight.
#include <cstdint>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "select_common.cuh"

namespace om {

// ------------------------------------------------- accumulated weights --

struct AccumulateArgs {
    const void* weights;
    const float* score;
    const int32_t* lengths;
    float* out;
    int64_t w_batch, w_head, w_query, s_batch, s_head, o_batch, o_head;
    int64_t length;
    int kv_heads, share, queries;
    float decay;
};

__device__ __forceinline__ int64_t valid_length(const int32_t* lengths, int64_t b, int64_t length) {
    if (lengths == nullptr) return length;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < length ? n : length;
}

// One thread per cache entry.
template <typename T>
__global__ void __launch_bounds__(256) accumulate_weights_kernel(AccumulateArgs a) {
    const int64_t b = blockIdx.y / a.kv_heads, h = blockIdx.y % a.kv_heads;
    const int64_t n = valid_length(a.lengths, b, a.length);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.length) return;
    float total = 0.0f;
    if (i < n) {
        const T* w = static_cast<const T*>(a.weights) + b * a.w_batch + h * a.share * a.w_head + i;
        for (int g = 0; g < a.share; ++g)
            for (int q = 0; q < a.queries; ++q) total += to_float(w[g * a.w_head + q * a.w_query]);
        if (a.score != nullptr) total += a.decay * a.score[b * a.s_batch + h * a.s_head + i];
    }
    a.out[b * a.o_batch + h * a.o_head + i] = total;
}

// ------------------------------------------------------------ selection --

struct EvictArgs {
    const float* score;
    const int32_t* lengths;
    int32_t* keep;
    int32_t* kept;
    int64_t s_batch, s_head;
    int length, heads, budget, first, last;
};

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kDigitBits = 11;
constexpr int kDigits = 1 << kDigitBits;

// A NaN score counts as -inf: it goes first.
__device__ __forceinline__ uint32_t evict_key(float s) { return score_image(s == s ? s : -INFINITY); }

// Sum of `mine` over the threads before, and over all of them.
__device__ __forceinline__ int block_scan(int mine, int* s_part, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += up;
    }
    __syncthreads();
    if (lane == 31) s_part[warp] = run;
    __syncthreads();
    int w = s_part[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += up;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + run - mine;
}

// One CTA per row (sequence and head).  The least key that stays is found
// digit by digit from the top (11 + 11 + 10 bits): a histogram of the keys
// that agree with the digits found so far gives the next one.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(EvictArgs a) {
    __shared__ int s_hist[kDigits];
    __shared__ int s_part[32];
    __shared__ int s_digit, s_above;
    const int64_t b = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
    const float* score = a.score + b * a.s_batch + h * a.s_head;
    int32_t* keep = a.keep + (int64_t)blockIdx.x * a.budget;
    const int n = (int)valid_length(a.lengths, b, a.length);
    if (h == 0 && threadIdx.x == 0) a.kept[b] = min(n, a.budget);
    if (n <= a.budget) {
        for (int i = threadIdx.x; i < a.budget; i += kSelectThreads) keep[i] = i < n ? i : -1;
        return;
    }
    const int lo = a.first, hi = n - a.last;
    int need = a.budget - a.first - a.last;  // still to be chosen among those that agree with `prefix`
    uint32_t prefix = 0, mask = 0;
    if (need > 0) {
        for (int shift = 21; shift >= -1; shift -= kDigitBits) {
            const int down = shift < 0 ? 0 : shift;
            const uint32_t digits = shift < 0 ? kDigits / 2 - 1 : kDigits - 1;
            for (int i = threadIdx.x; i < kDigits; i += kSelectThreads) s_hist[i] = 0;
            __syncthreads();
            for (int i = lo + threadIdx.x; i < hi; i += kSelectThreads) {
                const uint32_t k = evict_key(score[i]);
                if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> down) & digits], 1);
            }
            __syncthreads();
            // two digits a thread, from the greatest down
            const int top = kDigits - 1 - 2 * threadIdx.x;
            const int c0 = s_hist[top], c1 = s_hist[top - 1];
            int total;
            const int above = block_scan(c0 + c1, s_part, &total);
            if (above < need && need <= above + c0) s_digit = top, s_above = above;
            if (above + c0 < need && need <= above + c0 + c1) s_digit = top - 1, s_above = above + c0;
            __syncthreads();
            prefix |= (uint32_t)s_digit << down;
            mask |= digits << down;
            need -= s_above;
        }
    }
    // in order: the first ones, those above the least key, the first `need` equal to it, the last ones
    int done = 0, ties = 0;
    const bool any = a.budget > a.first + a.last;
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + threadIdx.x;
        bool sure = false, tie = false;
        if (i < n) {
            if (i < lo || i >= hi) {
                sure = true;
            } else if (any) {
                const uint32_t k = evict_key(score[i]);
                sure = k > prefix;
                tie = k == prefix;
            }
        }
        int all;
        const int tied = ties + block_scan(tie, s_part, &all);
        const bool stays = sure || (tie && tied < need);
        ties += all;
        const int at = done + block_scan(stays, s_part, &all);
        if (stays) keep[at] = i;
        done += all;
    }
}

// --------------------------------------------------------------- gather --

constexpr int kMaxArrays = 8;

struct GatherArgs {
    om_cache_array arrays[kMaxArrays];
    const int32_t* keep;
    int64_t slots;  // batch * heads * budget
    int64_t budget, length;
    int heads;
};

// One thread per vector of a kept entry.
template <typename V>
__device__ void gather_array(const GatherArgs& a, const om_cache_array& c) {
    const int per = (int)(c.entry_bytes / (int)sizeof(V));
    const int64_t total = a.slots * per, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t slot = i / per, piece = i % per, row = slot / a.budget, j = slot % a.budget;
        const int64_t b = row / a.heads, h = row % a.heads;
        const int32_t from = a.keep[slot];
        V v{};
        if (from >= 0 && from < a.length)
            v = *reinterpret_cast<const V*>(static_cast<const char*>(c.src) + b * c.src_batch + h * c.src_head +
                                            from * c.src_entry + piece * (int64_t)sizeof(V));
        *reinterpret_cast<V*>(static_cast<char*>(c.dst) + b * c.dst_batch + h * c.dst_head + j * c.dst_entry +
                              piece * (int64_t)sizeof(V)) = v;
    }
}

__global__ void __launch_bounds__(256) evict_gather_kernel(GatherArgs a) {
    const om_cache_array& c = a.arrays[blockIdx.y];
    const uint64_t low = reinterpret_cast<uintptr_t>(c.src) | reinterpret_cast<uintptr_t>(c.dst) |
                         (uint64_t)c.src_batch | (uint64_t)c.src_head | (uint64_t)c.src_entry |
                         (uint64_t)c.dst_batch | (uint64_t)c.dst_head | (uint64_t)c.dst_entry |
                         (uint64_t)c.entry_bytes;
    if ((low & 15) == 0) gather_array<uint4>(a, c);
    else if ((low & 3) == 0) gather_array<uint32_t>(a, c);
    else if ((low & 1) == 0) gather_array<uint16_t>(a, c);
    else gather_array<uint8_t>(a, c);
}

// Largest strides taken, so that no span of an array overflows 64 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxEntryStride = (int64_t)1 << 30;

// Bytes from the first to past the last of a strided array, or -1 when its
// entries share bytes (which an output's must not).
static int64_t strided_span(int64_t bytes, const int64_t (&count)[3], const int64_t (&stride)[3], bool* shared) {
    int64_t c[3] = {count[0], count[1], count[2]}, s[3] = {stride[0], stride[1], stride[2]};
    for (int i = 0; i < 3; ++i)  // least stride first
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                const int64_t ts = s[i], tc = c[i];
                s[i] = s[j], c[i] = c[j], s[j] = ts, c[j] = tc;
            }
    int64_t span = bytes;
    *shared = false;
    for (int i = 0; i < 3; ++i)
        if (c[i] > 1) {
            if (s[i] < span) *shared = true;
            span += s[i] * (c[i] - 1);
        }
    return span;
}

}  // namespace om

using namespace om;

extern "C" {

om_status om_accumulate_weights(int value_type, const void* weights, int64_t batch, int64_t q_heads, int64_t kv_heads,
                                int64_t queries, int64_t length, int64_t w_batch, int64_t w_head, int64_t w_query,
                                const float* score, int64_t s_batch, int64_t s_head, const int32_t* lengths,
                                float decay, float* out, int64_t o_batch, int64_t o_head, void* stream) {
    const int vb = value_bytes(value_type);
    if (vb == 0 || batch < 0 || kv_heads < 1 || q_heads < 1 || q_heads % kv_heads != 0 || queries < 0 || length < 0)
        return OM_EINVAL;
    for (const int64_t s : {w_batch, w_head, w_query, s_batch, s_head, o_batch, o_head})
        if (s < 0) return OM_EINVAL;
    if (length > INT32_MAX || queries > 65535 || q_heads > 65535 || batch > 65535 || batch * kv_heads > 65535)
        return OM_ERANGE;
    for (const int64_t s : {w_batch, w_head, w_query, s_batch, s_head, o_batch, o_head})
        if (s > kMaxStride) return OM_ERANGE;
    if (batch == 0 || length == 0) return OM_OK;
    if (out == nullptr || (queries > 0 && weights == nullptr) || misaligned(weights, vb) || misaligned4(score) ||
        misaligned4(lengths) || misaligned4(out))
        return OM_EINVAL;
    bool shared = false;
    const int64_t o_span = strided_span(length * 4, {batch, kv_heads, 1}, {o_batch * 4, o_head * 4, 0}, &shared);
    if (shared) return OM_EINVAL;
    const int64_t w_span = ((batch - 1) * w_batch + (q_heads - 1) * w_head + (queries - 1) * w_query + length) * vb;
    if (queries > 0 && overlaps(out, o_span, weights, w_span, 1)) return OM_EINVAL;
    if (lengths != nullptr && overlaps(out, o_span, lengths, batch * 4, 1)) return OM_EINVAL;
    if (score != nullptr && !(score == out && s_batch == o_batch && s_head == o_head) &&
        overlaps(out, o_span, score, ((batch - 1) * s_batch + (kv_heads - 1) * s_head + length) * 4, 1))
        return OM_EINVAL;
    AccumulateArgs a{weights, score, lengths, out,    w_batch, w_head,        w_query, s_batch, s_head, o_batch, o_head,
                     length,  (int)kv_heads, (int)(q_heads / kv_heads), (int)queries, decay};
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid((unsigned)((length + 255) / 256), (unsigned)(batch * kv_heads));
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        return traced(kKindEvict, st, [&] { accumulate_weights_kernel<decltype(v)><<<grid, 256, 0, st>>>(a); });
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_evict_select(const float* score, int64_t batch, int64_t heads, int64_t length, int64_t s_batch,
                          int64_t s_head, const int32_t* lengths, int64_t budget, int64_t first, int64_t last,
                          int32_t* keep, int32_t* kept, void* stream) {
    if (batch < 0 || heads < 1 || length < 0 || s_batch < 0 || s_head < 0 || budget < 1 || first < 0 || last < 0)
        return OM_EINVAL;
    if (first > budget || last > budget - first) return OM_EINVAL;
    if (length > INT32_MAX - 65536 || budget > INT32_MAX - 65536 || heads > 65535 || batch > 32767 ||
        s_batch > kMaxStride || s_head > kMaxStride)
        return OM_ERANGE;
    if (batch == 0) return OM_OK;
    if (keep == nullptr || kept == nullptr || (length > 0 && score == nullptr) || misaligned4(score) ||
        misaligned4(lengths) || misaligned4(keep) || misaligned4(kept))
        return OM_EINVAL;
    const int64_t span = (batch - 1) * s_batch + (heads - 1) * s_head + length, slots = batch * heads * budget;
    if (overlaps(keep, slots, kept, batch)) return OM_EINVAL;
    if (overlaps(keep, slots, score, span) || overlaps(kept, batch, score, span)) return OM_EINVAL;
    if (lengths != nullptr && (overlaps(keep, slots, lengths, batch) || overlaps(kept, batch, lengths, batch)))
        return OM_EINVAL;
    EvictArgs a{score, lengths, keep, kept, s_batch, s_head, (int)length, (int)heads, (int)budget, (int)first, (int)last};
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = traced(kKindEvict, st, [&] {
        evict_select_kernel<<<(unsigned)(batch * heads), kSelectThreads, 0, st>>>(a);
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_evict_gather(const int32_t* keep, int64_t batch, int64_t heads, int64_t budget, int64_t length,
                          const om_cache_array* arrays, int count, void* stream) {
    if (batch < 0 || heads < 1 || budget < 1 || length < 0 || count < 1 || arrays == nullptr) return OM_EINVAL;
    if (length > INT32_MAX || budget > INT32_MAX || heads > 65535 || batch > 32767 || count > kMaxArrays)
        return OM_ERANGE;
    if (batch == 0) return OM_OK;
    if (keep == nullptr || misaligned4(keep)) return OM_EINVAL;
    GatherArgs a{};
    const int64_t slots = batch * heads * budget;
    int64_t spans[kMaxArrays], src_spans[kMaxArrays];
    for (int i = 0; i < count; ++i) {
        const om_cache_array& c = arrays[i];
        if (c.entry_bytes < 1 || c.dst == nullptr || (length > 0 && c.src == nullptr)) return OM_EINVAL;
        if (c.entry_bytes > (1 << 24)) return OM_ERANGE;
        for (const int64_t s : {c.src_batch, c.src_head, c.src_entry, c.dst_batch, c.dst_head, c.dst_entry})
            if (s < 0) return OM_EINVAL;
        if (c.src_batch > kMaxStride || c.src_head > kMaxStride || c.dst_batch > kMaxStride ||
            c.dst_head > kMaxStride || c.src_entry > kMaxEntryStride || c.dst_entry > kMaxEntryStride)
            return OM_ERANGE;
        bool shared = false, ignored = false;
        spans[i] = strided_span(c.entry_bytes, {batch, heads, budget}, {c.dst_batch, c.dst_head, c.dst_entry}, &shared);
        if (shared) return OM_EINVAL;
        src_spans[i] = length > 0 ? strided_span(c.entry_bytes, {batch, heads, length},
                                                 {c.src_batch, c.src_head, c.src_entry}, &ignored)
                                  : 0;
        if (overlaps(c.dst, spans[i], keep, slots * 4, 1)) return OM_EINVAL;
        a.arrays[i] = c;
    }
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j)
            if (overlaps(a.arrays[i].dst, spans[i], a.arrays[j].src, src_spans[j], 1) ||
                (i < j && overlaps(a.arrays[i].dst, spans[i], a.arrays[j].dst, spans[j], 1)))
                return OM_EINVAL;
    a.keep = keep;
    a.slots = slots;
    a.budget = budget;
    a.length = length;
    a.heads = (int)heads;
    cudaStream_t st = (cudaStream_t)stream;
    DeviceState* d = nullptr;
    const om_status s = device_state(&d);
    if (s != OM_OK) return s;
    const dim3 grid((unsigned)(d->sm_count * 8), (unsigned)count);
    const cudaError_t e = traced(kKindEvict, st, [&] { evict_gather_kernel<<<grid, 256, 0, st>>>(a); });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

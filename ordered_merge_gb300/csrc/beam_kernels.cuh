// Kernels of om_beam_select and om_beam_gather: the best continuations of a
// beam search, and the beams' states moved to the beams that go on.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "select_common.cuh"

namespace om {

constexpr int kMaxBeams = 64;
constexpr int kMaxBeamTop = 64;

// ------------------------------------------------------------ selection --

constexpr int kBeamThreadBits = 8, kBeamThreads = 1 << kBeamThreadBits;
constexpr int kBeamWarps = kBeamThreads / 32;
constexpr int kBeamGroups = 128;       // pairs of threads, of whose maxima the top-th bounds the selection
constexpr int kBeamCandidates = 512;   // entries of a slice that may reach that bound
constexpr int kBeamEach = 16;          // words of a chunk for each thread
constexpr int kBeamGroup = 8;          // of them are looked at together
constexpr int kBeamChunk = kBeamThreads * kBeamEach;
constexpr int kBeamMaxStages = 4;      // chunks in shared memory
constexpr int kBeamStageBytes = kBeamChunk * 4 + 32;
constexpr int kBeamCluster = 8;
// Continuations of all slices times slices up to which the best are found by counting,
// each its greater ones, instead of by one warp that takes a winner after the other (whole
// calls, counted and taken: 8 slices of 32, 14.8 and 18.2 us; 10 of 20, 16.3 and 17.6; but 12
// of 24, 24.5 and 20.5, 16 of 16, 12.7 and 12.2, 8 of 64, 30.2 and 28.8, 64 of 8, 35.1 and 20.1).
constexpr int kBeamCounted = 2048;

struct BeamArgs {
    const void* logits;
    const float* scores;      // nullptr: all zero
    const uint8_t* finished;  // nullptr: none
    int64_t batch_stride, beam_stride;
    int beams, vocab, top, end_id;
    int parts, slice;  // a row is cut into `parts` slices of `slice` logits (a multiple of 8)
    int stages;        // of the ring
    float* out_scores;
    int32_t* out_parents;
    int32_t* out_tokens;
    uint32_t* err;
};

// The logits of a word: two of 16 bits, or one.
template <typename T>
struct WordOf {
    static constexpr int kPer = 4 / (int)sizeof(T);
    static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // -inf in every place of a word
    static constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : kBf16 ? 0xff80ff80u : 0xfc00fc00u;
    // Lowest bits of a float that no value of T uses (all equal in an image: not compared).
    static constexpr int kSpare = sizeof(T) == 4 ? 0 : kBf16 ? 16 : 13;
    static constexpr uint64_t kKeyBits = ~((((uint64_t)1 << kSpare) - 1) << 32);
};

// The greater of two words, value by value; NaN loses against any number.
__device__ __forceinline__ uint32_t word_max(uint32_t x, uint32_t y, float) {
    return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
}
__device__ __forceinline__ uint32_t word_max(uint32_t x, uint32_t y, __nv_bfloat16) {
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
    return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t word_max(uint32_t x, uint32_t y, __half) {
    const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
    return *reinterpret_cast<const uint32_t*>(&m);
}
// The first value of a word, and the second (32 bits have one).
__device__ __forceinline__ float2 word_values(uint32_t w, float) { return make_float2(__uint_as_float(w), -INFINITY); }
__device__ __forceinline__ float2 word_values(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 word_values(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Order-preserving image of a double that is not NaN; 0 is free.
__device__ __forceinline__ uint64_t score_image64(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double image64_score(uint64_t u) {
    return __longlong_as_double((int64_t)(u >> 63 ? u ^ 0x8000000000000000ull : ~u));
}
__device__ __forceinline__ float image_score(uint32_t u) {
    return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u);
}
// Greater logit first, then the lower token; 0: none.
__device__ __forceinline__ uint64_t beam_key(float x, uint32_t token) {
    return (uint64_t)score_image(x) << 32 | (uint32_t)~token;
}

struct BeamShared {
    uint64_t full[kBeamMaxStages];
    uint64_t key[kBeamCandidates];
    double lse[kMaxBeams];
    float2 base[kMaxBeams];    // of each unit: the sum of exp(x - base), base in two parts
    uint64_t sum[kMaxBeams];   // (a float)
    float score[kMaxBeams];    // (first CTA) of each beam, and whether it is finished
    uint8_t ended[kMaxBeams];
    uint32_t group_key[kBeamGroups];
    float warp_max[kBeamWarps];
    float warp_scale[kBeamWarps];
    float warp_sum[kBeamWarps];
    float most;       // of the slice
    int slow;         // its sum is to be made again
    uint32_t bound;   // image of a lower bound of the slice's top-th greatest
    int found;        // logits that reach the bound
    int eights;       // eights that hold some
    uint32_t eight[2 * kBeamThreads];  // which, times 256, and whose
    int count;        // (settling) those counted
    int ties[kBeamWarps];
    int stop;         // a wait has run out (1), and thread 0 has waited for the other stages (2)
    int live, dead;   // units of this CTA that have logits to look at, and others
    uint8_t unit[kMaxBeams];  // the former from the front, the latter from the back
};
// After it the ring's stages and, in the first CTA of a cluster, the units' lists,
// [units][top] keys, then the images of the continuations' scores in the same places.

__device__ __forceinline__ uint32_t cluster_index() {
    uint32_t i;
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(i));
    return i;
}

// The two halves of a meeting of the cluster that hands no data on.  (The half that
// does waits for a trip to memory, 2.3 us while all CTAs' first chunks are on their way.)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// A word pair of CTA `rank`'s shared memory, at the address p has in this CTA's.
__device__ __forceinline__ void store_peer(uint64_t* p, uint32_t rank, uint64_t v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// What a unit found, to the first CTA.
__device__ __forceinline__ void store_stats(BeamShared& s, int unit, float base, float rest, float sum) {
    store_peer(reinterpret_cast<uint64_t*>(&s.base[unit]), 0, pack2(base, rest));
    store_peer(&s.sum[unit], 0, (uint64_t)__float_as_uint(sum));
}

// A slice of a row: its first logit and how many.
template <typename T>
struct BeamSlice {
    const T* row;
    int first, n;

    __device__ __forceinline__ BeamSlice(const BeamArgs& a, int64_t b, int unit) {
        const int beam = unit / a.parts, part = unit - beam * a.parts;
        row = static_cast<const T*>(a.logits) + b * a.batch_stride + beam * a.beam_stride;
        first = min(part * a.slice, a.vocab);
        n = min(a.slice, a.vocab - first);
    }
    __device__ __forceinline__ int words() const { return (n + WordOf<T>::kPer - 1) / WordOf<T>::kPer; }
    __device__ __forceinline__ int chunks() const { return (words() + kBeamChunk - 1) / kBeamChunk; }
    // NaN as -inf
    __device__ __forceinline__ float at(int i) const { return fmaxf(to_float(row[first + i]), -INFINITY); }
    // Word w, -inf past the end, NaN as -inf.  Loads without branches, so that several go together.
    __device__ __forceinline__ uint32_t word(int w) const {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row + first) + (uintptr_t)w * 4;
        const int left = n - w * WordOf<T>::kPer;
        const uint32_t* at = reinterpret_cast<const uint32_t*>(p & ~(uintptr_t)3);
        const bool odd = sizeof(T) == 2 && (p & 2) != 0;
        uint32_t v = left > 0 ? at[0] : WordOf<T>::kNone;
        const uint32_t up = odd && left > 1 ? at[1] : 0u;
        v = odd && left > 0 ? __byte_perm(v, up, 0x5432) : v;
        if (sizeof(T) == 2 && left == 1) v = (v & 0xffffu) | (WordOf<T>::kNone & 0xffff0000u);
        return word_max(v, WordOf<T>::kNone, T{});
    }
};

// The top-th greatest key of a slice too full of near values for the candidates'
// room: its bits one after another, each by a count over the slice.  All threads.
template <typename T>
__device__ __noinline__ uint64_t settle_edge(const BeamSlice<T>& slice, int top, BeamShared& s) {
    uint64_t edge = 0;
    for (int bit = 63; bit >= 0; bit = bit == 32 + WordOf<T>::kSpare ? 31 : bit - 1) {
        const uint64_t want = edge | 1ull << bit;
        int mine = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < slice.n; i += kBeamThreads) {
            const float x = slice.at(i);
            mine += x > -INFINITY && (beam_key(x, slice.first + i) & WordOf<T>::kKeyBits) >= want;
        }
        if (threadIdx.x == 0) s.count = 0;
        __syncthreads();
        mine = __reduce_add_sync(0xffffffffu, mine);
        if ((threadIdx.x & 31) == 0 && mine != 0) atomicAdd(&s.count, mine);
        __syncthreads();
        if (s.count >= top) edge = want;
        __syncthreads();
    }
    return edge;
}

// x * y + z of two at once.
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(x), "l"(y), "l"(z));
    return p;
}

// What a thread keeps of the words it has seen, 8 at a time ("eights"): the greatest
// maxima of eights, where the first two were, and the sum of 2^(x log2e - scale).  The
// scale is its first maximum times log2e, rounded (what the rounding does cancels
// when sums are joined by their scales), and moves only when logits leave the range
// that a float can take from there: to move it with every new maximum cost as much
// as the rest.  Beyond kBeamPlain it no longer says anything, and NaN spoils the
// sum: such slices are summed once more, slowly.
constexpr float kBeamPlain = 1e6f;

struct BeamRunning {
    float most = -INFINITY, second = -INFINITY, third = -INFINITY;
    int where = 0, next = 0;  // the eights of `most` and `second`
    float scale = -kBeamPlain * kLog2e, limit = 60.0f - kBeamPlain;
    uint64_t sum[2] = {0, 0};  // each of first values and second values (of two zeros)

    template <typename T>
    __device__ __forceinline__ void add(const uint32_t (&w)[kBeamGroup], int index, T) {
        uint32_t top = WordOf<T>::kNone;
#pragma unroll
        for (int i = 0; i < kBeamGroup; ++i) top = word_max(top, w[i], T{});
        const float2 both = word_values(top, T{});
        const float best = fmaxf(both.x, both.y);
        if (best > limit) {  // once, as a rule
            const float to = best * kLog2e, down = exp2_fast(scale - to);
#pragma unroll
            for (int i = 0; i < 2; ++i) sum[i] = mul2(sum[i], pack2(down, down));
            scale = to, limit = best + 60.0f;
        }
        third = fmaxf(third, fminf(best, second));
        next = best > most ? where : best > second ? index : next;
        second = fmaxf(second, fminf(best, most));
        where = best > most ? index : where;
        most = fmaxf(most, best);
        const uint64_t log2e = pack2(kLog2e, kLog2e), less = pack2(-scale, -scale);
        constexpr int kStep = 2 / WordOf<T>::kPer;  // words of two logits
#pragma unroll
        for (int i = 0; i < kBeamGroup; i += kStep) {
            const float2 v = word_values(w[i], T{});
            const uint64_t x = kStep == 1 ? pack2(v.x, v.y) : pack2(v.x, __uint_as_float(w[i + kStep - 1]));
            const float2 e = unpack2(fma2(x, log2e, less));
            add2(sum[(i / kStep) & 1], pack2(exp2_fast(e.x), exp2_fast(e.y)));
        }
    }
    __device__ __forceinline__ float total() const {
        const float2 x = unpack2(sum[0]), y = unpack2(sum[1]);
        return (x.x + y.x) + (x.y + y.y);
    }
};

// A thread's words of a chunk of `words`, word i of which starts `offset` bytes into
// the stage and 4 i on.  Which words a thread has does not depend on the row's
// address, so that equal rows have equal sums and equal continuations tie.
template <typename T, bool ODD>  // ODD: 16-bit logits between two words
__device__ __forceinline__ void beam_whole_chunk(const uint32_t* s, int chunk, BeamRunning& run) {
    constexpr int W = kBeamGroup;
#pragma unroll
    for (int j = 0; j < kBeamEach / W; ++j) {
        uint32_t w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = s[(j * W + i) * kBeamThreads];
        if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = __byte_perm(w[i], s[(j * W + i) * kBeamThreads + 1], 0x5432);
        }
        run.add(w, chunk * (kBeamEach / W) + j, T{});
    }
}
template <typename T>
__device__ __forceinline__ void beam_last_chunk(const uint32_t* s, bool odd, int logits, int chunk, BeamRunning& run) {
    constexpr int W = kBeamGroup;
    const int words = (logits + WordOf<T>::kPer - 1) / WordOf<T>::kPer;
#pragma unroll 1
    for (int j = 0; j < kBeamEach / W; ++j) {
        uint32_t w[W];
        if (j * W * kBeamThreads >= words) break;
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int at = (j * W + i) * kBeamThreads + (int)threadIdx.x;
            w[i] = WordOf<T>::kNone;
            if (at < words) {
                w[i] = s[(j * W + i) * kBeamThreads];
                const bool half = sizeof(T) == 2 && 2 * at + 1 == logits;  // its second value is none of the row's
                if (odd) w[i] = __byte_perm(w[i], half ? 0u : s[(j * W + i) * kBeamThreads + 1], 0x5432);
                if (half) w[i] = (w[i] & 0xffffu) | (WordOf<T>::kNone & 0xffff0000u);
            }
        }
        run.add(w, chunk * (kBeamEach / W) + j, T{});
    }
}

// U words, `step` apart, from `first` on: loaded together, then what of them reaches
// the bound (exceeds it: STRICT) one by one.
template <typename T, bool STRICT, int U, typename F>
__device__ __forceinline__ void look_at(const BeamSlice<T>& slice, float bound, BeamShared& s, F&& word_of) {
    auto reaches = [&](float x) { return STRICT ? x > bound : x >= bound && x > -INFINITY; };
    uint32_t w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) w[i] = slice.word(word_of(i));
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const float2 x = word_values(w[i], T{});
        auto keep = [&](float v, int second) {
            const int at = atomicAdd(&s.found, 1);
            if (at < kBeamCandidates) s.key[at] = beam_key(v, slice.first + word_of(i) * WordOf<T>::kPer + second);
        };
        if (reaches(x.x)) keep(x.x, 0);
        if (WordOf<T>::kPer == 2 && reaches(x.y)) keep(x.y, 1);
    }
}

// The one or two eights of a thread that hold what reaches the bound are listed, and
// read again by all threads, a word each; where a thread has more, its warp reads all of
// its words.  A warp with many such threads leaves the slice to crowded_slice.
constexpr int kBeamCrowd = 8;

template <typename T, bool STRICT>
__device__ __forceinline__ void look_again(const BeamSlice<T>& slice, const BeamRunning& run, float bound, BeamShared& s) {
    auto reaches = [&](float x) { return STRICT ? x > bound : x >= bound && x > -INFINITY; };
    const int lane = threadIdx.x & 31, words = slice.words();
    unsigned todo = __ballot_sync(0xffffffffu, reaches(run.third));
    if (__popc(todo) > kBeamCrowd) {
        if (lane == 0) atomicAdd(&s.found, kBeamCandidates + 1);
        todo = 0;
    } else if (!(todo >> lane & 1) && reaches(run.most)) {
        const int at = atomicAdd(&s.eights, reaches(run.second) ? 2 : 1);
        s.eight[at] = (uint32_t)run.where << 8 | threadIdx.x;
        if (reaches(run.second)) s.eight[at + 1] = (uint32_t)run.next << 8 | threadIdx.x;
    }
    for (; todo != 0; todo &= todo - 1) {
        const int from = ((int)threadIdx.x & ~31) + __ffs(todo) - 1 + lane * kBeamThreads;
        for (int w = from; w < words; w += 64 * kBeamGroup * kBeamThreads)
            look_at<T, STRICT, 2 * kBeamGroup>(slice, bound, s, [&](int i) { return w + i * 32 * kBeamThreads; });
    }
    __syncthreads();
    const int all = s.eights * kBeamGroup;
    auto word_of = [&](int i) {
        const uint32_t e = s.eight[min(i, all - 1) / kBeamGroup];
        const int word = ((int)(e >> 8) * kBeamGroup + i % kBeamGroup) * kBeamThreads + (int)(e & 255);
        return i < all ? word : words;
    };
    if (all <= kBeamThreads) {
        if ((int)threadIdx.x < all) look_at<T, STRICT, 1>(slice, bound, s, [&](int) { return word_of(threadIdx.x); });
    } else if (s.found <= kBeamCandidates) {
        for (int i0 = threadIdx.x; i0 < all; i0 += 4 * kBeamThreads)
            look_at<T, STRICT, 4>(slice, bound, s, [&](int i) { return word_of(i0 + i * kBeamThreads); });
    }
}

// How many of n numbers (or equal ones before it) are greater than number c of them,
// by 2^bits neighbouring threads together.  Whole warps.
__device__ __forceinline__ int place_of(const uint64_t* numbers, int n, int c, int bits) {
    const int lanes = 1 << bits;
    const uint64_t mine = numbers[min(c, n - 1)];
    int place = 0;
#pragma unroll 4
    for (int o = (int)threadIdx.x & (lanes - 1); o < n; o += lanes) place += numbers[o] + (o < c) > mine;
    for (int d = 1; d < lanes; d <<= 1) place += __shfl_xor_sync(0xffffffffu, place, d);
    return place;
}
// The same of continuations whose rows are cut: equal images of one beam go by their keys
// (logit, then token), which a great score may have rounded together; others, and those of
// no continuation, by their places.
__device__ __forceinline__ int place_of_cut(const uint64_t* images, const uint64_t* keys, int n, int per, int c, int bits) {
    const int lanes = 1 << bits, own = min(c, n - 1), beam = own / per;
    const uint64_t mine = images[own];
    int place = 0;
#pragma unroll 4
    for (int o = (int)threadIdx.x & (lanes - 1); o < n; o += lanes) {
        const uint64_t image = images[o];
        bool before = image + (o < c) > mine;
        if (image == mine && mine != 0 && o != own && o / per == beam) before = keys[o] > keys[own];
        place += before;
    }
    for (int d = 1; d < lanes; d <<= 1) place += __shfl_xor_sync(0xffffffffu, place, d);
    return place;
}
// As many threads for each of n as there are, in bits.
__device__ __forceinline__ int place_bits(int n) { return min(max(__clz(max(n - 1, 1)) - (32 - kBeamThreadBits), 0), 5); }

// The candidates of a slice of which too many reach the bound.  Most often these are
// ties with the bound itself (rows of one value; of few values and a low one for what
// is masked): then fewer than `top` exceed it, and the first of the ties, in order,
// fill up.  All threads; returns how many keys there are.
template <typename T>
__device__ __noinline__ int crowded_slice(const BeamSlice<T>& slice, const BeamRunning& run, float bound, int top, BeamShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();  // all have read s.found
    if (threadIdx.x == 0) s.found = 0, s.eights = 0;
    __syncthreads();
    look_again<T, true>(slice, run, bound, s);
    __syncthreads();
    int have = s.found;
    if (have >= top && have <= kBeamCandidates) return have;
    if (have < top) {
        for (int i0 = 0; i0 < slice.n && have < top && bound > -INFINITY; i0 += kBeamThreads) {
            const int i = i0 + (int)threadIdx.x;
            const unsigned ties = __ballot_sync(0xffffffffu, i < slice.n && slice.at(i) == bound);
            if (lane == 0) s.ties[warp] = __popc(ties);
            __syncthreads();
            int before = have, all = 0;
            for (int w = 0; w < kBeamWarps; ++w) before += w < warp ? s.ties[w] : 0, all += s.ties[w];
            before += __popc(ties & ((1u << lane) - 1));
            if ((ties >> lane & 1) && before < top) s.key[before] = beam_key(bound, slice.first + i);
            have = min(have + all, top);
            __syncthreads();
        }
        return have;
    }
    const uint64_t edge = settle_edge(slice, top, s);
    if (threadIdx.x == 0) s.found = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < slice.n; i += kBeamThreads) {
        const float x = slice.at(i);
        const uint64_t key = beam_key(x, slice.first + i);
        if (x > -INFINITY && (key & WordOf<T>::kKeyBits) >= edge) {
            const int at = atomicAdd(&s.found, 1);  // `top` of them: keys differ
            if (at < kBeamCandidates) s.key[at] = key;
        }
    }
    __syncthreads();
    return min(s.found, kBeamCandidates);
}

// The end of a slice: its maximum, its sum of exponentials and its `top` greatest
// logits in order, into place `unit` of the first CTA.  All threads.
//
// Of the maxima of 128 pairs of threads the top-th greatest is a lower bound of the
// slice's top-th greatest logit, and only threads whose own maximum reaches it hold
// any that do: few more than `top`.  They look again, and what reaches the bound is
// put in order by counting.
template <typename T>
__device__ __forceinline__ void beam_slice_end(const BeamArgs& a, const BeamSlice<T>& slice, int unit, const BeamRunning& run,
                                               uint64_t* lists, BeamShared& s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float m = run.most;
    // groups are ranked by their maxima, the last bits given up for the group's number: all differ
    const float group_max = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t group_key = (score_image(group_max) & ~(uint32_t)(kBeamGroups - 1)) | (threadIdx.x >> 1);
    if ((threadIdx.x & 1) == 0) s.group_key[threadIdx.x >> 1] = group_key;
    // NaN stays NaN in these, to be seen at the end
    const float most = warp_max(m), scale = warp_max(run.scale);
    const float all = warp_sum(run.total() * exp2_fast(run.scale - scale));
    if (lane == 0) s.warp_max[warp] = most, s.warp_scale[warp] = scale, s.warp_sum[warp] = all;
    if (threadIdx.x == 0) s.found = 0, s.eights = 0, s.bound = 0xffffffffu;
    __syncthreads();
    {  // two threads a group, each comparing with half of the groups
        int rank = 0;
        const uint4* others = reinterpret_cast<const uint4*>(s.group_key) + (threadIdx.x & 1) * (kBeamGroups / 8);
#pragma unroll 4
        for (int i = 0; i < kBeamGroups / 8; ++i) {
            const uint4 o = others[i];
            rank += (o.x > group_key) + (o.y > group_key) + (o.z > group_key) + (o.w > group_key);
        }
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        // the least maximum of those groups: a logit of the slice
        const uint32_t least = __reduce_min_sync(0xffffffffu, rank < a.top ? score_image(group_max) : 0xffffffffu);
        if (lane == 0) atomicMin(&s.bound, least);
    }
    if (warp == kBeamWarps - 1) {
        const float wm = warp_max(lane < kBeamWarps ? s.warp_max[lane] : -INFINITY);
        const float ws = lane < kBeamWarps ? s.warp_scale[lane] : -INFINITY, top_scale = warp_max(ws);
        const float sum = warp_sum(lane < kBeamWarps ? s.warp_sum[lane] * exp2_fast(ws - top_scale) : 0.0f);
        if (lane == 0) {
            s.most = wm;
            s.slow = wm > -INFINITY && !(fabsf(wm) <= kBeamPlain && sum > 0.0f && sum < INFINITY);
            // the scale over log2e, in two floats
            constexpr double kBack = 1.0 / (double)kLog2e;
            constexpr float kBackHigh = (float)kBack, kBackLow = (float)(kBack - (double)kBackHigh);
            const float base = top_scale * kBackHigh, rest = fmaf(top_scale, kBackHigh, -base) + top_scale * kBackLow;
            if (wm > -INFINITY) store_stats(s, unit, base, rest, sum);
            else store_stats(s, unit, -INFINITY, 0.0f, 0.0f);
        }
    }
    __syncthreads();
    const float bound = image_score(s.bound);
    look_again<T, false>(slice, run, bound, s);
    __syncthreads();
    if (s.slow) {
        float sum = 0.0f;
#pragma unroll 4
        for (int i = threadIdx.x; i < slice.n; i += kBeamThreads) {
            const float x = slice.at(i);
            if (x > -INFINITY) sum += exp2_fast((x - s.most) * kLog2e);
        }
        sum = warp_sum(sum);
        if (lane == 0) s.warp_sum[warp] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            float all_warps = 0.0f;
            for (int i = 0; i < kBeamWarps; ++i) all_warps += s.warp_sum[i];
            store_stats(s, unit, s.most, 0.0f, all_warps);
        }
    }
    int found = s.found;
    if (found > kBeamCandidates) found = crowded_slice(slice, run, bound, a.top, s);
    uint64_t* list = lists + unit * a.top;
    const int bits = place_bits(found), own = (int)threadIdx.x >> bits;
    for (int c0 = 0; c0 < found; c0 += kBeamThreads >> bits) {
        const int c = c0 + own, place = place_of(s.key, found, c, bits);
        if (c < found && place < a.top && own << bits == (int)threadIdx.x) store_peer(list + place, 0, s.key[c]);
    }
    for (int r = found + threadIdx.x; r < a.top; r += kBeamThreads) store_peer(list + r, 0, 0ull);
    __syncthreads();  // s is used again
}

// A stage's wait has run out (om_device_error says so; the outputs are none then): no more
// copies are asked for, and those of the other stages get as long to end.
__device__ __noinline__ void ring_stops(const BeamArgs& a, int stage, uint32_t phase, BeamShared& s) {
    if (s.stop != 1) return;
    for (int i = 1; i < a.stages; ++i)
        mbar_wait_bounded(&s.full[(stage + i) % a.stages], phase ^ (stage + i >= a.stages), a.err);
    s.stop = 2;
}

// Bytes of BeamShared before the ring.
__host__ __device__ constexpr int beam_ring_offset() { return ((int)sizeof(BeamShared) + 127) / 128 * 128; }

// A cluster to each sequence; its slices ("units", beam by beam) go to the CTAs in
// turn.  A CTA streams the chunks of its slices through a ring in shared memory,
// filled by bulk copies (of whole aligned 16 bytes around a chunk, whatever the
// row's address), each thread keeping a running maximum and sum of its words.  The
// first CTA joins the slices: the beams' logarithms of their sums, the scores of
// the slices' best continuations in 64 bits, and the best of all.
//
// 64 sequences of 8 beams over 131071 bf16 logits, 0.13 GB: 34.2 us, of which 20 would
// stream it at the memory's rate.  The first loads take 2.5, the stream 18 on SMs with
// three of the 512 CTAs and 21 (27 at most) on those with four, a slice's bound and its
// candidates, read once more, 3, the cluster's meeting and the joining 3.  One prompt of 4
// beams is that chain, about 8 us.
// (Vectors loaded straight into registers, rows realigned by shifts: 70 us.)
template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 4) beam_select_kernel(const BeamArgs a) {
    wait_for_stream();
    extern __shared__ __align__(128) unsigned char s_raw[];
    BeamShared& s = *reinterpret_cast<BeamShared*>(s_raw);
    unsigned char* ring = s_raw + beam_ring_offset();
    uint64_t* lists = reinterpret_cast<uint64_t*>(ring + a.stages * kBeamStageBytes);
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    const int64_t b = cluster_index();
    const int units = a.beams * a.parts;
    const uint64_t policy = l2_policy_evict_first();
    // thread 0: slices to come, where the next copy starts, how many there are of its slice, their bytes and the last one's
    int live = 0, dead = 0, next_slice = 0, copies = 0;
    uint32_t bytes = 0, last_bytes = 0;
    uintptr_t from = 0;
    auto fill = [&](int stage) {
        if (copies == 0) {
            if (next_slice >= live) return;
            const BeamSlice<T> slice(a, b, s.unit[next_slice++]);
            from = reinterpret_cast<uintptr_t>(slice.row + slice.first);
            const uint32_t skip = (uint32_t)(from & 15);
            from -= skip, copies = slice.chunks();
            bytes = kBeamChunk * 4 + (skip != 0 ? 16 : 0);
            last_bytes = (uint32_t)((int64_t)slice.n * (int)sizeof(T) - (int64_t)(copies - 1) * (kBeamChunk * 4) + skip + 15) & ~15u;
        }
        const uint32_t now = --copies == 0 ? last_bytes : bytes;
        mbar_arrive_expect_tx(&s.full[stage], now);
        bulk_copy_g2s(ring + stage * kBeamStageBytes, reinterpret_cast<const void*>(from), now, &s.full[stage], policy);
        from += kBeamChunk * 4;
    };
    if (threadIdx.x < 32) {  // the slices of this CTA that have logits to look at
        if (threadIdx.x == 0) {
            for (int i = 0; i < a.stages; ++i) mbar_init(&s.full[i], 1);
            fence_barrier_init();
        }
        for (int u0 = (int)rank; u0 < units; u0 += 32 * (int)ctas) {
            const int u = u0 + (int)threadIdx.x * (int)ctas;
            bool looks = false;
            if (u < units) {
                const int beam = u / a.parts;
                const float score = a.scores == nullptr ? 0.0f : a.scores[b * a.beams + beam];
                const bool ended = a.finished != nullptr && a.finished[b * a.beams + beam] != 0;
                looks = !ended && score > -INFINITY && u % a.parts * a.slice < a.vocab;
            }
            const unsigned there = __ballot_sync(0xffffffffu, looks);
            if (looks) s.unit[live + __popc(there & ((1u << threadIdx.x) - 1))] = (uint8_t)u;
            const unsigned rest = __ballot_sync(0xffffffffu, u < units && !looks);
            if (rest >> threadIdx.x & 1) s.unit[kMaxBeams - 1 - dead - __popc(rest & ((1u << threadIdx.x) - 1))] = (uint8_t)u;
            live += __popc(there), dead += __popc(rest);
        }
        __syncwarp();
        if (threadIdx.x == 0) {
            s.live = live, s.dead = dead, s.stop = 0;
            for (int i = 0; i < a.stages; ++i) fill(i);
        }
    } else if (rank == 0 && (int)threadIdx.x - 32 < a.beams) {  // for the end
        const int i = (int)threadIdx.x - 32;
        s.score[i] = a.scores == nullptr ? 0.0f : a.scores[b * a.beams + i];
        s.ended[i] = a.finished != nullptr && a.finished[b * a.beams + i] != 0;
    }
    __syncthreads();
    if (ctas > 1) cluster_arrive();  // and wait before the first store to the first CTA's shared memory
    live = s.live;
    int stage = 0;
    uint32_t phase = 0;
    for (int k = 0; k < live; ++k) {
        const int unit = s.unit[k];
        const BeamSlice<T> slice(a, b, unit);
        const int chunks = slice.chunks();
        BeamRunning run;
        const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(slice.row + slice.first) & 15);  // chunks are whole 16 bytes
        const uint32_t* words = reinterpret_cast<const uint32_t*>(ring + (skip & ~3u)) + threadIdx.x;
        const bool odd = skip & 2;
        int left = slice.n;
        for (int c = 0; c < chunks; ++c, left -= kBeamChunk * WordOf<T>::kPer) {
            if (!mbar_wait_or_stop(&s.full[stage], phase, a.err, &s.stop) && threadIdx.x == 0) {
                ring_stops(a, stage, phase, s);
                copies = 0, next_slice = live;  // nothing more to fill with
            }
            const uint32_t* mine = words + stage * (kBeamStageBytes / 4);
            if (left < kBeamChunk * WordOf<T>::kPer) beam_last_chunk<T>(mine, odd, left, c, run);
            else if (sizeof(T) == 2 && odd) beam_whole_chunk<T, sizeof(T) == 2>(mine, c, run);
            else beam_whole_chunk<T, false>(mine, c, run);
            __syncthreads();
            if (threadIdx.x == 0) fill(stage);
            if (++stage == a.stages) stage = 0, phase ^= 1;
        }
        if (k == 0 && ctas > 1) cluster_wait();
        beam_slice_end<T>(a, slice, unit, run, lists, s);
    }
    if (live == 0 && ctas > 1) cluster_wait();
    dead = s.dead;
    for (int i = threadIdx.x; i < dead * (a.top + 1); i += kBeamThreads) {
        const int unit = s.unit[kMaxBeams - 1 - i / (a.top + 1)], r = i % (a.top + 1);
        if (r < a.top) store_peer(lists + unit * a.top + r, 0, 0ull);
        else store_stats(s, unit, -INFINITY, 0.0f, 0.0f);
    }
    if (ctas > 1) {
        cluster_sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }
    uint64_t* images = lists + units * a.top;
    if (threadIdx.x < a.beams) {
        const int i = threadIdx.x;
        float2 most = s.base[i * a.parts];
        for (int p = 1; p < a.parts; ++p) {
            const float2 base = s.base[i * a.parts + p];
            if (base.x > most.x) most = base;
        }
        float sum = 0.0f;
        for (int p = 0; p < a.parts; ++p) {
            const float part = __uint_as_float((uint32_t)s.sum[i * a.parts + p]);
            const float2 base = s.base[i * a.parts + p];
            if (base.x > -INFINITY) sum += part * (base.x == most.x && base.y == most.y ? 1.0f : exp2_fast(((base.x - most.x) + (base.y - most.y)) * kLog2e));
        }
        // the logarithm of a sum as its exponent's and its fraction's, of which only the latter is rounded to 32 bits
        const int exponent = (int)(__float_as_uint(sum) >> 23) - 127;
        const float fraction = __uint_as_float((__float_as_uint(sum) & 0x7fffffu) | 0x3f800000u);
        s.lse[i] = sum > 0.0f ? (double)most.x + ((double)(most.y + logf(fraction)) + exponent * 0.6931471805599453) : (double)NAN;
    }
    __syncthreads();
    const int n = units * a.top, per = a.top * a.parts;
    for (int c = threadIdx.x; c < n; c += kBeamThreads) {
        const int beam = c / per;
        uint64_t image = 0;
        if (lists[c] != 0) {
            const double v = (double)s.score[beam] + ((double)image_score((uint32_t)(lists[c] >> 32)) - s.lse[beam]);
            if ((float)v > -INFINITY) image = score_image64(v);
        }
        if (c == beam * per && s.ended[beam]) {
            lists[c] = (uint32_t)~(uint32_t)a.end_id;
            if (s.score[beam] > -INFINITY) image = score_image64((double)s.score[beam]);
        }
        images[c] = image;
    }
    __syncthreads();
    if (n * units <= kBeamCounted) {
        // the place of a continuation is the number of those before it
        const int bits = place_bits(n), own = (int)threadIdx.x >> bits;
        for (int c0 = 0; c0 < n; c0 += kBeamThreads >> bits) {
            const int c = c0 + own;
            const int place = a.parts > 1 ? place_of_cut(images, lists, n, per, c, bits) : place_of(images, n, c, bits);
            if (c >= n || place >= a.top || own << bits != (int)threadIdx.x) continue;
            const uint64_t mine = images[c];
            const int64_t to = b * a.top + place;
            a.out_scores[to] = mine != 0 ? (float)image64_score(mine) : -INFINITY;
            a.out_parents[to] = mine != 0 ? c / per : -1;
            a.out_tokens[to] = mine != 0 ? (int32_t)~(uint32_t)lists[c] : -1;
        }
        return;
    }
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    int at[2];
    uint64_t head[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int u = lane + 32 * i;
        at[i] = u * a.top;
        head[i] = u < units ? images[at[i]] : 0;
    }
    for (int k = 0; k < a.top; ++k) {
        const uint64_t mine = head[1] > head[0] ? head[1] : head[0];
        const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32));
        const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(mine >> 32) == hi ? (uint32_t)mine : 0);
        const uint64_t best = (uint64_t)hi << 32 | lo;
        const int64_t to = b * a.top + k;
        if (best == 0) {
            for (int r = k + lane; r < a.top; r += 32) {
                a.out_scores[b * a.top + r] = -INFINITY;
                a.out_parents[b * a.top + r] = -1;
                a.out_tokens[b * a.top + r] = -1;
            }
            break;
        }
        const unsigned in0 = __ballot_sync(0xffffffffu, head[0] == best);
        const unsigned in1 = __ballot_sync(0xffffffffu, head[1] == best);
        int win = in0 != 0 ? __ffs(in0) - 1 : __ffs(in1) - 1;
        if (a.parts > 1 && (in0 & (in0 - 1)) != 0) {  // slices of one beam (16 units at most then): by their keys
            const bool same = (in0 >> lane & 1) && lane / a.parts == win / a.parts;
            const uint64_t key = same ? lists[at[0]] : 0;
            const uint32_t key_hi = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
            const uint32_t key_lo = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == key_hi ? (uint32_t)key : 0);
            win = __ffs(__ballot_sync(0xffffffffu, same && key == ((uint64_t)key_hi << 32 | key_lo))) - 1;
        }
        if (lane == win) {
            const int i = in0 != 0 ? 0 : 1;
            const int from = i == 0 ? at[0] : at[1];
            a.out_scores[to] = (float)image64_score(best);
            a.out_parents[to] = (lane + 32 * i) / a.parts;
            a.out_tokens[to] = (int32_t)~(uint32_t)lists[from];
            const bool more = (from + 1) % a.top != 0;
            const uint64_t next = more ? images[from + 1] : 0;
            if (i == 0) at[0] = from + 1, head[0] = next;
            else at[1] = from + 1, head[1] = next;
        }
    }
}

// --------------------------------------------------------------- gather --

constexpr int kMaxBeamArrays = 64;
constexpr int kBeamGatherThreads = 128;
constexpr int kBeamsInRegisters = 16;

struct BeamGatherShape {
    const int32_t *parents, *starts, *lengths;
    int64_t entries, rows;  // rows: batch * heads
    int beams, heads, count, parts, in_place;
};
// MOST: arrays that the launch carries (what it carries costs its caller time).
template <int MOST>
struct BeamGatherArgs : BeamGatherShape {
    om_beam_array arrays[MOST];
    unsigned char vector[MOST];
};
constexpr int kFewBeamArrays = 4;

// A column of the beams (the same bytes of one entry in each) belongs to one
// thread, which loads what its beams get before it stores any of it: so the move
// works in place for every map of beams to parents, with no barrier.  A beam
// that keeps its own place is not touched in place.
//
// Bound by memory: 64 beams' keys and values of 8 heads, 2.5 K entries of 256 bytes each
// on average, 1.11 GB, 165 us (6.7 TB/s, the copy rate).
// BEAMS: beams loaded together (all of them in place).  STAGED: in place with
// more than that many, through shared memory.
template <typename V, int BEAMS, bool STAGED>
__device__ __forceinline__ void gather_columns(const BeamGatherShape& a, const om_beam_array& c, int64_t b, int64_t h,
                                               int part, int64_t lo, int64_t hi) {
    extern __shared__ __align__(16) unsigned char s_stage[];
    const int64_t per = c.entry_bytes / (int)sizeof(V), total = (hi - lo) * per;
    const char* src = static_cast<const char*>(c.src) + b * c.src_batch + h * c.src_head + lo * c.src_entry;
    char* dst = static_cast<char*>(c.dst) + b * c.dst_batch + h * c.dst_head + lo * c.dst_entry;
    const int32_t* parents = a.parents + b * a.beams;
    const bool whole = c.src_entry == c.entry_bytes && c.dst_entry == c.entry_bytes;
    for (int64_t i = (int64_t)part * kBeamGatherThreads + threadIdx.x; i < total; i += (int64_t)a.parts * kBeamGatherThreads) {
        int64_t from = i * (int)sizeof(V), to = from;
        if (!whole) {
            const int64_t entry = total <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
            const int64_t piece = (i - entry * per) * (int)sizeof(V);
            from = entry * c.src_entry + piece;
            to = entry * c.dst_entry + piece;
        }
        if constexpr (STAGED) {
            V* mine = reinterpret_cast<V*>(s_stage) + threadIdx.x;
            for (int j = 0; j < a.beams; ++j) {
                const int p = parents[j];
                if (p != j && (unsigned)p < (unsigned)a.beams)
                    mine[j * kBeamGatherThreads] = *reinterpret_cast<const V*>(src + p * c.src_beam + from);
            }
            for (int j = 0; j < a.beams; ++j) {
                const int p = parents[j];
                if (p != j && (unsigned)p < (unsigned)a.beams)
                    *reinterpret_cast<V*>(dst + j * c.dst_beam + to) = mine[j * kBeamGatherThreads];
            }
        } else {
            for (int j0 = 0; j0 < a.beams; j0 += BEAMS) {
                V v[BEAMS];
                unsigned moved = 0;
#pragma unroll
                for (int j = 0; j < BEAMS; ++j) {
                    const int p = j0 + j < a.beams ? parents[j0 + j] : -1;
                    v[j] = V{};
                    if ((unsigned)p < (unsigned)a.beams && !(a.in_place && p == j0 + j)) {
                        v[j] = *reinterpret_cast<const V*>(src + p * c.src_beam + from);
                        moved |= 1u << j;
                    }
                }
#pragma unroll
                for (int j = 0; j < BEAMS; ++j)
                    if (moved >> j & 1) *reinterpret_cast<V*>(dst + (j0 + j) * c.dst_beam + to) = v[j];
            }
        }
    }
}

template <int BEAMS, bool STAGED, int MOST>
__global__ void __launch_bounds__(kBeamGatherThreads) beam_gather_kernel(const __grid_constant__ BeamGatherArgs<MOST> a) {
    wait_for_stream();
    const int64_t job = blockIdx.x / a.parts;
    const int part = (int)(blockIdx.x - job * a.parts), k = (int)(job / a.rows);
    const int64_t row = job - k * a.rows, b = row / a.heads, h = row - b * a.heads;
    int64_t lo = a.starts == nullptr ? 0 : a.starts[b], hi = a.lengths == nullptr ? a.entries : a.lengths[b];
    if (lo < 0) lo = 0;
    if (hi > a.entries) hi = a.entries;
    switch (a.vector[k]) {
        case 16: gather_columns<uint4, BEAMS, STAGED>(a, a.arrays[k], b, h, part, lo, hi); break;
        case 4: gather_columns<uint32_t, BEAMS, STAGED>(a, a.arrays[k], b, h, part, lo, hi); break;
        case 2: gather_columns<unsigned short, BEAMS, STAGED>(a, a.arrays[k], b, h, part, lo, hi); break;
        default: gather_columns<unsigned char, BEAMS, STAGED>(a, a.arrays[k], b, h, part, lo, hi); break;
    }
}

}  // namespace om

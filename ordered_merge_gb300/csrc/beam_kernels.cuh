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

constexpr int kBeamThreads = 512;
constexpr int kBeamGroups = kBeamThreads / 4;  // groups of 4 threads, of whose maxima the top-th bounds the selection
constexpr int kBeamCandidates = 1024;          // entries of a slice that may reach that bound
constexpr int kBeamUnroll = 4;                 // vectors in flight per thread
constexpr int kBeamCluster = 16;

struct BeamArgs {
    const void* logits;
    const float* scores;      // nullptr: all zero
    const uint8_t* finished;  // nullptr: none
    int64_t batch_stride, beam_stride;
    int beams, vocab, top, end_id;
    int parts, slice;  // a row is cut into `parts` slices of `slice` logits (a multiple of 8)
    float* out_scores;
    int32_t* out_parents;
    int32_t* out_tokens;
};

// A row's logits in vectors of 16 bytes from its first one on, whatever the
// row's address: what thread t sums does not depend on it, so that equal rows
// have equal sums, and equal continuations tie.
template <typename T>
struct RowVectors {
    static constexpr int kPer = 16 / (int)sizeof(T);
    const char* base;  // the row's address rounded down to 16 bytes
    uint32_t shift;    // and the bytes it lies after that
    uint32_t n;        // logits

    __device__ __forceinline__ RowVectors(const T* row, int logits) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row);
        base = reinterpret_cast<const char*>(p & ~(uintptr_t)15);
        shift = (uint32_t)(p & 15);
        n = (uint32_t)logits;
    }
    // -inf in every place of a word
    static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    static constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : kBf16 ? 0xff80ff80u : 0xfc00fc00u;
    // Lowest bits of a float that no value of T uses (all equal in an image: not compared).
    static constexpr int kSpare = sizeof(T) == 4 ? 0 : kBf16 ? 16 : 13;
    static constexpr uint64_t kKeyBits = ~((((uint64_t)1 << kSpare) - 1) << 32);

    // Vector j (logits j * kPer ...), -inf past the row's end.  Reads the 16 aligned bytes
    // around each logit, nothing beyond.
    __device__ __forceinline__ uint4 load(uint32_t j) const {
        const uint4* p = reinterpret_cast<const uint4*>(base) + j;
        const uint32_t left = n > j * kPer ? n - j * kPer : 0;  // logits from here on
        uint4 v = make_uint4(kNone, kNone, kNone, kNone);
        if (left == 0) return v;
        v = *p;
        if (shift != 0) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (left * (uint32_t)sizeof(T) > 16 - shift) w = p[1];
            // the 16 bytes from `shift` on
            uint32_t x[8] = {v.x, v.y, v.z, v.w, w.x, w.y, w.z, w.w};
            if (shift & 8) {
#pragma unroll
                for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
            }
            if (shift & 4) {
#pragma unroll
                for (int i = 0; i < 5; ++i) x[i] = x[i + 1];
            }
            if (shift & 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
            }
            v = make_uint4(x[0], x[1], x[2], x[3]);
        }
        if (left < kPer) {
            uint32_t* x = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                constexpr uint32_t in_word = 4 / sizeof(T);
                if (i * in_word >= left) x[i] = kNone;
                else if (in_word == 2 && i * in_word + 1 == left) x[i] = (x[i] & 0xffffu) | (kNone & 0xffff0000u);
            }
        }
        return v;
    }
};
// The logits of a vector as floats, NaN as -inf (a maximum takes the operand that is a number).
__device__ __forceinline__ void logits_of(const uint4& v, float (&x)[4], float) {
    const uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = fmaxf(__uint_as_float(w[i]), -INFINITY);
}
__device__ __forceinline__ void logits_of(const uint4& v, float (&x)[8], __nv_bfloat16) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v);
    const __nv_bfloat162 low = __float2bfloat162_rn(-INFINITY);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 m = __hmax2(w[i], low);
        const uint32_t u = *reinterpret_cast<const uint32_t*>(&m);
        x[2 * i] = __uint_as_float(u << 16);
        x[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
    }
}
__device__ __forceinline__ void logits_of(const uint4& v, float (&x)[8], __half) {
    const __half2* w = reinterpret_cast<const __half2*>(&v);
    const __half2 low = __float2half2_rn(-INFINITY);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(__hmax2(w[i], low));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

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
    float warp_max[kBeamThreads / 32];
    float warp_sum[kBeamThreads / 32];
    float group_max[kBeamGroups];
    float bound;
    int near;         // threads whose maximum reaches the bound
    int found;        // logits that reach it
    int count;        // (settling) those counted
    uint16_t who[kBeamThreads];
    uint64_t key[kBeamCandidates];
    float2 stats[kMaxBeams];   // of each unit: maximum, sum of exp(x - maximum)
    double lse[kMaxBeams];
    float score[kMaxBeams];
};
// After it, in the first CTA of a cluster: the units' lists, [units][top] keys,
// then the images of the continuations' scores in the same places.

// A word pair of CTA `rank`'s shared memory, at the address p has in this CTA's.
__device__ __forceinline__ void store_peer(uint64_t* p, uint32_t rank, uint64_t v) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}

// The top-th greatest key of a slice too full of equal or near values for the
// candidates' room (rows of one value, of few values not masked by the type's
// lowest): its bits one after another, each by a count over the slice.  All threads.
template <typename T>
__device__ __noinline__ uint64_t settle_edge(const RowVectors<T>& row, uint32_t v0, uint32_t v1, int top, BeamShared& s) {
    constexpr int N = RowVectors<T>::kPer;
    uint64_t edge = 0;
    for (int bit = 63; bit >= 0; bit = bit == 32 + RowVectors<T>::kSpare ? 31 : bit - 1) {
        const uint64_t want = edge | 1ull << bit;
        int mine = 0;
        for (uint32_t j = v0 + threadIdx.x; j < v1; j += kBeamThreads) {
            float x[N];
            logits_of(row.load(j), x, T{});
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = beam_key(x[i], j * N + i) & RowVectors<T>::kKeyBits;
                mine += x[i] > -INFINITY && key >= want;
            }
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

// One slice of a row: its maximum, its sum of exponentials and its `top`
// greatest logits in order, into place `unit` of the first CTA.  All threads.
//
// Each thread streams its vectors once, keeping a running maximum and sum.  Of
// the maxima of 128 groups of threads the top-th greatest is a lower bound of the
// slice's top-th greatest logit, and only threads whose own maximum reaches it
// hold any that do: few more than `top`.  Their vectors are read again, a warp to
// each such thread, and what reaches the bound is put in order by counting.
template <typename T>
__device__ __forceinline__ void beam_slice(const BeamArgs& a, const T* logits, int part, int unit, uint64_t* lists,
                                           BeamShared& s) {
    constexpr int N = RowVectors<T>::kPer, U = kBeamUnroll;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const RowVectors<T> row(logits, a.vocab);
    const uint32_t v0 = (uint32_t)part * (uint32_t)(a.slice / N);
    const uint32_t all = (uint32_t)((a.vocab + N - 1) / N), v1 = min(v0 + (uint32_t)(a.slice / N), all);

    float m = -INFINITY;
    uint64_t sum2 = pack2(0.0f, 0.0f);
    for (uint32_t j0 = v0 + threadIdx.x; j0 < v1; j0 += kBeamThreads * U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t j = j0 + u * kBeamThreads;
            v[u] = row.load(j < v1 ? j : 0xffffffffu / N);
        }
        float x[U][N], best = m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            logits_of(v[u], x[u], T{});
#pragma unroll
            for (int i = 0; i < N; ++i) best = fmaxf(best, x[u][i]);
        }
        if (best > m) {
            const float down = exp2_fast((m - best) * kLog2e);
            sum2 = mul2(sum2, pack2(down, down));
            m = best;
        }
        if (m > -INFINITY) {
            const uint64_t less = pack2(-m, -m), log2e = pack2(kLog2e, kLog2e);
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    uint64_t d = pack2(x[u][i], x[u][i + 1]);
                    add2(d, less);
                    const float2 e = unpack2(mul2(d, log2e));
                    add2(sum2, pack2(exp2_fast(e.x), exp2_fast(e.y)));
                }
        }
    }
    const float2 halves = unpack2(sum2);
    float sum = halves.x + halves.y;

    // the slice's maximum and sum, and the groups' maxima
    float g = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((threadIdx.x & 3) == 0) s.group_max[threadIdx.x >> 2] = g;
    const float most = warp_max(g);
    sum = m > -INFINITY ? sum * exp2_fast((m - most) * kLog2e) : 0.0f;
    sum = warp_sum(sum);
    if (lane == 0) s.warp_max[warp] = most, s.warp_sum[warp] = sum;
    if (threadIdx.x == 0) s.near = 0, s.found = 0;
    __syncthreads();
    if (warp == 0) {
        constexpr int W = kBeamThreads / 32;
        const float wm = lane < W ? s.warp_max[lane] : -INFINITY;
        const float top_max = warp_max(wm);
        const float ws = warp_sum(lane < W && wm > -INFINITY ? s.warp_sum[lane] * exp2_fast((wm - top_max) * kLog2e) : 0.0f);
        if (lane == 0) store_peer(reinterpret_cast<uint64_t*>(&s.stats[unit]), 0, pack2(top_max, ws));
    }
    if (threadIdx.x < kBeamGroups) {
        const float mine = s.group_max[threadIdx.x];
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < kBeamGroups; i += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&s.group_max[i]);
            const float other[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                rank += other[k] > mine || (other[k] == mine && i + k < (int)threadIdx.x);
        }
        if (rank == a.top - 1) s.bound = mine;
    }
    __syncthreads();
    const float bound = s.bound;
    if (m >= bound && m > -INFINITY) s.who[atomicAdd(&s.near, 1)] = (uint16_t)threadIdx.x;
    __syncthreads();
    const int near = s.near;
    for (int k = warp; k < near; k += kBeamThreads / 32) {
        for (uint32_t j = v0 + s.who[k] + lane * kBeamThreads; j < v1; j += 32 * kBeamThreads) {
            float x[N];
            logits_of(row.load(j), x, T{});
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (x[i] >= bound && x[i] > -INFINITY) {
                    const int at = atomicAdd(&s.found, 1);
                    if (at < kBeamCandidates) s.key[at] = beam_key(x[i], j * N + i);
                }
        }
    }
    __syncthreads();
    int found = s.found;
    if (found > kBeamCandidates) {
        const uint64_t edge = settle_edge(row, v0, v1, a.top, s);
        if (threadIdx.x == 0) s.found = 0;
        __syncthreads();
        for (uint32_t j = v0 + threadIdx.x; j < v1; j += kBeamThreads) {
            float x[N];
            logits_of(row.load(j), x, T{});
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = beam_key(x[i], j * N + i);
                if (x[i] > -INFINITY && (key & RowVectors<T>::kKeyBits) >= edge) {
                    const int at = atomicAdd(&s.found, 1);  // `top` of them: keys differ
                    if (at < kBeamCandidates) s.key[at] = key;
                }
            }
        }
        __syncthreads();
        found = min(s.found, kBeamCandidates);
    }
    uint64_t* list = lists + unit * a.top;
    for (int c = threadIdx.x; c < found; c += kBeamThreads) {
        const uint64_t mine = s.key[c];
        int rank = 0;
        for (int o = 0; o < found; ++o) rank += s.key[o] > mine;
        if (rank < a.top) store_peer(list + rank, 0, mine);
    }
    for (int r = found + threadIdx.x; r < a.top; r += kBeamThreads) store_peer(list + r, 0, 0ull);
    __syncthreads();  // s is used again
}

// A cluster to each sequence; its slices ("units", beam by beam) go to the CTAs in
// turn, and the first CTA joins them: the beams' logarithms of their sums, the
// scores of the slices' best continuations in 64 bits, and the lists merged by one
// warp, a winner at a time.
template <typename T>
__global__ void __launch_bounds__(kBeamThreads, 2) beam_select_kernel(const BeamArgs a) {
    wait_for_stream();
    extern __shared__ __align__(16) unsigned char s_raw[];
    BeamShared& s = *reinterpret_cast<BeamShared*>(s_raw);
    uint64_t* lists = reinterpret_cast<uint64_t*>(s_raw + sizeof(BeamShared));
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    const int64_t b = blockIdx.x / ctas;
    const int units = a.beams * a.parts;
    if (ctas > 1) cluster_sync();  // the first CTA has started: its shared memory may be written
    for (int u = (int)rank; u < units; u += (int)ctas) {
        const int beam = u / a.parts, part = u - beam * a.parts;
        const float score = a.scores == nullptr ? 0.0f : a.scores[b * a.beams + beam];
        const bool ended = a.finished != nullptr && a.finished[b * a.beams + beam] != 0;
        // a beam that has ended, or whose score is -inf or NaN, has no logits to look at
        if (ended || !(score > -INFINITY)) {
            for (int r = threadIdx.x; r < a.top; r += kBeamThreads) store_peer(lists + u * a.top + r, 0, 0ull);
            if (threadIdx.x == 0) store_peer(reinterpret_cast<uint64_t*>(&s.stats[u]), 0, pack2(-INFINITY, 0.0f));
            continue;
        }
        const T* row = static_cast<const T*>(a.logits) + b * a.batch_stride + beam * a.beam_stride;
        beam_slice<T>(a, row, part, u, lists, s);
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
        float most = -INFINITY;
        for (int p = 0; p < a.parts; ++p) most = fmaxf(most, s.stats[i * a.parts + p].x);
        float sum = 0.0f;
        for (int p = 0; p < a.parts; ++p) {
            const float2 st = s.stats[i * a.parts + p];
            if (st.x > -INFINITY) sum += st.y * exp2_fast((st.x - most) * kLog2e);
        }
        s.lse[i] = (double)most + log((double)sum);
        s.score[i] = a.scores == nullptr ? 0.0f : a.scores[b * a.beams + i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < units * a.top; c += kBeamThreads) {
        const int beam = c / a.top / a.parts;
        uint64_t image = 0;
        if (lists[c] != 0) {
            const double v = (double)s.score[beam] + ((double)image_score((uint32_t)(lists[c] >> 32)) - s.lse[beam]);
            if ((float)v > -INFINITY) image = score_image64(v);
        }
        if (c % (a.top * a.parts) == 0 && a.finished != nullptr && a.finished[b * a.beams + beam] != 0) {
            lists[c] = (uint32_t)~(uint32_t)a.end_id;
            if (s.score[beam] > -INFINITY) image = score_image64((double)s.score[beam]);
        }
        images[c] = image;
    }
    __syncthreads();
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
        const int win = in0 != 0 ? __ffs(in0) - 1 : __ffs(in1) - 1;
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

struct BeamGatherArgs {
    om_beam_array arrays[kMaxBeamArrays];
    unsigned char vector[kMaxBeamArrays];
    const int32_t *parents, *starts, *lengths;
    int64_t entries, rows;  // rows: batch * heads
    int beams, heads, count, parts, in_place;
};

// A column of the beams (the same bytes of one entry in each) belongs to one
// thread, which loads what its beams get before it stores any of it: so the move
// works in place for every map of beams to parents, with no barrier.  A beam
// that keeps its own place is not touched in place.
//
// Bound by memory.
// BEAMS: beams loaded together (all of them in place).  STAGED: in place with
// more than that many, through shared memory.
template <typename V, int BEAMS, bool STAGED>
__device__ __forceinline__ void gather_columns(const BeamGatherArgs& a, const om_beam_array& c, int64_t b, int64_t h,
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

template <int BEAMS, bool STAGED>
__global__ void __launch_bounds__(kBeamGatherThreads) beam_gather_kernel(const __grid_constant__ BeamGatherArgs a) {
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

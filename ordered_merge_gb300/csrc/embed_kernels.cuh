// Kernels of om_embed_lookup and om_embed_lookup_backward: rows of a table by
// token, and the table's gradient by sorted tokens.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "select_common.cuh"

namespace om {

// A token as a row of the table, or -1 where it is none of its rows.
__device__ __forceinline__ int64_t embed_row(const void* ids, int wide, int64_t i, int64_t rows) {
    const int64_t id = wide ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
    return id >= 0 && id < rows ? id : -1;
}

// N values of type T as one vector.
template <typename T, int N>
struct alignas(sizeof(T) * N) ValueVec {
    T v[N];
};

// 16 bytes stored past the caches' usual order: they are not read again soon.
template <typename T, int N>
__device__ __forceinline__ void store_streaming(ValueVec<T, N>* p, const ValueVec<T, N>& v) {
    static_assert(sizeof(v) == 16, "one vector");
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
}

// 16 of 32 bytes, from byte `shift` (a multiple of two) below 16 on.
__device__ __forceinline__ uint4 shifted_vector(const uint4& low, const uint4& high, uint32_t shift) {
    uint32_t w[8] = {low.x, low.y, low.z, low.w, high.x, high.y, high.z, high.w};
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = shift & 8 ? w[k + 2] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = shift & 4 ? w[k + 1] : w[k];
    const uint32_t bits = 8 * (shift & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// --------------------------------------------------------------- lookup --

struct EmbedArgs {
    const void* table;
    const void* ids;
    void* out;
    int64_t rows, n, table_stride, out_stride;  // strides in values
    int width, wide;
    float scale;
};

constexpr int kEmbedThreads = 64;
constexpr int kEmbedUnroll = 4;

// CTAs of two warps take a tile of 256 vectors: several short rows or a piece of
// a long one.  All tokens first, then all vectors: two trips to memory.
//
// Bound by memory: 65536 rows of 2048 bf16 out of 131072, 0.41 GB with each row that
// is asked for read once, 71.7 us (5.7 TB/s; CTAs of 64 to 256 threads and 2 to 8
// vectors a thread come to the same or more).
template <typename T>
__global__ void __launch_bounds__(kEmbedThreads) embed_lookup_kernel(const EmbedArgs a) {
    wait_for_stream();
    constexpr int N = 16 / (int)sizeof(T);
    using V = ValueVec<T, N>;
    const int per = a.width / N;
    const uint32_t total_tile = kEmbedThreads * kEmbedUnroll;
    int64_t token[kEmbedUnroll];
    int piece[kEmbedUnroll];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
        const int64_t i = (int64_t)blockIdx.x * total_tile + u * kEmbedThreads + threadIdx.x;
        const int64_t t = i <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
        token[u] = t;
        piece[u] = (int)(i - t * per) * N;
    }
    int64_t row[kEmbedUnroll];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) row[u] = token[u] < a.n ? embed_row(a.ids, a.wide, token[u], a.rows) : -1;
    V v[kEmbedUnroll];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
#pragma unroll
        for (int k = 0; k < N; ++k) v[u].v[k] = from_float<T>(0.0f);
        if (row[u] >= 0) {
            const T* from = static_cast<const T*>(a.table) + row[u] * a.table_stride + piece[u];
            const uint4 bits = load_once(reinterpret_cast<const uint4*>(from));  // volatile, so that all are on their way together (75.8 us otherwise)
            v[u] = *reinterpret_cast<const V*>(&bits);
        }
    }
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
        if (token[u] >= a.n) continue;
        if (row[u] >= 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[u].v[k] = from_float<T>(to_float(v[u].v[k]) * a.scale);
        }
        store_streaming(reinterpret_cast<V*>(static_cast<T*>(a.out) + token[u] * a.out_stride + piece[u]), v[u]);
    }
}

// The same for rows that 16-byte vectors do not fit: a thread writes a whole aligned
// vector of the output, from the one or two aligned vectors of the table that hold its
// bytes; at a row's ends value by value.  65536 rows of 2047 bf16 122 us, of 2044 121 (by
// single values 527, by vectors of 8 bytes 264); 32768 of 2047 f32 117 (264), of 2046 116 (133).
template <typename T>
__global__ void __launch_bounds__(kEmbedThreads) embed_lookup_odd_kernel(const EmbedArgs a) {
    wait_for_stream();
    constexpr int kValues = 16 / (int)sizeof(T);
    const int64_t length = (int64_t)a.width * (int)sizeof(T);
    const int per = (int)((length + 30) / 16);  // vectors that a row touches, at most
    int64_t token[kEmbedUnroll];
    int piece[kEmbedUnroll];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
        const int64_t i = (int64_t)blockIdx.x * (kEmbedThreads * kEmbedUnroll) + u * kEmbedThreads + threadIdx.x;
        token[u] = i <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)per) : i / per;
        piece[u] = (int)(i - token[u] * per);
    }
    int64_t row[kEmbedUnroll];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) row[u] = token[u] < a.n ? embed_row(a.ids, a.wide, token[u], a.rows) : -1;
    uint4 low[kEmbedUnroll], high[kEmbedUnroll];
    uint32_t shift[kEmbedUnroll];
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
        const uintptr_t to = reinterpret_cast<uintptr_t>(static_cast<T*>(a.out) + token[u] * a.out_stride);
        const uintptr_t from = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.table) + row[u] * a.table_stride);
        // of the table what the output's vector holds; it may begin before the row
        const int64_t offset = (int64_t)piece[u] * 16 - (int64_t)(to & 15);
        const uintptr_t first = (from + offset) & ~(uintptr_t)15;
        shift[u] = (uint32_t)(from + offset) & 15;
        low[u] = high[u] = make_uint4(0, 0, 0, 0);
        if (row[u] >= 0 && offset < length) {  // only vectors that hold some of the row
            if (first + 16 > from && first < from + length) low[u] = *reinterpret_cast<const uint4*>(first);
            if (shift[u] != 0 && first + 16 < from + length) high[u] = reinterpret_cast<const uint4*>(first)[1];
        }
    }
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
        if (token[u] >= a.n) continue;
        T* to = static_cast<T*>(a.out) + token[u] * a.out_stride;
        const int64_t offset = (int64_t)piece[u] * 16 - (int64_t)(reinterpret_cast<uintptr_t>(to) & 15);
        if (offset >= length) continue;
        const uint4 bits = shifted_vector(low[u], high[u], shift[u]);
        ValueVec<T, kValues> v = *reinterpret_cast<const ValueVec<T, kValues>*>(&bits);
        if (a.scale != 1.0f && row[u] >= 0) {
#pragma unroll
            for (int k = 0; k < kValues; ++k) v.v[k] = from_float<T>(to_float(v.v[k]) * a.scale);
        }
        T* at = to + offset / (int)sizeof(T);
        if (offset >= 0 && offset + 16 <= length) {
            store_streaming(reinterpret_cast<ValueVec<T, kValues>*>(at), v);
        } else {
#pragma unroll
            for (int k = 0; k < kValues; ++k)
                if (offset + k * (int)sizeof(T) >= 0 && offset + k * (int)sizeof(T) < length) at[k] = v.v[k];
        }
    }
}

// ------------------------------------------------------------- gradient --
//
// The tokens are sorted stably; the rows of equal tokens are then neighbours, and
// are summed in their order.  The same launch writes the zeros of the rows that no
// token asks for; a last one joins the pieces of long runs.

struct EmbedBackArgs {
    const void* grad;
    const void* ids;
    void* grad_table;
    uint32_t *keys, *slots;            // tokens sorted (rows: none of the table's), and where they stand
    uint32_t *other_keys, *other_slots;  // (sorting) the passes' other side
    float* partial;  // sums of the pieces of long runs
    int64_t n, rows, grad_stride, table_stride;
    int width, wide, accumulate;
    int tiles;            // column tiles of a row
    int window;           // sorted places of a warp
    int piece_bits;       // tokens of a long run that one warp sums: 1 << piece_bits
    int passes, bits;     // (sorting) digits of a key and bits of a digit
    int64_t sum_ctas;     // CTAs that sum; those after them write zeros
    int zero_rows;        // rows of a warp of them
    float scale;
};

// Tokens of a run that one warp sums (a power of two of them): of few tokens, and of many.
constexpr int kEmbedPieceBits = 5;
constexpr int kEmbedLongPieceBits = 7;

// ---- the sort: one cluster, least digit first
//
// As in the grouping of slots by id: a place is the sum of the places of lower
// digits, those of its own in the chunks of the CTAs before, in the parts of the
// warps before, and before it in its warp's part.  Counts go through the cluster's
// shared memory.  A chunk is put in order in shared memory and leaves it in runs of
// equal digits.
//
// Bound by the 16 SMs that a cluster has: 65537 tokens, two digits of 9 bits, 25.9 us,
// of which ranking takes 10.5 (nine votes for 32 tokens), counting 2.6, the cluster's
// meetings and sums 6.  (Stores straight from the lanes, a line each: 27.1.)
constexpr int kEmbedCluster = 16;
constexpr int kEmbedSortThreads = 1024;
constexpr int kEmbedSortWarps = kEmbedSortThreads / 32;
constexpr int kEmbedDigits = 512;
// Shared memory for a CTA's chunk of the tokens: the counts, and the chunk in order.
inline size_t embed_sort_smem(int64_t chunk) { return (size_t)(kEmbedSortWarps + 3) * kEmbedDigits * 4 + (size_t)chunk * 8; }

struct EmbedDigits {
    const EmbedBackArgs& a;
    const uint32_t *keys, *slots;  // nullptr: the tokens themselves
    int shift;

    // Two words of place i; written by other CTAs of the cluster, so past the L1 cache.
    __device__ __forceinline__ uint32_t key(int64_t i) const {
        if (keys != nullptr) return (uint32_t)load_l2(reinterpret_cast<const int*>(keys + i));
        const int64_t row = embed_row(a.ids, a.wide, i, a.rows);
        return row >= 0 ? (uint32_t)row : (uint32_t)a.rows;
    }
    __device__ __forceinline__ uint32_t slot(int64_t i) const {
        return slots != nullptr ? (uint32_t)load_l2(reinterpret_cast<const int*>(slots + i)) : (uint32_t)i;
    }
    __device__ __forceinline__ int digit(uint32_t key) const { return (int)(key >> shift) & ((1 << a.bits) - 1); }
};

__global__ void __launch_bounds__(kEmbedSortThreads) embed_sort_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    extern __shared__ int s_next[];  // [warps][digits]: a warp's counts, then its next place less the CTA's first
    __shared__ int2 s_part[kEmbedSortWarps];
    int* s_count = s_next + kEmbedSortWarps * kEmbedDigits;
    int* s_first = s_count + kEmbedDigits;  // a digit's first place, less its first in the chunk
    int* s_local = s_first + kEmbedDigits;  // and that
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t chunk = (a.n + kEmbedCluster - 1) / kEmbedCluster;
    const int64_t lo = min((int64_t)rank * chunk, a.n), hi = min(lo + chunk, a.n);
    const int64_t part = ((hi - lo + kEmbedSortWarps - 1) / kEmbedSortWarps + 31) / 32 * 32;
    const int64_t wlo = min(lo + warp * part, hi), whi = min(wlo + part, hi);
    int* next = s_next + warp * kEmbedDigits;
    uint32_t* s_key = reinterpret_cast<uint32_t*>(s_local + kEmbedDigits);
    uint32_t* s_slot = s_key + chunk;
    constexpr int U = 4;
    for (int pass = 0; pass < a.passes; ++pass) {
        // the last pass ends in keys and slots
        const bool even = (a.passes - 1 - pass) % 2 == 0;
        const EmbedDigits from{a, pass == 0 ? nullptr : even ? a.other_keys : a.keys,
                               pass == 0 ? nullptr : even ? a.other_slots : a.slots, pass * a.bits};
        uint32_t* to_keys = even ? a.keys : a.other_keys;
        uint32_t* to_slots = even ? a.slots : a.other_slots;
        for (int d = lane; d < kEmbedDigits / 4; d += 32) reinterpret_cast<int4*>(next)[d] = make_int4(0, 0, 0, 0);
        __syncwarp();
        for (int64_t i0 = wlo + lane; i0 < whi; i0 += 32 * U) {
            uint32_t key[U];
#pragma unroll
            for (int u = 0; u < U; ++u) key[u] = i0 + 32 * u < whi ? from.key(i0 + 32 * u) : 0;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + 32 * u < whi) atomicAdd(&next[from.digit(key[u])], 1);
        }
        __syncthreads();
        if (threadIdx.x < kEmbedDigits) {
            int run = 0;
#pragma unroll 8
            for (int w = 0; w < kEmbedSortWarps; ++w) {
                const int c = s_next[w * kEmbedDigits + threadIdx.x];
                s_next[w * kEmbedDigits + threadIdx.x] = run;
                run += c;
            }
            s_count[threadIdx.x] = run;
        }
        cluster_sync();
        // a digit's total, what lies before this CTA's, and the sums of both over lower digits
        int total = 0, before = 0, mine = 0, run = 0, local = 0;
        if (threadIdx.x < kEmbedDigits) {
            mine = s_count[threadIdx.x];
            int count[kEmbedCluster];
#pragma unroll
            for (uint32_t r = 0; r < kEmbedCluster; ++r) count[r] = peer_word(s_count + threadIdx.x, r);
#pragma unroll
            for (uint32_t r = 0; r < kEmbedCluster; ++r) total += count[r], before += r < rank ? count[r] : 0;
            run = total, local = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, run, d), up_local = __shfl_up_sync(0xffffffffu, local, d);
                if (lane >= d) run += up, local += up_local;
            }
            if (lane == 31) s_part[warp] = make_int2(run, local);
        }
        __syncthreads();
        if (threadIdx.x < kEmbedDigits) {
            const int2 sums = lane < warp ? s_part[lane] : make_int2(0, 0);  // 16 warps at most
            const int lower = __reduce_add_sync(0xffffffffu, sums.x) + run - total;
            const int lower_local = __reduce_add_sync(0xffffffffu, sums.y) + local - mine;
            s_local[threadIdx.x] = lower_local;
            s_first[threadIdx.x] = lower + before - lower_local;
        }
        __syncthreads();
        const unsigned before_me = (1u << lane) - 1;
        for (int64_t i0 = wlo; i0 < whi; i0 += 32 * U) {
            uint32_t key[U], slot[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + 32 * u + lane;
                key[u] = i < whi ? from.key(i) : 0;
                slot[u] = i < whi ? from.slot(i) : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + 32 * u >= whi) break;
                const bool live = i0 + 32 * u + lane < whi;
                const int g = from.digit(key[u]);
                unsigned same = __ballot_sync(0xffffffffu, live);
#pragma unroll
                for (int bit = 0; bit < 9; ++bit) {
                    const bool one = g >> bit & 1;
                    same &= __ballot_sync(0xffffffffu, one) ^ (one ? 0u : 0xffffffffu);
                }
                const int place = __popc(same & before_me);
                const int at = next[g] + place;
                __syncwarp();
                if (live && place == 0) next[g] = at + __popc(same);
                __syncwarp();
                if (live) s_key[s_local[g] + at] = key[u], s_slot[s_local[g] + at] = slot[u];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < (int)(hi - lo); i += kEmbedSortThreads) {
            const uint32_t key = s_key[i];
            const int to = s_first[from.digit(key)] + i;
            __stcg(to_keys + to, key);
            __stcg(to_slots + to, s_slot[i]);
        }
        __threadfence();
        cluster_sync();  // what this pass wrote the next one reads; no CTA leaves, or counts anew, before
    }
}

// The same for few tokens, by all SMs and without a pass over digits: the place of
// a token is the number of smaller ones and of equal ones before it.  A CTA counts
// for 32 tokens, a lane each; its warps share out what they are compared with, which
// lies in shared memory.  4096 tokens: 5.5 us; by a cluster's digits 12, and with one
// CTA's in shared memory 10.
constexpr int64_t kEmbedSmallMost = 8192;
constexpr int kEmbedSmallThreads = 512;

__global__ void __launch_bounds__(kEmbedSmallThreads) embed_sort_small_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    extern __shared__ __align__(16) uint32_t s_key[];  // all keys, then the warps' counts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = (int)a.n, i0 = blockIdx.x * 32, i = i0 + lane;
    const int whole = (n + 31) / 32 * 32;
    for (int j = threadIdx.x; j < whole; j += kEmbedSmallThreads) {
        const int64_t row = j < n ? embed_row(a.ids, a.wide, j, a.rows) : 0;
        s_key[j] = j >= n ? 0xffffffffu : row >= 0 ? (uint32_t)row : (uint32_t)a.rows;  // past the end: smaller than none
    }
    __syncthreads();
    const uint32_t mine = s_key[i];
    int count = 0;
    // 32 at a time: those before mine count when equal, those after do not
    for (int b = warp; b < whole / 32; b += kEmbedSmallThreads / 32) {
        const uint4* other = reinterpret_cast<const uint4*>(s_key + 32 * b);
        if (32 * b == i0) {
            for (int k = 0; k < 32; ++k) count += s_key[i0 + k] < mine || (s_key[i0 + k] == mine && k < lane);
        } else {
            const bool before = 32 * b < i0;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint4 v = other[q];
                if (before) count += (v.x <= mine) + (v.y <= mine) + (v.z <= mine) + (v.w <= mine);
                else count += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
            }
        }
    }
    int* s_count = reinterpret_cast<int*>(s_key + whole);
    s_count[threadIdx.x] = count;
    __syncthreads();
    if (warp == 0 && i < n) {
        int place = 0;
#pragma unroll
        for (int w = 0; w < kEmbedSmallThreads / 32; ++w) place += s_count[w * 32 + lane];
        a.keys[place] = mine;
        a.slots[place] = (uint32_t)i;
    }
}

// Sort keys for more tokens than one cluster sorts.
__global__ void __launch_bounds__(256) embed_keys_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.n) return;
    const int64_t row = embed_row(a.ids, a.wide, i, a.rows);
    a.keys[i] = row >= 0 ? (uint32_t)row : (uint32_t)a.rows;
    a.slots[i] = (uint32_t)i;
}

// ---- sums

constexpr int kEmbedSumThreads = 128;
constexpr int kEmbedSumRows = 16;  // rows of a warp in flight

// Copies a vector into shared memory in the background.
__device__ __forceinline__ void copy_async(uint4* to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of the groups committed last are on their way.
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// First sorted place whose key is at least `key`, in [lo, hi].
__device__ __forceinline__ int64_t first_place(const uint32_t* keys, int64_t lo, int64_t hi, uint32_t key) {
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// The same for one key by a warp, which looks at 32 places at a time.
__device__ __forceinline__ int64_t first_place_warp(const uint32_t* keys, int64_t lo, int64_t hi, uint32_t key) {
    const int lane = threadIdx.x & 31;
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, probe = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, probe < hi && keys[probe] < key);
        const int n = __popc(below);  // probes rise, so the first n of them are below
        if (n == 0) return lo;
        hi = min(hi, lo + n * step);
        lo = lo + (n - 1) * step + 1;
    }
    return lo;
}

// The slot of a piece's sum in `partial`: pieces start at multiples of their length from
// their run's start, so at most one piece that goes on a run and one that starts a
// long run start in the same places between two multiples.
__device__ __forceinline__ int64_t piece_slot(const EmbedBackArgs& a, int64_t at, bool first) {
    return 2 * (at >> a.piece_bits) + first;
}

// N sums of a lane to a row of the table's gradient (scaled), or as they are.
template <typename O, int N>
__device__ __forceinline__ void store_sums(const EmbedBackArgs& a, uint32_t row, int column, const float (&sum)[N]) {
    constexpr int W = N * (int)sizeof(O) > 16 ? 16 / (int)sizeof(O) : N;  // values of a store
    using V = ValueVec<O, W>;
    O* out = static_cast<O*>(a.grad_table) + (int64_t)row * a.table_stride + column;
#pragma unroll
    for (int p = 0; p < N; p += W) {
        V v;
        if (a.accumulate) v = *reinterpret_cast<const V*>(out + p);
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float x = sum[p + k] * a.scale;
            v.v[k] = from_float<O>(a.accumulate ? to_float(v.v[k]) + x : x);
        }
        *reinterpret_cast<V*>(out + p) = v;
    }
}

// Zeros in those rows of a warp's share that no token asks for.
template <typename O, bool ODD>
__device__ __forceinline__ void zero_rows(const EmbedBackArgs& a, int64_t warp) {
    constexpr int W = 16 / (int)sizeof(O);  // values of a store
    using V = ValueVec<O, W>;
    const int lane = threadIdx.x & 31;
    const int64_t lo = warp * a.zero_rows, mine = lo + lane;
    if (lo >= a.rows) return;
    // the sorted tokens from the first of these rows on: mostly few, or none
    const int64_t at = first_place_warp(a.keys, 0, a.n, (uint32_t)lo);
    const uint32_t key = at + lane < a.n ? a.keys[at + lane] : 0xffffffffu;
    const uint32_t there = __reduce_or_sync(0xffffffffu, key - (uint32_t)lo < 32 ? 1u << (key - (uint32_t)lo) : 0u);
    bool absent = lane < a.zero_rows && mine < a.rows && !(there >> lane & 1);
    if (__shfl_sync(0xffffffffu, key, 31) < lo + a.zero_rows && absent) {  // more than 32 tokens ask for them
        const int64_t p = first_place(a.keys, at, a.n, (uint32_t)mine);
        absent = p == a.n || a.keys[p] != (uint32_t)mine;
    }
    V none;
#pragma unroll
    for (int k = 0; k < W; ++k) none.v[k] = from_float<O>(0.0f);
    for (unsigned todo = __ballot_sync(0xffffffffu, absent); todo != 0; todo &= todo - 1) {
        O* out = static_cast<O*>(a.grad_table) + (lo + __ffs(todo) - 1) * a.table_stride;
        int from = 0;  // what lies before the first whole vector
        if constexpr (ODD) {
            from = min((int)(-reinterpret_cast<uintptr_t>(out) & 15) / (int)sizeof(O), a.width);
            if (lane < from) out[lane] = none.v[0];
            const int rest = (a.width - from) % W;
            if (lane < rest) out[a.width - rest + lane] = none.v[0];
        }
        for (int c = from + lane * W, end = a.width - W; c <= end; c += 32 * W) store_streaming(reinterpret_cast<V*>(out + c), none);
    }
}

// A warp looks after the pieces that start in its window of sorted places, for a
// tile of 32 N columns.  A piece is a run of equal tokens, or 32 (128)
// places of a longer one, counted from its start; so those of a window are
// neighbours, and the warp streams their rows, 16 in flight through shared memory
// (each lane copies and reads its own vectors: no barrier), adding each to the sum
// in its order and putting the sum away where a piece ends: to the table, or, for
// pieces of a longer run, to `partial`.
//
// ODD: rows that 16-byte vectors do not fit come in as the aligned vectors that hold
// them, 33 for the 32 of a tile, and each lane shifts its columns out of two; sums go out
// through shared memory, neighbouring lanes' value by value.  (32784 rows of 2047 bf16 to
// as many rows 88 us, by single values 201; of 2046 to f32 98, by two values 122.)
//
// Zeros: a warp searches the sorted tokens for its rows.
//
// Bound by memory: 65537 tokens into 131072 rows of 2048, bf16 to f32, 1.34 GB, 188 us
// (7.1 TB/s).  (Rows in registers, eight at a time, took 128 us for the sums alone,
// which take 83 so; the zeros apart from them, beside the sort, as much in all.)
template <typename T, typename O, bool ODD>
__global__ void __launch_bounds__(kEmbedSumThreads) embed_sum_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    if ((int64_t)blockIdx.x >= a.sum_ctas) {
        zero_rows<O, ODD>(a, ((int64_t)blockIdx.x - a.sum_ctas) * (kEmbedSumThreads / 32) + (threadIdx.x >> 5));
        return;
    }
    constexpr int N = 16 / (int)sizeof(T), D = kEmbedSumRows, R = ODD ? 33 : 32;
    using V = ValueVec<T, N>;
    // a warp's ring and, ODD, the sums on their way out
    __shared__ uint4 s_ring[kEmbedSumThreads / 32][D * R + (ODD ? 8 * N : 0)];
    const int lane = threadIdx.x & 31;
    uint4* ring = &s_ring[threadIdx.x >> 5][lane];
    const int64_t warp = (int64_t)blockIdx.x * (kEmbedSumThreads / 32) + (threadIdx.x >> 5);
    const int64_t w = warp / a.tiles, lo = w * a.window;
    if (lo >= a.n) return;
    const int column = (int)(warp - w * a.tiles) * (32 * N) + lane * N;
    const bool inside = column < a.width;
    const T* grad = static_cast<const T*>(a.grad) + column;
    float sum[N];
    int64_t at = -1;  // where the piece being summed starts, its token, and whether it starts its run
    uint32_t row = 0;
    bool run_start = false;
#pragma unroll
    for (int n = 0; n < N; ++n) sum[n] = 0.0f;
    auto put_away = [&](uint32_t next_key) {
        if (at < 0) return;
        if constexpr (ODD) {  // neighbouring lanes store neighbouring values
            float* all = reinterpret_cast<float*>(&s_ring[threadIdx.x >> 5][D * R]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < N; ++k) all[lane * N + k] = sum[k];
            __syncwarp();
            const bool whole_run = run_start && next_key != row;
            const int first = column - lane * N, most = min(32 * N, a.width - first);
            O* table = static_cast<O*>(a.grad_table) + (int64_t)row * a.table_stride + first;
            float* part = a.partial + piece_slot(a, at, run_start) * a.width + first;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int c = 32 * k + lane;
                if (c >= most) break;
                if (whole_run) table[c] = from_float<O>(a.accumulate ? to_float(table[c]) + all[c] * a.scale : all[c] * a.scale);
                else part[c] = all[c];
            }
            return;
        }
        if (!inside) return;
        if (run_start && next_key != row) {
            store_sums<O, N>(a, row, column, sum);
        } else {
            float* out = a.partial + piece_slot(a, at, run_start) * a.width + column;
#pragma unroll
            for (int k = 0; k < N; ++k) out[k] = sum[k];
        }
    };
    for (int64_t base = lo;; base += 32) {
        const int64_t mine = base + lane;
        uint32_t key = 0xffffffffu, slot = 0;
        bool starts = false, first = false;
        if (mine < a.n) {
            key = a.keys[mine];
            slot = a.slots[mine];
            first = mine == 0 || a.keys[mine - 1] != key;
            starts = first;
        }
        const unsigned outside = __ballot_sync(0xffffffffu, key >= (uint32_t)a.rows);
        const unsigned firsts = __ballot_sync(0xffffffffu, first);
        // Further pieces of a long run among these places: only of the run that the first
        // one is in the midst of (one that starts here has its next piece 32 places on at least).
        const uint32_t key0 = __shfl_sync(0xffffffffu, key, 0);
        if (!(firsts & 1) && key0 < (uint32_t)a.rows) {
            // where that run started, if it was in the 32 places before, or else by a search
            const int64_t back = max(base - 32, (int64_t)0);
            const unsigned there = __ballot_sync(0xffffffffu, back + lane < base && a.keys[back + lane] != key0);
            int64_t run;
            if (there != 0) run = back + 32 - __clz(there);
            else run = first_place_warp(a.keys, 0, back, key0);
            if (mine < a.n && key == key0 && !first) starts = ((mine - run) & ((1 << a.piece_bits) - 1)) == 0;
        }
        const unsigned start = __ballot_sync(0xffffffffu, starts);
        const unsigned window = base > lo ? 0u : a.window >= 32 ? 0xffffffffu : (1u << a.window) - 1;
        const unsigned stops = (start & ~window) | outside;
        const int stop = stops != 0 ? __ffs(stops) - 1 : 32;
        int r = 0;
        if (at < 0) {
            r = (start & window & ~outside) != 0 ? __ffs(start & window & ~outside) - 1 : 32;
            if (r > stop || r == 32) return;  // no piece starts here
        }
        const int count = stop - r;
        auto fetch = [&](int i) {
            const uint32_t from = __shfl_sync(0xffffffffu, slot, (r + i) & 31);
            if constexpr (ODD) {  // the aligned vectors that hold some of the row's part
                const uintptr_t row_at = reinterpret_cast<uintptr_t>(static_cast<const T*>(a.grad) + (int64_t)from * a.grad_stride);
                const uintptr_t end = row_at + (uintptr_t)a.width * sizeof(T);
                const uintptr_t first = (row_at + (uintptr_t)(column - lane * N) * sizeof(T)) & ~(uintptr_t)15;
                if (i < count && first + 16 * lane < end)
                    copy_async(ring + (i % D) * R, reinterpret_cast<const uint4*>(first) + lane);
                if (i < count && lane == 0 && first + 512 < end)
                    copy_async(ring + (i % D) * R + 32, reinterpret_cast<const uint4*>(first) + 32);
            } else {
                if (i < count && inside)
                    copy_async(ring + (i % D) * R, reinterpret_cast<const uint4*>(grad + (int64_t)from * a.grad_stride));
            }
            copy_commit();
        };
        for (int i = 0; i < D; ++i) fetch(i);
        for (int i = 0; i < count; ++i) {
            copy_wait<D - 1>();
            uint4 bits;
            if constexpr (ODD) {
                __syncwarp();  // other lanes' copies
                const uint32_t from = __shfl_sync(0xffffffffu, slot, r + i);
                const uint32_t low_bits = (uint32_t)reinterpret_cast<uintptr_t>(grad) + from * (uint32_t)(a.grad_stride * (int)sizeof(T));
                bits = shifted_vector(ring[(i % D) * R], ring[(i % D) * R + 1], low_bits & 15);
                __syncwarp();  // the vectors are copied over next
            } else {
                bits = ring[(i % D) * R];
            }
            const V v = *reinterpret_cast<const V*>(&bits);
            const uint32_t k = __shfl_sync(0xffffffffu, key, r + i);
            if (start >> (r + i) & 1) {
                put_away(k);
                at = base + r + i, row = k, run_start = firsts >> (r + i) & 1;
#pragma unroll
                for (int n = 0; n < N; ++n) sum[n] = 0.0f;
            }
            if (inside) {
#pragma unroll
                for (int n = 0; n < N; ++n) sum[n] += to_float(v.v[n]);
            }
            fetch(i + D);
        }
        if (stop < 32) {
            put_away(__shfl_sync(0xffffffffu, key, stop));
            return;
        }
    }
}

// Long runs: the pieces' sums in order.  A run longer than a piece
// holds a multiple of its length after its start; the first of them is the one
// whose CTA adds them.  A CTA looks at a few multiples, and each of its warps has
// 128 columns.  13 us for the 65537 tokens above, of a run of 3000 and many shorter
// ones: a chain of loads, most of them from memory.
constexpr int kEmbedJoinThreads = 128;
constexpr int kEmbedJoinColumns = 4 * kEmbedJoinThreads;  // four to a lane
constexpr int kEmbedJoinPlaces = 4;

template <typename O>
__global__ void __launch_bounds__(kEmbedJoinThreads) embed_join_kernel(const EmbedBackArgs a, int tiles) {
    wait_for_stream();
    const int lane = threadIdx.x & 31, piece = 1 << a.piece_bits;
    const int64_t group = blockIdx.x / tiles;
    const int column = (int)(blockIdx.x - group * tiles) * kEmbedJoinColumns + (int)(threadIdx.x >> 5) * 128 + lane;
    bool mine = false;
    if (lane < kEmbedJoinPlaces) {
        const int64_t at = (group * kEmbedJoinPlaces + lane + 1) * piece, lo = at - piece;
        if (at < a.n) {
            const uint32_t key = a.keys[at], last = a.keys[at - 1], low = a.keys[lo];
            const uint32_t lower = lo > 0 ? a.keys[lo - 1] : 0xffffffffu;
            mine = key < (uint32_t)a.rows && last == key && !(low == key && lower == key);
        }
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, mine); todo != 0; todo &= todo - 1) {
        const int64_t at = (group * kEmbedJoinPlaces + __ffs(todo)) * piece;
        const uint32_t key = a.keys[at];
        const int64_t start = first_place_warp(a.keys, at - piece, at, key);
        const int64_t end = first_place_warp(a.keys, at, a.n, key + 1);
        if (end - start <= piece) continue;
        const int64_t pieces = (end - start + piece - 1) >> a.piece_bits;
        // piece p starts in the block of places p blocks after the run's start
        const float* first = a.partial + piece_slot(a, start, true) * a.width;
        const float* others = a.partial + piece_slot(a, start, false) * a.width;
        const int64_t step = 2 * (int64_t)a.width;
        float sum[4] = {};
        constexpr int U = 16;
        for (int64_t p = 0; p < pieces; p += U) {
            float v[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[u][k] = p + u < pieces && column + 32 * k < a.width
                                  ? (p + u == 0 ? first : others + (p + u) * step)[column + 32 * k]
                                  : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < 4; ++k) sum[k] += v[u][k];
        }
        O* out = static_cast<O*>(a.grad_table) + (int64_t)key * a.table_stride;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = column + 32 * k;
            if (c >= a.width) continue;
            const float x = sum[k] * a.scale;
            out[c] = from_float<O>(a.accumulate ? to_float(out[c]) + x : x);
        }
    }
}

}  // namespace om

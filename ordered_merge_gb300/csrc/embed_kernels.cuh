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

// N values of type T as one vector, the widest that the addresses allow.
template <typename T, int N>
struct alignas(sizeof(T) * N) ValueVec {
    T v[N];
};

// --------------------------------------------------------------- lookup --

struct EmbedArgs {
    const void* table;
    const void* ids;
    void* out;
    int64_t rows, n, table_stride, out_stride;  // strides in values
    int width, wide;
    int tiles, tile_vectors;  // of a row, and vectors of a tile
    float scale;
};

constexpr int kEmbedThreads = 64;
constexpr int kEmbedUnroll = 4;

// CTAs of two warps take a tile of 256 vectors: several short rows or a piece of
// a long one.  All tokens first, then all vectors: two trips to memory.
template <typename T, int N>
__global__ void __launch_bounds__(kEmbedThreads) embed_lookup_kernel(const EmbedArgs a) {
    wait_for_stream();
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
        if (row[u] >= 0)
            v[u] = *reinterpret_cast<const V*>(static_cast<const T*>(a.table) + row[u] * a.table_stride + piece[u]);
    }
#pragma unroll
    for (int u = 0; u < kEmbedUnroll; ++u) {
        if (token[u] >= a.n) continue;
        if (row[u] >= 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[u].v[k] = from_float<T>(to_float(v[u].v[k]) * a.scale);
        }
        *reinterpret_cast<V*>(static_cast<T*>(a.out) + token[u] * a.out_stride + piece[u]) = v[u];
    }
}

// ------------------------------------------------------------- gradient --

struct EmbedBackArgs {
    const void* grad;
    const void* ids;
    void* grad_table;
    uint32_t *keys, *slots;  // tokens sorted (rows: none of the table's), and where they stand
    float* partial;          // sums of the pieces of long runs
    int64_t n, rows, grad_stride, table_stride;
    int width, wide, accumulate;
    int tiles;               // column tiles of a row
    int window;              // sorted places of a warp
    int64_t sum_ctas, zero_rows;  // CTAs that sum, and rows that a zeroing warp looks after
    float scale;
};

constexpr int kEmbedBackThreads = 128;
constexpr int kEmbedPiece = 64;  // tokens of a run that one warp sums
constexpr int kEmbedTile = 1024;  // columns of a warp

// Sort keys: tokens that are no row of the table come last.
__global__ void __launch_bounds__(256) embed_keys_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.n) return;
    const int64_t row = embed_row(a.ids, a.wide, i, a.rows);
    a.keys[i] = row >= 0 ? (uint32_t)row : (uint32_t)a.rows;
    a.slots[i] = (uint32_t)i;
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

// A lane's columns of a tile: vectors of N values, 32 vectors a step, C of them.
template <typename T, int N>
struct EmbedLane {
    static constexpr int kSteps = kEmbedTile / (32 * N);
};

// The sum of `count` sorted places' rows, in their order, for a lane's columns.
// Two rows at a time are in flight.
template <typename T, int N>
__device__ __forceinline__ void sum_run(const EmbedBackArgs& a, int64_t at, int count, int column,
                                        float (&sum)[kEmbedTile / 32]) {
    constexpr int S = EmbedLane<T, N>::kSteps;
    using V = ValueVec<T, N>;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kEmbedTile / 32; ++k) sum[k] = 0.0f;
    for (int r = 0; r < count; ++r) {
        const T* row = static_cast<const T*>(a.grad) + (int64_t)a.slots[at + r] * a.grad_stride + column;
        V v[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int c = (s * 32 + lane) * N;
            if (column + c < a.width) v[s] = *reinterpret_cast<const V*>(row + c);
            else
#pragma unroll
                for (int k = 0; k < N; ++k) v[s].v[k] = from_float<T>(0.0f);
        }
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int k = 0; k < N; ++k) sum[s * N + k] += to_float(v[s].v[k]);
    }
}

// A row of the table's gradient from its sum.
template <typename O, int N>
__device__ __forceinline__ void store_row(const EmbedBackArgs& a, uint32_t row, int column, int steps,
                                          const float (&sum)[kEmbedTile / 32]) {
    const int lane = threadIdx.x & 31;
    using V = ValueVec<O, N>;
    O* out = static_cast<O*>(a.grad_table) + (int64_t)row * a.table_stride + column;
#pragma unroll
    for (int s = 0; s < kEmbedTile / (32 * N); ++s) {
        const int c = (s * 32 + lane) * N;
        if (column + c >= a.width) continue;
        V v;
        if (a.accumulate) v = *reinterpret_cast<const V*>(out + c);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const float x = sum[s * N + k] * a.scale;
            v.v[k] = from_float<O>(a.accumulate ? to_float(v.v[k]) + x : x);
        }
        *reinterpret_cast<V*>(out + c) = v;
    }
}

// The slot of a piece's sum in `partial`: pieces start at multiples of
// kEmbedPiece from their run's start, so at most one piece that goes on a run and
// one that starts a long run start in the same kEmbedPiece places.
__device__ __forceinline__ int64_t piece_slot(int64_t at, bool first) { return 2 * (at / kEmbedPiece) + first; }

// Sums: a warp looks after `window` sorted places and the column tiles of one
// tile; for each place that starts a run of equal tokens, or a further piece of a
// long run, it sums the run (or the piece) in order.  Short runs go straight to
// the table, pieces of long ones to `partial`.
// Zeros: rows that no token asks for, found by a search of the sorted tokens.
template <typename T, typename O, int N>
__global__ void __launch_bounds__(kEmbedBackThreads) embed_sum_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (kEmbedBackThreads / 32) + (threadIdx.x >> 5);
    if ((int64_t)blockIdx.x >= a.sum_ctas) {
        const int64_t zero = warp - a.sum_ctas * (kEmbedBackThreads / 32);
        const int64_t lo = zero * a.zero_rows, mine = lo + lane;
        if (lo >= a.rows) return;
        bool absent = false;
        if (lane < a.zero_rows && mine < a.rows) {
            const int64_t at = first_place(a.keys, 0, a.n, (uint32_t)mine);
            absent = at == a.n || a.keys[at] != (uint32_t)mine;
        }
        unsigned todo = __ballot_sync(0xffffffffu, absent);
        using V = ValueVec<O, N>;
        V none;
#pragma unroll
        for (int k = 0; k < N; ++k) none.v[k] = from_float<O>(0.0f);
        while (todo != 0) {
            const int r = __ffs(todo) - 1;
            todo &= todo - 1;
            O* out = static_cast<O*>(a.grad_table) + (lo + r) * a.table_stride;
            for (int c = lane * N; c < a.width; c += 32 * N) *reinterpret_cast<V*>(out + c) = none;
        }
        return;
    }
    const int64_t w = warp / a.tiles;
    const int column = (int)(warp - w * a.tiles) * kEmbedTile;
    const int64_t lo = w * a.window, mine = lo + lane;
    if (lo >= a.n) return;
    // does a piece start at this lane's place, and is it its run's first?
    uint32_t key = (uint32_t)a.rows;
    bool starts = false, first = false;
    if (lane < a.window && mine < a.n) {
        key = a.keys[mine];
        first = mine == 0 || a.keys[mine - 1] != key;
        starts = first;
        if (!first && mine >= kEmbedPiece && a.keys[mine - kEmbedPiece] == key)
            starts = (mine - first_place(a.keys, 0, mine, key)) % kEmbedPiece == 0;
        if (key >= (uint32_t)a.rows) starts = false;
    }
    unsigned todo = __ballot_sync(0xffffffffu, starts);
    const unsigned firsts = __ballot_sync(0xffffffffu, first);
    while (todo != 0) {
        const int r = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t at = lo + r;
        const uint32_t row = __shfl_sync(0xffffffffu, key, r);
        // places from here on with the same token, kEmbedPiece + 1 at most
        int count = 0;
#pragma unroll
        for (int k = 0; k < kEmbedPiece; k += 32) {
            if (count != k) break;
            const int64_t p = at + k + lane;
            const unsigned same = __ballot_sync(0xffffffffu, p < a.n && a.keys[p] == row);
            count += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
        }
        const bool is_first = firsts >> r & 1;
        const bool more = count == kEmbedPiece && at + kEmbedPiece < a.n && a.keys[at + kEmbedPiece] == row;
        float sum[kEmbedTile / 32];
        sum_run<T, N>(a, at, count, column, sum);
        if (is_first && !more) {
            store_row<O, N>(a, row, column, 0, sum);
        } else {
            float* out = a.partial + piece_slot(at, is_first) * a.width + column;
#pragma unroll
            for (int s = 0; s < EmbedLane<T, N>::kSteps; ++s) {
                const int c = (s * 32 + lane) * N;
#pragma unroll
                for (int k = 0; k < N; ++k)
                    if (column + c + k < a.width) out[c + k] = sum[s * N + k];
            }
        }
    }
}

// Long runs: the pieces' sums in order.  A run of more than kEmbedPiece places
// holds a multiple of kEmbedPiece after its start; the first of them is its CTA.
template <typename O>
__global__ void __launch_bounds__(256) embed_join_kernel(const EmbedBackArgs a) {
    wait_for_stream();
    const int64_t q = blockIdx.x / a.tiles;
    const int column = (int)(blockIdx.x - q * a.tiles) * kEmbedTile;
    const int64_t at = (q + 1) * kEmbedPiece;
    if (at >= a.n) return;
    const uint32_t key = a.keys[at];
    if (key >= (uint32_t)a.rows || a.keys[at - 1] != key) return;
    const int64_t lo = at - kEmbedPiece;
    if (lo > 0 && a.keys[lo] == key && a.keys[lo - 1] == key) return;  // an earlier multiple lies inside the run
    int64_t start = first_place(a.keys, lo, at, key);
    const int64_t end = first_place(a.keys, at, a.n, key + 1);
    if (end - start <= kEmbedPiece) return;
    const int64_t pieces = (end - start + kEmbedPiece - 1) / kEmbedPiece;
    for (int c = column + (int)threadIdx.x; c < min(column + kEmbedTile, a.width); c += 256) {
        float sum = a.partial[piece_slot(start, true) * a.width + c];
        for (int64_t p = 1; p < pieces; ++p)
            sum += a.partial[piece_slot(start + p * kEmbedPiece, false) * a.width + c];
        O* out = static_cast<O*>(a.grad_table) + (int64_t)key * a.table_stride + c;
        sum *= a.scale;
        *out = from_float<O>(a.accumulate ? to_float(*out) + sum : sum);
    }
}

}  // namespace om

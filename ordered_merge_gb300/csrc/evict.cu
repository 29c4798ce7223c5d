// om_accumulate_weights / om_evict_select / om_evict_gather: eviction from a
// cache by accumulated attention weight.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "select_common.cuh"
#include "strided.cuh"

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

// The values of a 16-byte vector added to their sums.
__device__ __forceinline__ void add_vector(uint64_t (&sum)[2], const uint4& w, float) {
    add2(sum[0], pack2(__uint_as_float(w.x), __uint_as_float(w.y)));
    add2(sum[1], pack2(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ void add_word(uint64_t& sum, uint32_t w, __nv_bfloat16) {
    add2(sum, pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
}
__device__ __forceinline__ void add_word(uint64_t& sum, uint32_t w, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    add2(sum, pack2(f.x, f.y));
}
template <typename T>
__device__ __forceinline__ void add_vector(uint64_t (&sum)[4], const uint4& w, T) {
    add_word(sum[0], w.x, T{});
    add_word(sum[1], w.y, T{});
    add_word(sum[2], w.z, T{});
    add_word(sum[3], w.w, T{});
}

// The vector that starts `skip` values (of type T) into a lane's w and goes on
// in the next lane's.  All lanes of the warp, with one skip.
template <typename T>
__device__ __noinline__ uint4 shifted(uint4 w, int skip) {
    uint32_t x[5] = {w.x, w.y, w.z, w.w, 0};
    if (skip != 0) {
        uint32_t y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __shfl_down_sync(0xffffffffu, x[i], 1);
        const int words = skip * (int)sizeof(T) / 4;
        x[4] = y[0];
        if (words == 1) x[0] = x[1], x[1] = x[2], x[2] = x[3], x[3] = y[0], x[4] = y[1];
        else if (words == 2) x[0] = x[2], x[1] = x[3], x[2] = y[0], x[3] = y[1], x[4] = y[2];
        else if (words == 3) x[0] = x[3], x[1] = y[0], x[2] = y[1], x[3] = y[2], x[4] = y[3];
        if (sizeof(T) == 2 && (skip & 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __funnelshift_r(x[i], x[i + 1], 16);
        }
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

constexpr int kAccMaxWarps = 8;
// Rows in flight per warp, and warps per SM: 8 x 24 for aligned rows and 4 x 32
// for odd ones were the best of 2 to 12 rows and 16 to 40 warps (64 x 8 cache
// heads of 8192 bf16 entries, eight rows each: 17.4 us against 17.8 with 4 x 32;
// 8 of 65539 f16 entries, 128 rows each: 28.8 against 29.8 with 8 x 24).
constexpr int acc_unroll(bool aligned) { return aligned ? 8 : 4; }
constexpr int acc_warps(bool aligned) { return aligned ? 24 : 32; }

// Rows that go one after another into one 32-bit sum.  Their sum is then added to
// the tile's, so that the error grows with 128 + rows / 128 and not with the rows
// (65536 equal ones: up to 1e-3 of the sum in one, 8e-6 so).
constexpr int kSumRows = 128;
static_assert(kSumRows % acc_unroll(true) == 0 && kSumRows % acc_unroll(false) == 0, "whole batches");

// A warp sums rows over one tile of entries, V = 16 bytes' worth per lane; the
// rows of a tile (share * queries of them) are split over 2^log_split warps of
// the CTA, whose sums are then added in the order of the warps.  The order of
// addition is fixed by the shapes, the strides, the rows' places within 16 bytes
// and the number of SMs (which the split goes by).
//
// Rows may start at any element (ALIGNED: all start on 16 bytes).  A lane loads
// the aligned 16 bytes that its part of the row begins in and adds them up as
// they lie; only when the rows' offset `skip` from that boundary changes are
// the sums added to the tile's entries, `skip` values further left.  Rows V
// queries apart have the same offset, so each warp walks its rows in the order
// (query mod V, head, query), in which the offset changes least often; where
// it changes within a batch of U rows, each vector is shifted into place with
// words of the next lane's.  The tile is then 31 lanes wide, as the last lane's
// vector reaches past it.  A vector that holds no value of the row's valid
// part is not loaded.
//
// DIRECT: one warp a tile, and aligned outputs: the lanes write their sums
// themselves, with no turn through shared memory.
//
// Bound by memory: every weight is read once.  64 x 8 cache heads of 8192 bf16
// entries, eight query heads each (90 MB): 16.6 us cold, 80 % of the copy rate,
// and 13.2 a pass with part of them left in L2; 8 cache heads of 65539 f16
// entries, 128 rows each, on odd addresses (138 MB): 28.5 us cold and 25.5 a pass,
// where each 16-byte vector of a warp also costs 67 instructions.
template <typename T, bool ALIGNED, bool DIRECT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, acc_warps(ALIGNED) / WARPS)
    accumulate_weights_kernel(AccumulateArgs a, int log_split) {
    wait_for_stream();
    constexpr int V = 16 / (int)sizeof(T), LANES = ALIGNED ? 32 : 31, TILE = LANES * V;
    constexpr int U = acc_unroll(ALIGNED);
    constexpr int STEP = ALIGNED ? 1 : V;  // queries between neighbours of the walk
    // Entry e of a tile is at (e mod V) * PITCH + e / V: the pitch keeps both
    // the lanes' writes and the reads of consecutive entries off each other's banks.
    constexpr int PITCH = 32 + 32 / V;
    __shared__ float s_sum[DIRECT ? 1 : WARPS][V * PITCH];
    if (DIRECT) log_split = 0;
    const int split = 1 << log_split, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp & (split - 1);
    const int wide = (WARPS >> log_split) * TILE;  // entries of this CTA
    const unsigned b = blockIdx.y / (unsigned)a.kv_heads, h = blockIdx.y - b * (unsigned)a.kv_heads;
    const int64_t n = valid_length(a.lengths, b, a.length);
    const int64_t first = (int64_t)blockIdx.x * wide;
    const int live = (int)max((int64_t)0, min(n - first, (int64_t)wide));  // valid ones among them
    const int there = (int)min(a.length - first, (int64_t)wide);
    const int c0 = (warp >> log_split) * TILE;  // this warp's first one
    const int64_t rows = (int64_t)a.share * a.queries;
    const int r0 = (int)(rows * part >> log_split), r1 = (int)(rows * (part + 1) >> log_split);
    const float* score = a.score == nullptr ? nullptr : a.score + b * a.s_batch + h * a.s_head + first;
    float* out = a.out + b * a.o_batch + h * a.o_head + first;
    // the old scores this thread will need, so that they arrive meanwhile
    float old[V];
#pragma unroll
    for (int k = 0; k < V; ++k) old[k] = 0.0f;
    if (score != nullptr) {
        if (DIRECT) {
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                const int j = c0 + lane * V + k;
                if (j + 3 < live) {
                    const float4 x = load_once(reinterpret_cast<const float4*>(score + j));
                    old[k] = x.x, old[k + 1] = x.y, old[k + 2] = x.z, old[k + 3] = x.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (j + i < live) old[k + i] = score[j + i];
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k * WARPS * 32 + (int)threadIdx.x < live) old[k] = load_once(score + k * WARPS * 32 + threadIdx.x);
        }
    }
    uint64_t sum[V / 2];
#pragma unroll
    for (int v = 0; v < V / 2; ++v) sum[v] = 0;
    uint64_t whole[V / 2];  // DIRECT: the blocks of rows before
#pragma unroll
    for (int v = 0; v < V / 2; ++v) whole[v] = 0;
    int cur = -1;  // offset, in values, of what `sum` holds
    bool fresh = true;
    // adds the sums to the tile's entries; entries left of it or past its end are other tiles'
    auto settle = [&] {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane * V + v - cur;
            float* at = &s_sum[warp][(e & (V - 1)) * PITCH + e / V];
            const float2 two = unpack2(sum[v / 2]);
            const float x = v & 1 ? two.y : two.x;
            if (e >= 0) *at = fresh ? x : *at + x;
        }
#pragma unroll
        for (int v = 0; v < V / 2; ++v) sum[v] = 0;
        fresh = false;
        __syncwarp();
    };
    if (c0 < live && r0 < r1) {
        constexpr int64_t size = (int64_t)sizeof(T);
        const char* base = reinterpret_cast<const char*>(static_cast<const T*>(a.weights) + b * a.w_batch +
                                                         (int64_t)h * a.share * a.w_head + first + c0);
        // the r0-th row of the walk: class c = query mod STEP, head g, query q
        int c = 0, before = r0, in_class = (a.queries + STEP - 1) / STEP, g = 0, q = 0;
        if (r0 > 0) {
            while (before >= a.share * in_class) {
                before -= a.share * in_class;
                ++c;
                in_class = (a.queries - c + STEP - 1) / STEP;
            }
            g = before / in_class;
            q = c + (before - g * in_class) * STEP;
        }
        const char* head = base + (g * a.w_head + c * a.w_query) * size;  // query c of head g
        const char* at = base + (g * a.w_head + q * a.w_query) * size;
        const int64_t step = STEP * a.w_query * size;
        const int room = (int)min(n - first - c0 - lane * V, (int64_t)1 << 20);  // valid from this lane's first on
        const int n_rows = r1 - r0;
        for (int r = 0; r < n_rows; r += U) {
            uint4 w[U];
            int skip[U], changes = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = make_uint4(0, 0, 0, 0);
                skip[u] = u > 0 ? skip[u - 1] : 0;
                if (r + u < n_rows) {
                    if (!ALIGNED) skip[u] = (int)(reinterpret_cast<uintptr_t>(at) & 15) / (int)sizeof(T);
                    if (room + skip[u] > 0)
                        w[u] = load_once(reinterpret_cast<const uint4*>(at - skip[u] * (int)sizeof(T)) + lane);
                    at += step;
                    q += STEP;
                    if (q >= a.queries) {
                        if (ALIGNED || ++g < a.share) {
                            head += a.w_head * size;
                        } else {
                            g = 0;
                            ++c;
                            head = base + c * a.w_query * size;
                        }
                        q = c;
                        at = head;
                    }
                }
                changes |= skip[u] ^ skip[0];
            }
            const int want = changes == 0 ? skip[0] : 0;  // 0 where ALIGNED
            if (cur != want || r % kSumRows == 0) {
                if (DIRECT) {
#pragma unroll
                    for (int v = 0; v < V / 2; ++v) add2(whole[v], sum[v]), sum[v] = 0;
                } else if (cur >= 0) {
                    settle();
                }
                cur = want;
            }
            if (ALIGNED || changes == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) add_vector(sum, w[u], T{});
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) add_vector(sum, shifted<T>(w[u], skip[u]), T{});
            }
        }
    }
    if (DIRECT) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const int j = c0 + lane * V + k;
            add2(sum[k / 2], whole[k / 2]), add2(sum[k / 2 + 1], whole[k / 2 + 1]);
            const float2 lo = unpack2(sum[k / 2]), hi = unpack2(sum[k / 2 + 1]);
            float x[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (score != nullptr) x[i] += a.decay * old[k + i];
                if (j + i >= live) x[i] = 0.0f;
            }
            if (j + 3 < there) {
                __stcs(reinterpret_cast<float4*>(out + j), make_float4(x[0], x[1], x[2], x[3]));
            } else {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (j + i < there) out[j + i] = x[i];
            }
        }
        return;
    }
    if (cur < 0) cur = 0;
    settle();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int j = k * WARPS * 32 + threadIdx.x;
        if (j >= there) break;
        float total = 0.0f;
        if (j < live) {
            const int t = j / TILE, e = j - t * TILE;
            const float* p = &s_sum[t << log_split][(e & (V - 1)) * PITCH + e / V];
            for (int w = 0; w < split; ++w) total += p[w * V * PITCH];
            if (score != nullptr) total += a.decay * old[k];
        }
        __stcs(out + j, total);
    }
}

template <typename T, bool ALIGNED>
static void launch_accumulate_split(const AccumulateArgs& a, dim3 grid, int log_split, bool direct, cudaStream_t st) {
    if (ALIGNED && direct) launch_early(accumulate_weights_kernel<T, ALIGNED, ALIGNED, 2>, grid, 2 * 32, 0, st, a, 0);
    else if (log_split <= 1) launch_early(accumulate_weights_kernel<T, ALIGNED, false, 2>, grid, 2 * 32, 0, st, a, log_split);
    else if (log_split == 2) launch_early(accumulate_weights_kernel<T, ALIGNED, false, 4>, grid, 4 * 32, 0, st, a, log_split);
    else launch_early(accumulate_weights_kernel<T, ALIGNED, false, 8>, grid, 8 * 32, 0, st, a, log_split);
}

template <typename T>
static cudaError_t launch_accumulate(const AccumulateArgs& a, int64_t batch, int sm_count, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t rows = (int64_t)a.share * a.queries;
    const uint64_t low = reinterpret_cast<uintptr_t>(a.weights) / sizeof(T) | (uint64_t)a.w_batch |
                         (uint64_t)a.w_head | (uint64_t)a.w_query;
    const bool aligned = low % V == 0;
    const int64_t tile = (aligned ? 32 : 31) * V, tiles = (a.length + tile - 1) / tile * batch * a.kv_heads;
    // as few warps a tile as fill the GPU with 32 warps an SM, while each has a batch of 8 rows
    int log_split = 0;
    while ((1 << log_split) < kAccMaxWarps && rows >= 16 << log_split && tiles << log_split < 32 * (int64_t)sm_count)
        ++log_split;
    uint64_t low4 = reinterpret_cast<uintptr_t>(a.out) / 4 | (uint64_t)a.o_batch | (uint64_t)a.o_head;
    if (a.score != nullptr) low4 |= reinterpret_cast<uintptr_t>(a.score) / 4 | (uint64_t)a.s_batch | (uint64_t)a.s_head;
    const bool direct = log_split == 0 && low4 % 4 == 0;
    const int64_t wide = (log_split == 0 ? 2 : 1) * tile;
    const dim3 grid((unsigned)((a.length + wide - 1) / wide), (unsigned)(batch * a.kv_heads));
    return counted([&] {
        if (aligned) launch_accumulate_split<T, true>(a, grid, log_split, direct, st);
        else launch_accumulate_split<T, false>(a, grid, log_split, direct, st);
    });
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

constexpr int kSelectStep = 128;  // keys a warp takes at a time, four consecutive ones per lane
constexpr int kDigitBits = 11;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kCoarse = kDigits / 32;
constexpr int kPasses = 3;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 48 * 1024;  // keys a CTA can hold in shared memory (192 KB)

// A NaN score counts as -inf: it goes first.
__device__ __forceinline__ uint32_t evict_key(float s) { return score_image(s == s ? s : -INFINITY); }

// The key of an entry that stays whatever its score; above that of +inf.
constexpr uint32_t kKeyStays = 0xffffffffu;

// Finds, among 32 * P counts held P per lane with the greatest place in lane 0's
// first, the place at which the sum from the top reaches `need`; *over is the
// sum above it.
template <int P>
__device__ __forceinline__ int place_of(const int (&c)[P], int need, int* over) {
    const int lane = threadIdx.x & 31;
    int mine = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) mine += c[j];
    int run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += up;
    }
    const int owner = __ffs(__ballot_sync(0xffffffffu, run >= need)) - 1;
    int above = run - mine, place = lane * P;
#pragma unroll
    for (int j = 0; j + 1 < P; ++j)
        if (above + c[j] < need) above += c[j], ++place;
        else break;
    *over = __shfl_sync(0xffffffffu, above, owner & 31);
    return __shfl_sync(0xffffffffu, place, owner & 31);
}

template <int WARPS>
struct SelectShared {
    __align__(16) int hist[kPasses][kDigits];
    int coarse[kPasses][kCoarse];  // sums of 32 digits each
    int above[WARPS], equal[WARPS];  // kept for sure / on the edge, in the warps before
    int total[2];                                  // the same of the CTA
    int digit, over;
};

// One cluster of 1 to 8 CTAs per row (sequence and head); CTA r takes the r-th
// contiguous part of it, and warp w of the CTA the w-th part of that, so that
// ranks in the row follow from sums over the CTAs and warps before.
//
// The row's least key that stays is found digit by digit from the top (11 + 11
// + 10 bits): a histogram of the keys that agree with the digits found so far,
// summed over the cluster, gives the next one.  Keys are read from memory
// once and kept in shared memory (CACHED), unless the part is too long for it.
// Places past the row's end hold key 0, which is below every score's and so
// never reached.
//
// Bound by its chain: each of the three digits is a pass over the keys, a meeting
// of the cluster and a search of the sums.  32 rows of 131072 entries (16.8 MB)
// take 22 us, 8 rows of 4096 8.0; the bytes alone would take 2.5 and 0.02.
template <bool CACHED, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 32 / WARPS) evict_select_kernel(EvictArgs a) {
    wait_for_stream();
    using Shared = SelectShared<WARPS>;
    constexpr int kThreads = WARPS * 32;
    extern __shared__ __align__(16) unsigned char s_raw[];
    Shared& s = *reinterpret_cast<Shared*>(s_raw);
    uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_raw + sizeof(Shared));
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    // with one CTA its own barrier and loads do, which are shorter
    auto meet = [&] {
        if (ctas > 1) cluster_sync();
        else __syncthreads();
    };
    auto word_of = [&](const int* p, uint32_t r) { return ctas > 1 ? peer_word(p, r) : *p; };
    const int64_t row = blockIdx.x / ctas, b = row / a.heads, h = row % a.heads;
    const float* score = a.score + b * a.s_batch + h * a.s_head;
    int32_t* keep = a.keep + row * a.budget;
    const int n = (int)valid_length(a.lengths, b, a.length);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (h == 0 && rank == 0 && threadIdx.x == 0) a.kept[b] = min(n, a.budget);
    if (n <= a.budget) {  // the whole cluster leaves here
        for (int i = (int)rank * kThreads + threadIdx.x; i < a.budget; i += (int)ctas * kThreads)
            keep[i] = i < n ? i : -1;
        return;
    }
    for (int i = threadIdx.x; i < kPasses * kDigits / 4; i += kThreads)
        reinterpret_cast<int4*>(&s.hist[0][0])[i] = make_int4(0, 0, 0, 0);
    const int warps = (int)ctas * WARPS;
    const int per_warp = (((n + warps - 1) / warps) + kSelectStep - 1) / kSelectStep * kSelectStep;
    const int64_t w0 = ((int64_t)rank * WARPS + warp) * per_warp;
    const int lo = (int)min(w0, (int64_t)n), hi = (int)min(w0 + per_warp, (int64_t)n);
    uint32_t* mine = s_keys + warp * per_warp;
    const bool aligned = (reinterpret_cast<uintptr_t>(score) & 15) == 0;  // lo is a multiple of 4

    auto fetch = [&](int i) {  // scores i .. i + 3
        if (aligned && i + 3 < hi) return *reinterpret_cast<const float4*>(score + i);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < hi) x.x = score[i];
        if (i + 1 < hi) x.y = score[i + 1];
        if (i + 2 < hi) x.z = score[i + 2];
        if (i + 3 < hi) x.w = score[i + 3];
        return x;
    };
    auto keys_of = [&](int i, float4 x) {  // their keys
        uint4 k = make_uint4(evict_key(x.x), evict_key(x.y), evict_key(x.z), evict_key(x.w));
        uint32_t* p = &k.x;
        if (i < a.first || i + 4 > n - a.last) {
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = i + j >= hi ? 0u : i + j < a.first || i + j >= n - a.last ? kKeyStays : p[j];
        }
        return k;
    };
    auto keys_at = [&](int i0) {
        if (CACHED) return *reinterpret_cast<const uint4*>(mine + (i0 - lo) + 4 * lane);
        return keys_of(i0 + 4 * lane, fetch(i0 + 4 * lane));
    };
    __syncthreads();

    int need = a.budget;  // still to be chosen among the keys that agree with `prefix`
    uint32_t prefix = 0, mask = 0;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? kDigits / 2 - 1 : kDigits - 1;
        auto count = [&](uint32_t k) {
            if (pass == 0 || (k & mask) == prefix) atomicAdd(&s.hist[pass][(k >> shift) & digits], 1);
        };
        if (pass == 0) {
            constexpr int U = 8;  // loads in flight per lane
            for (int i0 = lo; i0 < hi; i0 += kSelectStep * U) {
                float4 x[U];
#pragma unroll
                for (int u = 0; u < U; ++u) x[u] = fetch(i0 + u * kSelectStep + 4 * lane);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int at = i0 + u * kSelectStep;
                    if (at < hi) {
                        const uint4 k = keys_of(at + 4 * lane, x[u]);
                        if (CACHED) *reinterpret_cast<uint4*>(mine + (at - lo) + 4 * lane) = k;
                        count(k.x), count(k.y), count(k.z), count(k.w);
                    }
                }
            }
        } else {
            for (int i0 = lo; i0 < hi; i0 += kSelectStep) {
                const uint4 k = keys_at(i0);
                count(k.x), count(k.y), count(k.z), count(k.w);
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kCoarse / WARPS; ++j) {
            const int at = warp * (kCoarse / WARPS) + j;
            const int c = __reduce_add_sync(0xffffffffu, s.hist[pass][at * 32 + lane]);
            if (lane == 0) s.coarse[pass][at] = c;
        }
        meet();
        // first which 32 digits, then which of them, both summed over the cluster
        if (warp == 0) {
            constexpr int C = kCoarse / 32;
            int c[C] = {}, f[1] = {0}, over, more;
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r)
                if (r < ctas) {
#pragma unroll
                    for (int j = 0; j < C; ++j) c[j] += word_of(&s.coarse[pass][kCoarse - 1 - (lane * C + j)], r);
                }
            const int top = kCoarse - 1 - place_of(c, need, &over);
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r)
                if (r < ctas) f[0] += word_of(&s.hist[pass][top * 32 + 31 - lane], r);
            const int fine = 31 - place_of(f, need - over, &more);
            if (lane == 0) s.digit = top * 32 + fine, s.over = over + more;
        }
        __syncthreads();
        prefix |= (uint32_t)s.digit << shift;
        mask |= digits << shift;
        need -= s.over;
    }

    // how many of each warp's and each CTA's part stay: above the edge for sure, and on it
    int above = 0, equal = 0;
    for (int i0 = lo; i0 < hi; i0 += kSelectStep) {
        const uint4 k = keys_at(i0);
        above += (k.x > prefix) + (k.y > prefix) + (k.z > prefix) + (k.w > prefix);
        equal += (k.x == prefix) + (k.y == prefix) + (k.z == prefix) + (k.w == prefix);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) s.above[warp] = above, s.equal[warp] = equal;
    __syncthreads();
    if (warp == 0) {
        const int x = lane < WARPS ? s.above[lane] : 0, y = lane < WARPS ? s.equal[lane] : 0;
        int rx = x, ry = y;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int ux = __shfl_up_sync(0xffffffffu, rx, d), uy = __shfl_up_sync(0xffffffffu, ry, d);
            if (lane >= d) rx += ux, ry += uy;
        }
        if (lane < WARPS) s.above[lane] = rx - x, s.equal[lane] = ry - y;
        if (lane == 31) s.total[0] = rx, s.total[1] = ry;
    }
    meet();
    int gone_above = s.above[warp], gone_equal = s.equal[warp];  // before this warp's part, in the row
    for (uint32_t r = 0; r < rank; ++r) {
        gone_above += peer_word(&s.total[0], r);
        gone_equal += peer_word(&s.total[1], r);
    }
    if (ctas > 1) cluster_sync();  // no CTA leaves while another reads its totals
    constexpr int U = 4;  // steps whose counts are summed together, a byte each (at most 128)
    for (int i0 = lo; i0 < hi; i0 += kSelectStep * U) {
        uint4 k[U];
        uint32_t sures = 0, ties = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = i0 + u * kSelectStep;
            k[u] = at < hi ? keys_at(at) : make_uint4(0, 0, 0, 0);
            const uint32_t* p = &k[u].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p[j] > prefix) sures += 1u << (8 * u);
                if (p[j] == prefix) ties += 1u << (8 * u);
            }
        }
        uint32_t run_s = sures, run_t = ties, all_t = 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, run_s, d);
            if (lane >= d) run_s += up;
        }
        const uint32_t all_s = __shfl_sync(0xffffffffu, run_s, 31);
        run_s -= sures;
        if (__any_sync(0xffffffffu, ties != 0)) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t up = __shfl_up_sync(0xffffffffu, run_t, d);
                if (lane >= d) run_t += up;
            }
            all_t = __shfl_sync(0xffffffffu, run_t, 31);
            run_t -= ties;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t* p = &k[u].x;
            const int i = i0 + u * kSelectStep + 4 * lane;
            int32_t* out = keep + (gone_above + min(gone_equal, need) + (int)(run_s >> (8 * u) & 255));
            if ((all_t >> (8 * u) & 255) == 0) {  // nothing on the edge in this step
                if ((sures >> (8 * u) & 255) != 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (p[j] > prefix) *out++ = i + j;
                }
            } else {
                int tied = gone_equal + (int)(run_t >> (8 * u) & 255);
                out += min(tied, need) - min(gone_equal, need);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // of the keys on the edge the first `need` of the row stay
                    const bool tie = p[j] == prefix;
                    if (p[j] > prefix || (tie && tied < need)) *out++ = i + j;
                    tied += tie;
                }
            }
            gone_above += (int)(all_s >> (8 * u) & 255);
            gone_equal += (int)(all_t >> (8 * u) & 255);
        }
    }
}

// Shared memory of the selection for `keys` cached keys per CTA.
template <int WARPS>
static size_t select_smem(int64_t keys) {
    return sizeof(SelectShared<WARPS>) + (size_t)keys * 4;
}

// Entries up to which a row's CTA has 8 warps instead of 16 where there are more
// rows than SMs: 1024 rows of 2048 entries 17.6 us against 29.4, of 4096 20.7
// against 32.3, but 512 of 8192 22.7 against 21.1, and 150 of 4096 8.6 against 8.4.
constexpr int64_t kSelectShort = 4096;

// Once per device: the selection kernels' shared-memory limit.
static om_status prepare_select(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        for (auto* kern : {evict_select_kernel<true, 16>, evict_select_kernel<false, 16>, evict_select_kernel<true, 8>})
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)select_smem<16>(kMaxCached)) != cudaSuccess) {
                cudaGetLastError();
                return OM_ECUDA;
            }
        ready[d->dev] = true;
    }
    return OM_OK;
}

template <int WARPS>
static cudaError_t launch_select_warps(const EvictArgs& a, int64_t rows, int sm_count, cudaStream_t st) {
    // As many CTAs per row as fill the SMs (two CTAs each), but at least 8192 entries
    // a CTA: 8 rows of 16384 10.4 us, with 2048 11.9, with 16384 11.3; of 8192 8.7,
    // with 2048 10.2, with 4096 9.6.
    int ctas = 1;
    while (ctas < kMaxCluster && rows * ctas * 2 <= 2 * (int64_t)sm_count && a.length > ctas * 8192) ctas *= 2;
    const int64_t warps = ctas * WARPS;
    const int64_t per_warp = (((a.length + warps - 1) / warps) + kSelectStep - 1) / kSelectStep * kSelectStep;
    const int64_t keys = per_warp * WARPS;
    const bool cached = keys <= kMaxCached;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = select_smem<WARPS>(cached ? keys : 0);
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {early_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    auto* kern = evict_select_kernel<true, WARPS>;
    if constexpr (WARPS == 16) {
        if (!cached) kern = evict_select_kernel<false, WARPS>;
    }
    return counted([&] { cudaLaunchKernelEx(&cfg, kern, a); });
}

static cudaError_t launch_select(const EvictArgs& a, int64_t rows, int sm_count, cudaStream_t st) {
    return a.length <= kSelectShort && rows > sm_count ? launch_select_warps<8>(a, rows, sm_count, st)
                                    : launch_select_warps<16>(a, rows, sm_count, st);
}

// --------------------------------------------------------------- gather --

constexpr int kMaxArrays = 8;

struct GatherArgs {
    om_cache_array arrays[kMaxArrays];
    int first_cta[kMaxArrays];  // of each array; a row's entries are cut into tiles, one CTA each
    int tiles[kMaxArrays], tile_entries[kMaxArrays], vector[kMaxArrays];
    const int32_t* keep;
    int64_t length;
    int budget, heads, count;
};

constexpr int kGatherThreads = 64;
constexpr int kGatherUnroll = 4;  // vectors in flight per thread

// One tile of one row of one array: the CTA's threads take its vectors in turn.
// Bound by memory: 32 rows of 16384 kept entries of 256 + 256 + 4 bytes (0.54 GB)
// take 86 us, 93 % of the copy rate; CTAs of 256 threads take 94, of 128 86.
template <typename V>
__device__ __forceinline__ void gather_tile(const GatherArgs& a, const om_cache_array& c, int64_t row, int j0, int j1) {
    const int per = (int)(c.entry_bytes / (int)sizeof(V));
    const int64_t b = row / a.heads, h = row % a.heads;
    const char* src = static_cast<const char*>(c.src) + b * c.src_batch + h * c.src_head;
    char* dst = static_cast<char*>(c.dst) + b * c.dst_batch + h * c.dst_head;
    const int32_t* keep = a.keep + row * a.budget;
    const int total = (j1 - j0) * per;
    for (int i0 = threadIdx.x; i0 < total; i0 += kGatherThreads * kGatherUnroll) {
        V v[kGatherUnroll];
        int64_t to[kGatherUnroll];
        int32_t from[kGatherUnroll];
        int piece[kGatherUnroll];
        // all indices first, then all vectors: two trips to memory, not two for each vector
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int i = i0 + u * kGatherThreads, j = i / per;
            from[u] = i < total ? keep[j0 + j] : -1;
            piece[u] = (i - j * per) * (int)sizeof(V);
            to[u] = i < total ? (j0 + j) * c.dst_entry + piece[u] : -1;
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            v[u] = V{};
            if (from[u] >= 0 && from[u] < a.length)
                v[u] = load_once(reinterpret_cast<const V*>(src + from[u] * c.src_entry + piece[u]));
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u)
            if (to[u] >= 0) __stcs(reinterpret_cast<V*>(dst + to[u]), v[u]);
    }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const __grid_constant__ GatherArgs a) {
    wait_for_stream();
    int k = a.count - 1;
    while (k > 0 && (int)blockIdx.x < a.first_cta[k]) --k;
    const int t = (int)blockIdx.x - a.first_cta[k], row = t / a.tiles[k];
    const int j0 = (t - row * a.tiles[k]) * a.tile_entries[k];
    const int j1 = j0 + min(a.tile_entries[k], a.budget - j0);  // budgets go up to 2^31 - 1
    switch (a.vector[k]) {
        case 16: gather_tile<uint4>(a, a.arrays[k], row, j0, j1); break;
        case 4: gather_tile<uint32_t>(a, a.arrays[k], row, j0, j1); break;
        case 2: gather_tile<unsigned short>(a, a.arrays[k], row, j0, j1); break;
        default: gather_tile<unsigned char>(a, a.arrays[k], row, j0, j1); break;
    }
}

// ---- in place
//
// keep rises, so entry j comes from entry keep[j] >= j: a CTA, or a cluster of
// them, that walks a row from its start, storing a chunk only when all of it has
// been loaded, never overwrites what a later chunk needs, and may load the next
// chunk meanwhile.  Where there are few rows, entries are cut into `slices`
// columns of at least 64 bytes, and clusters of up to 8 CTAs take a column's
// chunks together.  An entry that stays where it is is not touched.
//
// Bound by the meetings between loading and storing, on cold inputs: 32 rows of
// 16384 kept of 131072 entries (keys and values of 256 bytes, a score) 94 us,
// 2 rows of 65536 47 us.  Into other memory these take 86 and 24 us, before
// anything is brought back.

constexpr int kInPlaceThreads = 512;

template <typename V>
__device__ __forceinline__ void gather_row_in_place(const GatherArgs& a, const om_cache_array& c, int64_t row,
                                                    int slice, int slices) {
    constexpr int U = kGatherUnroll;
    const unsigned per = (unsigned)(c.entry_bytes / (int)sizeof(V)) / (unsigned)slices;  // vectors of an entry here
    const int64_t b = row / a.heads, h = row % a.heads;
    char* base = static_cast<char*>(c.dst) + b * c.dst_batch + h * c.dst_head + (int64_t)slice * per * sizeof(V);
    const int32_t* keep = a.keep + row * a.budget;
    const unsigned total = (unsigned)a.budget * per, ctas = cluster_size();
    const unsigned first = cluster_rank() * kInPlaceThreads + threadIdx.x, stride = ctas * kInPlaceThreads;
    struct Chunk {
        V v[U];
        int64_t to[U];
    };
    auto load = [&](unsigned i0, Chunk& x) {
        int32_t from[U];
        unsigned piece[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned i = i0 + u * stride + first, j = i / per;
            from[u] = i < total ? keep[j] : (int32_t)j;
            piece[u] = (i - j * per) * (unsigned)sizeof(V);
            x.to[u] = from[u] != (int32_t)j ? j * c.dst_entry + piece[u] : -1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x.v[u] = V{};
            if (x.to[u] >= 0 && from[u] >= 0 && from[u] < a.length)
                x.v[u] = *reinterpret_cast<const V*>(base + from[u] * c.dst_entry + piece[u]);
        }
    };
    Chunk now, next;
    load(0, now);
    for (unsigned i0 = 0; i0 < total; i0 += U * stride) {
        const bool more = total - i0 > U * stride;
        if (more) load(i0 + U * stride, next);
        // the whole of `now` has been loaded
        if (ctas > 1) cluster_sync();
        else __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (now.to[u] >= 0) *reinterpret_cast<V*>(base + now.to[u]) = now.v[u];
        if (more) now = next;
        else break;
    }
}

// first_cta, tiles: as for the other kernel, for clusters, a tile being a slice of a row.
__global__ void __launch_bounds__(kInPlaceThreads) evict_gather_in_place_kernel(const __grid_constant__ GatherArgs a) {
    wait_for_stream();
    const int cluster = (int)(blockIdx.x / cluster_size());
    int k = a.count - 1;
    while (k > 0 && cluster < a.first_cta[k]) --k;
    const int t = cluster - a.first_cta[k], row = t / a.tiles[k], slice = t - row * a.tiles[k];
    switch (a.vector[k]) {
        case 16: gather_row_in_place<uint4>(a, a.arrays[k], row, slice, a.tiles[k]); break;
        case 4: gather_row_in_place<uint32_t>(a, a.arrays[k], row, slice, a.tiles[k]); break;
        case 2: gather_row_in_place<unsigned short>(a, a.arrays[k], row, slice, a.tiles[k]); break;
        default: gather_row_in_place<unsigned char>(a, a.arrays[k], row, slice, a.tiles[k]); break;
    }
}

// Bytes of the vectors that every address of the array allows.
static int gather_vector(const om_cache_array& c) {
    const uint64_t low = reinterpret_cast<uintptr_t>(c.src) | reinterpret_cast<uintptr_t>(c.dst) |
                         (uint64_t)c.src_batch | (uint64_t)c.src_head | (uint64_t)c.src_entry |
                         (uint64_t)c.dst_batch | (uint64_t)c.dst_head | (uint64_t)c.dst_entry |
                         (uint64_t)c.entry_bytes;
    return (low & 15) == 0 ? 16 : (low & 3) == 0 ? 4 : (low & 1) == 0 ? 2 : 1;
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
    if (length > INT32_MAX || queries > 65535 || q_heads > 65535 || batch > 65535 || batch * kv_heads > 65535 ||
        q_heads / kv_heads * queries > INT32_MAX - 64)
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
        arrays_meet(out, o_span, length * 4, {batch, kv_heads, 1}, {o_batch * 4, o_head * 4, 0}, score,
                    ((batch - 1) * s_batch + (kv_heads - 1) * s_head + length) * 4, length * 4, {batch, kv_heads, 1},
                    {s_batch * 4, s_head * 4, 0}))
        return OM_EINVAL;
    AccumulateArgs a{weights, score, lengths, out,    w_batch, w_head,        w_query, s_batch, s_head, o_batch, o_head,
                     length,  (int)kv_heads, (int)(q_heads / kv_heads), (int)queries, decay};
    DeviceState* d = nullptr;
    const om_status s = device_state(&d);
    if (s != OM_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e =
        with_value_type(value_type, [&](auto v) { return launch_accumulate<decltype(v)>(a, batch, d->sm_count, st); });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_evict_select(const float* score, int64_t batch, int64_t heads, int64_t length, int64_t s_batch,
                          int64_t s_head, const int32_t* lengths, int64_t budget, int64_t first, int64_t last,
                          int32_t* keep, int32_t* kept, void* stream) {
    if (batch < 0 || heads < 1 || length < 0 || s_batch < 0 || s_head < 0 || budget < 1 || first < 0 || last < 0)
        return OM_EINVAL;
    if (first > budget || last > budget - first) return OM_EINVAL;
    if (length > INT32_MAX - 65536 || budget > INT32_MAX - 65536 || heads > 65535 || batch > 32767 ||
        batch * heads > (1 << 27) || s_batch > kMaxStride || s_head > kMaxStride)
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
    DeviceState* d = nullptr;
    om_status ds = device_state(&d);
    if (ds == OM_OK) ds = prepare_select(d);
    if (ds != OM_OK) return ds;
    const cudaError_t e = launch_select(a, batch * heads, d->sm_count, st);
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
    int in_place = 0;
    for (int i = 0; i < count; ++i) {
        const om_cache_array& c = arrays[i];
        if (c.entry_bytes < 1 || c.dst == nullptr || (length > 0 && c.src == nullptr)) return OM_EINVAL;
        if (c.entry_bytes > (1 << 24)) return OM_ERANGE;
        for (const int64_t s : {c.src_batch, c.src_head, c.src_entry, c.dst_batch, c.dst_head, c.dst_entry})
            if (s < 0) return OM_EINVAL;
        if (c.src_batch > kMaxStride || c.src_head > kMaxStride || c.dst_batch > kMaxStride ||
            c.dst_head > kMaxStride || c.src_entry > kMaxEntryStride || c.dst_entry > kMaxEntryStride)
            return OM_ERANGE;
        bool shared = false, src_shared = false;
        spans[i] = strided_span(c.entry_bytes, {batch, heads, budget}, {c.dst_batch, c.dst_head, c.dst_entry}, &shared);
        if (shared) return OM_EINVAL;
        src_spans[i] = length > 0 ? strided_span(c.entry_bytes, {batch, heads, length},
                                                 {c.src_batch, c.src_head, c.src_entry}, &src_shared)
                                  : 0;
        if (overlaps(c.dst, spans[i], keep, slots * 4, 1)) return OM_EINVAL;
        if (c.src == c.dst && c.src_batch == c.dst_batch && c.src_head == c.dst_head && c.src_entry == c.dst_entry) {
            if (src_shared) return OM_EINVAL;  // rows would write into each other's entries
            ++in_place;
        }
        a.arrays[i] = c;
    }
    if (in_place != 0 && in_place != count) return OM_EINVAL;
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j) {
            const om_cache_array &c = a.arrays[i], &o = a.arrays[j];
            auto dst_meets = [&](const void* p, int64_t span, int64_t entries, int64_t sb, int64_t sh, int64_t se) {
                return span > 0 && arrays_meet(c.dst, spans[i], c.entry_bytes, {batch, heads, budget},
                                               {c.dst_batch, c.dst_head, c.dst_entry}, p, span, o.entry_bytes,
                                               {batch, heads, entries}, {sb, sh, se});
            };
            if (!(in_place && i == j) && dst_meets(o.src, src_spans[j], length, o.src_batch, o.src_head, o.src_entry))
                return OM_EINVAL;
            if (i < j && dst_meets(o.dst, spans[j], budget, o.dst_batch, o.dst_head, o.dst_entry)) return OM_EINVAL;
        }
    a.keep = keep;
    a.length = length;
    a.budget = (int)budget;
    a.heads = (int)heads;
    a.count = count;
    DeviceState* d = nullptr;
    const om_status s = device_state(&d);
    if (s != OM_OK) return s;
    int64_t ctas = 0;
    for (int i = 0; i < count; ++i) {
        a.vector[i] = gather_vector(a.arrays[i]);
        const int64_t per = a.arrays[i].entry_bytes / a.vector[i];
        if (in_place) {
            // columns of at least 64 bytes until there are two CTAs an SM
            int64_t slices = 1;
            while (batch * heads * count * slices < 2 * d->sm_count && per % (2 * slices) == 0 &&
                   per / (2 * slices) * a.vector[i] >= 64)
                slices *= 2;
            if (budget * per / slices > INT32_MAX) return OM_ERANGE;  // with a chunk more still 32 bits
            a.tiles[i] = (int)slices;
        } else {
            // tiles of about kGatherUnroll vectors per thread
            int64_t entries = kGatherThreads * kGatherUnroll / per;
            if (entries < 1) entries = 1;
            a.tile_entries[i] = (int)entries;
            a.tiles[i] = (int)((budget + entries - 1) / entries);
        }
        a.first_cta[i] = (int)ctas;
        ctas += batch * heads * a.tiles[i];
        if (ctas > INT32_MAX) return OM_ERANGE;
    }
    cudaStream_t st = (cudaStream_t)stream;
    unsigned cluster = 1;  // in place: CTAs to each column of a row
    while (in_place && cluster < kMaxCluster && ctas * cluster * 2 <= 2 * d->sm_count &&
           budget > (int64_t)cluster * kInPlaceThreads)
        cluster *= 2;
    const cudaError_t e = counted([&] {
        if (!in_place) {
            launch_early(evict_gather_kernel, (unsigned)ctas, kGatherThreads, 0, st, a);
            return;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas * cluster);
        cfg.blockDim = dim3(kInPlaceThreads);
        cfg.stream = st;
        cudaLaunchAttribute attr[2] = {early_attribute()};
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        cudaLaunchKernelEx(&cfg, evict_gather_in_place_kernel, a);
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

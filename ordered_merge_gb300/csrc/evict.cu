// om_accumulate_weights / om_evict_select / om_evict_gather: eviction from a
// cache by accumulated attention weight.
#include <cstdint>
#include <mutex>

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

// The two 16-bit values of a word, or the one 32-bit value, added to sums.
__device__ __forceinline__ void add_word(float* sum, uint32_t w, float) { sum[0] += __uint_as_float(w); }
__device__ __forceinline__ void add_word(float* sum, uint32_t w, __nv_bfloat16) {
    sum[0] += __uint_as_float(w << 16);
    sum[1] += __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void add_word(float* sum, uint32_t w, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    sum[0] += f.x;
    sum[1] += f.y;
}

constexpr int kAccWarps = 8;

// A warp sums rows over one tile of entries, V = 16 bytes' worth per lane; the
// rows of a tile (share * queries of them) are split over `split` warps of
// the CTA, whose sums are then added in the order of the warps, so the result
// depends on the shapes alone.
//
// Rows may start at any element (ALIGNED: all start on 16 bytes).  A lane loads
// the aligned 16 bytes that its part of the row begins in and adds them up as
// they lie; only when the rows' offset `skip` from that boundary changes are
// the sums added to the tile's entries, `skip` values further left.  Rows V
// queries apart have the same offset, so each warp walks its rows in the order
// (query mod V, head, query), in which the offset changes least often.  The
// tile is then 31 lanes wide, as the last lane's vector reaches past it.  A
// vector that holds no value of the row's valid part is not loaded.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(kAccWarps * 32) accumulate_weights_kernel(AccumulateArgs a, int split) {
    constexpr int V = 16 / (int)sizeof(T), LANES = ALIGNED ? 32 : 31, TILE = LANES * V, U = 8;
    __shared__ __align__(16) float s_sum[kAccWarps][32 * V];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % split;
    const int tiles = kAccWarps / split;  // of this CTA
    const int64_t b = blockIdx.y / a.kv_heads, h = blockIdx.y % a.kv_heads;
    const int64_t n = valid_length(a.lengths, b, a.length);
    const int64_t first = (int64_t)blockIdx.x * tiles * TILE;
    const int64_t c0 = first + (warp / split) * TILE;
    const int rows = a.share * a.queries;
    const int r0 = (int)((int64_t)rows * part / split), r1 = (int)((int64_t)rows * (part + 1) / split);
    // the old scores this thread will need, so that they arrive meanwhile
    float old[V];
    const float* score = a.score == nullptr ? nullptr : a.score + b * a.s_batch + h * a.s_head;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int j = k * kAccWarps * 32 + threadIdx.x;
        old[k] = 0.0f;
        if (score != nullptr && j < tiles * TILE && first + j < n) old[k] = __ldcs(score + first + j);
    }
    float sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f;
    if (!ALIGNED) {
#pragma unroll
        for (int v = 0; v < V; ++v) s_sum[warp][lane * V + v] = 0.0f;
        __syncwarp();
    }
    if (c0 < n && r0 < r1) {
        const char* base = reinterpret_cast<const char*>(static_cast<const T*>(a.weights) + b * a.w_batch +
                                                         h * a.share * a.w_head + c0);
        // the r0-th row of the walk: class c = query mod V, head g, query q
        int c = 0, before = r0;
        int in_class = (a.queries + V - 1) / V;  // queries of class c
        while (before >= a.share * in_class) {
            before -= a.share * in_class;
            ++c;
            in_class = (a.queries - c + V - 1) / V;
        }
        int g = before / in_class, q = c + (before - g * in_class) * V;
        int cur = 0;  // offset, in values, of what `sum` holds
        for (int r = r0; r < r1; r += U) {
            uint4 w[U];
            int skip[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                w[u] = make_uint4(0, 0, 0, 0);
                skip[u] = -1;
                if (r + u < r1) {
                    const char* at = base + (g * a.w_head + q * a.w_query) * (int64_t)sizeof(T);
                    if ((q += V) >= a.queries) {
                        if (++g == a.share) g = 0, ++c;
                        q = c;
                    }
                    skip[u] = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(at) & 15) / (int)sizeof(T);
                    if (c0 + lane * V - skip[u] < n)
                        w[u] = __ldcs(reinterpret_cast<const uint4*>(at - skip[u] * (int)sizeof(T)) + lane);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!ALIGNED && skip[u] >= 0 && skip[u] != cur) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (lane * V + v >= cur) s_sum[warp][lane * V + v - cur] += sum[v];
                        sum[v] = 0.0f;
                    }
                    __syncwarp();
                    cur = skip[u];
                }
                add_word(sum, w[u].x, T{});
                add_word(sum + V / 4, w[u].y, T{});
                add_word(sum + V / 2, w[u].z, T{});
                add_word(sum + 3 * V / 4, w[u].w, T{});
            }
        }
        if (!ALIGNED) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (lane * V + v >= cur) s_sum[warp][lane * V + v - cur] += sum[v];
        }
    }
    if (ALIGNED) {
#pragma unroll
        for (int v = 0; v < V; v += 4)
            *reinterpret_cast<float4*>(&s_sum[warp][lane * V + v]) =
                make_float4(sum[v], sum[v + 1], sum[v + 2], sum[v + 3]);
    }
    __syncthreads();
    float* out = a.out + b * a.o_batch + h * a.o_head;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int j = k * kAccWarps * 32 + threadIdx.x;
        const int64_t i = first + j;
        if (j >= tiles * TILE || i >= a.length) break;
        float total = 0.0f;
        if (i < n) {
            const int t = j / TILE, col = j - t * TILE;
            for (int w = 0; w < split; ++w) total += s_sum[t * split + w][col];
            if (score != nullptr) total += a.decay * old[k];
        }
        __stcs(out + i, total);
    }
}

template <typename T>
static cudaError_t launch_accumulate(const AccumulateArgs& a, int64_t batch, cudaStream_t st) {
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t rows = (int64_t)a.share * a.queries;
    int split = 1;  // at least 8 rows a warp: one batch of its loads
    while (split < kAccWarps && rows >= 16 * split) split *= 2;
    const uint64_t low = reinterpret_cast<uintptr_t>(a.weights) / sizeof(T) | (uint64_t)a.w_batch |
                         (uint64_t)a.w_head | (uint64_t)a.w_query;
    const bool aligned = low % V == 0;
    const int64_t wide = (int64_t)(kAccWarps / split) * (aligned ? 32 : 31) * V;
    const dim3 grid((unsigned)((a.length + wide - 1) / wide), (unsigned)(batch * a.kv_heads));
    return traced(kKindEvict, st, [&] {
        if (aligned) accumulate_weights_kernel<T, true><<<grid, kAccWarps * 32, 0, st>>>(a, split);
        else accumulate_weights_kernel<T, false><<<grid, kAccWarps * 32, 0, st>>>(a, split);
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

constexpr int kSelectThreads = 512;
constexpr int kSelectStep = 128;  // keys a warp takes at a time, four consecutive ones per lane
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kDigitBits = 11;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kPasses = 3;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 48 * 1024;  // keys a CTA can hold in shared memory (192 KB)

// A NaN score counts as -inf: it goes first.
__device__ __forceinline__ uint32_t evict_key(float s) { return score_image(s == s ? s : -INFINITY); }

// The key of an entry that stays whatever its score; above that of +inf.
constexpr uint32_t kKeyStays = 0xffffffffu;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster; orders their shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word, or four, of CTA `rank`'s shared memory, at the address p has in this CTA's.
__device__ __forceinline__ int peer_word(const int* p, uint32_t rank) {
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ int4 peer_words(const int* p, uint32_t rank) {
    uint32_t at;
    int4 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// Sum of `mine` over the threads before.
__device__ __forceinline__ int block_before(int mine, int* s_part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += up;
    }
    if (lane == 31) s_part[warp] = run;
    __syncthreads();
    int w = lane < kSelectWarps ? s_part[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += up;
    }
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return (warp > 0 ? before : 0) + run - mine;
}

struct SelectShared {
    __align__(16) int hist[kPasses][kDigits];
    int part[kPasses][kSelectWarps];
    int above[kSelectWarps], equal[kSelectWarps];  // kept for sure / on the edge, in the warps before
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
template <bool CACHED>
__global__ void __launch_bounds__(kSelectThreads, 2) evict_select_kernel(EvictArgs a) {
    extern __shared__ __align__(16) unsigned char s_raw[];
    SelectShared& s = *reinterpret_cast<SelectShared*>(s_raw);
    uint32_t* s_keys = reinterpret_cast<uint32_t*>(s_raw + sizeof(SelectShared));
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int64_t row = blockIdx.x / ctas, b = row / a.heads, h = row % a.heads;
    const float* score = a.score + b * a.s_batch + h * a.s_head;
    int32_t* keep = a.keep + row * a.budget;
    const int n = (int)valid_length(a.lengths, b, a.length);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (h == 0 && rank == 0 && threadIdx.x == 0) a.kept[b] = min(n, a.budget);
    if (n <= a.budget) {  // the whole cluster leaves here
        for (int i = (int)rank * kSelectThreads + threadIdx.x; i < a.budget; i += (int)ctas * kSelectThreads)
            keep[i] = i < n ? i : -1;
        return;
    }
    for (int i = threadIdx.x; i < kPasses * kDigits / 4; i += kSelectThreads)
        reinterpret_cast<int4*>(&s.hist[0][0])[i] = make_int4(0, 0, 0, 0);
    const int warps = (int)ctas * kSelectWarps;
    const int per_warp = (((n + warps - 1) / warps) + kSelectStep - 1) / kSelectStep * kSelectStep;
    const int64_t w0 = ((int64_t)rank * kSelectWarps + warp) * per_warp;
    const int lo = (int)min(w0, (int64_t)n), hi = (int)min(w0 + per_warp, (int64_t)n);
    uint32_t* mine = s_keys + warp * per_warp;
    const bool aligned = (reinterpret_cast<uintptr_t>(score) & 15) == 0;  // lo is a multiple of 4

    auto fetch = [&](int i) {  // scores i .. i + 3
        if (aligned && i + 3 < hi) return __ldg(reinterpret_cast<const float4*>(score + i));
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < hi) x.x = __ldg(score + i);
        if (i + 1 < hi) x.y = __ldg(score + i + 1);
        if (i + 2 < hi) x.z = __ldg(score + i + 2);
        if (i + 3 < hi) x.w = __ldg(score + i + 3);
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
            constexpr int U = 4;  // loads in flight per lane
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
        cluster_sync();
        // four digits a thread, from the greatest down, summed over the cluster
        const int low = kDigits - 4 - 4 * threadIdx.x;
        int4 c = make_int4(0, 0, 0, 0);
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            if (r < ctas) {
                const int4 p = peer_words(&s.hist[pass][low], r);
                c.x += p.x, c.y += p.y, c.z += p.z, c.w += p.w;
            }
        }
        int above = block_before(c.x + c.y + c.z + c.w, s.part[pass]);
        if (above < need && need <= above + c.x + c.y + c.z + c.w) {  // one thread
            int digit = low + 3;
            if (need > above + c.w) {
                above += c.w, --digit;
                if (need > above + c.z) {
                    above += c.z, --digit;
                    if (need > above + c.y) above += c.y, --digit;
                }
            }
            s.digit = digit;
            s.over = above;
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
        const int x = lane < kSelectWarps ? s.above[lane] : 0, y = lane < kSelectWarps ? s.equal[lane] : 0;
        int rx = x, ry = y;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int ux = __shfl_up_sync(0xffffffffu, rx, d), uy = __shfl_up_sync(0xffffffffu, ry, d);
            if (lane >= d) rx += ux, ry += uy;
        }
        if (lane < kSelectWarps) s.above[lane] = rx - x, s.equal[lane] = ry - y;
        if (lane == 31) s.total[0] = rx, s.total[1] = ry;
    }
    cluster_sync();
    int gone_above = s.above[warp], gone_equal = s.equal[warp];  // before this warp's part, in the row
    for (uint32_t r = 0; r < rank; ++r) {
        gone_above += peer_word(&s.total[0], r);
        gone_equal += peer_word(&s.total[1], r);
    }
    cluster_sync();  // no CTA leaves while another reads its totals
    for (int i0 = lo; i0 < hi; i0 += kSelectStep) {
        const uint4 k = keys_at(i0);
        const uint32_t* p = &k.x;
        // a lane's counts of both kinds in one word (at most 128 each a step), summed over the lanes before
        uint32_t both = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) both += (p[j] > prefix ? 1u : 0u) + (p[j] == prefix ? 1u << 16 : 0u);
        uint32_t run = both;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += up;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, run, 31);
        run -= both;
        int at = gone_above + (int)(run & 0xffff), ties = gone_equal + (int)(run >> 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // of the keys on the edge the first `need` of the row stay
            const bool tie = p[j] == prefix, sure = p[j] > prefix;
            if (sure || (tie && ties < need)) keep[at + min(ties, need)] = i0 + 4 * lane + j;
            at += sure;
            ties += tie;
        }
        gone_above += (int)(all & 0xffff);
        gone_equal += (int)(all >> 16);
    }
}

// Shared memory of the selection for `keys` cached keys per CTA.
static size_t select_smem(int64_t keys) { return sizeof(SelectShared) + (size_t)keys * 4; }

// Once per device: the selection kernel's shared-memory limit.
static om_status prepare_select(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        for (auto* kern : {evict_select_kernel<true>, evict_select_kernel<false>})
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)select_smem(kMaxCached)) != cudaSuccess) {
                cudaGetLastError();
                return OM_ECUDA;
            }
        ready[d->dev] = true;
    }
    return OM_OK;
}

static cudaError_t launch_select(const EvictArgs& a, int64_t rows, int sm_count, cudaStream_t st) {
    // As many CTAs per row as fill the SMs (two CTAs each), but at least 2048 entries a CTA.
    int ctas = 1;
    while (ctas < kMaxCluster && rows * ctas * 2 <= 2 * (int64_t)sm_count && a.length > ctas * 2048) ctas *= 2;
    const int64_t warps = ctas * kSelectWarps;
    const int64_t per_warp = (((a.length + warps - 1) / warps) + kSelectStep - 1) / kSelectStep * kSelectStep;
    const int64_t keys = per_warp * kSelectWarps;
    const bool cached = keys <= kMaxCached;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * ctas));
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = select_smem(cached ? keys : 0);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kern = cached ? evict_select_kernel<true> : evict_select_kernel<false>;
    return traced(kKindEvict, st, [&] { cudaLaunchKernelEx(&cfg, kern, a); });
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

constexpr int kGatherThreads = 256;
constexpr int kGatherUnroll = 4;  // vectors in flight per thread

// One tile of one row of one array: the CTA's threads take its vectors in turn.
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
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u) {
            const int i = i0 + u * kGatherThreads;
            v[u] = V{};
            to[u] = -1;
            if (i < total) {
                const int j = i / per, piece = (i - j * per) * (int)sizeof(V);
                const int32_t from = __ldg(keep + j0 + j);
                to[u] = (j0 + j) * c.dst_entry + piece;
                if (from >= 0 && from < a.length)
                    v[u] = __ldcs(reinterpret_cast<const V*>(src + from * c.src_entry + piece));
            }
        }
#pragma unroll
        for (int u = 0; u < kGatherUnroll; ++u)
            if (to[u] >= 0) __stcs(reinterpret_cast<V*>(dst + to[u]), v[u]);
    }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const __grid_constant__ GatherArgs a) {
    int k = a.count - 1;
    while (k > 0 && (int)blockIdx.x < a.first_cta[k]) --k;
    const int t = (int)blockIdx.x - a.first_cta[k], row = t / a.tiles[k];
    const int j0 = (t - row * a.tiles[k]) * a.tile_entries[k], j1 = min(j0 + a.tile_entries[k], a.budget);
    switch (a.vector[k]) {
        case 16: gather_tile<uint4>(a, a.arrays[k], row, j0, j1); break;
        case 4: gather_tile<uint32_t>(a, a.arrays[k], row, j0, j1); break;
        case 2: gather_tile<unsigned short>(a, a.arrays[k], row, j0, j1); break;
        default: gather_tile<unsigned char>(a, a.arrays[k], row, j0, j1); break;
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
    const cudaError_t e =
        with_value_type(value_type, [&](auto v) { return launch_accumulate<decltype(v)>(a, batch, st); });
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
    a.length = length;
    a.budget = (int)budget;
    a.heads = (int)heads;
    a.count = count;
    int64_t ctas = 0;
    for (int i = 0; i < count; ++i) {
        // tiles of about kGatherUnroll vectors per thread
        a.vector[i] = gather_vector(a.arrays[i]);
        const int64_t per = a.arrays[i].entry_bytes / a.vector[i];
        int64_t entries = kGatherThreads * kGatherUnroll / per;
        if (entries < 1) entries = 1;
        a.tile_entries[i] = (int)entries;
        a.tiles[i] = (int)((budget + entries - 1) / entries);
        a.first_cta[i] = (int)ctas;
        ctas += batch * heads * a.tiles[i];
        if (ctas > INT32_MAX) return OM_ERANGE;
    }
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = traced(
        kKindEvict, st, [&] { evict_gather_kernel<<<(unsigned)ctas, kGatherThreads, 0, st>>>(a); });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

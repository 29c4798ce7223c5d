// om_group_by_id: the stable grouping of slots by a small integer id.
#include <cstdint>
#include <mutex>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "select_common.cuh"

namespace om {

constexpr int kMaxGroups = 1024;
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr unsigned kGroupCluster8 = 8;  // CTAs of a cluster at most

// Ids outside [0, groups) form one more group after the others.
__device__ __forceinline__ int group_of(int32_t id, int groups) {
    return (uint32_t)id < (uint32_t)groups ? id : groups;
}

struct GroupArgs {
    const int32_t* ids;
    int64_t n;
    int groups;
    int32_t* offsets;
    int32_t* order;
    int32_t* place;
    int chunk, longer;  // n over the CTAs, and the remainder: the first `longer` chunks have one slot more

    // First slot of CTA c's chunk.
    __device__ __forceinline__ int64_t start(unsigned c) const {
        return (int64_t)chunk * c + min(c, (unsigned)longer);
    }
};

// Every thread of the cooperative grid.  A function of its own, because inlined
// the thread that waits for the other CTAs stayed apart from its warp
// afterwards, and the warp ran everything twice.
__device__ __noinline__ void grid_barrier() { cooperative_groups::this_grid().sync(); }

// How the CTAs of a call learn of each other's counts.
enum GroupWay {
    kGroupLone,     // one CTA
    kGroupCluster,  // a cluster of 2 to 8: from each other's shared memory
    kGroupGrid      // a cooperative grid: through the chunks of `place`
};

// A slot's place is the sum of: the slots of lower groups, those of its own in
// the chunks of the CTAs before, in the parts of the warps before, and before
// it in its own warp's part.  Chunks and parts are contiguous, so equal ids
// keep their order.
//
// kGroupGrid takes no scratch memory: CTA c leaves its counts at the start of
// its own chunk of `place` (2 * (groups + 1) words); one warp per group turns
// the column of a group into the sums over the CTAs before, and leaves the
// group's total beside each; then every CTA needs its own chunk only, which it
// overwrites at the end.
//
// What bounds it: for few slots the chain of loads and barriers, 4 us of which
// one CTA needs for its first loads; for many the two grid barriers (1.4 us
// each) and counting and ranking, about 150 instructions per 32 slots.  Measured,
// times of the kernel: 512 slots of 256 groups 4.0 us, 32768 7.6 us, 1.05 M of
// 128 16.4 us.  Writing `order` from a chunk put in order in shared memory first,
// in runs, was no faster (16.5 us).
// BITS: of the greatest group, `groups` itself.
template <int WAY, int BITS>
__global__ void __launch_bounds__(kGroupThreads) group_by_id_kernel(GroupArgs a) {
    wait_for_stream();
    extern __shared__ int s_next[];  // [warps][E]: a warp's counts, then its next place less the CTA's first
    __shared__ int s_part[kGroupWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = a.groups + 1;
    int* s_count = s_next + warps * E;  // [E]: the CTA's counts
    int* s_first = s_count + E;         // [E]: the CTA's first place of each group
    const unsigned ctas = gridDim.x;
    const int64_t lo = a.start(blockIdx.x), hi = a.start(blockIdx.x + 1);
    // each warp's part of the chunk, in steps of 32 slots
    const int part = ((int)(hi - lo) / warps + 32) & ~31;
    const int64_t wlo = min(lo + (int64_t)warp * part, hi), whi = min(wlo + part, hi);
    int* next = s_next + warp * E;
    for (int g = lane; g < E; g += 32) next[g] = 0;
    __syncwarp();
    constexpr int U = 8;  // loads in flight per lane
    for (int64_t i0 = wlo + lane; i0 < whi; i0 += 32 * U) {
        int32_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = i0 + 32 * u < whi ? a.ids[i0 + 32 * u] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + 32 * u < whi) atomicAdd(&next[group_of(id[u], a.groups)], 1);
    }
    __syncthreads();
    // counts to sums over the warps before
    for (int g = threadIdx.x; g < E; g += blockDim.x) {
        int run = 0;
        for (int w0 = 0; w0 < warps; w0 += 8) {
            int c[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) c[k] = w0 + k < warps ? s_next[(w0 + k) * E + g] : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (w0 + k < warps) s_next[(w0 + k) * E + g] = run;
                run += c[k];
            }
        }
        s_count[g] = run;
        if (WAY == kGroupGrid) __stcg(a.place + lo + g, run);
    }
    if (WAY == kGroupCluster) cluster_sync();
    if (WAY == kGroupGrid) {
        grid_barrier();
        for (int g = warp * (int)ctas + (int)blockIdx.x; g < E; g += warps * (int)ctas) {
            constexpr int R = 5;  // 160 CTAs at a time
            int before = 0;
            for (unsigned c0 = 0; c0 < ctas; c0 += 32 * R) {
                int count[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const unsigned c = c0 + 32 * r + lane;
                    count[r] = c < ctas ? load_l2(a.place + a.start(c) + g) : 0;
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const unsigned c = c0 + 32 * r + lane;
                    int run = count[r];
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int up = __shfl_up_sync(0xffffffffu, run, d);
                        if (lane >= d) run += up;
                    }
                    if (c < ctas) __stcg(a.place + a.start(c) + g, before + run - count[r]);
                    before += __shfl_sync(0xffffffffu, run, 31);
                }
            }
            for (unsigned c = lane; c < ctas; c += 32) __stcg(a.place + a.start(c) + E + g, before);
        }
        grid_barrier();
    }

    // where each group starts, and the CTA's slots of it
    int start = 0;
    for (int g0 = 0; g0 < E; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x;
        int total = 0, before = 0;
        if (g < E) {
            if (WAY == kGroupGrid) {
                before = load_l2(a.place + lo + g);
                total = load_l2(a.place + lo + E + g);
            } else if (WAY == kGroupCluster) {
#pragma unroll
                for (unsigned r = 0; r < kGroupCluster8; ++r) {
                    const int count = r < ctas ? peer_word(s_count + g, r) : 0;
                    total += count;
                    before += r < blockIdx.x ? count : 0;
                }
            } else {
                total = s_count[g];
            }
        }
        int run = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += up;
        }
        if (lane == 31) s_part[warp] = run;
        __syncthreads();
        int sums = lane < warps ? s_part[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sums, d);
            if (lane >= d) sums += up;
        }
        const int earlier = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
        const int first = start + (warp > 0 ? earlier : 0) + run - total;
        start += __shfl_sync(0xffffffffu, sums, 31);
        if (g < E) {
            if (blockIdx.x == 0) a.offsets[g] = first;  // the last one, of the ids outside, ends the others
            s_first[g] = first + before;
        }
        __syncthreads();
    }
    if (WAY == kGroupCluster) cluster_sync();  // no CTA leaves, or writes, while another reads its counts

    const int32_t* ids = a.ids + lo;
    int32_t* place = a.place + lo;
    const int r1 = (int)(whi - lo);
    const unsigned before_me = (1u << lane) - 1;
    for (int r0 = (int)(wlo - lo) + lane; r0 - lane < r1; r0 += 32 * U) {
        int32_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = r0 + 32 * u < r1 ? ids[r0 + 32 * u] : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = r0 + 32 * u;
            if (r - lane >= r1) break;
            const bool live = r < r1;
            const int g = group_of(id[u], a.groups);
            // the lanes with the same group, one bit of it at a time: a vote each (the
            // hardware's match of whole words made the whole call a tenth longer)
            unsigned same = __ballot_sync(0xffffffffu, live);
#pragma unroll
            for (int bit = 0; bit < BITS; ++bit) {
                const bool one = g & (1 << bit);
                same &= __ballot_sync(0xffffffffu, one) ^ (one ? 0u : 0xffffffffu);
            }
            const int rank = __popc(same & before_me);
            int at = next[g] + rank;
            __syncwarp();
            if (live && rank == 0) next[g] = at + __popc(same);
            __syncwarp();
            if (live) {
                at += s_first[g];
                a.order[at] = (int32_t)(lo + r);
                place[r] = at;
            }
        }
    }
}

template <int BITS>
static auto group_kernel(int way) {
    return way == kGroupLone      ? group_by_id_kernel<kGroupLone, BITS>
           : way == kGroupCluster ? group_by_id_kernel<kGroupCluster, BITS>
                                  : group_by_id_kernel<kGroupGrid, BITS>;
}

// Once per device: the kernel's shared-memory limit.
static om_status prepare_group(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        for (auto* kern : {group_by_id_kernel<kGroupLone, 8>, group_by_id_kernel<kGroupLone, 11>,
                           group_by_id_kernel<kGroupCluster, 8>, group_by_id_kernel<kGroupCluster, 11>,
                           group_by_id_kernel<kGroupGrid, 8>, group_by_id_kernel<kGroupGrid, 11>})
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (kGroupWarps + 2) * (kMaxGroups + 1) * 4) != cudaSuccess) {
                cudaGetLastError();
                return OM_ECUDA;
            }
        ready[d->dev] = true;
    }
    return OM_OK;
}

// Slots up to which one CTA, and one cluster, does the call: 2048 slots of 64
// groups 4.6 us alone, 5.1 in a cluster; 4096 6.3 and 5.2, 8192 of 128 10.0 and
// 5.3; 49152 of 256 9.1 in a cluster, 9.9 in a grid; 65536 11.5 and 10.0.
constexpr int64_t kGroupLoneSlots = 2048;
constexpr int64_t kGroupClusterSlots = 49152;
// Least slots of a CTA of several (8192 slots in 8 CTAs 5.3 us, in 4 5.9; 4096 of
// 64 groups in 4 5.2 us, in 2 5.8, in 8 5.0).
constexpr int64_t kGroupLeastChunk = 1024;

}  // namespace om

using namespace om;

extern "C" {

om_status om_group_by_id(const int32_t* ids, int64_t n, int64_t groups, int32_t* offsets, int32_t* order,
                         int32_t* place, void* stream) {
    if (n < 0 || groups < 1) return OM_EINVAL;
    if (n > INT32_MAX || groups > kMaxGroups) return OM_ERANGE;
    if (offsets == nullptr || (n > 0 && (ids == nullptr || order == nullptr || place == nullptr))) return OM_EINVAL;
    for (const void* p : {(const void*)ids, (const void*)offsets, (const void*)order, (const void*)place})
        if (misaligned4(p)) return OM_EINVAL;
    if (overlaps(order, n, ids, n) || overlaps(place, n, ids, n) || overlaps(order, n, place, n) ||
        overlaps(offsets, groups + 1, ids, n) || overlaps(offsets, groups + 1, order, n) ||
        overlaps(offsets, groups + 1, place, n))
        return OM_EINVAL;
    DeviceState* d = nullptr;
    om_status s = device_state(&d);
    if (s == OM_OK) s = prepare_group(d);
    if (s != OM_OK) return s;
    int way = kGroupLone, warps = kGroupWarps;
    int64_t ctas = 1;
    if (n <= kGroupLoneSlots) {
        if (n <= 128 * (kGroupWarps - 1)) warps = (int)(n / 128) + 1;  // a warp per 128 slots
    } else if (n <= kGroupClusterSlots) {
        way = kGroupCluster;
        for (ctas = 2; ctas < kGroupCluster8 && ctas * kGroupLeastChunk < n; ctas *= 2) {}
    } else {
        // a chunk holds at least the two words per group that its CTA exchanges
        way = kGroupGrid;
        ctas = n / (2 * (groups + 1) > kGroupLeastChunk ? 2 * (groups + 1) : kGroupLeastChunk);
        if (ctas > d->sm_count) ctas = d->sm_count;
    }
    GroupArgs a{ids, n, (int)groups, offsets, order, place, (int)(n / ctas), (int)(n % ctas)};
    cudaStream_t st = (cudaStream_t)stream;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = (size_t)(warps + 2) * (groups + 1) * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    if (way == kGroupGrid) {
        attr[0].id = cudaLaunchAttributeCooperative;
        attr[0].val.cooperative = 1;
    } else {
        attr[0] = early_attribute();
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)ctas;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = way == kGroupCluster ? 2 : 1;
    auto* kern = group_kernel<8>(way);
    if (groups >= 256) kern = group_kernel<11>(way);
    const cudaError_t e = counted([&] { cudaLaunchKernelEx(&cfg, kern, a); });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

// om_group_by_id: the stable grouping of slots by a small integer id.
#include <cstdint>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "select_common.cuh"

namespace om {

constexpr int kMaxGroups = 1024;

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
    int32_t* counts;  // [groups + 1][ctas]: slots of a group in a CTA's chunk, then the slots in the chunks before
    int32_t* totals;  // [groups + 1]
    int64_t chunk;    // slots per CTA
};

constexpr int kGroupThreads = 512;
constexpr int kGroupWarps = kGroupThreads / 32;

// Slots of each group in each CTA's chunk.
__global__ void __launch_bounds__(kGroupThreads) group_count_kernel(GroupArgs a) {
    __shared__ int s_count[kMaxGroups + 1];
    for (int g = threadIdx.x; g <= a.groups; g += kGroupThreads) s_count[g] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
    for (int64_t i = lo + threadIdx.x; i < hi; i += kGroupThreads) atomicAdd(&s_count[group_of(a.ids[i], a.groups)], 1);
    __syncthreads();
    for (int g = threadIdx.x; g <= a.groups; g += kGroupThreads) a.counts[(int64_t)g * gridDim.x + blockIdx.x] = s_count[g];
}

// One warp per group: its counts become the sums over the chunks before.
__global__ void __launch_bounds__(128) group_scan_kernel(GroupArgs a, int ctas) {
    const int g = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (g > a.groups) return;
    int before = 0;
    for (int c0 = 0; c0 < ctas; c0 += 32) {
        const int c = c0 + lane;
        const int mine = c < ctas ? a.counts[(int64_t)g * ctas + c] : 0;
        int run = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += up;
        }
        if (c < ctas) a.counts[(int64_t)g * ctas + c] = before + run - mine;
        before += __shfl_sync(0xffffffffu, run, 31);
    }
    if (lane == 0) a.totals[g] = before;
}

// Places of a chunk's slots.  Each warp takes a contiguous part of the chunk,
// so that a slot's rank in its group is: the group's start, the group's slots
// in the chunks and warps before, and those before it in its own warp.
__global__ void __launch_bounds__(kGroupThreads) group_place_kernel(GroupArgs a) {
    extern __shared__ int s_next[];  // [kGroupWarps][groups + 1]
    __shared__ int s_part[kGroupWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.groups + 1;
    for (int i = threadIdx.x; i < kGroupWarps * E; i += kGroupThreads) s_next[i] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * a.chunk, hi = min(lo + a.chunk, a.n);
    const int64_t part = (((hi - lo + kGroupWarps - 1) / kGroupWarps) + 31) & ~(int64_t)31;
    const int64_t wlo = min(lo + warp * part, hi), whi = min(wlo + part, hi);
    int* next = s_next + warp * E;
    for (int64_t i = wlo + lane; i < whi; i += 32) atomicAdd(&next[group_of(a.ids[i], a.groups)], 1);
    __syncthreads();
    // starts of the groups: exclusive sum of the totals, E values over the threads in order
    int start = 0;
    for (int g0 = 0; g0 < E; g0 += kGroupThreads) {
        const int g = g0 + threadIdx.x;
        int mine = 0, before = 0;
        if (g < E) {
            if (gridDim.x > 1) {
                mine = a.totals[g];
                before = a.counts[(int64_t)g * gridDim.x + blockIdx.x];
            } else {
                for (int w = 0; w < kGroupWarps; ++w) mine += s_next[w * E + g];
            }
        }
        int run = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += up;
        }
        if (lane == 31) s_part[warp] = run;
        __syncthreads();
        int earlier = 0, all = 0;
        for (int w = 0; w < kGroupWarps; ++w) {
            if (w < warp) earlier += s_part[w];
            all += s_part[w];
        }
        const int first = start + earlier + run - mine;
        if (g < E) {
            if (blockIdx.x == 0) a.offsets[g] = first;  // the last one, of the ids outside, ends the others
            int at = first + before;
            for (int w = 0; w < kGroupWarps; ++w) {
                const int c = s_next[w * E + g];
                s_next[w * E + g] = at;
                at += c;
            }
        }
        start += all;
        __syncthreads();
    }
    for (int64_t i0 = wlo; i0 < whi; i0 += 32) {
        const int64_t i = i0 + lane;
        const unsigned live = __ballot_sync(0xffffffffu, i < whi);
        if (i < whi) {
            const int g = group_of(a.ids[i], a.groups);
            const unsigned same = __match_any_sync(live, g);
            const int at = next[g] + __popc(same & ((1u << lane) - 1));
            __syncwarp(live);
            if (lane == __ffs(same) - 1) next[g] += __popc(same);
            a.order[at] = (int32_t)i;
            a.place[i] = at;
        }
        __syncwarp();
    }
}

// Slots per CTA below which one CTA does the whole call.
constexpr int64_t kGroupOneCta = 8192;

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
    if (s != OM_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    const size_t smem = (size_t)kGroupWarps * (groups + 1) * 4;
    if (cudaFuncSetAttribute(group_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kGroupWarps * (kMaxGroups + 1) * 4) != cudaSuccess)
        return OM_ECUDA;
    GroupArgs a{ids, n, (int)groups, offsets, order, place, nullptr, nullptr, n > 0 ? n : 1};
    int64_t ctas = 1;
    if (n > kGroupOneCta) {
        const int64_t most = d->sm_count;
        ctas = (n + 2047) / 2048;
        if (ctas > most) ctas = most;
        a.chunk = (((n + ctas - 1) / ctas) + 31) & ~(int64_t)31;
        ctas = (n + a.chunk - 1) / a.chunk;
    }
    cudaError_t e = cudaSuccess;
    int32_t* scratch = nullptr;
    if (ctas > 1) {
        cudaMemPool_t pool = nullptr;
        s = scratch_pool(d, &pool);
        if (s != OM_OK) return s;
        e = scratch_alloc(pool, reinterpret_cast<void**>(&scratch), (size_t)(groups + 1) * (ctas + 1) * 4, st);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return OM_ENOMEM;
        }
        a.totals = scratch;
        a.counts = scratch + groups + 1;
        e = traced(kKindGroup, st, [&] { group_count_kernel<<<(unsigned)ctas, kGroupThreads, 0, st>>>(a); });
        if (e == cudaSuccess)
            e = traced(kKindGroup, st,
                       [&] { group_scan_kernel<<<(unsigned)(groups + 4) / 4, 128, 0, st>>>(a, (int)ctas); });
    }
    if (e == cudaSuccess)
        e = traced(kKindGroup, st, [&] { group_place_kernel<<<(unsigned)ctas, kGroupThreads, smem, st>>>(a); });
    if (scratch != nullptr) scratch_free(scratch, st);
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

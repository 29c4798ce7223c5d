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

// A slot's place is the sum of: the slots of lower groups, those of its own in
// the chunks of the CTAs before, in the parts of the warps before, and before
// it in its own warp's part.  Chunks and parts are contiguous, so equal ids
// keep their order.
//
// One CTA, or a cooperative grid whose CTAs exchange their counts through the
// start of their own chunk of `place` (2 * (groups + 1) words), which they
// overwrite only at the end: no scratch memory.  CTA c leaves its counts there;
// one warp per group turns the column of a group into the sums over the CTAs
// before, and leaves the group's total beside each; then every CTA needs its
// own chunk only.  (Every CTA reading every other's counts took 12 us more.)
__global__ void __launch_bounds__(kGroupThreads) group_by_id_kernel(GroupArgs a) {
    extern __shared__ int s_next[];  // [warps][groups + 1]: counts, then the next place
    __shared__ int s_part[kGroupWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, E = a.groups + 1;
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
        for (int u = 0; u < U; ++u) id[u] = i0 + 32 * u < whi ? __ldg(a.ids + i0 + 32 * u) : 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + 32 * u < whi) atomicAdd(&next[group_of(id[u], a.groups)], 1);
    }
    __syncthreads();

    int32_t* mine = a.place + lo;  // this CTA's words of the exchange
    if (ctas > 1) {
        for (int g = threadIdx.x; g < E; g += blockDim.x) {
            int count = 0;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) count += s_next[w * E + g];
            __stcg(mine + g, count);
        }
        cooperative_groups::this_grid().sync();
        for (int g = warp * (int)ctas + (int)blockIdx.x; g < E; g += warps * (int)ctas) {
            constexpr int R = 4;  // loads of a column in flight per lane
            int before = 0;
            for (unsigned c0 = 0; c0 < ctas; c0 += 32 * R) {
                int count[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const unsigned c = c0 + 32 * r + lane;
                    count[r] = c < ctas ? __ldcg(a.place + a.start(c) + g) : 0;
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
        cooperative_groups::this_grid().sync();
    }

    // where each group starts, then where each warp's slots of it do
    int start = 0;
    for (int g0 = 0; g0 < E; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x;
        int total = 0, before = 0;
        if (g < E) {
            if (ctas > 1) {
                before = __ldcg(mine + g);
                total = __ldcg(mine + E + g);
            } else {
#pragma unroll 8
                for (int w = 0; w < warps; ++w) total += s_next[w * E + g];
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
            int at = first + before;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) {
                const int c = s_next[w * E + g];
                s_next[w * E + g] = at;
                at += c;
            }
        }
        __syncthreads();
    }
    const int bits = 32 - __clz(a.groups);  // of the greatest group, `groups` itself
    for (int64_t i0 = wlo; i0 < whi; i0 += 32 * U) {
        int32_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = i0 + 32 * u + lane < whi ? __ldg(a.ids + i0 + 32 * u + lane) : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + 32 * u >= whi) break;
            const int64_t i = i0 + 32 * u + lane;
            const bool live = i < whi;
            const int g = live ? group_of(id[u], a.groups) : 0;
            // the lanes with the same group, one bit of it at a time (a vote each; the
            // hardware's match of whole words takes far longer: 7.5 us of 1 M slots' 22)
            unsigned same = __ballot_sync(0xffffffffu, live);
            for (int bit = 0; bit < bits; ++bit) {
                const bool one = g >> bit & 1;
                const unsigned ones = __ballot_sync(0xffffffffu, one);
                same &= one ? ones : ~ones;
            }
            int at = 0;
            if (live) at = next[g] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (live && lane == __ffs(same) - 1) next[g] += __popc(same);
            __syncwarp();
            if (live) {
                a.order[at] = (int32_t)i;
                a.place[i] = at;
            }
        }
    }
}

// Once per device: the kernel's shared-memory limit.
static om_status prepare_group(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        if (cudaFuncSetAttribute(group_by_id_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kGroupWarps * (kMaxGroups + 1) * 4) != cudaSuccess) {
            cudaGetLastError();
            return OM_ECUDA;
        }
        ready[d->dev] = true;
    }
    return OM_OK;
}

// Least slots of a CTA of several; and the slots up to which one CTA does the
// call alone, without the exchange: 4096 slots of 256 groups 7.2 us (two CTAs
// 14), 8192 of 128 10.3 (four 10.8).
constexpr int64_t kGroupLeastChunk = 2048;
constexpr int64_t kGroupLone = 8192;

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
    // a chunk holds at least the two words per group that its CTA exchanges
    int64_t least = 2 * (groups + 1);
    if (least < kGroupLeastChunk) least = kGroupLeastChunk;
    int64_t ctas = n / least;
    if (ctas > d->sm_count) ctas = d->sm_count;
    if (n < kGroupLone) ctas = 1;
    if (ctas < 1) ctas = 1;
    GroupArgs a{ids, n, (int)groups, offsets, order, place, (int)(n / ctas), (int)(n % ctas)};
    // a lone CTA takes a warp per 128 slots
    int warps = kGroupWarps;
    if (ctas == 1 && n <= 128 * (kGroupWarps - 1)) warps = (int)(n / 128) + 1;
    cudaStream_t st = (cudaStream_t)stream;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(warps * 32);
    cfg.dynamicSmemBytes = (size_t)warps * (groups + 1) * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 1 : 0;
    const cudaError_t e = traced(kKindGroup, st, [&] { cudaLaunchKernelEx(&cfg, group_by_id_kernel, a); });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

// Shared by the ordered-selection operators (route.cu, group.cu, evict.cu):
// value types, the order-preserving integer image of a score and warp
// reductions.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "ordmerge.h"

namespace om {

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// Order-preserving image of a float that is not NaN: a < b exactly when
// image(a) < image(b), and -0 and +0 share one image (adding +0 makes -0
// positive), so equal scores tie.  -inf maps to 0x007fffff, hence 0 is free
// for "no candidate".
__device__ __forceinline__ uint32_t score_image(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// Two floats in one register pair, added or multiplied at once.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    return p;
}
__device__ __forceinline__ float2 unpack2(uint64_t p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ void add2(uint64_t& sum, uint64_t x) {
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sum) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
    uint64_t p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(x), "l"(y));
    return p;
}

// ---- thread-block clusters

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
// Every thread of every CTA of the cluster; orders their shared memory.  Not the
// .aligned form: nothing promises that a warp is whole where this is inlined.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// A word of CTA `rank`'s shared memory, at the address p has in this CTA's.
__device__ __forceinline__ int peer_word(const int* p, uint32_t rank) {
    uint32_t at;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Launches through `launch` (a callable issuing exactly one kernel) and counts
// it for om_launch_count; om_trace_* keep no kind for these kernels.
template <typename F>
cudaError_t counted(F&& launch) {
    launch();
    return trace_end(TraceRec{0, nullptr, nullptr}, false, nullptr);
}

// ---- launches that overlap the end of the stream's work
//
// A kernel launched by launch_early may be given to the SMs while the kernel
// before it in the stream still drains; wait_for_stream, its first statement,
// holds it back until that one has ended and its writes are visible.  Then it
// lets the next such kernel come, which waits in its turn.
//
// Its inputs may thus be written during its life, so it reads them by ordinary
// loads and by those below, never by the read-only path (__ldg), which takes
// memory that nobody writes while the kernel lives, and which the compiler may
// lift over the wait.

__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

// Loads with a cache hint; volatile, so that they stay behind the wait.
// load_once: what is read once (evicted first).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(__cvta_generic_to_global(p)));
    return v;
}
__device__ __forceinline__ float4 load_once(const float4* p) {
    float4 v;
    asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(__cvta_generic_to_global(p)));
    return v;
}
__device__ __forceinline__ float load_once(const float* p) {
    float v;
    asm volatile("ld.global.cs.f32 %0, [%1];" : "=f"(v) : "l"(__cvta_generic_to_global(p)));
    return v;
}
__device__ __forceinline__ uint32_t load_once(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)));
    return v;
}
__device__ __forceinline__ unsigned short load_once(const unsigned short* p) {
    unsigned short v;
    asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(v) : "l"(__cvta_generic_to_global(p)));
    return v;
}
__device__ __forceinline__ unsigned char load_once(const unsigned char* p) {
    uint32_t v;
    asm volatile("ld.global.cs.u8 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)));
    return (unsigned char)v;
}
// load_l2: a word that another CTA of this launch has written (past the L1 cache).
__device__ __forceinline__ int load_l2(const int* p) {
    int v;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(__cvta_generic_to_global(p)) : "memory");
    return v;
}

// The attribute of such a launch.
inline cudaLaunchAttribute early_attribute() {
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

template <typename... Ps, typename... As>
void launch_early(void (*kern)(Ps...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, As... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = early_attribute();
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kern, args...);
}

inline int value_bytes(int value_type) {
    switch (value_type) {
        case OM_VALUE_F32: return 4;
        case OM_VALUE_BF16:
        case OM_VALUE_F16: return 2;
        default: return 0;
    }
}

// Calls f with a value of the C++ type behind value_type (already checked).
template <typename F>
auto with_value_type(int value_type, F&& f) {
    switch (value_type) {
        case OM_VALUE_F32: return f(float{});
        case OM_VALUE_BF16: return f(__nv_bfloat16{});
        default: return f(__half{});
    }
}

}  // namespace om

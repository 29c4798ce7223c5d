// om_expert_mlp: argument checks, scratch and launches.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "expert_kernels.cuh"
#include "select_common.cuh"
#include "strided.cuh"

namespace om {

// Calls f with a value of the 16-bit type behind value_type (already checked).
template <typename F>
static auto with_half_type(int value_type, F&& f) {
    return value_type == OM_VALUE_BF16 ? f(__nv_bfloat16{}) : f(__half{});
}

constexpr int kFewTiles = 2, kManyTiles = 8;  // tokens of an expert taken at once, in eights

static constexpr size_t up_smem(int mats, int tiles) { return (size_t)kExpertWarps * mats * 8 * tiles * kExpertRows * 4; }

template <typename T>
static auto up_kernel(bool gated, bool many) {
    return gated ? (many ? expert_up_kernel<T, true, kManyTiles> : expert_up_kernel<T, true, kFewTiles>)
                 : (many ? expert_up_kernel<T, false, kManyTiles> : expert_up_kernel<T, false, kFewTiles>);
}

// Once per device: the kernels' shared-memory limits.
static om_status prepare_experts(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        bool ok = true;
        auto limit = [&](auto* kern, size_t bytes) {
            ok = ok && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
        };
        for (const bool gated : {false, true}) {
            limit(up_kernel<__half>(gated, true), up_smem(2, kManyTiles));
            limit(up_kernel<__nv_bfloat16>(gated, true), up_smem(2, kManyTiles));
        }
        if (!ok) {
            cudaGetLastError();
            return OM_ECUDA;
        }
        ready[d->dev] = true;
    }
    return OM_OK;
}

// Rows of any size and address.
template <typename T>
static cudaError_t launch_odd_rows(ExpertArgs a, int sm_count, cudaStream_t st) {
    const bool gated = a.gate != nullptr;
    a.by_slot = a.slots < a.experts;
    const bool many = a.slots > 8 * a.experts;
    const int tiles = many ? kManyTiles : kFewTiles;
    const dim3 grid((unsigned)((a.inner + kExpertRows - 1) / kExpertRows), (unsigned)std::min(a.slots, a.experts));
    cudaError_t e = counted([&] {
        launch_early(up_kernel<T>(gated, many), grid, kExpertWarps * 32, up_smem(gated ? 2 : 1, tiles), st, a);
    });
    if (e != cudaSuccess) return e;
    const int64_t rows = (a.hidden + kExpertRows - 1) / kExpertRows;
    unsigned ctas = 1;
    while (ctas < kExpertCluster && rows * ctas < 3 * (int64_t)sm_count) ctas *= 2;
    // pieces of the experts' columns: enough for every warp of the cluster, of four steps at least
    const int experts = std::min(a.slots, a.experts), steps = (a.inner + 31) / 32;
    a.parts = std::max(1, std::min((int)(ctas * kExpertWarps) / experts, steps / 4));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * ctas);
    cfg.blockDim = dim3(kExpertWarps * 32);
    cfg.dynamicSmemBytes = (size_t)kExpertWarps * a.tokens * kExpertRows * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {early_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return counted([&] { cudaLaunchKernelEx(&cfg, expert_down_kernel<T>, a); });
}

// Rows of whole aligned vectors.
template <typename T>
static cudaError_t launch_layer(const ExpertArgs& a, int sm_count, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sm_count * kLayerCtas));
    cfg.blockDim = dim3(kLayerThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {};
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kern = a.gate != nullptr ? expert_layer_kernel<T, true> : expert_layer_kernel<T, false>;
    return counted([&] { cudaLaunchKernelEx(&cfg, kern, a); });
}

}  // namespace om

using namespace om;

extern "C" {

om_status om_expert_mlp(int value_type, const void* x, int64_t tokens, int64_t hidden, int64_t x_stride,
                        const int32_t* ids, const float* weights, int64_t picks, int64_t experts, int64_t inner,
                        const void* up, int64_t up_expert, int64_t up_row, const void* gate, int64_t gate_expert,
                        int64_t gate_row, const void* down, int64_t down_expert, int64_t down_row, int act, void* out,
                        int64_t out_stride, void* stream) {
    if (value_type != OM_VALUE_BF16 && value_type != OM_VALUE_F16) return OM_EINVAL;
    if (tokens < 0 || hidden < 1 || picks < 1 || experts < 1 || inner < 1 || act < OM_ACT_SILU || act > OM_ACT_RELU)
        return OM_EINVAL;
    const int64_t strides[] = {x_stride, up_expert, up_row, gate_expert, gate_row, down_expert, down_row, out_stride};
    for (const int64_t s : strides)
        if (s < 0) return OM_EINVAL;
    if (tokens > kExpertMaxTokens || picks > kExpertMaxPicks || experts > kExpertMaxExperts || hidden > (1 << 20) ||
        inner > (1 << 20))
        return OM_ERANGE;
    for (const int64_t s : strides)
        if (s > kMaxStride) return OM_ERANGE;
    if (tokens == 0) return OM_OK;
    if (x == nullptr || ids == nullptr || weights == nullptr || up == nullptr || down == nullptr || out == nullptr ||
        misaligned4(ids) || misaligned4(weights) || (tokens > 1 && out_stride < hidden))
        return OM_EINVAL;
    for (const void* p : {x, up, gate, down, (const void*)out})
        if (misaligned(p, 2)) return OM_EINVAL;
    const int64_t slots = tokens * picks, out_span = ((tokens - 1) * out_stride + hidden) * 2;
    if (overlaps(out, out_span, x, ((tokens - 1) * x_stride + hidden) * 2, 1) || overlaps(out, out_span, ids, slots * 4, 1) ||
        overlaps(out, out_span, weights, slots * 4, 1) ||
        overlaps(out, out_span, up, ((experts - 1) * up_expert + (inner - 1) * up_row + hidden) * 2, 1) ||
        (gate != nullptr &&
         overlaps(out, out_span, gate, ((experts - 1) * gate_expert + (inner - 1) * gate_row + hidden) * 2, 1)) ||
        overlaps(out, out_span, down, ((experts - 1) * down_expert + (hidden - 1) * down_row + inner) * 2, 1))
        return OM_EINVAL;
    DeviceState* d = nullptr;
    om_status s = device_state(&d);
    if (s == OM_OK) s = prepare_experts(d);
    cudaMemPool_t pool = nullptr;
    if (s == OM_OK) s = scratch_pool(d, &pool);
    if (s != OM_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    ExpertArgs a{};
    a.x = x, a.ids = ids, a.weights = weights, a.up = up, a.gate = gate, a.down = down, a.out = out;
    // a stride that takes no step says nothing about alignment
    auto stride = [](int64_t count, int64_t s) { return count > 1 ? s : 0; };
    a.x_stride = stride(tokens, x_stride), a.out_stride = out_stride;
    a.up_expert = stride(experts, up_expert), a.up_row = stride(inner, up_row);
    a.gate_expert = stride(experts, gate_expert), a.gate_row = stride(inner, gate_row);
    a.down_expert = stride(experts, down_expert), a.down_row = stride(hidden, down_row);
    a.tokens = (int)tokens, a.picks = (int)picks, a.slots = (int)slots, a.experts = (int)experts;
    a.hidden = (int)hidden, a.inner = (int)inner, a.inner_pad = (int)((inner + 7) / 8 * 8), a.act = act;
    // whole vectors where every row starts on 16 bytes and holds a multiple of them
    bool vec = hidden % 8 == 0 && inner % 8 == 0;
    for (const int64_t v : {a.x_stride, a.up_expert, a.up_row, a.gate_expert, a.gate_row, a.down_expert, a.down_row})
        vec = vec && v % 8 == 0;
    for (const void* p : {x, up, gate, down}) vec = vec && !misaligned(p, 16);
    const size_t half = (size_t)slots * a.inner_pad * 2;  // a multiple of 16
    cudaError_t e = scratch_alloc(pool, &a.high, 2 * half + (vec ? (size_t)slots * hidden * 4 : 0), st);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return OM_ENOMEM;
    }
    a.low = static_cast<char*>(a.high) + half;
    a.each = reinterpret_cast<float*>(static_cast<char*>(a.high) + 2 * half);
    e = with_half_type(value_type, [&](auto v) {
        using T = decltype(v);
        return vec ? launch_layer<T>(a, d->sm_count, st) : launch_odd_rows<T>(a, d->sm_count, st);
    });
    scratch_free(a.high, st);
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

// om_beam_select / om_beam_gather: argument checks and launches.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "beam_kernels.cuh"
#include "select_common.cuh"
#include "strided.cuh"

namespace om {

static size_t beam_smem(int stages, int64_t units, int64_t top) {
    return (size_t)beam_ring_offset() + (size_t)stages * kBeamStageBytes + (size_t)(units * top) * 16;
}

// Least logits of a slice: 16 for each thread.
constexpr int64_t kBeamLeastSlice = kBeamThreads * 16;

// Once per device: the kernels' shared memory.
static om_status prepare_beam(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        bool ok = true;
        for (auto* kern : {beam_select_kernel<float>, beam_select_kernel<__nv_bfloat16>, beam_select_kernel<__half>})
            ok = ok &&
                 cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)beam_smem(kBeamMaxStages, kMaxBeams, kMaxBeamTop)) == cudaSuccess &&
                 cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
        for (const void* kern : {(const void*)beam_gather_kernel<kBeamsInRegisters, true, kFewBeamArrays>,
                                 (const void*)beam_gather_kernel<kBeamsInRegisters, true, kMaxBeamArrays>})
            ok = ok && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kMaxBeams * kBeamGatherThreads * 16) == cudaSuccess;
        if (!ok) {
            cudaGetLastError();
            return OM_ECUDA;
        }
        ready[d->dev] = true;
    }
    return OM_OK;
}

template <typename T>
static cudaError_t launch_beam(BeamArgs a, int64_t batch, int sm_count, cudaStream_t st) {
    // CTAs of a cluster: as many as fill the SMs (two each), while slices stay long enough;
    // 16 only for few sequences with much to read.  (8 and 16: 1 x 4 x 131071 bf16 12.4
    // and 11.0 us, 4 x 8 17.5 and 17.0, but 1 x 4 x 32768 8.1 and 8.3, 8 x 8 x 131071 17.8
    // and 21.7, 16 x 8 x 50021 13.7 and 23.3.)
    const int64_t most = a.beams * std::max<int64_t>(1, a.vocab / kBeamLeastSlice);
    const bool wide = batch <= 4 && (int64_t)a.beams * a.vocab > kBeamCluster * (int64_t)32768;
    int ctas = 1;
    while (ctas < (wide ? 2 * kBeamCluster : kBeamCluster) && batch * ctas < 2 * (int64_t)sm_count && ctas < most) ctas *= 2;
    a.parts = std::max(1, ctas / a.beams);
    a.slice = (int)((((int64_t)a.vocab + a.parts - 1) / a.parts + 7) / 8 * 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * ctas));
    cfg.blockDim = dim3(kBeamThreads);
    // chunks on their way: two where there are four CTAs an SM, else four
    a.stages = batch * ctas > 2 * (int64_t)sm_count ? 2 : kBeamMaxStages;
    cfg.dynamicSmemBytes = beam_smem(a.stages, (int64_t)a.beams * a.parts, a.top);
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {early_attribute()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return counted([&] { cudaLaunchKernelEx(&cfg, beam_select_kernel<T>, a); });
}

// Bytes of the vectors that every address of the array allows.
static int beam_vector(const om_beam_array& c) {
    uint64_t low = reinterpret_cast<uintptr_t>(c.src) | reinterpret_cast<uintptr_t>(c.dst) | (uint64_t)c.entry_bytes;
    for (const int64_t s : {c.src_batch, c.src_beam, c.src_head, c.src_entry, c.dst_batch, c.dst_beam, c.dst_head,
                            c.dst_entry})
        low |= (uint64_t)s;
    return (low & 15) == 0 ? 16 : (low & 3) == 0 ? 4 : (low & 1) == 0 ? 2 : 1;
}

template <int MOST>
static cudaError_t launch_gather(const BeamGatherShape& shape, const om_beam_array* arrays, int64_t ctas, cudaStream_t st) {
    BeamGatherArgs<MOST> a;
    static_cast<BeamGatherShape&>(a) = shape;
    for (int i = 0; i < shape.count; ++i) a.arrays[i] = arrays[i], a.vector[i] = (unsigned char)beam_vector(arrays[i]);
    const bool staged = a.in_place && a.beams > kBeamsInRegisters;
    auto* kern = staged                          ? beam_gather_kernel<kBeamsInRegisters, true, MOST>
                 : a.beams <= 4                  ? beam_gather_kernel<4, false, MOST>
                 : (a.beams <= 8 || !a.in_place) ? beam_gather_kernel<8, false, MOST>
                                                 : beam_gather_kernel<kBeamsInRegisters, false, MOST>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = early_attribute();
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kBeamGatherThreads);
    cfg.dynamicSmemBytes = staged ? (size_t)a.beams * kBeamGatherThreads * 16 : 0;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return counted([&] { cudaLaunchKernelEx(&cfg, kern, a); });
}

}  // namespace om

using namespace om;

extern "C" {

om_status om_beam_select(int value_type, const void* logits, int64_t batch, int64_t beams, int64_t vocab,
                         int64_t batch_stride, int64_t beam_stride, const float* scores, const uint8_t* finished,
                         int64_t end_id, int top, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                         void* stream) {
    const int vb = value_bytes(value_type);
    if (vb == 0 || batch < 0 || beams < 1 || vocab < 1 || top < 1 || batch_stride < 0 || beam_stride < 0)
        return OM_EINVAL;
    if (finished != nullptr && (end_id < 0 || end_id >= vocab)) return OM_EINVAL;
    if (beams > kMaxBeams || top > kMaxBeamTop || vocab > (1 << 30) || batch > (1 << 24) || batch_stride > kMaxStride ||
        beam_stride > kMaxStride || too_far(batch, batch_stride))
        return OM_ERANGE;
    if (batch == 0) return OM_OK;
    if (logits == nullptr || out_scores == nullptr || out_parents == nullptr || out_tokens == nullptr ||
        misaligned(logits, vb) || misaligned4(scores) || misaligned4(out_scores) || misaligned4(out_parents) ||
        misaligned4(out_tokens))
        return OM_EINVAL;
    const int64_t span = ((batch - 1) * batch_stride + (beams - 1) * beam_stride + vocab) * vb, slots = batch * top * 4;
    const void* outs[3] = {out_scores, out_parents, out_tokens};
    for (int i = 0; i < 3; ++i) {
        if (overlaps(outs[i], slots, logits, span, 1)) return OM_EINVAL;
        if (scores != nullptr && overlaps(outs[i], slots, scores, batch * beams * 4, 1)) return OM_EINVAL;
        if (finished != nullptr && overlaps(outs[i], slots, finished, batch * beams, 1)) return OM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], slots, outs[j], slots, 1)) return OM_EINVAL;
    }
    DeviceState* d = nullptr;
    om_status s = device_state(&d);
    if (s == OM_OK) s = prepare_beam(d);
    if (s != OM_OK) return s;
    const BeamArgs a{logits, scores,     finished,    batch_stride, beam_stride, (int)beams, (int)vocab, top,
                     (int)end_id, 1, 0, 0, out_scores, out_parents, out_tokens, d->err};
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        return launch_beam<decltype(v)>(a, batch, d->sm_count, (cudaStream_t)stream);
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_beam_gather(const int32_t* parents, int64_t batch, int64_t beams, int64_t heads, int64_t entries,
                         const int32_t* starts, const int32_t* lengths, const om_beam_array* arrays, int count,
                         void* stream) {
    if (batch < 0 || beams < 1 || heads < 1 || entries < 0 || count < 1 || arrays == nullptr) return OM_EINVAL;
    if (beams > kMaxBeams || heads > 65535 || batch > 32767 || entries > INT32_MAX || count > kMaxBeamArrays)
        return OM_ERANGE;
    if (batch == 0 || entries == 0) return OM_OK;
    if (parents == nullptr || misaligned4(parents) || misaligned4(starts) || misaligned4(lengths)) return OM_EINVAL;
    int64_t spans[kMaxBeamArrays], src_spans[kMaxBeamArrays], bytes = 0;
    const int64_t counts[4] = {batch, beams, heads, entries};
    int in_place = 0;
    for (int i = 0; i < count; ++i) {
        const om_beam_array& c = arrays[i];
        if (c.entry_bytes < 1 || c.src == nullptr || c.dst == nullptr) return OM_EINVAL;
        const int64_t from[4] = {c.src_batch, c.src_beam, c.src_head, c.src_entry};
        const int64_t to[4] = {c.dst_batch, c.dst_beam, c.dst_head, c.dst_entry};
        for (int k = 0; k < 4; ++k)
            if (from[k] < 0 || to[k] < 0) return OM_EINVAL;
        if (c.entry_bytes > kMaxEntryStride || c.src_entry > kMaxEntryStride || c.dst_entry > kMaxEntryStride)
            return OM_ERANGE;
        for (int k = 0; k < 3; ++k)
            if (from[k] > kMaxStride || to[k] > kMaxStride) return OM_ERANGE;
        bool shared = false, src_shared = false;
        spans[i] = strided_span(c.entry_bytes, counts, to, &shared);
        src_spans[i] = strided_span(c.entry_bytes, counts, from, &src_shared);
        if (shared) return OM_EINVAL;
        if (overlaps(c.dst, spans[i], parents, batch * beams * 4, 1)) return OM_EINVAL;
        for (const int32_t* p : {starts, lengths})
            if (p != nullptr && overlaps(c.dst, spans[i], p, batch * 4, 1)) return OM_EINVAL;
        bool same = c.src == c.dst;
        for (int k = 0; k < 4; ++k) same = same && (from[k] == to[k] || counts[k] == 1);
        in_place += same;
        bytes = std::max(bytes, c.entry_bytes / beam_vector(c) * entries);  // columns of a row
    }
    if (in_place != 0 && in_place != count) return OM_EINVAL;
    for (int i = 0; i < count; ++i)
        for (int j = 0; j < count; ++j) {
            const om_beam_array &c = arrays[i], &o = arrays[j];
            auto dst_meets = [&](const void* p, int64_t span, int64_t sb, int64_t sn, int64_t sh, int64_t se) {
                return arrays_meet(c.dst, spans[i], c.entry_bytes, counts, {c.dst_batch, c.dst_beam, c.dst_head, c.dst_entry},
                                   p, span, o.entry_bytes, counts, {sb, sn, sh, se});
            };
            if (!in_place && dst_meets(o.src, src_spans[j], o.src_batch, o.src_beam, o.src_head, o.src_entry))
                return OM_EINVAL;
            if (i < j && dst_meets(o.dst, spans[j], o.dst_batch, o.dst_beam, o.dst_head, o.dst_entry)) return OM_EINVAL;
        }
    DeviceState* d = nullptr;
    om_status s = device_state(&d);
    if (s == OM_OK) s = prepare_beam(d);
    if (s != OM_OK) return s;
    // CTAs of a row: four waves of 8 an SM over all rows, but a column a thread at most
    const int64_t jobs = batch * heads * count;
    const int64_t parts = std::min((bytes + kBeamGatherThreads - 1) / kBeamGatherThreads,
                                   std::max<int64_t>(1, 32 * (int64_t)d->sm_count / jobs));
    if (jobs * parts > INT32_MAX) return OM_ERANGE;
    const BeamGatherShape shape{parents, starts,     lengths, entries,    batch * heads, (int)beams,
                                (int)heads, count, (int)parts, in_place != 0};
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = count <= kFewBeamArrays ? launch_gather<kFewBeamArrays>(shape, arrays, jobs * parts, st)
                                                  : launch_gather<kMaxBeamArrays>(shape, arrays, jobs * parts, st);
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

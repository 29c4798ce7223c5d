// om_embed_lookup / om_embed_lookup_backward: argument checks, scratch and launches.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "embed_kernels.cuh"
#include "select_common.cuh"
#include "strided.cuh"

namespace om {

// Whether every row of T at p consists of whole aligned vectors of 16 bytes.
template <typename T>
static bool whole_vectors(const void* p, int64_t stride, int64_t width) {
    constexpr int N = 16 / (int)sizeof(T);
    return !misaligned(p, 16) && stride % N == 0 && width % N == 0;
}

template <typename T>
static cudaError_t launch_lookup(EmbedArgs a, cudaStream_t st) {
    constexpr int kMost = 16 / (int)sizeof(T);
    const bool whole = whole_vectors<T>(a.table, a.table_stride, a.width) && whole_vectors<T>(a.out, a.out_stride, a.width);
    const int64_t vectors = a.n * (whole ? a.width / kMost : ((int64_t)a.width * (int)sizeof(T) + 30) / 16);
    const int64_t ctas = (vectors + kEmbedThreads * kEmbedUnroll - 1) / (kEmbedThreads * kEmbedUnroll);
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    auto* kern = whole ? embed_lookup_kernel<T> : embed_lookup_odd_kernel<T>;
    return counted([&] { launch_early(kern, (unsigned)ctas, kEmbedThreads, 0, st, a); });
}

// Tokens up to which pieces of long runs are short: 4096 tokens, half of them of one
// row, take 35.1 us in pieces of 32, 45.8 of 128; 65537 take 305 and 245.
constexpr int64_t kEmbedFewTokens = 16384;

// Tokens that one cluster sorts; more take the library's merge sort.
constexpr int64_t kEmbedSortMost = 1 << 18;

// Once per device: clusters of 16, and the sort's shared memory.
static om_status prepare_embed(const DeviceState* d) {
    static std::mutex mu;
    static bool ready[128];
    std::lock_guard<std::mutex> lk(mu);
    if (!ready[d->dev]) {
        if (cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)embed_sort_smem(kEmbedSortMost / kEmbedCluster)) !=
                cudaSuccess) {
            cudaGetLastError();
            return OM_ECUDA;
        }
        ready[d->dev] = true;
    }
    return OM_OK;
}

template <typename T, typename O>
static cudaError_t launch_backward(EmbedBackArgs a, int sm_count, cudaStream_t st) {
    constexpr int kMostT = 16 / (int)sizeof(T);
    cudaError_t e = cudaSuccess;
    if (a.n > 0 && a.n <= kEmbedSortMost) {
        int bits = 1;
        while (bits < 31 && (a.rows >> bits) != 0) ++bits;  // of the greatest key, `rows`
        a.passes = (bits + 8) / 9;
        a.bits = (bits + a.passes - 1) / a.passes;
        if (a.n <= kEmbedSmallMost) {
            const unsigned blocks = (unsigned)((a.n + 31) / 32);
            const size_t smem = (size_t)blocks * 32 * 4 + kEmbedSmallThreads * 4;
            e = counted([&] { launch_early(embed_sort_small_kernel, blocks, kEmbedSmallThreads, smem, st, a); });
        } else {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kEmbedCluster);
            cfg.blockDim = dim3(kEmbedSortThreads);
            cfg.dynamicSmemBytes = embed_sort_smem((a.n + kEmbedCluster - 1) / kEmbedCluster);
            cfg.stream = st;
            cudaLaunchAttribute attr[2] = {early_attribute()};
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = kEmbedCluster;
            attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            e = counted([&] { cudaLaunchKernelEx(&cfg, embed_sort_kernel, a); });
        }
        if (e != cudaSuccess) return e;
    } else if (a.n > 0) {
        e = counted([&] { launch_early(embed_keys_kernel, (unsigned)((a.n + 255) / 256), 256, 0, st, a); });
        if (e != cudaSuccess) return e;
        const om_status s = om_merge_sort_u32(a.keys, a.slots, a.n, st);
        if (s != OM_OK) return s == OM_ENOMEM ? cudaErrorMemoryAllocation : cudaErrorUnknown;
    }
    const bool whole = whole_vectors<T>(a.grad, a.grad_stride, a.width) &&
                       whole_vectors<O>(a.grad_table, a.table_stride, a.width);
    a.tiles = (a.width + 32 * kMostT - 1) / (32 * kMostT);
    // sorted places of a warp: as few as leave at most 96 warps to an SM, four waves of the
    // 24 that its shared memory holds
    a.window = 4;
    while (a.window < 32 && a.n * a.tiles / a.window > 96 * (int64_t)sm_count) a.window *= 2;
    const int64_t per = kEmbedSumThreads / 32;
    a.sum_ctas = ((a.n + a.window - 1) / a.window * a.tiles + per - 1) / per;
    a.zero_rows = 32;
    while (a.zero_rows > 4 && a.rows / a.zero_rows < 32 * (int64_t)sm_count) a.zero_rows /= 2;
    const int64_t zeros = a.accumulate ? 0 : (a.rows + a.zero_rows - 1) / a.zero_rows;
    const int64_t ctas = a.sum_ctas + (zeros + per - 1) / per;
    if (ctas == 0) return e;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    auto* kern = whole ? embed_sum_kernel<T, O, false> : embed_sum_kernel<T, O, true>;
    e = counted([&] { launch_early(kern, (unsigned)ctas, kEmbedSumThreads, 0, st, a); });
    const int64_t joins = (a.n - 1) >> a.piece_bits;  // multiples of a piece's length in (0, n)
    if (e == cudaSuccess && joins > 0) {
        const int tiles = (a.width + kEmbedJoinColumns - 1) / kEmbedJoinColumns;
        const int64_t groups = (joins + kEmbedJoinPlaces - 1) / kEmbedJoinPlaces;
        e = counted([&] { launch_early(embed_join_kernel<O>, (unsigned)(groups * tiles), kEmbedJoinThreads, 0, st, a, tiles); });
    }
    return e;
}

}  // namespace om

using namespace om;

extern "C" {

om_status om_embed_lookup(int value_type, const void* table, int64_t rows, int64_t width, int64_t table_stride,
                          const void* ids, int id_bytes, int64_t n, float scale, void* out, int64_t out_stride,
                          void* stream) {
    const int vb = value_bytes(value_type);
    if (vb == 0 || rows < 0 || width < 1 || table_stride < 0 || out_stride < 0 || n < 0 || (id_bytes != 4 && id_bytes != 8))
        return OM_EINVAL;
    if (rows > INT32_MAX - 1 || n > INT32_MAX || width > (1 << 24) || table_stride > kMaxStride || out_stride > kMaxStride ||
        too_far(rows, table_stride) || too_far(n, out_stride))
        return OM_ERANGE;
    if (n == 0) return OM_OK;
    if ((rows > 0 && table == nullptr) || ids == nullptr || out == nullptr || misaligned(table, vb) ||
        misaligned(ids, id_bytes) || misaligned(out, vb) || (n > 1 && out_stride < width))
        return OM_EINVAL;
    const int64_t span = ((n - 1) * out_stride + width) * vb;
    if (overlaps(out, span, ids, n * id_bytes, 1)) return OM_EINVAL;
    if (rows > 0 && overlaps(out, span, table, ((rows - 1) * table_stride + width) * vb, 1)) return OM_EINVAL;
    if ((n * width + kEmbedThreads * kEmbedUnroll - 1) / (kEmbedThreads * kEmbedUnroll) > INT32_MAX) return OM_ERANGE;
    DeviceState* d = nullptr;
    const om_status s = device_state(&d);
    if (s != OM_OK) return s;
    const EmbedArgs a{table, ids, out, rows, n, table_stride, out_stride, (int)width, id_bytes == 8, scale};
    const cudaError_t e =
        with_value_type(value_type, [&](auto v) { return launch_lookup<decltype(v)>(a, (cudaStream_t)stream); });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_embed_lookup_backward(int value_type, const void* grad, int64_t n, int64_t width, int64_t grad_stride,
                                   const void* ids, int id_bytes, int64_t rows, float scale, int accumulate,
                                   int table_type, void* grad_table, int64_t table_stride, void* stream) {
    const int vb = value_bytes(value_type), ob = value_bytes(table_type);
    if (vb == 0 || ob == 0 || (table_type != value_type && table_type != OM_VALUE_F32) || rows < 0 || width < 1 ||
        grad_stride < 0 || table_stride < 0 || n < 0 || (id_bytes != 4 && id_bytes != 8))
        return OM_EINVAL;
    if (rows > INT32_MAX - 1 || n > (1 << 30) || width > (1 << 20) || grad_stride > kMaxStride || table_stride > kMaxStride ||
        too_far(rows, table_stride) || too_far(n, grad_stride))
        return OM_ERANGE;
    if (rows == 0) return OM_OK;
    if (grad_table == nullptr || misaligned(grad_table, ob) || (rows > 1 && table_stride < width)) return OM_EINVAL;
    if (n > 0 && (grad == nullptr || ids == nullptr || misaligned(grad, vb) || misaligned(ids, id_bytes))) return OM_EINVAL;
    const int64_t span = ((rows - 1) * table_stride + width) * ob;
    if (n > 0 && (overlaps(grad_table, span, grad, ((n - 1) * grad_stride + width) * vb, 1) ||
                  overlaps(grad_table, span, ids, n * id_bytes, 1)))
        return OM_EINVAL;
    if ((n + 3) / 4 * ((width + 31) / 32) > (int64_t)INT32_MAX) return OM_ERANGE;
    DeviceState* d = nullptr;
    om_status s = device_state(&d);
    if (s == OM_OK) s = prepare_embed(d);
    if (s != OM_OK) return s;
    EmbedBackArgs a{};
    a.grad = grad, a.ids = ids, a.grad_table = grad_table;
    a.n = n, a.rows = rows, a.grad_stride = grad_stride, a.table_stride = table_stride;
    a.width = (int)width, a.wide = id_bytes == 8, a.accumulate = accumulate != 0, a.scale = scale;
    cudaStream_t st = (cudaStream_t)stream;
    unsigned char* scratch = nullptr;
    const size_t list = ((size_t)n * 4 + 255) & ~(size_t)255;
    a.piece_bits = n <= kEmbedFewTokens ? kEmbedPieceBits : kEmbedLongPieceBits;
    const size_t sums = n > 1 << a.piece_bits ? (size_t)(2 * (((n - 1) >> a.piece_bits) + 1)) * (size_t)width * 4 : 0;
    if (n > 0) {
        cudaMemPool_t pool = nullptr;
        s = scratch_pool(d, &pool);
        if (s != OM_OK) return s;
        const int lists = n <= kEmbedSortMost ? 4 : 2;
        const cudaError_t e = scratch_alloc(pool, reinterpret_cast<void**>(&scratch), lists * list + sums, st);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return OM_ENOMEM;
        }
        unsigned char* at = scratch;
        a.keys = reinterpret_cast<uint32_t*>(at), at += list;
        a.slots = reinterpret_cast<uint32_t*>(at), at += list;
        if (lists == 4) {
            a.other_keys = reinterpret_cast<uint32_t*>(at), at += list;
            a.other_slots = reinterpret_cast<uint32_t*>(at), at += list;
        }
        a.partial = reinterpret_cast<float*>(at);
    }
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        using T = decltype(v);
        return table_type == value_type ? launch_backward<T, T>(a, d->sm_count, st) : launch_backward<T, float>(a, d->sm_count, st);
    });
    if (scratch != nullptr) scratch_free(scratch, st);
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

// Host checks of strided arrays (caches, states): whether an array's entries
// share bytes, and whether two arrays meet.
#pragma once

#include <algorithm>
#include <cstdint>

#include "api_internal.cuh"

namespace om {

// Largest strides taken, so that no span of an array overflows 64 bits.
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxEntryStride = (int64_t)1 << 30;

// Whether `count` steps of `stride` go further than any array (and than 64 bits hold with others beside).
inline bool too_far(int64_t count, int64_t stride) { return count > 1 && stride > ((int64_t)1 << 58) / (count - 1); }

// Bytes from the first to past the last of a strided array whose entries have
// `bytes` bytes; *shared says whether entries share bytes (which an output's must not).
template <int N>
int64_t strided_span(int64_t bytes, const int64_t (&count)[N], const int64_t (&stride)[N], bool* shared) {
    int64_t c[N], s[N];
    for (int i = 0; i < N; ++i) c[i] = count[i], s[i] = stride[i];
    for (int i = 0; i < N; ++i)  // least stride first
        for (int j = i + 1; j < N; ++j)
            if (s[j] < s[i]) std::swap(s[i], s[j]), std::swap(c[i], c[j]);
    int64_t span = bytes;
    *shared = false;
    for (int i = 0; i < N; ++i)
        if (c[i] > 1) {
            if (s[i] < span) *shared = true;
            span += s[i] * (c[i] - 1);
        }
    return span;
}

// Two strided arrays of the same dimensions: of each their counts and strides in bytes.
struct DimPair {
    int64_t count_a, stride_a, count_b, stride_b;
};

// Whether an element of a and one of b share a byte, b's first one being `delta`
// bytes after a's; dims greatest stride first.  Rows of one stride can only meet
// at the few multiples of it that bring their insides together.  A yes may be
// wrong where strides differ, a no never is.
inline bool rows_meet(int64_t delta, const DimPair* dim, int dims, int64_t bytes_a, int64_t bytes_b) {
    int64_t in_a = bytes_a, in_b = bytes_b;  // spans of the dimensions below the first
    for (int i = 1; i < dims; ++i) {
        in_a += dim[i].stride_a * (dim[i].count_a - 1);
        in_b += dim[i].stride_b * (dim[i].count_b - 1);
    }
    if (dims == 0) return delta < in_a && -delta < in_b;
    if (delta >= in_a + dim->stride_a * (dim->count_a - 1) || -delta >= in_b + dim->stride_b * (dim->count_b - 1))
        return false;
    const int64_t s = dim->stride_a;
    if (s != dim->stride_b || s == 0 || (in_a + in_b) / s > 4) return true;
    // row i of a and row i + k of b
    const int64_t low = std::max((-in_b - delta) / s - 1, -(dim->count_a - 1));
    const int64_t high = std::min((in_a - delta) / s + 1, dim->count_b - 1);
    for (int64_t k = low; k <= high; ++k)
        if (rows_meet(delta + k * s, dim + 1, dims - 1, bytes_a, bytes_b)) return true;
    return false;
}

// The same of arrays at a and b, whose spans are known.
template <int N>
bool arrays_meet(const void* a, int64_t span_a, int64_t bytes_a, const int64_t (&count_a)[N],
                 const int64_t (&stride_a)[N], const void* b, int64_t span_b, int64_t bytes_b,
                 const int64_t (&count_b)[N], const int64_t (&stride_b)[N]) {
    if (!overlaps(a, span_a, b, span_b, 1)) return false;
    DimPair dim[N];
    int dims = 0;
    for (int i = 0; i < N; ++i)
        if (count_a[i] > 1 || count_b[i] > 1) dim[dims++] = {count_a[i], stride_a[i], count_b[i], stride_b[i]};
    std::sort(dim, dim + dims, [](const DimPair& x, const DimPair& y) { return x.stride_a > y.stride_a; });
    return rows_meet((int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)), dim, dims, bytes_a,
                     bytes_b);
}

}  // namespace om

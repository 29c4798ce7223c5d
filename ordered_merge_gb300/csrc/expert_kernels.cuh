// Kernels of om_expert_mlp: the routed experts' layers for a few tokens.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "select_common.cuh"

namespace om {

constexpr int kExpertMaxTokens = 64;
constexpr int kExpertMaxPicks = 32;
constexpr int kExpertMaxExperts = 1024;
constexpr int kExpertWarps = 8;
constexpr int kExpertRows = 16;    // weight rows of a CTA: the height of one matrix instruction
constexpr int kExpertUnroll = 4;   // steps of 32 columns whose weights are in flight
constexpr int kExpertCluster = 8;

enum ExpertAct { kActSilu = 0, kActGelu = 1, kActRelu = 2 };

struct ExpertArgs {
    const void* x;
    const int32_t* ids;
    const float* weights;
    const void *up, *gate, *down;
    void *high, *low;  // [slots][inner_pad]: the activations, and what their rounding left
    void* out;
    int64_t x_stride, out_stride;
    int64_t up_expert, up_row, gate_expert, gate_row, down_expert, down_row;  // strides in values
    int tokens, picks, slots, experts, hidden, inner, inner_pad, act;
    int by_slot;  // first kernel: CTAs by slot (the first of its expert works), not by expert
    int parts;    // second kernel: pieces of an expert's columns
};

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1, __half) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A product over 32 columns, two instructions: lane (g, t) = (lane / 4, lane % 4)
// holds 8 neighbouring columns (8t ...) of weight rows g and g + 8 and of token g.
// Which column an instruction takes for which does not matter as long as both
// sides agree, so every lane loads whole 16-byte vectors of a row.
template <typename T>
__device__ __forceinline__ void mma_step(float (&d)[4], const uint4& a, const uint4& b, const uint4& x) {
    mma_16x8x16(d, a.x, b.x, a.y, b.y, x.x, x.y, T{});
    mma_16x8x16(d, a.z, b.z, a.w, b.w, x.z, x.w, T{});
}

// 8 values of a row of `columns` from column k on, zeros past its end.
// VEC: rows are aligned to 16 bytes and columns a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load8(const T* row, int k, int columns) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (VEC) {
        if (k < columns) v = *reinterpret_cast<const uint4*>(row + k);
    } else {
        const unsigned short* p = reinterpret_cast<const unsigned short*>(row) + k;
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = k + i < columns ? p[i] : 0;
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    return v;
}

// The next slots, from `from` on, whose id is e: up to `most` of them into list (in
// order), and where to go on.  All lanes of a warp.
__device__ __forceinline__ int next_slots(const int32_t* ids, int slots, int e, int& from, int most, uint16_t* list) {
    const int lane = threadIdx.x & 31;
    int count = 0;
    while (from < slots && count < most) {
        const int q = from + lane;
        unsigned same = __ballot_sync(0xffffffffu, q < slots && ids[q] == e);
        const int before = __popc(same & ((1u << lane) - 1));
        if ((same >> lane & 1) && count + before < most) list[count + before] = (uint16_t)q;
        const int found = __popc(same);
        if (count + found > most) {  // go on at the first that found no room
            for (int k = count; k < most; ++k) same &= same - 1;
            from += __ffs(same) - 1;
            count = most;
        } else {
            from += 32;
            count += found;
        }
    }
    __syncwarp();
    return count;
}

__device__ __forceinline__ float activate(float x, int act) {
    if (act == kActSilu) return x / (1.0f + expf(-x));
    if (act == kActGelu) return 0.5f * x * (1.0f + erff(x * 0.70710678118654752f));
    return x > 0.0f || x != x ? x : 0.0f;
}

// First kernel: the activations act(gate x) * (up x), or act(up x), of every slot
// whose id is an expert.  A CTA takes 16 rows of one expert, its eight warps every
// eighth step of 32 columns of them, and its tokens 8 NT at a time; the warps' sums
// meet in shared memory.  With at most a few tokens to an expert the weights'
// bytes bound it: each is read once, straight from memory to the instruction's
// registers, 16 bytes a lane, and the tokens' rows come from the caches.  The
// tensor work is small beside that, so mma.sync does.
template <typename T, bool GATED, int NT, bool VEC>
__global__ void __launch_bounds__(kExpertWarps * 32) expert_up_kernel(const ExpertArgs a) {
    wait_for_stream();
    constexpr int MATS = GATED ? 2 : 1, COLS = 8 * NT, U = VEC ? kExpertUnroll : 1;
    extern __shared__ __align__(16) float s_sum[];  // [warps][MATS][COLS][16]
    __shared__ uint16_t s_list[COLS];
    __shared__ int s_count, s_from;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int first_row = blockIdx.x * kExpertRows;
    const int e = a.by_slot ? a.ids[blockIdx.y] : (int)blockIdx.y;
    if ((unsigned)e >= (unsigned)a.experts) return;
    const T* up = static_cast<const T*>(a.up) + e * a.up_expert;
    const T* gate = static_cast<const T*>(a.gate) + e * a.gate_expert;
    const int r0 = first_row + g, r1 = r0 + 8;
    const T* rows[2 * MATS] = {up + (int64_t)min(r0, a.inner - 1) * a.up_row, up + (int64_t)min(r1, a.inner - 1) * a.up_row};
    if (GATED) {
        rows[2 * MATS - 2] = gate + (int64_t)min(r0, a.inner - 1) * a.gate_row;
        rows[2 * MATS - 1] = gate + (int64_t)min(r1, a.inner - 1) * a.gate_row;
    }
    const int steps = (a.hidden + 31) / 32;
    for (int from = 0;;) {
        if (warp == 0) {
            const int n = next_slots(a.ids, a.slots, e, from, COLS, s_list);
            if (lane == 0) s_count = n, s_from = from;
        }
        __syncthreads();
        const int count = s_count;
        from = s_from;
        if (count == 0) return;
        if (a.by_slot && s_list[0] < blockIdx.y) return;  // the expert is its first slot's CTA's
        const T* tokens[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int c = 8 * n + g;
            tokens[n] = c < count ? static_cast<const T*>(a.x) + (int64_t)(s_list[c] / a.picks) * a.x_stride : nullptr;
        }
        float d[MATS][NT][4] = {};
        for (int s0 = warp; s0 < steps; s0 += kExpertWarps * U) {
            uint4 w[U][2 * MATS];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (s0 + u * kExpertWarps) * 32 + 8 * t;
#pragma unroll
                for (int m = 0; m < 2 * MATS; ++m) w[u][m] = load8<T, VEC>(rows[m], k, a.hidden);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (s0 + u * kExpertWarps) * 32 + 8 * t;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (8 * n >= count) break;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (tokens[n] != nullptr) x = load8<T, VEC>(tokens[n], k, a.hidden);
                    mma_step<T>(d[0][n], w[u][0], w[u][1], x);
                    if (GATED) mma_step<T>(d[MATS - 1][n], w[u][2 * MATS - 2], w[u][2 * MATS - 1], x);
                }
            }
        }
        // lane's sums: rows g, g and g + 8, g + 8, tokens 2t, 2t + 1
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float* to = s_sum + ((warp * MATS + m) * COLS + 8 * n + 2 * t) * kExpertRows + g;
                to[0] = d[m][n][0], to[kExpertRows] = d[m][n][1];
                to[8] = d[m][n][2], to[kExpertRows + 8] = d[m][n][3];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < count * kExpertRows; i += kExpertWarps * 32) {
            const int c = i / kExpertRows, r = first_row + i % kExpertRows;
            float v[MATS] = {};
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int k = 0; k < kExpertWarps; ++k) v[m] += s_sum[(k * MATS + m) * COLS * kExpertRows + i];
            if (r < a.inner) {
                const float act = GATED ? activate(v[MATS - 1], a.act) * v[0] : activate(v[0], a.act);
                // two roundings hold the value to 16 (bf16) or 22 bits, so that the second
                // product loses nothing that its sums in 32 bits keep
                const T high = from_float<T>(act);
                const T low = from_float<T>(isinf(to_float(high)) ? 0.0f : act - to_float(high));
                const int64_t at = (int64_t)s_list[c] * a.inner_pad + r;
                static_cast<T*>(a.high)[at] = high;
                static_cast<T*>(a.low)[at] = low;
            }
        }
        if (from >= a.slots) return;
        __syncthreads();
    }
}

// Second kernel: y = sum over a token's slots of weight * down[e] a.  A cluster
// takes 16 rows of the output; its warps share out the experts that any slot asks
// for (cut into `parts` pieces of their columns where there are few), each adding
// what its items give to its own sums of all tokens in shared memory; these are
// added in a fixed order, over the CTAs of the cluster through its shared memory.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kExpertWarps * 32) expert_down_kernel(const ExpertArgs a) {
    wait_for_stream();
    constexpr int U = VEC ? kExpertUnroll : 1, NT = 2, COLS = 8 * NT;
    extern __shared__ __align__(16) float s_sum[];  // [warps][tokens][16]
    __shared__ float s_tile[kExpertWarps][COLS][kExpertRows];
    __shared__ uint16_t s_list[kExpertWarps][COLS];
    __shared__ uint16_t s_expert[kExpertMaxExperts];
    __shared__ unsigned s_asked[kExpertMaxExperts / 32];
    __shared__ int s_experts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const uint32_t ctas = cluster_size(), rank = cluster_rank();
    const int first_row = (int)(blockIdx.x / ctas) * kExpertRows;
    for (int i = threadIdx.x; i < kExpertMaxExperts / 32; i += kExpertWarps * 32) s_asked[i] = 0;
    for (int i = threadIdx.x; i < kExpertWarps * a.tokens * kExpertRows; i += kExpertWarps * 32) s_sum[i] = 0.0f;
    __syncthreads();
    for (int q = threadIdx.x; q < a.slots; q += kExpertWarps * 32) {
        const int e = a.ids[q];
        if ((unsigned)e < (unsigned)a.experts) atomicOr(&s_asked[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (warp == 0) {  // the experts asked for, rising
        const unsigned mine = s_asked[lane];
        int run = __popc(mine);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int upper = __shfl_up_sync(0xffffffffu, run, d);
            if (lane >= d) run += upper;
        }
        int at = run - __popc(mine);
        for (unsigned left = mine; left != 0; left &= left - 1) s_expert[at++] = (uint16_t)(32 * lane + __ffs(left) - 1);
        if (lane == 31) s_experts = run;
    }
    __syncthreads();
    const int items = s_experts * a.parts, steps = (a.inner + 31) / 32, piece = (steps + a.parts - 1) / a.parts;
    const int r0 = min(first_row + g, a.hidden - 1), r1 = min(first_row + g + 8, a.hidden - 1);
    float* sums = s_sum + warp * a.tokens * kExpertRows;
    for (int i = (int)rank * kExpertWarps + warp; i < items; i += (int)ctas * kExpertWarps) {
        const int e = s_expert[i / a.parts], s_lo = i % a.parts * piece, s_hi = min(s_lo + piece, steps);
        const T* down = static_cast<const T*>(a.down) + e * a.down_expert;
        const T *row0 = down + (int64_t)r0 * a.down_row, *row1 = down + (int64_t)r1 * a.down_row;
        for (int from = 0; from < a.slots;) {
            const int count = next_slots(a.ids, a.slots, e, from, COLS, s_list[warp]);
            if (count == 0) break;
            const T *high[NT], *low[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int c = 8 * n + g;
                high[n] = c < count ? static_cast<const T*>(a.high) + (int64_t)s_list[warp][c] * a.inner_pad : nullptr;
                low[n] = c < count ? static_cast<const T*>(a.low) + (int64_t)s_list[warp][c] * a.inner_pad : nullptr;
            }
            float d[NT][4] = {};
            for (int s0 = s_lo; s0 < s_hi; s0 += U) {
                uint4 w[U][2];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = s0 + u < s_hi ? (s0 + u) * 32 + 8 * t : a.inner;
                    w[u][0] = load8<T, VEC>(row0, k, a.inner);
                    w[u][1] = load8<T, VEC>(row1, k, a.inner);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = s0 + u < s_hi ? (s0 + u) * 32 + 8 * t : a.inner;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (8 * n >= count) break;
                        uint4 h = make_uint4(0, 0, 0, 0), l = h;
                        if (high[n] != nullptr) h = load8<T, VEC>(high[n], k, a.inner), l = load8<T, VEC>(low[n], k, a.inner);
                        mma_step<T>(d[n], w[u][0], w[u][1], h);
                        mma_step<T>(d[n], w[u][0], w[u][1], l);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float* to = &s_tile[warp][8 * n + 2 * t][g];
                to[0] = d[n][0], to[kExpertRows] = d[n][1], to[8] = d[n][2], to[kExpertRows + 8] = d[n][3];
            }
            __syncwarp();
            // one slot after another: a token may ask for an expert twice
            if (lane < kExpertRows)
                for (int c = 0; c < count; ++c) {
                    const int q = s_list[warp][c];
                    sums[q / a.picks * kExpertRows + lane] += a.weights[q] * s_tile[warp][c][lane];
                }
            __syncwarp();
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * kExpertRows; i += kExpertWarps * 32) {
        float y = s_sum[i];
#pragma unroll
        for (int w = 1; w < kExpertWarps; ++w) y += s_sum[w * a.tokens * kExpertRows + i];
        s_sum[i] = y;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    // the CTAs of the cluster take the tokens in turn
    for (int i = (int)rank * kExpertWarps * 32 + (int)threadIdx.x; i < a.tokens * kExpertRows; i += (int)ctas * kExpertWarps * 32) {
        float y = 0.0f;
        for (uint32_t r = 0; r < ctas; ++r) y += __int_as_float(peer_word(reinterpret_cast<const int*>(s_sum + i), r));
        const int token = i / kExpertRows, row = first_row + i % kExpertRows;
        if (row < a.hidden) static_cast<T*>(a.out)[token * a.out_stride + row] = from_float<T>(y);
    }
    if (ctas > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

}  // namespace om

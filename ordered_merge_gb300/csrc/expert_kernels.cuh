// Kernels of om_expert_mlp: the routed experts' layers for a few tokens.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "select_common.cuh"

namespace om {

constexpr int kExpertMaxTokens = 64;
constexpr int kExpertMaxPicks = 32;
constexpr int kExpertMaxExperts = 1024;
constexpr int kExpertWarps = 8;
constexpr int kExpertRows = 16;    // weight rows of a CTA: the height of one matrix instruction
constexpr int kExpertCluster = 8;

// 16 bytes that other CTAs of this launch have written (past the L1 cache).
__device__ __forceinline__ uint4 load_l2(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(__cvta_generic_to_global(p))
                 : "memory");
    return v;
}

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
    int by_slot;  // expert_up_kernel: CTAs by slot (the first of its expert works), not by expert
    int parts;    // expert_down_kernel: pieces of an expert's columns
    float* each;  // expert_layer_kernel: [slots][hidden], what each slot adds to its token
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

// 8 values of a row of `columns` from column k on, zeros past its end, one by one.
template <typename T>
__device__ __forceinline__ uint4 load8(const T* row, int k, int columns) {
    const unsigned short* p = reinterpret_cast<const unsigned short*>(row) + k;
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = k + i < columns ? p[i] : 0;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
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
    // 1 + erf(y) as erfc(-y): the sum would cancel in 32 bits far below zero (6 % of it at x = -5)
    if (act == kActGelu) return 0.5f * x * erfcf(x * -0.70710678118654752f);
    return x > 0.0f || x != x ? x : 0.0f;
}

// An activation goes to the second product as two values of the weights' type, each with
// sums of its own: itself rounded, and what that left.  In bf16 the pair is within 2^-16 of
// it, 2^-8 of what the output's rounding may take.  In f16 it is within 2^-22; f16's smallest
// step, 2^-24, would spoil that for activations below 1/8, so the second value is kept times
// 2^11: 2^-22 down to activations of 2^-14, and 2^-36 at most beneath.  (Times 2^12, what the
// greatest activations leave would overflow.)  Times are as with one sum and no factor: 12
// tokens of 4 of 32 experts, 2000 x 1400 f16, 59.7 us.
template <typename T>
constexpr float kRestScale = std::is_same<T, __half>::value ? 2048.0f : 1.0f;
// The sum of both.  An infinite weight makes the first one infinite; what was left has any
// sign there, or is zero, and says nothing.
template <typename T>
__device__ __forceinline__ float pair_sum(float first, float rest) {
    return isinf(first) ? first : first + rest * (1.0f / kRestScale<T>);
}
template <typename T>
__device__ __forceinline__ void store_pair(const ExpertArgs& a, int64_t at, float h) {
    const T high = from_float<T>(h);
    // beyond f16's range the first value is infinite, and nothing is left
    const float rest = isinf(to_float(high)) ? 0.0f : h - to_float(high);
    static_cast<T*>(a.high)[at] = high;
    static_cast<T*>(a.low)[at] = from_float<T>(rest * kRestScale<T>);
}

// ---- rows that no 16-byte copy can take (odd sizes, strides or addresses): two
// kernels whose lanes load value by value

// First the activations act(gate x) * (up x), or act(up x), of every slot whose id
// is an expert.  A CTA takes 16 rows of one expert, its eight warps every eighth
// step of 32 columns of them, and its tokens 8 NT at a time; the warps' sums meet
// in shared memory.
template <typename T, bool GATED, int NT>
__global__ void __launch_bounds__(kExpertWarps * 32) expert_up_kernel(const ExpertArgs a) {
    wait_for_stream();
    constexpr int MATS = GATED ? 2 : 1, COLS = 8 * NT;
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
        for (int s = warp; s < steps; s += kExpertWarps) {
            const int k = s * 32 + 8 * t;
            uint4 w[2 * MATS];
#pragma unroll
            for (int m = 0; m < 2 * MATS; ++m) w[m] = load8<T>(rows[m], k, a.hidden);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (8 * n >= count) break;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (tokens[n] != nullptr) x = load8<T>(tokens[n], k, a.hidden);
                mma_step<T>(d[0][n], w[0], w[1], x);
                if (GATED) mma_step<T>(d[MATS - 1][n], w[2 * MATS - 2], w[2 * MATS - 1], x);
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
                store_pair<T>(a, (int64_t)s_list[c] * a.inner_pad + r, act);
            }
        }
        if (from >= a.slots) return;
        __syncthreads();
    }
}

// Then y = sum over a token's slots of weight * down[e] a.  A cluster
// takes 16 rows of the output; its warps share out the experts that any slot asks
// for (cut into `parts` pieces of their columns where there are few), each adding
// what its items give to its own sums of all tokens in shared memory; these are
// added in a fixed order, over the CTAs of the cluster through its shared memory.
//
// Bound by the latency of single values: both kernels for one token of 8 of 64 gated
// experts, 2047 x 1023 f16, take 58 us (aligned rows 29), 12 tokens of 4 of 32, 2001 x
// 1399, 245, 64 of 8 of 64, 1023 x 511, 170, 64 of 4 of 16, 2047 x 1023, 287 (aligned 79).
// In the 64 registers of four CTAs an SM a few bytes spill; three without: 15 % slower.
template <typename T>
__global__ void __launch_bounds__(kExpertWarps * 32) expert_down_kernel(const ExpertArgs a) {
    wait_for_stream();
    constexpr int NT = 2, COLS = 8 * NT;
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
            float d[2][NT][4] = {};
            for (int s = s_lo; s < s_hi; ++s) {
                const int k = s * 32 + 8 * t;
                const uint4 w0 = load8<T>(row0, k, a.inner), w1 = load8<T>(row1, k, a.inner);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (8 * n >= count) break;
                    uint4 h = make_uint4(0, 0, 0, 0), l = h;
                    if (high[n] != nullptr) h = load8<T>(high[n], k, a.inner), l = load8<T>(low[n], k, a.inner);
                    mma_step<T>(d[0][n], w0, w1, h);
                    mma_step<T>(d[1][n], w0, w1, l);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) d[0][n][i] = pair_sum<T>(d[0][n][i], d[1][n][i]);
                float* to = &s_tile[warp][8 * n + 2 * t][g];
                to[0] = d[0][n][0], to[kExpertRows] = d[0][n][1], to[8] = d[0][n][2], to[kExpertRows + 8] = d[0][n][3];
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

// ---- the layer in one launch
//
// With a few tokens to an expert the weights' bytes bound the layer: each is to be
// read once, at the memory's rate.  Two CTAs an SM, all at once (a cooperative
// launch), take items of 16 or 32 weight rows of one expert in turn; a block of an
// item is 1024 columns, of which each of the eight warps has every eighth step of
// 32.  A lane loads its 16 bytes of the rows straight into the registers that the
// tensor instructions take (16 rows by 8 tokens; mma.sync: at 64 tokens the tensor
// work is a few percent of what it can do, and 8 columns waste least), all of a
// block at once, and the next block's before the sums of this one are put together
// in shared memory: of a whole block 64 KB a CTA are on their way in the first product, 32
// in the second (one tile of rows, beside which each token has two).
// Bound by memory where many experts are read: 64 tokens through 8 of 128 gated
// experts of 2048 x 1024, 1.59 GB, 257 us (6.2 TB/s, 91 % of the copy rate).  (Rings in
// shared memory were slower: filled by bulk copies of 512-byte pieces of rows, 90
// cycles apiece, 984 us, by 16-byte copies of producer warps 327.)  One token, 0.1 GB,
// 28.7 us: 10 and 5 of them at the copy rate, the rest the launch and first loads (5),
// the barriers (2.5), uneven shares of 512 items among 304 CTAs (3) and the last sums.
//
// An expert with more than 8 tokens takes its weights again, from the L2 cache: 64
// tokens of 4 of 16 experts 79 us (16 tokens at a time 82, 32 at a time 95), of 8
// of 64 experts 169 (180, 283).
//
// First all items of the up (and gate) products, then, after a barrier of the
// grid, those of the down products, whose first weights are asked for inside the
// barrier; each slot's products go to `each`, and after another barrier a token's
// slots are added in their order.

constexpr int kLayerSteps = 4;                                     // of a warp in a block
constexpr int kLayerColumns = 32 * kExpertWarps * kLayerSteps;     // of a block
constexpr int kLayerThreads = kExpertWarps * 32;
constexpr int kLayerCtas = 2;     // of an SM: they need their 128 registers a thread
constexpr int kLayerTokens = 8;   // taken at once

struct LayerShared {
    uint16_t order[kExpertMaxTokens * kExpertMaxPicks];  // the slots, by expert
    uint16_t expert[kExpertMaxExperts];                  // the experts asked for, rising
    uint16_t start[kExpertMaxExperts + 1];               // and where their slots start
    int count[kExpertMaxExperts];
    int experts;
};

// The two halves of a barrier of the grid; all threads.  What a thread loads between
// them does not hold up the arrival (2.7 us of 31 where the next weights were asked for
// before it).  Functions of their own: inlined, the thread that waits stays apart from
// its warp afterwards.
__device__ __noinline__ unsigned layer_arrive() { return cooperative_groups::this_grid().barrier_arrive(); }
__device__ __noinline__ void layer_wait(unsigned token) { cooperative_groups::this_grid().barrier_wait(static_cast<unsigned&&>(token)); }

// One of the two products: its weights, their shape and the rows that they meet.
template <typename T, bool SECOND, bool GATED, int TILES>
struct LayerProduct {
    const ExpertArgs& a;
    static constexpr int kMats = GATED ? 2 : 1;       // matrices that give 16 TILES / kMats rows each
    static constexpr int kRows = 16 * TILES / kMats;  // rows of the result in an item
    static constexpr int kSets = SECOND ? 2 : 1;      // rows of a token, and sums
    static constexpr bool kSecond = SECOND;
    __device__ __forceinline__ int columns() const { return SECOND ? a.inner : a.hidden; }
    __device__ __forceinline__ int result() const { return SECOND ? a.hidden : a.inner; }
    __device__ __forceinline__ int64_t row_stride(int m) const { return SECOND ? a.down_row : m == 0 ? a.up_row : a.gate_row; }
    __device__ __forceinline__ const T* expert(int m, int e) const {
        if (SECOND) return static_cast<const T*>(a.down) + e * a.down_expert;
        return m == 0 ? static_cast<const T*>(a.up) + e * a.up_expert : static_cast<const T*>(a.gate) + e * a.gate_expert;
    }
    __device__ __forceinline__ const T* token(int slot) const {
        if (!SECOND) return static_cast<const T*>(a.x) + slot / a.picks * a.x_stride;
        return static_cast<const T*>(a.high) + (int64_t)slot * a.inner_pad;
    }
};

// A warp's way through the blocks of a product.
template <typename T, int TILES, typename P>
struct LayerWork {
    static constexpr int S = kLayerSteps;
    const P& p;
    const LayerShared& s;
    const int tiles, items, columns;
    int item, tile, expert, q, end, c;  // the block: first slot in order, those of its expert, first column
    const T* rows[TILES];               // this lane's, in the tiles, at its columns of the first step
    const T* token;                     // and of its token, if there is one
    uint4 w[S][TILES][2], x[S][P::kSets];

    __device__ __forceinline__ LayerWork(const P& product, const LayerShared& shared)
        : p(product), s(shared), tiles((product.result() + P::kRows - 1) / P::kRows), items(shared.experts * tiles),
          columns(product.columns()) {
        item = (int)blockIdx.x;
        if (here()) start_item();
    }
    __device__ __forceinline__ int lane_column() const { return 32 * (int)(threadIdx.x >> 5) + 8 * (int)(threadIdx.x & 3); }
    __device__ __forceinline__ bool here() const { return item < items; }
    __device__ __forceinline__ bool last_columns() const { return c + kLayerColumns >= columns; }
    __device__ __forceinline__ int count() const { return min(kLayerTokens, end - q); }
    __device__ __forceinline__ void start_item() {
        const int k = item / tiles;
        tile = item - k * tiles, expert = s.expert[k], q = s.start[k], end = s.start[k + 1], c = 0;
        const int g = (int)(threadIdx.x & 31) >> 2;
#pragma unroll
        for (int m = 0; m < TILES; ++m) {  // rows past the matrix's end are its last one again: they are not stored
            const int row = min(tile * P::kRows + (P::kMats == 1 ? 16 * m : 0) + g, p.result() - 1);
            const int mat = P::kMats == 1 ? 0 : m;
            rows[m] = p.expert(mat, expert) + row * p.row_stride(mat) + lane_column();
        }
        start_tokens();
    }
    __device__ __forceinline__ void start_tokens() {
        const int i = q + ((int)(threadIdx.x & 31) >> 2);
        token = i < end ? p.token(s.order[i]) + lane_column() : nullptr;
    }
    __device__ __forceinline__ void next() {
        c += kLayerColumns;
        if (c < columns) return;
        c = 0, q += kLayerTokens;
        if (q < end) {
            start_tokens();
            return;
        }
        item += (int)gridDim.x;
        if (here()) start_item();
    }
    // From a lane's row to the one 8 below it, or 0 where that is past the end.
    __device__ __forceinline__ int64_t second_row(int m) const {
        const int row = tile * P::kRows + (P::kMats == 1 ? 16 * m : 0) + ((int)(threadIdx.x & 31) >> 2);
        return row + 8 < p.result() ? 8 * p.row_stride(P::kMats == 1 ? 0 : m) : 0;
    }
    __device__ __forceinline__ void load_weights() {
        const int left = columns - c - lane_column();
#pragma unroll
        for (int m = 0; m < TILES; ++m) {
            const int64_t below = second_row(m);
#pragma unroll
            for (int u = 0; u < S; ++u) {
                const int k = u * 32 * kExpertWarps;
                w[u][m][0] = w[u][m][1] = make_uint4(0, 0, 0, 0);
                if (k < left) {
                    w[u][m][0] = load_once(reinterpret_cast<const uint4*>(rows[m] + c + k));
                    w[u][m][1] = load_once(reinterpret_cast<const uint4*>(rows[m] + below + c + k));
                }
            }
        }
    }
    // Behind the barrier of the grid h is there; other SMs wrote it, so past the L1 cache.
    __device__ __forceinline__ void load_tokens() {
#pragma unroll
        for (int u = 0; u < S; ++u)
#pragma unroll
            for (int set = 0; set < P::kSets; ++set) {
                const int k = c + u * 32 * kExpertWarps;
                x[u][set] = make_uint4(0, 0, 0, 0);
                if (token == nullptr || k + lane_column() >= columns) continue;
                const T* from = token + k + (set == 0 ? 0 : static_cast<const T*>(p.a.low) - static_cast<const T*>(p.a.high));
                if constexpr (P::kSecond) x[u][set] = load_l2(reinterpret_cast<const uint4*>(from));
                else x[u][set] = *reinterpret_cast<const uint4*>(from);
            }
    }
    __device__ __forceinline__ void multiply(float (&d)[P::kSets][TILES][4]) {
        const int warp_column = c + 32 * (int)(threadIdx.x >> 5);
#pragma unroll
        for (int u = 0; u < S; ++u) {
            if (warp_column + u * 32 * kExpertWarps >= columns) break;
#pragma unroll
            for (int set = 0; set < P::kSets; ++set)
#pragma unroll
                for (int m = 0; m < TILES; ++m) mma_step<T>(d[set][m], w[u][m][0], w[u][m][1], x[u][set]);
        }
    }
};

// All blocks of a product; done(slot in order, first row, sums of the TILES tiles)
// takes an item's sums.  The first block's weights are there.
template <typename T, int TILES, typename P, typename F>
__device__ __forceinline__ void layer_product(LayerWork<T, TILES, P>& work, float* sums, int& turn, F&& done) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    float d[P::kSets][TILES][4] = {};
    while (work.here()) {
        work.multiply(d);
        const bool last = work.last_columns();
        const int q = work.q, count = work.count(), row = work.tile * P::kRows;
        work.next();
        if (work.here()) work.load_weights(), work.load_tokens();
        if (!last) continue;
        // lane's sums: rows g, g and g + 8, g + 8, tokens 2t, 2t + 1.  Two turns of the memory:
        // one barrier an item.
        float* mine = sums + turn * kExpertWarps * TILES * kLayerTokens * kExpertRows;
        turn ^= 1;
#pragma unroll
        for (int m = 0; m < TILES; ++m) {
            if constexpr (P::kSets == 2) {
#pragma unroll
                for (int i = 0; i < 4; ++i) d[0][m][i] = pair_sum<T>(d[0][m][i], d[1][m][i]), d[1][m][i] = 0.0f;
            }
            float* to = mine + ((warp * TILES + m) * kLayerTokens + 2 * t) * kExpertRows + g;
            to[0] = d[0][m][0], to[kExpertRows] = d[0][m][1];
            to[8] = d[0][m][2], to[kExpertRows + 8] = d[0][m][3];
            d[0][m][0] = d[0][m][1] = d[0][m][2] = d[0][m][3] = 0.0f;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < count * kExpertRows; i += kLayerThreads) {
            float v[TILES];
#pragma unroll
            for (int m = 0; m < TILES; ++m) {
                v[m] = 0.0f;
#pragma unroll
                for (int k = 0; k < kExpertWarps; ++k) v[m] += mine[(k * TILES + m) * kLayerTokens * kExpertRows + i];
            }
            done(q + i / kExpertRows, row + i % kExpertRows, v);
        }
    }
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kLayerThreads, kLayerCtas) expert_layer_kernel(const ExpertArgs a) {
    wait_for_stream();
    // 16-row tiles of an item: up and gate, or two of up; one of down, beside whose 16 rows
    // each token has two (items of 32 rows were 1 to 5 % slower)
    constexpr int UP = 2, DOWN = 1;
    __shared__ float s_sums[2 * kExpertWarps * UP * kLayerTokens * kExpertRows];
    __shared__ LayerShared s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the slots by expert
    for (int e = threadIdx.x; e < kExpertMaxExperts; e += kLayerThreads) s.count[e] = 0;
    __syncthreads();
    for (int q = threadIdx.x; q < a.slots; q += kLayerThreads) {
        const int e = a.ids[q];
        if ((unsigned)e < (unsigned)a.experts) atomicAdd(&s.count[e], 1);
    }
    __syncthreads();
    if (warp == 0) {  // 32 experts a round
        int slots = 0, asked = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int c = s.count[e0 + lane];
            const unsigned there = __ballot_sync(0xffffffffu, c != 0);
            if (there == 0) continue;
            int run = c;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, run, d);
                if (lane >= d) run += up;
            }
            if (c != 0) {
                const int at = asked + __popc(there & ((1u << lane) - 1));
                s.expert[at] = (uint16_t)(e0 + lane);
                s.start[at] = (uint16_t)(slots + run - c);
                s.count[e0 + lane] = slots + run - c;
            }
            asked += __popc(there);
            slots += __shfl_sync(0xffffffffu, run, 31);
        }
        if (lane == 0) s.experts = asked, s.start[asked] = (uint16_t)slots;
    }
    __syncthreads();
    for (int q = threadIdx.x; q < a.slots; q += kLayerThreads) {  // in any order: a slot's values do not depend on it
        const int e = a.ids[q];
        if ((unsigned)e < (unsigned)a.experts) s.order[atomicAdd(&s.count[e], 1)] = (uint16_t)q;
    }
    __syncthreads();

    int turn = 0;
    {
        const LayerProduct<T, false, GATED, UP> product{a};
        LayerWork<T, UP, LayerProduct<T, false, GATED, UP>> work(product, s);
        if (work.here()) work.load_weights(), work.load_tokens();
        layer_product<T, UP>(work, s_sums, turn, [&](int q, int row, const float (&v)[UP]) {
            const int64_t to = (int64_t)s.order[q] * a.inner_pad;
#pragma unroll
            for (int m = 0; m < (GATED ? 1 : UP); ++m) {
                const int r = row + 16 * m;
                if (r >= a.inner) break;
                const float act = GATED ? activate(v[UP - 1], a.act) * v[0] : activate(v[m], a.act);
                store_pair<T>(a, to + r, act);
            }
        });
    }
    {
        const LayerProduct<T, true, false, DOWN> product{a};
        LayerWork<T, DOWN, LayerProduct<T, true, false, DOWN>> work(product, s);
        const unsigned token = layer_arrive();
        if (work.here()) work.load_weights();
        layer_wait(token);
        if (work.here()) work.load_tokens();
        layer_product<T, DOWN>(work, s_sums, turn, [&](int q, int row, const float (&v)[DOWN]) {
            const int slot = s.order[q];
#pragma unroll
            for (int m = 0; m < DOWN; ++m)
                if (row + 16 * m < a.hidden) __stcg(a.each + (int64_t)slot * a.hidden + row + 16 * m, v[m]);
        });
    }
    layer_wait(layer_arrive());
    const int64_t all = (int64_t)a.tokens * a.hidden;
    for (int64_t i = (int64_t)blockIdx.x * kLayerThreads + threadIdx.x; i < all; i += (int64_t)gridDim.x * kLayerThreads) {
        const int token = (int)(i / a.hidden), row = (int)(i - (int64_t)token * a.hidden);
        float y = 0.0f;
        constexpr int U = 8;
        for (int j = 0; j < a.picks; j += U) {
            float weight[U], v[U];
            bool there[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = token * a.picks + min(j + u, a.picks - 1);
                there[u] = j + u < a.picks && (unsigned)a.ids[q] < (unsigned)a.experts;
                weight[u] = a.weights[q];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t q = token * a.picks + j + u;
                v[u] = there[u] ? __int_as_float(load_l2(reinterpret_cast<const int*>(a.each + q * a.hidden + row))) : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (there[u]) y += weight[u] * v[u];
        }
        static_cast<T*>(a.out)[token * a.out_stride + row] = from_float<T>(y);
    }
}

}  // namespace om

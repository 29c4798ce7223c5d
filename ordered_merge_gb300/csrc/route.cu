// om_route_topk / om_route_topk_backward: routing of tokens to experts.
#include <cstdint>

#include <cuda_runtime.h>

#include "api_internal.cuh"
#include "select_common.cuh"

namespace om {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;        // one lane per pick
constexpr int kMaxExpertGroups = 32;  // one lane per group

struct RouteArgs {
    const void* logits;
    int64_t tokens;
    int64_t row_stride;
    const float* bias;
    int32_t* ids;
    float* weights;
    int experts, score, groups, group_picks, group_best, top_k, renorm;
    float scale;
};

constexpr int kRouteWarps = 8;

// The renormalised sigmoid weights are s_i / sum s with s = 1 / (1 + e^-x).
// Dividing every s by e^low, low = min(largest picked x, 0), leaves the
// quotient as it is and keeps the numerators from vanishing together when
// every picked logit is far below zero.  (x >= 0 implies low == 0.)
__device__ __forceinline__ float shifted_sigmoid(float x, float low) {
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - low) / (1.0f + expf(x));
}

__device__ __forceinline__ float sigmoid(float x) {
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x) / (1.0f + expf(x));
}

// One warp per token; lane l holds the experts l, l + 32, ...
template <typename T, int R>
__global__ void __launch_bounds__(kRouteWarps * 32) route_topk_kernel(RouteArgs a) {
    __shared__ float s_choice[kRouteWarps][R * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* logits = static_cast<const T*>(a.logits);
    const bool by_logit = a.bias == nullptr && (a.groups == 1 || a.group_best == 1);
    const bool need_sum = a.score == OM_SCORE_SOFTMAX && (!a.renorm || !by_logit);
    const float kNone = -INFINITY;

    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        const T* row = logits + t * a.row_stride;
        float x[R];
        float top = kNone;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = r * 32 + lane;
            x[r] = e < a.experts ? to_float(row[e]) : kNone;
            top = fmaxf(top, x[r]);  // a NaN is passed over
        }
        top = warp_max(top);
        float sum = 1.0f;
        if (need_sum) {
            float part = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (x[r] > kNone) part += expf(x[r] - top);
            sum = warp_sum(part);
        }
        // what the experts are chosen by: the logit itself where its order is the score's
        uint32_t key[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = r * 32 + lane;
            float c = x[r];
            if (!by_logit && x[r] > kNone) {
                c = a.score == OM_SCORE_SOFTMAX ? expf(x[r] - top) / sum : sigmoid(x[r]);
                if (a.bias != nullptr) c += a.bias[e];
            }
            const bool open = x[r] > kNone && c > kNone;  // false for NaN too
            key[r] = open ? score_image(c) : 0u;
            if (a.groups > 1) s_choice[warp][e] = open ? c : kNone;
        }
        if (a.groups > 1) {
            __syncwarp();
            const int size = a.experts / a.groups;
            uint32_t gkey = 0;
            if (lane < a.groups) {
                float b0 = kNone, b1 = kNone;
                for (int i = 0; i < size; ++i) {
                    const float c = s_choice[warp][lane * size + i];
                    b1 = fmaxf(b1, fminf(b0, c));
                    b0 = fmaxf(b0, c);
                }
                if (b0 > kNone) gkey = score_image(a.group_best == 2 && b1 > kNone ? b0 + b1 : b0);
            }
            uint32_t picked = 0;
            for (int i = 0; i < a.group_picks; ++i) {
                const uint32_t best = __reduce_max_sync(0xffffffffu, gkey);
                if (best == 0) break;
                const int g = __ffs(__ballot_sync(0xffffffffu, gkey == best)) - 1;
                picked |= 1u << g;
                if (lane == g) gkey = 0;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = r * 32 + lane;
                if (e < a.experts && !((picked >> (e / size)) & 1)) key[r] = 0;
            }
            __syncwarp();
        }
        // the picks, best first: lane j keeps the j-th
        int my_id = -1;
        float my_x = kNone;
        for (int j = 0; j < a.top_k; ++j) {
            uint32_t best = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) best = max(best, key[r]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0) break;
            int at = kMaxExperts;
            float xv = 0.0f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r)
                if (key[r] == best) at = r * 32 + lane, xv = x[r];
            const int first = __reduce_min_sync(0xffffffffu, (unsigned)at);
            xv = __shfl_sync(0xffffffffu, xv, first & 31);
            if (lane == j) my_id = first, my_x = xv;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r * 32 + lane == first) key[r] = 0;
        }
        float w = 0.0f;
        if (a.renorm) {
            const float best = warp_max(my_x);
            const float low = fminf(best, 0.0f);
            if (my_id >= 0) w = a.score == OM_SCORE_SOFTMAX ? expf(my_x - best) : shifted_sigmoid(my_x, low);
            const float total = warp_sum(w);
            if (my_id >= 0) w = w / total;
        } else if (my_id >= 0) {
            w = a.score == OM_SCORE_SOFTMAX ? expf(my_x - top) / sum : sigmoid(my_x);
        }
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = my_id;
            a.weights[t * a.top_k + lane] = w * a.scale;
        }
    }
}

struct RouteBackArgs {
    const void* logits;
    int64_t tokens;
    int64_t row_stride;
    const int32_t* ids;
    const float* grad_weights;
    void* grad_logits;
    int experts, score, top_k, renorm;
    float scale;
};

// One warp per token; lane l holds the experts l, l + 32, ... and, for
// l < top_k, the l-th pick.
template <typename T, int R>
__global__ void __launch_bounds__(kRouteWarps * 32) route_topk_backward_kernel(RouteBackArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* logits = static_cast<const T*>(a.logits);
    T* grad = static_cast<T*>(a.grad_logits);
    const bool dense = a.score == OM_SCORE_SOFTMAX && !a.renorm;  // every logit moves the weights
    const float kNone = -INFINITY;

    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kRouteWarps) {
        const T* row = logits + t * a.row_stride;
        int id = -1;
        float g = 0.0f, px = kNone;
        if (lane < a.top_k) {
            id = a.ids[t * a.top_k + lane];
            if (id < 0 || id >= a.experts) id = -1;
            if (id >= 0) {
                g = a.grad_weights[t * a.top_k + lane] * a.scale;
                px = to_float(row[id]);
                if (!(px > kNone)) id = -1;  // masked: no pick of the forward call
            }
        }
        float s[R];
        float top = 0.0f, sum = 1.0f;
        if (dense) {
            top = kNone;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int e = r * 32 + lane;
                s[r] = e < a.experts ? to_float(row[e]) : kNone;
                top = fmaxf(top, s[r]);
            }
            top = warp_max(top);
            float part = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[r] = s[r] > kNone ? expf(s[r] - top) : 0.0f;
                part += s[r];
            }
            sum = warp_sum(part);
        }
        // w: the pick's weight before scale; v: its logit's gradient, less what `dense` subtracts everywhere
        float w = 0.0f, v = 0.0f, dot = 0.0f;
        if (a.renorm) {
            const float best = warp_max(px);
            const float low = fminf(best, 0.0f);
            if (id >= 0) w = a.score == OM_SCORE_SOFTMAX ? expf(px - best) : shifted_sigmoid(px, low);
            const float total = warp_sum(w);
            if (id >= 0) w = w / total;
            dot = warp_sum(id >= 0 ? g * w : 0.0f);
            if (id >= 0) v = w * (g - dot);
            if (id >= 0 && a.score == OM_SCORE_SIGMOID) v *= sigmoid(-px);
        } else if (dense) {
            if (id >= 0) w = expf(px - top) / sum;
            dot = warp_sum(id >= 0 ? g * w : 0.0f);
            v = w * (g - dot);
        } else if (id >= 0) {
            v = g * sigmoid(px) * sigmoid(-px);
        }
        float out[R];
#pragma unroll
        for (int r = 0; r < R; ++r) out[r] = dense && s[r] != 0.0f ? -(s[r] / sum) * dot : 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int pid = __shfl_sync(0xffffffffu, id, j);
            const float pv = __shfl_sync(0xffffffffu, v, j);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (pid == r * 32 + lane) out[r] = pv;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e = r * 32 + lane;
            if (e < a.experts) grad[t * a.experts + e] = from_float<T>(out[r]);
        }
    }
}

// Calls f with the number of experts per lane as a constant.
template <typename F>
static cudaError_t with_lane_experts(int experts, F&& f) {
    if (experts <= 32) return f(std::integral_constant<int, 1>{});
    if (experts <= 64) return f(std::integral_constant<int, 2>{});
    if (experts <= 128) return f(std::integral_constant<int, 4>{});
    if (experts <= 256) return f(std::integral_constant<int, 8>{});
    if (experts <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

static unsigned route_grid(int64_t tokens) {
    const int64_t blocks = (tokens + kRouteWarps - 1) / kRouteWarps;
    return (unsigned)(blocks < (1 << 20) ? blocks : (1 << 20));
}

// Checks shared by both directions.
static om_status route_check(int value_type, const void* logits, int64_t tokens, int64_t experts, int64_t row_stride,
                             int score, int top_k) {
    const int vb = value_bytes(value_type);
    if (vb == 0 || (score != OM_SCORE_SOFTMAX && score != OM_SCORE_SIGMOID)) return OM_EINVAL;
    if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts) return OM_EINVAL;
    if (experts > kMaxExperts || top_k > kMaxTopK) return OM_ERANGE;
    if (tokens > 1 && row_stride < 0) return OM_EINVAL;
    if (tokens > ((int64_t)1 << 40) || row_stride > ((int64_t)1 << 40)) return OM_ERANGE;
    if (tokens > 0 && (logits == nullptr || misaligned(logits, vb))) return OM_EINVAL;
    return OM_OK;
}

}  // namespace om

using namespace om;

extern "C" {

om_status om_route_topk(int value_type, const void* logits, int64_t tokens, int64_t experts, int64_t row_stride,
                        const float* bias, int score, int groups, int group_picks, int group_best, int top_k,
                        int renorm, float scale, int32_t* ids, float* weights, void* stream) {
    const om_status s = route_check(value_type, logits, tokens, experts, row_stride, score, top_k);
    if (s != OM_OK) return s;
    if (groups < 1 || experts % groups != 0 || group_picks < 1 || group_picks > groups ||
        (group_best != 1 && group_best != 2) || top_k > group_picks * (experts / groups))
        return OM_EINVAL;
    if (groups > kMaxExpertGroups) return OM_ERANGE;
    if (tokens == 0) return OM_OK;
    if (ids == nullptr || weights == nullptr || misaligned4(bias) || misaligned4(ids) || misaligned4(weights))
        return OM_EINVAL;
    const int vb = value_bytes(value_type);
    const int64_t span = ((tokens - 1) * row_stride + experts) * vb, out = tokens * top_k * 4;
    if (overlaps(ids, out, weights, out, 1)) return OM_EINVAL;
    for (const void* o : {(const void*)ids, (const void*)weights})
        if (overlaps(o, out, logits, span, 1) || (bias && overlaps(o, out, bias, experts * 4, 1))) return OM_EINVAL;
    RouteArgs a{logits, tokens, row_stride, bias, ids, weights, (int)experts, score, groups, group_picks, group_best,
                top_k, renorm != 0, scale};
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        return with_lane_experts((int)experts, [&](auto r) {
            return traced(kKindRoute, st, [&] {
                route_topk_kernel<decltype(v), decltype(r)::value><<<route_grid(tokens), kRouteWarps * 32, 0, st>>>(a);
            });
        });
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

om_status om_route_topk_backward(int value_type, const void* logits, int64_t tokens, int64_t experts,
                                 int64_t row_stride, const int32_t* ids, const float* grad_weights, int score,
                                 int top_k, int renorm, float scale, void* grad_logits, void* stream) {
    const om_status s = route_check(value_type, logits, tokens, experts, row_stride, score, top_k);
    if (s != OM_OK) return s;
    if (tokens == 0) return OM_OK;
    const int vb = value_bytes(value_type);
    if (ids == nullptr || grad_weights == nullptr || grad_logits == nullptr || misaligned4(ids) ||
        misaligned4(grad_weights) || misaligned(grad_logits, vb))
        return OM_EINVAL;
    const int64_t span = ((tokens - 1) * row_stride + experts) * vb, out = tokens * experts * vb;
    if (overlaps(grad_logits, out, logits, span, 1) || overlaps(grad_logits, out, ids, tokens * top_k * 4, 1) ||
        overlaps(grad_logits, out, grad_weights, tokens * top_k * 4, 1))
        return OM_EINVAL;
    RouteBackArgs a{logits, tokens, row_stride, ids, grad_weights, grad_logits, (int)experts, score, top_k,
                    renorm != 0, scale};
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = with_value_type(value_type, [&](auto v) {
        return with_lane_experts((int)experts, [&](auto r) {
            return traced(kKindRoute, st, [&] {
                route_topk_backward_kernel<decltype(v), decltype(r)::value>
                    <<<route_grid(tokens), kRouteWarps * 32, 0, st>>>(a);
            });
        });
    });
    return e == cudaSuccess ? OM_OK : cuda_fail(e);
}

}  // extern "C"

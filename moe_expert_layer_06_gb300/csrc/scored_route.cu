// Scored routing: sigmoid or softmax scores, a selection bias, expert groups,
// top-k, renormalised and scaled weights; and the gradient of the weights.
//
//   s_e = sigmoid(l_e) | softmax(l)_e,  c_e = s_e + b_e,
//   idx = top-k of c over the best groups,  w_j = scale * s_j [/ sum_i s_i].
//
// One warp per token.
#include <math.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 4;  // tokens per CTA

struct RouteArgs {
    const float* partials;  // [ksplit][T][E] logits (added in order)
    int ksplit;
    const float* bias;      // [E] or null
    int T, E, k;
    int sigmoid, n_groups, topk_groups, top2, renormalize;
    float scale;
    float* logits_out;      // or null
    int32_t* topk_idx;
    float* topk_w;
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Largest (value, lowest index) over the warp; index 0x7fffffff: none.
__device__ __forceinline__ void warp_best(double& v, int& i) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const double ov = __shfl_xor_sync(0xffffffffu, v, d);
        const int oi = __shfl_xor_sync(0xffffffffu, i, d);
        if (oi != 0x7fffffff && (i == 0x7fffffff || ov > v || (ov == v && oi < i))) {
            v = ov;
            i = oi;
        }
    }
}

// A NaN logit masks its expert as -inf does.
__device__ __forceinline__ float masked_logit(float l) { return l == l ? l : -INFINITY; }

__device__ __forceinline__ float sigmoid_f(float l) { return 1.0f / (1.0f + expf(-l)); }

// Renormalised share of the selected experts: lane j < k holds logit l_j.
// s_j / sum s_i relative to the largest: exp(l) for a softmax; for a sigmoid
// exp(min(l, 0)) / (1 + exp(-|l|)), whose small factor exp(min(l, 0)) is taken
// relative to the row's largest.  A row of masked logits gets 0.
__device__ __forceinline__ float share_of(float l, bool in, int sigmoid) {
    const float low = in ? (sigmoid ? fminf(l, 0.0f) : l) : -INFINITY;
    const float m = warp_max(low);
    float e = low == m ? 1.0f : expf(low - m);
    if (sigmoid) e /= 1.0f + expf(-fabsf(l));
    if (!in || l == -INFINITY) e = 0.0f;
    const float sum = warp_sum(e);
    return sum > 0.0f ? e / sum : 0.0f;
}

// exp(l - mx) with the limit at infinite logits (l = mx = inf gives 1)
__device__ __forceinline__ float exp_rel(float l, float mx) { return l == mx ? 1.0f : expf(l - mx); }

__global__ void __launch_bounds__(kWarps * 32) scored_topk_kernel(const RouteArgs a) {
    pdl_begin();
    extern __shared__ double c_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double* c = c_all + (size_t)warp * a.E;
    const size_t slice = (size_t)a.T * a.E;
    for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
        const float* row = a.partials + (size_t)t * a.E;
        float* lo = a.logits_out ? a.logits_out + (size_t)t * a.E : nullptr;
        auto logit = [&](int e) {
            float l = row[e];
            for (int s = 1; s < a.ksplit; ++s) l += row[(size_t)s * slice + e];
            return l;
        };
        float mx = -INFINITY;
        for (int e = lane; e < a.E; e += 32) {
            const float l = logit(e);
            if (lo) lo[e] = l;
            c[e] = masked_logit(l);
            mx = fmaxf(mx, masked_logit(l));
        }
        mx = warp_max(mx);
        double den = 0.0;
        if (!a.sigmoid) {
            for (int e = lane; e < a.E; e += 32)
                if (c[e] != -INFINITY) den += c[e] == mx ? 1.0 : exp(c[e] - (double)mx);
            den = warp_sum(den);
        }
        for (int e = lane; e < a.E; e += 32) {
            const double l = c[e];
            if (l == -INFINITY) continue;
            double s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : (l == mx ? 1.0 : exp(l - (double)mx)) / den;
            if (a.bias) s += a.bias[e];
            c[e] = s;
        }
        __syncwarp();
        uint32_t kept = 0xffffffffu;
        const int gs = a.E / a.n_groups;
        if (a.topk_groups < a.n_groups) {
            double b0 = -INFINITY, b1 = -INFINITY;
            if (lane < a.n_groups) {
                for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
                    const double v = c[e];
                    if (v > b0) {
                        b1 = b0;
                        b0 = v;
                    } else if (v > b1) {
                        b1 = v;
                    }
                }
                if (a.top2 && b1 != -INFINITY) b0 += b1;
            }
            kept = 0;
            for (int r = 0; r < a.topk_groups; ++r) {
                double v = b0;
                int i = lane < a.n_groups && !((kept >> lane) & 1u) ? lane : 0x7fffffff;
                warp_best(v, i);
                kept |= 1u << i;
            }
        }
        // lane j keeps the j-th selected expert; taken experts are marked NaN
        int mine = -1;
        for (int j = 0; j < a.k; ++j) {
            double v = 0.0;
            int i = 0x7fffffff;
            for (int e = lane; e < a.E; e += 32) {
                const double u = c[e];
                if (u != u || !((kept >> (e / gs)) & 1u)) continue;
                if (i == 0x7fffffff || u > v) {
                    v = u;
                    i = e;
                }
            }
            warp_best(v, i);
            if ((i & 31) == lane) c[i] = NAN;
            if (lane == j) mine = i;
        }
        const bool in = lane < a.k;
        const float l = in ? masked_logit(logit(mine)) : -INFINITY;
        float w;
        if (a.renormalize) w = share_of(l, in, a.sigmoid);
        else if (l == -INFINITY) w = 0.0f;
        else w = a.sigmoid ? sigmoid_f(l) : (float)(exp_rel(l, mx) / den);
        if (in) {
            a.topk_idx[(size_t)t * a.k + lane] = mine;
            a.topk_w[(size_t)t * a.k + lane] = a.scale * w;
        }
        __syncwarp();
    }
}

// One warp per token: lane j < k holds the j-th selected expert.
__global__ void __launch_bounds__(kWarps * 32) scored_backward_kernel(const float* __restrict__ logits,
                                                                      const int32_t* __restrict__ topk_idx,
                                                                      const float* __restrict__ dw, int T, int E,
                                                                      int k, int sigmoid, int renormalize, float scale,
                                                                      float* __restrict__ dl, DevStatus st) {
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int t = blockIdx.x * kWarps + warp; t < T; t += gridDim.x * kWarps) {
        const float* row = logits + (size_t)t * E;
        float* out = dl + (size_t)t * E;
        int e = lane < k ? topk_idx[(size_t)t * k + lane] : -1;
        const bool in = e >= 0 && e < E;
        if (lane < k && !in) raise_status(st, kStatusInvalidExpert);
        const float g = in ? dw[(size_t)t * k + lane] : 0.0f;
        const float l = in ? masked_logit(row[e]) : -INFINITY;
        const bool live = l != -INFINITY;
        const float rest = sigmoid && live ? 1.0f / (1.0f + expf(l)) : 1.0f;  // 1 - sigmoid(l)
        float d;  // gradient through the selected scores
        if (renormalize) {
            const float w = share_of(l, in, sigmoid);
            d = scale * w * (g - warp_sum(w * g)) * rest;
        } else if (sigmoid) {
            d = live ? scale * g * sigmoid_f(l) * rest : 0.0f;
        } else {
            float mx = -INFINITY;
            for (int i = lane; i < E; i += 32) mx = fmaxf(mx, masked_logit(row[i]));
            mx = warp_max(mx);
            float den = 0.0f;
            for (int i = lane; i < E; i += 32) {
                const float v = masked_logit(row[i]);
                if (v != -INFINITY) den += exp_rel(v, mx);
            }
            den = warp_sum(den);
            const float p = live ? exp_rel(l, mx) / den : 0.0f;
            const float dot = warp_sum(scale * g * p);
            for (int i = lane; i < E; i += 32) {
                const float v = masked_logit(row[i]);
                out[i] = v == -INFINITY ? 0.0f : -(exp_rel(v, mx) / den) * dot;
            }
            __syncwarp();
            if (live) out[e] = p * (scale * g - dot);
            __syncwarp();
            continue;
        }
        for (int i = lane; i < E; i += 32) out[i] = 0.0f;
        __syncwarp();
        if (in) out[e] = d;
        __syncwarp();
    }
}

int check_router(const moe_shape_t* s, const moe_router_t* r, int T) {
    if (int rc = api_check_shape(s, T)) return rc;
    if (!r) return api_fail(MOE_ERR_INVALID_ARG, "router is NULL");
    if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
        return api_fail(MOE_ERR_INVALID_ARG, "bad score %d", r->score);
    if (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2)
        return api_fail(MOE_ERR_INVALID_ARG, "bad group_score %d", r->group_score);
    if (r->renormalize != 0 && r->renormalize != 1)
        return api_fail(MOE_ERR_INVALID_ARG, "renormalize %d is not 0 or 1", r->renormalize);
    if (!isfinite(r->scale)) return api_fail(MOE_ERR_INVALID_ARG, "scale is not finite");
    if (r->n_groups < 1 || r->n_groups > 32 || s->n_experts % r->n_groups)
        return api_fail(MOE_ERR_INVALID_ARG, "n_groups %d must divide n_experts and be in [1, 32]", r->n_groups);
    if (r->topk_groups < 1 || r->topk_groups > r->n_groups)
        return api_fail(MOE_ERR_INVALID_ARG, "topk_groups %d not in [1, n_groups]", r->topk_groups);
    if ((int64_t)r->topk_groups * (s->n_experts / r->n_groups) < s->top_k)
        return api_fail(MOE_ERR_INVALID_ARG, "top_k %d exceeds the experts of %d groups", s->top_k, r->topk_groups);
    return MOE_OK;
}

int grid_for(int T) {
    const long want = ((long)T + kWarps - 1) / kWarps;
    const long cap = (long)num_sms() * 16;
    return (int)(want < cap ? want : cap);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_route_scored(const moe_shape_t* shape, const moe_router_t* router, int T, const void* x,
                     const void* w_router, const float* select_bias, const float* logits_in, float* logits_out,
                     int32_t* topk_idx, float* topk_w, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_router(shape, router, T);
    if (rc) return rc;
    if (T == 0) return MOE_OK;
    PdlScope pdl((long)T * shape->top_k);
    if ((rc = api_need(topk_idx, "topk_idx", 4)) || (rc = api_need(topk_w, "topk_w", 4))) return rc;
    if (logits_out && (rc = api_need(logits_out, "logits_out", 4))) return rc;
    if (select_bias && (rc = api_need(select_bias, "select_bias", 4))) return rc;
    RouteArgs a;
    a.partials = logits_in;
    a.ksplit = 1;
    if (logits_in) {
        if ((rc = api_need(logits_in, "logits_in", 4))) return rc;
    } else {
        if ((rc = api_need(x, "x")) || (rc = api_need(w_router, "w_router"))) return rc;
        if ((rc = api_router_gemm(shape, T, x, w_router, ws, ws_bytes, &a.ksplit,
                                  reinterpret_cast<cudaStream_t>(stream))))
            return rc;
        a.partials = static_cast<const float*>(ws);
    }
    a.bias = select_bias;
    a.T = T;
    a.E = shape->n_experts;
    a.k = shape->top_k;
    a.sigmoid = router->score == MOE_SCORE_SIGMOID;
    a.n_groups = router->n_groups;
    a.topk_groups = router->topk_groups;
    a.top2 = router->group_score == MOE_GROUP_TOP2;
    a.renormalize = router->renormalize;
    a.scale = router->scale;
    a.logits_out = logits_out;
    a.topk_idx = topk_idx;
    a.topk_w = topk_w;
    const cudaError_t e = launch_pdl(scored_topk_kernel, dim3(grid_for(T)), dim3(kWarps * 32),
                                     (size_t)kWarps * a.E * sizeof(double), reinterpret_cast<cudaStream_t>(stream), a);
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "scored top-k launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

int moe_route_scored_backward(const moe_shape_t* shape, const moe_router_t* router, int T, const float* logits,
                              const int32_t* topk_idx, const float* d_topk_w, float* d_logits, void* stream) {
    int rc = check_router(shape, router, T);
    if (rc) return rc;
    if (T == 0) return MOE_OK;
    PdlScope pdl((long)T * shape->top_k);
    if ((rc = api_need(logits, "logits", 4)) || (rc = api_need(topk_idx, "topk_idx", 4)) ||
        (rc = api_need(d_topk_w, "d_topk_w", 4)) || (rc = api_need(d_logits, "d_logits", 4)))
        return rc;
    DevStatus st;
    if ((rc = api_device_status(&st))) return rc;
    const cudaError_t e =
        launch_pdl(scored_backward_kernel, dim3(grid_for(T)), dim3(kWarps * 32), 0,
                   reinterpret_cast<cudaStream_t>(stream), logits, topk_idx, d_topk_w, T, shape->n_experts,
                   shape->top_k, (int)(router->score == MOE_SCORE_SIGMOID), (int)router->renormalize, router->scale,
                   d_logits, st);
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "scored backward launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

}  // extern "C"

// Scored routing: sigmoid or softmax scores, a selection bias, expert groups,
// top-k, renormalised and scaled weights; and the gradient of the weights.
//
//   s_e = sigmoid(l_e) | softmax(l)_e,  c_e = s_e + b_e,
//   idx = top-k of c over the best groups,  w_j = scale * s_j [/ sum_i s_i].
//
// One warp per token.  Lane maxima give a threshold that few logits pass; those
// candidates are ranked against one another, so the cost hardly grows with k.
// The selection is made on fp32 values whose error is bounded; a row where two
// values that decide the selection or its order lie within that bound of one
// another is decided again in fp64 (about one row in a thousand).
#include <float.h>
#include <math.h>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kWarps = 4;  // tokens per CTA
constexpr int kCand = 64;  // candidates of one row (two per lane)

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
__device__ __forceinline__ float share_term(float l, float top, int sigmoid) {
    const float low = sigmoid ? fminf(l, 0.0f) : l;
    const float e = low == top ? 1.0f : expf(low - top);
    return sigmoid ? e / (1.0f + expf(-fabsf(l))) : e;
}

__device__ __forceinline__ float share_of(float l, bool in, int sigmoid) {
    const float m = warp_max(in ? (sigmoid ? fminf(l, 0.0f) : l) : -INFINITY);
    const float e = in && l != -INFINITY ? share_term(l, m, sigmoid) : 0.0f;
    const float sum = warp_sum(e);
    return sum > 0.0f ? e / sum : 0.0f;
}

// exp(l - mx) with the limit at infinite logits (l = mx = inf gives 1)
__device__ __forceinline__ float exp_rel(float l, float mx) { return l == mx ? 1.0f : expf(l - mx); }

// The j-th selected expert's weight on lane j < k (mine: its id), written out.  mx, den:
// the softmax statistics of the row (weights that are not renormalised).
__device__ __forceinline__ void write_selection(const RouteArgs& a, int t, int lane, int mine, float l, float mx,
                                                float den) {
    const bool in = lane < a.k;
    float w;
    if (a.renormalize) w = share_of(l, in, a.sigmoid);
    else if (l == -INFINITY) w = 0.0f;
    else w = a.sigmoid ? sigmoid_f(l) : exp_rel(l, mx) / den;
    if (in) {
        a.topk_idx[(size_t)t * a.k + lane] = mine;
        a.topk_w[(size_t)t * a.k + lane] = a.scale * w;
    }
}

__device__ __forceinline__ float logit_at(const RouteArgs& a, int t, int e) {
    const float* p = a.partials + (size_t)t * a.E + e;
    float l = *p;
    for (int s = 1; s < a.ksplit; ++s) l += p[(size_t)s * a.T * a.E];
    return l;
}

// One row in fp64 from its logits, k arg-max rounds: rows that fp32 cannot decide, and
// shapes outside the fast kernel's layout.  c: E doubles of this warp's shared memory.
__device__ __noinline__ void select_fp64(const RouteArgs& a, int t, double* c) {
    const int lane = threadIdx.x & 31;
    float mx = -INFINITY;
    for (int e = lane; e < a.E; e += 32) {
        const float l = masked_logit(logit_at(a, t, e));
        c[e] = l;
        mx = fmaxf(mx, l);
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
    const float l = lane < a.k ? masked_logit(logit_at(a, t, mine)) : -INFINITY;
    write_selection(a, t, lane, mine, l, mx, (float)den);
    __syncwarp();
}

__global__ void __launch_bounds__(kWarps * 32) scored_topk_fp64_kernel(const __grid_constant__ RouteArgs a) {
    pdl_begin();
    extern __shared__ double c_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
        if (a.logits_out)
            for (int e = lane; e < a.E; e += 32) a.logits_out[(size_t)t * a.E + e] = logit_at(a, t, e);
        select_fp64(a, t, c_all + (size_t)warp * a.E);
    }
}

// Monotone map of a float (no NaN) to an unsigned word that is never 0.
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 1 / (1 + exp(-l)) from the hardware's approximate 2^x and reciprocal.
__device__ __forceinline__ float fast_sigmoid(float l) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.442695041f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// Reductions over the LPT consecutive lanes of one token (every lane gets the result).
template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
    if constexpr (LPT == 32) {
        return __reduce_max_sync(0xffffffffu, v);
    } else {
#pragma unroll
        for (int d = LPT / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

template <int LPT>
__device__ __forceinline__ float token_max(float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

template <int LPT>
__device__ __forceinline__ bool token_any(bool p) {
    const uint32_t b = __ballot_sync(0xffffffffu, p);
    if (LPT == 32) return b != 0;
    return ((b >> (threadIdx.x & 31 & ~(LPT - 1))) & ((1u << (LPT & 31)) - 1u)) != 0;
}

// fp64 scratch of a warp: a row, or a value per candidate.
__host__ __device__ __forceinline__ int scratch_doubles(int E) { return E > kCand ? E : kCand; }

// What the fp32 selection value of an expert is.
enum KeyKind : int {
    kKeyLogit,    // the logit itself: orders as the score does, and exactly (no bias, no sum of two)
    kKeySigmoid,  // sigmoid + bias
    kKeySoftmax,  // softmax + bias
};

// LPT lanes per token (32 / LPT tokens per warp).  A token's lanes are laid out by
// groups: lpg (a power of two) lanes per group, PER consecutive experts per lane; what
// passes the group's end is empty (key 0).
template <int LPT, int PER, int KIND>
__global__ void __launch_bounds__(kWarps * 32) scored_topk_kernel(const __grid_constant__ RouteArgs a, int lpg, int vec) {
    pdl_begin();
    constexpr int TPW = 32 / LPT;                // tokens per warp
    // experts per block maximum: at least 32 blocks of a full row, at most 8 experts each
    constexpr int BLK = PER * LPT >= 256 ? 8 : PER * LPT >= 64 ? PER * LPT / 32 : 1;
    constexpr int NB = PER / BLK;
    extern __shared__ double c_all[];
    __shared__ __align__(16) uint32_t cand_all[kWarps * TPW][kCand];
    __shared__ uint16_t cand_e_all[kWarps * TPW][kCand];
    __shared__ uint16_t sorted_all[kWarps * TPW][kCand];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & (LPT - 1), slot = lane / LPT;
    uint32_t* cand = cand_all[warp * TPW + slot];      // keys of the candidates, in expert order
    uint16_t* cand_e = cand_e_all[warp * TPW + slot];  // their experts
    uint16_t* sorted = sorted_all[warp * TPW + slot];  // candidate of each rank
    const int gs = a.E / a.n_groups;
    const int group = sub / lpg;
    const int in_group = (sub & (lpg - 1)) * PER;  // first of this lane's experts within its group
    const int n_mine = group < a.n_groups ? min(PER, max(0, gs - in_group)) : 0;
    const int e0 = group * gs + in_group;
    const bool grouped = a.topk_groups < a.n_groups;
    const bool stats = KIND == kKeySoftmax || (!a.sigmoid && !a.renormalize);
    // bias, a lane's experts together and lanes apart by PER + 4 words (16-byte reads without bank conflicts)
    double* scratch = c_all + (size_t)warp * scratch_doubles(a.E);
    float* bias = reinterpret_cast<float*>(c_all + (size_t)kWarps * scratch_doubles(a.E));
    if (KIND != kKeyLogit) {
        if (warp == 0 && lane < LPT)
            for (int i = 0; i < PER; ++i) bias[sub * (PER + 4) + i] = a.bias && i < n_mine ? a.bias[e0 + i] : 0.0f;
        __syncthreads();
    }

    float l[PER];
    auto load = [&](int t) {
        const float* p = a.partials + (size_t)t * a.E + e0;
        const int n = t < a.T ? n_mine : 0;
        if (PER >= 4 && vec) {
            // rows and groups are whole float4s, so a lane's experts are too
#pragma unroll
            for (int i = 0; i < PER; i += 4)
                if (i < n) {
                    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
                    l[i] = v.x;
                    l[(i + 1) % PER] = v.y;
                    l[(i + 2) % PER] = v.z;
                    l[(i + 3) % PER] = v.w;
                }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < n) l[i] = p[i];
            for (int s = 1; s < a.ksplit; ++s) {
                p += (size_t)a.T * a.E;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (i < n) l[i] += p[i];
            }
        }
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = 0.0f;
    const int stride = gridDim.x * kWarps * TPW;
    int tw = (blockIdx.x * kWarps + warp) * TPW;  // the warp's first token
    load(tw + slot);
    for (; tw < a.T; tw += stride) {
        const int t = tw + slot;
        const bool alive = t < a.T;
        if (a.logits_out && alive) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < n_mine) a.logits_out[(size_t)t * a.E + e0 + i] = l[i];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) l[i] = masked_logit(l[i]);
        float mx = -INFINITY, den = 1.0f;
        if (KIND == kKeyLogit && !a.sigmoid) {
            // beside an infinite logit every finite one has softmax 0: they tie
            bool inf = false;
#pragma unroll
            for (int i = 0; i < PER; ++i) inf |= i < n_mine && l[i] == INFINITY;
            if (token_any<LPT>(inf)) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (isfinite(l[i])) l[i] = -FLT_MAX;
            }
        }
        uint32_t key[PER];
        if (stats) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < n_mine) mx = fmaxf(mx, l[i]);
            mx = token_max<LPT>(mx);
            float part[PER];  // summed in pairs: log2(E) roundings
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                part[i] = i < n_mine && l[i] != -INFINITY ? exp_rel(l[i], mx) : 0.0f;
                if (KIND == kKeySoftmax) key[i] = __float_as_uint(part[i]);
            }
#pragma unroll
            for (int w = PER / 2; w > 0; w >>= 1)
#pragma unroll
                for (int i = 0; i < w; ++i) part[i] += part[i + w];
            den = token_sum<LPT>(part[0]);
        }
        const float inv_den = 1.0f / den;
#pragma unroll
        for (int i = 0; i < PER; i += (PER >= 4 ? 4 : 1)) {
            float b4[4];
            if (KIND != kKeyLogit) {
                if (PER >= 4) {
                    const float4 v = *reinterpret_cast<const float4*>(bias + sub * (PER + 4) + i);
                    b4[0] = v.x;
                    b4[1] = v.y;
                    b4[2] = v.z;
                    b4[3] = v.w;
                } else {
                    b4[0] = bias[sub * (PER + 4) + i];
                }
            }
#pragma unroll
            for (int u = 0; u < (PER >= 4 ? 4 : 1); ++u) {
                float c = l[i + u];
                if (KIND == kKeySigmoid) c = fast_sigmoid(c) + b4[u];
                if (KIND == kKeySoftmax) c = fmaf(__uint_as_float(key[i + u]), inv_den, b4[u]);
                if (KIND != kKeyLogit && l[i + u] == -INFINITY) c = -INFINITY;
                key[i + u] = i + u < n_mine ? key_of(c) : 0u;
            }
        }
        // the next row's loads run while this one is selected
        load(tw + stride + slot);

        // Bound of |fp32 value - exact value| before the bias is added.  Sigmoid: the
        // exponential is off by 2 + 1.18 |l| steps, which 1 / (1 + e) takes s (1 - s) of
        // (at most 0.63 steps of 2^-23), the sum and the reciprocal by 1.5 more: 3 in
        // all.  Softmax: 2 steps of the exponential, |l - mx| / 2 of its argument, those
        // of den (`rel` below), of 1 / den and the product, all relative to a value of
        // at most 1 / den: below 16.  The sum with the bias adds half a step.
        const float err = KIND == kKeyLogit ? 0.0f : 0x1p-23f * (KIND == kKeySigmoid ? 3.0f : 16.0f * inv_den);
        // exact scores: the softmax's sum in fp64, then one logit at a time
        double den64 = 0.0;
        auto sum64 = [&](bool need) {
            if (KIND != kKeySoftmax) return;
            double d = 0.0;
            if (need)
                for (int i = 0; i < n_mine; ++i) {
                    const float x = masked_logit(logit_at(a, t, e0 + i));
                    if (x != -INFINITY) d += x == mx ? 1.0 : exp((double)x - (double)mx);
                }
#pragma unroll
            for (int w = LPT / 2; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
            if (need) den64 = d;
        };
        auto score64 = [&](float x) -> double {
            if (KIND == kKeySoftmax) return (x == mx ? 1.0 : exp((double)x - (double)mx)) / den64;
            return 1.0 / (1.0 + exp(-(double)x));
        };
        bool unsure = false;
        if (grouped) {
            uint32_t k0 = 0, k1 = 0;  // the two largest of the group
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                k1 = max(k1, min(k0, key[i]));
                k0 = max(k0, key[i]);
            }
            for (int d = 1; d < lpg; d <<= 1) {
                const uint32_t o0 = __shfl_xor_sync(0xffffffffu, k0, d), o1 = __shfl_xor_sync(0xffffffffu, k1, d);
                k1 = max(max(k1, o1), min(k0, o0));
                k0 = max(k0, o0);
            }
            float g = k0 ? value_of(k0) : 0.0f;
            const bool two = a.top2 && k1 && value_of(k1) != -INFINITY;
            if (KIND != kKeyLogit && two) g += value_of(k1);
            const uint32_t gk = group < a.n_groups ? key_of(g) : 0u;
            int rank = 0;
            for (int o = 0; o < a.n_groups; ++o) {
                const uint32_t ok = __shfl_sync(0xffffffffu, gk, o * lpg, LPT);
                rank += ok > gk || (ok == gk && o < group) ? 1 : 0;
            }
            bool keep = group < a.n_groups && rank < a.topk_groups;
            if (KIND != kKeyLogit) {
                const float in = value_of(~token_max<LPT>(keep ? ~gk : 0u)), out = value_of(token_max<LPT>(keep ? 0u : gk));
                // (two groups without an unmasked expert tie exactly)
                const bool close = out != -INFINITY && in - out <= 4.0f * err + 0x1p-21f * fabsf(in);
                if (__any_sync(0xffffffffu, close)) {
                    // the group scores in fp64, from the experts that fp32 leaves for the two best
                    const float low = value_of(a.top2 && k1 ? k1 : k0);
                    const float margin = 2.0f * err + 0x1p-22f * fabsf(low);
                    double d0 = -INFINITY, d1 = -INFINITY;
                    sum64(close);
                    if (close && k0) {
                        for (int i = 0; i < n_mine; ++i) {
                            const float x = masked_logit(logit_at(a, t, e0 + i));
                            uint32_t ki = 0;
#pragma unroll
                            for (int u = 0; u < PER; ++u) ki = u == i ? key[u] : ki;
                            if (x == -INFINITY || value_of(ki) < low - margin) continue;
                            const double c = score64(x) + (double)bias[sub * (PER + 4) + i];
                            d1 = fmax(d1, fmin(d0, c));
                            d0 = fmax(d0, c);
                        }
                    }
                    for (int d = 1; d < lpg; d <<= 1) {
                        const double o0 = __shfl_xor_sync(0xffffffffu, d0, d), o1 = __shfl_xor_sync(0xffffffffu, d1, d);
                        d1 = fmax(fmax(d1, o1), fmin(d0, o0));
                        d0 = fmax(d0, o0);
                    }
                    if (a.top2 && d1 != -INFINITY) d0 += d1;
                    int exact = 0;
                    for (int o = 0; o < a.n_groups; ++o) {
                        const double od = __shfl_sync(0xffffffffu, d0, o * lpg, LPT);
                        exact += od > d0 || (od == d0 && o < group) ? 1 : 0;
                    }
                    if (close) keep = group < a.n_groups && exact < a.topk_groups;
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (!keep) key[i] = 0u;
        }
        // threshold: the (k+1)-th largest block maximum (the largest k+1 keys pass it)
        uint32_t m[NB];
#pragma unroll
        for (int q = 0; q < NB; ++q) {
            m[q] = 0;
#pragma unroll
            for (int i = 0; i < BLK; ++i) m[q] = max(m[q], key[q * BLK + i]);
        }
        uint32_t tau = 0, top = 0;
        for (int j = 0; j <= a.k; ++j) {
            uint32_t mine = m[0];
#pragma unroll
            for (int q = 1; q < NB; ++q) mine = max(mine, m[q]);
            tau = token_max<LPT>(mine);
            if (j == 0) top = tau;
#pragma unroll
            for (int q = 0; q < NB; ++q)
                if (m[q] == tau) m[q] = 0;
        }
        const float mag = fmaxf(fabsf(value_of(top)), tau ? fabsf(value_of(tau)) : 0.0f);
        const float eps = 2.0f * err + (KIND == kKeyLogit || mag == INFINITY ? 0.0f : 0x1p-22f * mag);
        if (KIND != kKeyLogit && tau && value_of(tau) != -INFINITY) tau = key_of(value_of(tau) - 2.0f * eps);
        if (tau == 0) tau = 1;
        // candidates in expert order
        int cnt = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) cnt += key[i] >= tau ? 1 : 0;
        int incl = cnt;
#pragma unroll
        for (int d = 1; d < LPT; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d, LPT);
            if (sub >= d) incl += o;
        }
        int n = __shfl_sync(0xffffffffu, incl, LPT - 1, LPT);
        if (n > kCand) {
            unsure = true;
            n = 0;
        }
        if (n > 0) {
            int at = incl - cnt;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (key[i] >= tau) {
                    cand[at] = key[i];
                    cand_e[at] = (uint16_t)(e0 + i);
                    ++at;
                }
            // whole vectors of four
            for (int q = n + sub; q < ((n + 3) & ~3); q += LPT) cand[q] = 0u;
        }
        __syncwarp();
        for (int q = sub; q < n; q += LPT) {
            // ties in expert order: an equal key at a lower position counts as larger
            const uint32_t mine = cand[q];
            int rank = 0;
            for (int o = 0; o < n; o += 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(cand + o);
                rank += v.x > mine || (v.x == mine && o < q) ? 1 : 0;
                rank += v.y > mine || (v.y == mine && o + 1 < q) ? 1 : 0;
                rank += v.z > mine || (v.z == mine && o + 2 < q) ? 1 : 0;
                rank += v.w > mine || (v.w == mine && o + 3 < q) ? 1 : 0;
            }
            sorted[rank] = (uint16_t)q;
        }
        __syncwarp();
        if (KIND != kKeyLogit) {
            // neighbours of the first k + 1 in order, too close for fp32?
            bool close = false;
            for (int j = sub; j < min(a.k, n - 1); j += LPT) {
                const float next = value_of(cand[sorted[j + 1]]);
                close |= next != -INFINITY && value_of(cand[sorted[j]]) - next <= eps;
            }
            const bool again = token_any<LPT>(close);
            if (__any_sync(0xffffffffu, again)) {
                // the candidates again in fp64 (every exact value above the k-th is among them), in
                // the warp's fp64 scratch: values and scores
                sum64(again);
                for (int w = 0; w < TPW; ++w) {
                    // one token of the warp after the other
                    const bool turn = again && slot == w;
                    if (turn)
                        for (int q = sub; q < n; q += LPT) {
                            const int e = cand_e[q];
                            const float x = masked_logit(logit_at(a, t, e));
                            scratch[q] = x == -INFINITY ? -INFINITY : score64(x) + (a.bias ? (double)a.bias[e] : 0.0);
                        }
                    __syncwarp();
                    if (turn)
                        for (int q = sub; q < n; q += LPT) {
                            int rank = 0;
                            for (int o = 0; o < n; ++o)
                                rank += scratch[o] > scratch[q] || (scratch[o] == scratch[q] && o < q) ? 1 : 0;
                            sorted[rank] = (uint16_t)q;
                        }
                    __syncwarp();
                }
            }
        }
        unsure = token_any<LPT>(unsure);
        // weights: lane sub holds the selected experts sub, sub + LPT, ... of its token
        constexpr int KPL = 32 / LPT;
        float lw[KPL], sh[KPL];
        int me[KPL];
        float low = -INFINITY;
#pragma unroll
        for (int q = 0; q < KPL; ++q) {
            const int j = sub + q * LPT;
            const bool in = j < a.k && alive && !unsure;
            me[q] = in ? cand_e[sorted[j]] : 0;
            lw[q] = in ? masked_logit(logit_at(a, t, me[q])) : -INFINITY;
            if (j < a.k) low = fmaxf(low, a.sigmoid ? fminf(lw[q], 0.0f) : lw[q]);
        }
        if (a.renormalize) {
            low = token_max<LPT>(low);
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < KPL; ++q) {
                sh[q] = 0.0f;
                if (lw[q] != -INFINITY) sh[q] = share_term(lw[q], low, a.sigmoid);
                sum += sh[q];
            }
            sum = token_sum<LPT>(sum);
            const float f = sum > 0.0f ? a.scale / sum : 0.0f;
#pragma unroll
            for (int q = 0; q < KPL; ++q) sh[q] *= f;
        } else {
#pragma unroll
            for (int q = 0; q < KPL; ++q) {
                sh[q] = 0.0f;
                if (lw[q] != -INFINITY) sh[q] = a.scale * (a.sigmoid ? sigmoid_f(lw[q]) : exp_rel(lw[q], mx) * inv_den);
            }
        }
        if (alive && !unsure) {
#pragma unroll
            for (int q = 0; q < KPL; ++q) {
                const int j = sub + q * LPT;
                if (j < a.k) {
                    a.topk_idx[(size_t)t * a.k + j] = me[q];
                    a.topk_w[(size_t)t * a.k + j] = sh[q];
                }
            }
        }
        uint32_t redo = __ballot_sync(0xffffffffu, alive && unsure && sub == 0);
        for (; redo; redo &= redo - 1)
            select_fp64(a, tw + (__ffs(redo) - 1) / LPT, scratch);
        __syncwarp();
    }
}

// The gradient of one row.  Lane j < k holds the j-th selected expert; V: float or float4,
// NV of them per lane (V vec = lane + 32 i of the row).  Sparse gradients (sigmoid, or
// renormalised) are zeros and k values; a softmax as it is reads the row once.
template <typename V, int NV>
__global__ void __launch_bounds__(kWarps * 32) scored_backward_kernel(const float* __restrict__ logits,
                                                                      const int32_t* __restrict__ topk_idx,
                                                                      const float* __restrict__ dw, int T, int E,
                                                                      int k, int sigmoid, int renormalize, float scale,
                                                                      float* __restrict__ dl, DevStatus st) {
    pdl_begin();
    constexpr int W = sizeof(V) / 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool dense = !sigmoid && !renormalize;
    const int nv = E / W;
    for (int t = blockIdx.x * kWarps + warp; t < T; t += gridDim.x * kWarps) {
        const float* row = logits + (size_t)t * E;
        float* out = dl + (size_t)t * E;
        const int e = lane < k ? topk_idx[(size_t)t * k + lane] : -1;
        const bool in = e >= 0 && e < E;
        if (lane < k && !in) raise_status(st, kStatusInvalidExpert);
        const float g = in ? dw[(size_t)t * k + lane] : 0.0f;
        const float l = in ? masked_logit(row[e]) : -INFINITY;
        const bool live = l != -INFINITY;
        if (!dense) {
            const float rest = sigmoid && live ? 1.0f / (1.0f + expf(l)) : 1.0f;  // 1 - sigmoid(l)
            float d;
            if (renormalize) {
                const float w = share_of(l, in, sigmoid);
                d = scale * w * (g - warp_sum(w * g)) * rest;
            } else {
                d = live ? scale * g * sigmoid_f(l) * rest : 0.0f;
            }
            V zero;
            float* z = reinterpret_cast<float*>(&zero);
#pragma unroll
            for (int u = 0; u < W; ++u) z[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane + 32 * i < nv) reinterpret_cast<V*>(out)[lane + 32 * i] = zero;
            __syncwarp();
            if (in) out[e] = d;
            continue;
        }
        V v[NV];
        float* p = reinterpret_cast<float*>(v);
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < nv) v[i] = reinterpret_cast<const V*>(row)[lane + 32 * i];
#pragma unroll
        for (int i = 0; i < NV * W; ++i) {
            p[i] = lane + 32 * (i / W) < nv ? masked_logit(p[i]) : -INFINITY;
            mx = fmaxf(mx, p[i]);
        }
        mx = warp_max(mx);
        float den = 0.0f;
#pragma unroll
        for (int i = 0; i < NV * W; ++i) {
            p[i] = p[i] == -INFINITY ? 0.0f : exp_rel(p[i], mx);
            den += p[i];
        }
        den = warp_sum(den);
        const float inv_den = den > 0.0f ? 1.0f / den : 0.0f;
        const float pe = live ? exp_rel(l, mx) * inv_den : 0.0f;
        const float dot = warp_sum(scale * g * pe);
#pragma unroll
        for (int i = 0; i < NV * W; ++i) p[i] *= -dot * inv_den;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < nv) reinterpret_cast<V*>(out)[lane + 32 * i] = v[i];
        __syncwarp();
        if (in) out[e] = pe * (scale * g - dot);
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

int grid_for(int T, int per_cta = kWarps) {
    const long want = ((long)T + per_cta - 1) / per_cta;
    const long cap = (long)num_sms() * 16;
    return (int)(want < cap ? want : cap);
}

template <int LPT, int PER>
cudaError_t launch_scored_per(const RouteArgs& a, int kind, int lpg, int vec, cudaStream_t stream) {
    const size_t smem = (size_t)kWarps * scratch_doubles(a.E) * sizeof(double) + LPT * (PER + 4) * sizeof(float);
    auto launch = [&](auto kern) {
        return launch_pdl(kern, dim3(grid_for(a.T, kWarps * (32 / LPT))), dim3(kWarps * 32), smem, stream, a, lpg, vec);
    };
    if (kind == kKeyLogit) return launch(scored_topk_kernel<LPT, PER, kKeyLogit>);
    if (kind == kKeySigmoid) return launch(scored_topk_kernel<LPT, PER, kKeySigmoid>);
    return launch(scored_topk_kernel<LPT, PER, kKeySoftmax>);
}

cudaError_t launch_scored(const RouteArgs& a, cudaStream_t stream) {
    const bool grouped = a.topk_groups < a.n_groups;
    const int kind = !a.bias && !(grouped && a.top2) ? kKeyLogit : a.sigmoid ? kKeySigmoid : kKeySoftmax;
    const int gs = a.E / a.n_groups;
    // lanes per group and experts per lane when a token has `lanes` lanes (0: does not fit)
    int lpg = 0;
    auto fit = [&](int lanes) {
        if (a.n_groups > lanes) return 0;
        lpg = lanes;
        while (lpg * a.n_groups > lanes) lpg >>= 1;
        return (gs + lpg - 1) / lpg;
    };
    const int vec = a.ksplit == 1 && gs % 4 == 0 && (reinterpret_cast<uintptr_t>(a.partials) & 15) == 0;
    // Two tokens per warp once every SM has dozens of tokens (65536 x 256: 77 against 88 us);
    // below, one per warp ends sooner (4096: 12 against 15 us).
    const int per16 = a.T >= 16384 ? fit(16) : 0;
    if (per16 > 4 && per16 <= 16 && a.k <= 31) {
        if (per16 <= 8) return launch_scored_per<16, 8>(a, kind, lpg, vec, stream);
        return launch_scored_per<16, 16>(a, kind, lpg, vec, stream);
    }
    const int per = fit(32);
    // more than 31 selected (no block left for the next one) or more experts than a lane holds
    if (a.k > 31 || per > 32)
        return launch_pdl(scored_topk_fp64_kernel, dim3(grid_for(a.T)), dim3(kWarps * 32),
                          (size_t)kWarps * a.E * sizeof(double), stream, a);
    if (per <= 1) return launch_scored_per<32, 1>(a, kind, lpg, vec, stream);
    if (per <= 2) return launch_scored_per<32, 2>(a, kind, lpg, vec, stream);
    if (per <= 4) return launch_scored_per<32, 4>(a, kind, lpg, vec, stream);
    if (per <= 8) return launch_scored_per<32, 8>(a, kind, lpg, vec, stream);
    if (per <= 16) return launch_scored_per<32, 16>(a, kind, lpg, vec, stream);
    return launch_scored_per<32, 32>(a, kind, lpg, vec, stream);
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
    const cudaError_t e = launch_scored(a, reinterpret_cast<cudaStream_t>(stream));
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
    const int E = shape->n_experts;
    // rows as float4s where they start on 16 bytes
    const bool vec = E % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(d_logits)) & 15) == 0;
    auto launch = [&](auto kern) {
        return launch_pdl(kern, dim3(grid_for(T)), dim3(kWarps * 32), 0, reinterpret_cast<cudaStream_t>(stream), logits,
                          topk_idx, d_topk_w, T, E, (int)shape->top_k, (int)(router->score == MOE_SCORE_SIGMOID),
                          (int)router->renormalize, router->scale, d_logits, st);
    };
    const cudaError_t e = !vec       ? launch(scored_backward_kernel<float, 32>)
                          : E <= 128 ? launch(scored_backward_kernel<float4, 1>)
                          : E <= 256 ? launch(scored_backward_kernel<float4, 2>)
                          : E <= 512 ? launch(scored_backward_kernel<float4, 4>)
                                     : launch(scored_backward_kernel<float4, 8>);
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "scored backward launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

}  // extern "C"

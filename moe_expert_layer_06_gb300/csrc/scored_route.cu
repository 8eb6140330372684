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
// another is decided again in fp64 (about one row in a thousand), as is a row with values of +inf.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "operators.cuh"

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
// shapes outside the fast kernel's layout.  c: E doubles of this warp's shared memory.  Where
// the scores order as the logits do (no bias, no sums of two) c stays the logits, as in the fast
// kernel: a sigmoid is 1 in fp64 too from a logit of 37 on, a softmax's small terms are 0.
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
    // (beside an infinite logit every other softmax is 0: they tie)
    const bool by_logit = !a.bias && !(a.top2 && a.topk_groups < a.n_groups) && (a.sigmoid || mx < INFINITY);
    for (int e = lane; e < a.E && !by_logit; e += 32) {
        const double l = c[e];
        if (l == -INFINITY) continue;
        double s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : (l == mx ? 1.0 : exp(l - (double)mx)) / den;
        if (a.bias) s += a.bias[e];
        c[e] = s == s ? s : -INFINITY;  // (a NaN bias keeps its expert out as one of -inf does)
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
    // Lane j keeps the j-th selected expert; taken experts are marked NaN, which nothing else is.
    // The kept groups hold k experts at least (check_router), so each round finds one.
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
        i = min(i, a.E - 1);  // (whatever the values: an index of the row)
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

// ---------------------------------------------------------------- the fast selection
// max of three in one instruction (NaN loses against a number)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <int N>
__device__ __forceinline__ float max_of(const float* v) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i + 1 < N; i += 2) m = max3(m, v[i], v[i + 1]);
    if (N % 2 == 0) m = fmaxf(m, v[N - 1]);
    return m;
}

__device__ __forceinline__ float fast_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// Reductions over the LPT consecutive lanes of one token (every lane gets the result).
template <int LPT>
__device__ __forceinline__ float token_max(float v) {
    if constexpr (LPT == 32) {
        float r;  // one instruction for the warp
        asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
        return r;
    } else {
#pragma unroll
        for (int d = LPT / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
}

template <int LPT>
__device__ __forceinline__ float token_sum(float v) {
#pragma unroll
    for (int d = LPT / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// What the fp32 selection value c of an expert is.
enum KeyKind : int {
    kKeyLogit,    // the logit itself: orders as the score does, and exactly (no bias, no sum of two)
    kKeySigmoid,  // sigmoid + bias
    kKeySoftmax,  // softmax + bias
};

// How a row lies in the lanes of its token: lpg (a power of two) lanes per group, `per`
// consecutive experts per lane; what passes the group's end is empty.
struct Layout {
    int gs, lpg, per;
};

// The exact score of one logit; den: the softmax's exact sum relative to mx.
__device__ __forceinline__ double score64(const RouteArgs& a, float l, float mx, double den) {
    if (a.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
    return (l == mx ? 1.0 : exp((double)l - (double)mx)) / den;
}

// The softmax's sum of row t in fp64, by the whole warp (1 for a sigmoid).
__device__ __forceinline__ double sum64(const RouteArgs& a, int t, float mx) {
    if (a.sigmoid) return 1.0;
    double d = 0.0;
#pragma unroll 4
    for (int e = threadIdx.x & 31; e < a.E; e += 32) {
        const float x = masked_logit(logit_at(a, t, e));
        d += x == mx ? 1.0 : exp((double)x - (double)mx);
    }
    return warp_sum(d);
}

// Row t, by the whole warp: which groups are kept, decided in fp64 from the experts that
// fp32 (values c of the row, off by `err` at most and half a step) leaves for the two best.
// 0: a group has more of them than kGroupCand (the row is left to select_fp64).
constexpr int kGroupCand = 4;
__device__ __noinline__ uint32_t resolve_groups(const RouteArgs& a, int t, const float* c, Layout lay, float mx, float err) {
    const int lane = threadIdx.x & 31;
    const double den = sum64(a, t, mx);
    double score = -INFINITY;
    bool over = false;
    if (lane < a.n_groups) {
        // the group's values: lpg lanes' rows of per + 4 floats
        float k0 = -INFINITY, k1 = -INFINITY;
        const float* row = c + lane * lay.lpg * (lay.per + 4);
        for (int l = 0; l < lay.lpg; ++l)
            for (int i = 0; i < lay.per; ++i) {  // (empty ones are -inf)
                const float v = fmaxf(row[l * (lay.per + 4) + i], -INFINITY);
                k1 = fmaxf(k1, fminf(k0, v));
                k0 = fmaxf(k0, v);
            }
        const float low = a.top2 && k1 != -INFINITY ? k1 : k0;
        const float from = low - 2.0f * err - 0x1p-21f * fabsf(low);
        // collected first, so that the lanes' evaluations run together (they are what takes time)
        int at[kGroupCand], n = 0;
        for (int l = 0; l < lay.lpg && k0 != -INFINITY; ++l)
            for (int i = 0; i < lay.per; ++i) {
                if (!(row[l * (lay.per + 4) + i] >= from)) continue;
#pragma unroll
                for (int q = 0; q < kGroupCand; ++q) at[q] = q == n ? lane * lay.gs + l * lay.per + i : at[q];
                ++n;
            }
        over = n > kGroupCand;
        double d0 = -INFINITY, d1 = -INFINITY;
#pragma unroll
        for (int q = 0; q < kGroupCand; ++q) {
            if (q >= n) continue;
            const double v = score64(a, masked_logit(logit_at(a, t, at[q])), mx, den) + (a.bias ? (double)a.bias[at[q]] : 0.0);
            d1 = fmax(d1, fmin(d0, v));
            d0 = fmax(d0, v);
        }
        score = d0;
        if (a.top2 && d1 != -INFINITY) score += d1;
    }
    __syncwarp();
    if (__any_sync(0xffffffffu, over)) return 0;
    int rank = 0;
    for (int o = 0; o < a.n_groups; ++o) {
        const double v = __shfl_sync(0xffffffffu, score, o);
        rank += v > score || (v == score && o < lane) ? 1 : 0;
    }
    return __ballot_sync(0xffffffffu, lane < a.n_groups && rank < a.topk_groups);
}

// Row t, by the whole warp: the order of its n <= 64 candidates (in ascending order of
// experts, e[]) in fp64; sorted[rank] = candidate.  v: 128 doubles.  A softmax's sum is
// first taken of fp32 exponentials (the rounding of l - mx made good, so 2 steps each; 1024
// fp64 ones take ten times as long), which decides unless two neighbours differ by no
// more than that error makes of the difference of their scores.
__device__ __noinline__ void resolve_order(const RouteArgs& a, int t, const uint16_t* e, int n, float mx, double* v,
                                           uint16_t* sorted) {
    const int lane = threadIdx.x & 31;
    double* s = v + kCand;
    double den = 1.0, rel = 0.0;
    if (!a.sigmoid) {
        den = 0.0;
        for (int i = lane; i < a.E; i += 32) {
            const float l = masked_logit(logit_at(a, t, i));
            const float x = l - mx, back = x + mx;
            const float rest = l == -INFINITY ? 0.0f : (l - back) - (mx - (back - x));
            den += (double)(expf(x) * (1.0f + rest));
        }
        den = warp_sum(den);
        rel = 0x1p-21;
    }
    for (bool again = true; again;) {
        for (int q = lane; q < n; q += 32) {
            s[q] = score64(a, masked_logit(logit_at(a, t, e[q])), mx, den);
            v[q] = s[q] + (a.bias ? (double)a.bias[e[q]] : 0.0);
        }
        __syncwarp();
        for (int q = lane; q < n; q += 32) {
            int rank = 0;
            for (int o = 0; o < n; ++o) rank += v[o] > v[q] || (v[o] == v[q] && o < q) ? 1 : 0;
            sorted[rank] = (uint16_t)q;
        }
        __syncwarp();
        bool open = false;
        if (rel > 0.0)
            for (int j = lane; j < min(a.k, n - 1); j += 32) {
                const int q = sorted[j];
                for (int i = j + 1; i < n; ++i) {
                    const int r = sorted[i];
                    const double gap = v[q] - v[r];
                    if (!(gap <= rel + 0x1p-45)) break;  // (scores are at most 1)
                    open |= gap <= rel * fabs(s[q] - s[r]) + 0x1p-45;
                }
            }
        again = __any_sync(0xffffffffu, open);
        if (again) {
            den = sum64(a, t, mx);
            rel = 0.0;
        }
    }
}

// Shared memory of a warp: two buffers of 32 lanes x `row` floats, or select_fp64's E doubles
// (resolve_order's 2 kCand doubles fit one buffer from rows of 8 floats, and both of less).
__host__ __device__ __forceinline__ int warp_smem(int E, int row) {
    const int b = 2 * 32 * row * 4, d = (E * 8 + 15) & ~15;
    return b > d ? b : d;
}

// LPT lanes per token, 32 / LPT tokens per warp.  Its time is instructions and the latency
// between them: 430 a token (65536 x 256 sigmoids in 8 groups), 23 us of the 51 if every cycle
// issued one; 16 warps an SM, all that 128 registers allow, issue in 53% of them.  Most of a
// token's (threshold, ranking, weights) cost the same for one token per warp or four, and the
// ones per expert are kept to the score and three more: a maximum of blocks, a comparison with
// the threshold and its bit.  Measured: 65536 x 256 51 us (29 where the logits decide), 8192 x
// 1024 softmax with a bias 30 us, one token 4.2 us.
template <int LPT, int PER, int KIND>
__global__ void __launch_bounds__(kWarps * 32)
    scored_topk_kernel(const __grid_constant__ RouteArgs a, int lpg, int vec) {
    pdl_begin();
    constexpr int TPW = 32 / LPT;  // tokens per warp
    // experts per block maximum: at least 32 blocks of a full row, at most 8 experts each
    constexpr int BLK = PER * LPT >= 256 ? 8 : PER * LPT >= 64 ? PER * LPT / 32 : 1;
    constexpr int NB = PER / BLK;
    constexpr int ROW = PER + 4;  // floats of a lane in shared memory (16-byte accesses without bank conflicts)
    extern __shared__ __align__(16) uint8_t dyn[];
    __shared__ __align__(16) float cand_all[kWarps * TPW][kCand];
    __shared__ uint16_t cand_e_all[kWarps * TPW][kCand];
    __shared__ uint16_t sorted_all[kWarps * TPW][kCand];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & (LPT - 1), slot = lane / LPT;
    float* cand = cand_all[warp * TPW + slot];         // values of the candidates, in expert order
    uint16_t* cand_e = cand_e_all[warp * TPW + slot];  // their experts
    uint16_t* sorted = sorted_all[warp * TPW + slot];  // candidate of each rank
    // Two buffers of 32 lanes x ROW: the logits, then the values of the warp's tokens, and
    // the logits of its next ones.  Also the fp64 scratch.
    const int warp_bytes = warp_smem(a.E, ROW);
    float* stage = reinterpret_cast<float*>(dyn + warp * warp_bytes);
    float* rows = stage;
    float* bias = reinterpret_cast<float*>(dyn + kWarps * warp_bytes);
    Layout lay;
    lay.gs = a.E / a.n_groups;
    lay.lpg = lpg;
    lay.per = PER;
    const int group = sub / lpg;
    const int in_group = (sub & (lpg - 1)) * PER;  // first of this lane's experts within its group
    const int n_mine = group < a.n_groups ? min(PER, max(0, lay.gs - in_group)) : 0;
    const int e0 = group * lay.gs + in_group;
    const bool grouped = a.topk_groups < a.n_groups;
    const bool stats = KIND == kKeySoftmax || (!a.sigmoid && !a.renormalize);
    auto bias_of = [&](int e) { return a.bias ? __ldg(a.bias + e) : 0.0f; };

    float c[PER];  // logits, then values
    // Whole float4s (vec): rows come by asynchronous 16-byte copies, coalesced, into the
    // places of their lanes, the next tokens' while these are selected.
    auto clear = [&]() {  // the empty places stay so
        for (int i = lane; i < 64 * ROW; i += 32) stage[i] = -INFINITY;
        __syncwarp();
    };
    int dst[PER >= 4 ? PER / 4 : 1];
    const int per_token = a.E / 4;
    if (PER >= 4 && vec) {
        if (a.E == LPT * PER) {  // no empty places: consecutive experts fill consecutive lanes
#pragma unroll
            for (int q = 0; q < (PER >= 4 ? PER / 4 : 1); ++q) {
                const int e = (lane + q * 32) * 4;
                dst[q] = e / PER * ROW + e % PER;
            }
        } else {
            clear();
        }
#pragma unroll
        for (int q = 0; q < (PER >= 4 ? PER / 4 : 1) && a.E != LPT * PER; ++q) {
            const int f = lane + q * 32, tok = f / per_token, e = (f - tok * per_token) * 4;
            const int g = e / lay.gs, i = e - g * lay.gs;
            dst[q] = tok < TPW ? (tok * LPT + g * lpg + i / PER) * ROW + i % PER : -1;
        }
    }
    auto prefetch = [&](int tw, int buf) {
        const float4* src = reinterpret_cast<const float4*>(a.partials + (size_t)tw * a.E);
        const int valid = min(TPW, a.T - tw) * per_token;  // float4s of tokens that exist
#pragma unroll
        for (int q = 0; q < (PER >= 4 ? PER / 4 : 1); ++q)
            if (dst[q] >= 0 && lane + q * 32 < valid)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(stage + buf * 32 * ROW + dst[q])),
                             "l"(src + lane + q * 32)
                             : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto load = [&](int t) {
        const float* p = a.partials + (size_t)t * a.E + e0;
        const int n = t < a.T ? n_mine : 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) c[i] = i < n ? p[i] : -INFINITY;
        for (int s = 1; s < a.ksplit; ++s) {
            p += (size_t)a.T * a.E;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < n) c[i] += p[i];
        }
    };
    const int stride = gridDim.x * kWarps * TPW;
    int tw = (blockIdx.x * kWarps + warp) * TPW;  // the warp's first token
    int buf = 0;
    if (PER >= 4 && vec && tw < a.T) prefetch(tw, 0);
    float bmax = -INFINITY;
    if (KIND != kKeyLogit) {
        if (warp == 0 && lane < LPT)
            for (int i = 0; i < PER; ++i) bias[sub * ROW + i] = a.bias && i < n_mine ? a.bias[e0 + i] : 0.0f;
        __syncthreads();
        for (int i = 0; i < n_mine; ++i) bmax = fmaxf(bmax, bias[sub * ROW + i]);
        bmax = token_max<LPT>(bmax);
    }
    for (; tw < a.T; tw += stride) {
        const int t = tw + slot;
        if (PER >= 4 && vec) {
            if (tw + stride < a.T) prefetch(tw + stride, buf ^ 1);
            else asm volatile("cp.async.commit_group;" ::: "memory");
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
            rows = stage + buf * 32 * ROW;
            const float* r = rows + lane * ROW;
#pragma unroll
            for (int i = 0; i < PER; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(r + i);
                c[i] = v.x;
                c[(i + 1) % PER] = v.y;
                c[(i + 2) % PER] = v.z;
                c[(i + 3) % PER] = v.w;
            }
            buf ^= 1;
            __syncwarp();
        } else {
            load(t);
        }
        const bool alive = t < a.T;
        if (a.logits_out && alive) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i < n_mine) a.logits_out[(size_t)t * a.E + e0 + i] = c[i];
        }
        // ---- values.  A NaN stays a NaN, which no maximum and no comparison takes: masked.
        bool unsure = !alive;  // the row is left to select_fp64 (or does not exist)
        float mx = 0.0f, inv_den = 1.0f;
        float e[KIND == kKeySoftmax ? PER : 1];
        if (stats) {
            mx = token_max<LPT>(max_of<PER>(c));
            unsure |= !(fabsf(mx) < INFINITY);  // an infinite logit, or none at all
            float part[PER];  // summed in pairs: log2(E) roundings
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                part[i] = fmaxf(fast_exp2((c[i] - mx) * kLog2e), 0.0f);
                if (KIND == kKeySoftmax) e[i % (KIND == kKeySoftmax ? PER : 1)] = part[i];
            }
#pragma unroll
            for (int w = PER / 2; w > 0; w >>= 1)
#pragma unroll
                for (int i = 0; i < w; ++i) part[i] += part[i + w];
            inv_den = 1.0f / token_sum<LPT>(part[0]);
        }
        if (KIND != kKeyLogit) {
#pragma unroll
            for (int i = 0; i < PER; i += (PER >= 4 ? 4 : 1)) {
                float b4[4];
                if (PER >= 4) {
                    const float4 v = *reinterpret_cast<const float4*>(bias + sub * ROW + i);
                    b4[0] = v.x;
                    b4[1] = v.y;
                    b4[2] = v.z;
                    b4[3] = v.w;
                } else {
                    b4[0] = bias[sub * ROW + i];
                }
#pragma unroll
                for (int u = 0; u < (PER >= 4 ? 4 : 1); ++u) {
                    // 2^-149 l: nothing beside the bias, but for -inf, which stays -inf (and +inf: see below)
                    const float base = fmaf(c[i + u], 0x1p-149f, b4[u]);
                    if (KIND == kKeySigmoid) c[i + u] = base + fast_rcp(1.0f + fast_exp2(c[i + u] * -kLog2e));
                    else c[i + u] = fmaf(e[(i + u) % (KIND == kKeySoftmax ? PER : 1)], inv_den, base);
                }
            }
        }
        // Bound of |c - exact| before the sum with the bias rounds (half a step).  Sigmoid: the
        // exponential is off by 2 steps and 1.5 |l| of its argument, which 1 / (1 + e) takes
        // s (1 - s) of (at most 0.75 steps of 2^-23), the sum and the reciprocal by 1.5
        // more: 3 in all.  Softmax: 2 steps of the exponential and 1.5 |l - mx| of its
        // argument (at most 0.6 of the value 1 / den), log2(1024) / 2 of the sum and 3 of
        // its terms, 2 of 1 / den and the product: 16.  Where a logit is near -FLT_MAX
        // 2^-149 of it adds 4 steps to its bias; only rows whose threshold is not above the
        // largest bias can select such an expert.
        const float err = KIND == kKeyLogit ? 0.0f : 0x1p-23f * (KIND == kKeySigmoid ? 3.0f : 16.0f * inv_den);

        // ---- groups
        float m[NB];
#pragma unroll
        for (int q = 0; q < NB; ++q) m[q] = max_of<BLK>(c + q * BLK);
        // Values of +inf are not what they stand for (an infinite logit's score is 1), and their
        // differences are NaN; so are sums beyond the largest float: such a row goes to select_fp64.
        auto any_lane = [&](bool p) {
            const uint32_t b = __ballot_sync(0xffffffffu, p);
            return LPT == 32 ? b != 0 : ((b >> (slot * LPT)) & ((1u << (LPT & 31)) - 1u)) != 0;
        };
        if (KIND != kKeyLogit) unsure |= any_lane(max_of<NB>(m) == INFINITY);
        auto write_rows = [&]() {
            float* r = rows + lane * ROW;
            if constexpr (PER >= 4) {
#pragma unroll
                for (int i = 0; i < PER; i += 4)
                    *reinterpret_cast<float4*>(r + i) = make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) r[i] = c[i];
            }
            __syncwarp();
        };
        write_rows();
        if (grouped) {
            float k0, k1 = -INFINITY;  // the two largest of the group
            if (KIND != kKeyLogit && a.top2) {
                k0 = -INFINITY;
                if constexpr (PER >= 2) {
#pragma unroll
                    for (int i = 0; i < PER; i += 2) {
                        const float x = fmaxf(c[i], -INFINITY), y = fmaxf(c[i + 1], -INFINITY);
                        const float hi = fmaxf(x, y);
                        k1 = max3(k1, fminf(x, y), fminf(k0, hi));
                        k0 = fmaxf(k0, hi);
                    }
                } else {
                    k0 = fmaxf(c[0], -INFINITY);
                }
            } else {
                k0 = fmaxf(max_of<NB>(m), -INFINITY);
            }
            for (int d = 1; d < lpg; d <<= 1) {
                const float o0 = __shfl_xor_sync(0xffffffffu, k0, d), o1 = __shfl_xor_sync(0xffffffffu, k1, d);
                k1 = max3(k1, o1, fminf(k0, o0));
                k0 = fmaxf(k0, o0);
            }
            const float g = KIND != kKeyLogit && a.top2 && k1 != -INFINITY ? k0 + k1 : k0;
            if (KIND != kKeyLogit && a.top2) unsure |= any_lane(fabsf(g) == INFINITY && k0 != -INFINITY);
            int rank = 0;
            for (int o = 0; o < a.n_groups; ++o) {
                const float v = __shfl_sync(0xffffffffu, g, o * lpg, LPT);
                rank += v > g || (v == g && o < group) ? 1 : 0;
            }
            bool keep = group < a.n_groups && rank < a.topk_groups;
            if (KIND != kKeyLogit) {
                const float in = -token_max<LPT>(keep ? -g : -INFINITY);
                const float out = token_max<LPT>(keep || group >= a.n_groups ? -INFINITY : g);
                // (two groups without an unmasked expert tie exactly)
                const float far = err + (out <= 2.0f * bmax + 0x1p-10f ? 0x1p-21f : 0.0f);
                const bool close = out != -INFINITY && in - out <= 4.0f * far + 0x1p-21f * fabsf(in);
                for (uint32_t todo = __ballot_sync(0xffffffffu, close && sub == 0 && !unsure); todo; todo &= todo - 1) {
                    const int s = (__ffs(todo) - 1) / LPT;
                    const uint32_t kept = resolve_groups(a, tw + s, rows + s * LPT * ROW, lay,
                                                         __shfl_sync(0xffffffffu, mx, s * LPT),
                                                         __shfl_sync(0xffffffffu, far, s * LPT));
                    if (slot == s) {
                        keep = group < a.n_groups && ((kept >> group) & 1u);
                        unsure |= kept == 0;
                    }
                }
            }
            if (!keep) {
#pragma unroll
                for (int q = 0; q < NB; ++q) m[q] = -INFINITY;
            }
        }
        // ---- threshold: the (k+1)-th largest block maximum (the largest k+1 values pass it)
        const bool mine_out = !(max_of<NB>(m) > -INFINITY);  // no expert of this lane can be selected
        float tau = INFINITY, top = -INFINITY;
        for (int j = 0; j <= a.k; ++j) {
            tau = token_max<LPT>(max_of<NB>(m));
            if (j == 0) top = tau;
#pragma unroll
            for (int q = 0; q < NB; ++q) m[q] = m[q] == tau ? -INFINITY : m[q];
        }
        float eps = 0.0f;
        if (KIND != kKeyLogit) {
            const float far = err + (tau <= bmax + 0x1p-10f ? 0x1p-21f : 0.0f);
            eps = 2.0f * far + 0x1p-22f * fmaxf(fabsf(top), tau > -INFINITY ? fabsf(tau) : 0.0f);
            tau -= 2.0f * eps;
        } else if (!a.sigmoid) {
            unsure |= top == INFINITY;  // beside an infinite logit every other has softmax 0: they tie
        }
        tau = fmaxf(tau, -FLT_MAX);
        // ---- candidates in expert order
        uint32_t part_bits[4] = {0, 0, 0, 0};
        auto mark = [&](int i, float v) {
            asm("{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\t@p or.b32 %0, %0, %3;\n\t}"
                : "+r"(part_bits[i & 3])
                : "f"(v), "f"(tau), "r"(1u << (i & 31)));
        };
        if constexpr (PER >= 4) {
#pragma unroll
            for (int i = 0; i < PER; i += 4) {  // from `rows`: the registers are free for the calls above
                const float4 v = *reinterpret_cast<const float4*>(rows + lane * ROW + i);
                mark(i, v.x);
                mark(i + 1, v.y);
                mark(i + 2, v.z);
                mark(i + 3, v.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) mark(i, rows[lane * ROW + i]);
        }
        uint32_t bits = (part_bits[0] | part_bits[1]) | (part_bits[2] | part_bits[3]);
        if (mine_out) bits = 0;
        const int cnt = __popc(bits);
        int incl = cnt;
#pragma unroll
        for (int d = 1; d < LPT; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, d, LPT);
            if (sub >= d) incl += o;
        }
        int n = __shfl_sync(0xffffffffu, incl, LPT - 1, LPT);
        if (unsure || n > kCand || n < a.k) {  // too many, or masked experts are among the selected
            unsure = true;
            n = 0;
            bits = 0;
        }
        for (int at = incl - cnt; bits; ++at, bits &= bits - 1) {
            const int i = __ffs(bits) - 1;
            cand[at] = rows[lane * ROW + i];
            cand_e[at] = (uint16_t)(e0 + i);
        }
        // whole vectors of four
        for (int q = n + sub; q < ((n + 3) & ~3); q += LPT) cand[q] = -INFINITY;
        __syncwarp();
        // ---- order: rank of each candidate among all
        bool dirty = false;  // the rows hold fp64 scratch
        bool tie = false;
        for (int q = sub; q < n; q += LPT) {
            const float mine = cand[q];
            int rank = 0, same = 0;
            for (int o = 0; o < n; o += 4) {
                const float4 v = *reinterpret_cast<const float4*>(cand + o);
                rank += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
                same += (v.x == mine) + (v.y == mine) + (v.z == mine) + (v.w == mine);
            }
            tie |= same > 1;
            sorted[rank] = (uint16_t)q;
        }
        if (__any_sync(0xffffffffu, tie)) {
            // ties in expert order: an equal value at a lower position goes first
            __syncwarp();
            for (int q = sub; q < n; q += LPT) {
                const float mine = cand[q];
                int rank = 0;
                for (int o = 0; o < n; ++o) rank += cand[o] > mine || (cand[o] == mine && o < q) ? 1 : 0;
                sorted[rank] = (uint16_t)q;
            }
        }
        __syncwarp();
        if (KIND != kKeyLogit) {
            // neighbours of the first k + 1 in order, too close for fp32?
            bool close = false;
            for (int j = sub; j < min(a.k, n - 1); j += LPT) {
                const int q = sorted[j];
                if (KIND == kKeySigmoid) {
                    close |= cand[q] - cand[sorted[j + 1]] <= eps;
                    continue;
                }
                // A softmax's error is relative to the scores: the pair's own, where eps takes the
                // largest of the row (all followers within eps: their scores differ).
                const float pq = fabsf(cand[q] - bias_of(cand_e[q]));
                for (int i = j + 1; i < n; ++i) {
                    const int r = sorted[i];
                    const float gap = cand[q] - cand[r];
                    if (!(gap <= eps)) break;
                    const float pr = fabsf(cand[r] - bias_of(cand_e[r]));
                    close |= gap <= eps - 2.0f * err + 0x1p-23f * 16.0f * (pq + pr);
                }
            }
            uint32_t todo = __ballot_sync(0xffffffffu, close);
            dirty = todo != 0;
            while (todo) {
                // (every exact value above the k-th is among the candidates)
                const int s = (__ffs(todo) - 1) / LPT, w = warp * TPW + s;
                resolve_order(a, tw + s, cand_e_all[w], __shfl_sync(0xffffffffu, n, s * LPT),
                              __shfl_sync(0xffffffffu, mx, s * LPT), reinterpret_cast<double*>(rows), sorted_all[w]);
                todo &= ~(((LPT == 32 ? 0u : 1u << (LPT & 31)) - 1u) << (s * LPT));
            }
        }
        // ---- weights: lane sub holds the selected experts sub, sub + LPT, ... of its token
        for (int j0 = 0; j0 < (a.renormalize ? 1 : a.k); j0 += LPT) {
            if (!a.renormalize) {
                const int j = j0 + sub;
                if (j < a.k && !unsure) {
                    const int id = cand_e[sorted[j]];
                    const float l = logit_at(a, t, id);
                    a.topk_idx[(size_t)t * a.k + j] = id;
                    a.topk_w[(size_t)t * a.k + j] = a.scale * (a.sigmoid ? sigmoid_f(l) : exp_rel(l, mx) * inv_den);
                }
            } else {
                constexpr int KPL = 32 / LPT;
                float l[KPL], sh[KPL];
                float low = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int q = 0; q < KPL; ++q) {
                    l[q] = -INFINITY;
                    const int j = sub + q * LPT;
                    if (j < a.k && !unsure) {
                        const int id = cand_e[sorted[j]];
                        l[q] = logit_at(a, t, id);
                        a.topk_idx[(size_t)t * a.k + j] = id;
                        low = fmaxf(low, a.sigmoid ? fminf(l[q], 0.0f) : l[q]);
                    }
                }
                low = token_max<LPT>(low);
#pragma unroll
                for (int q = 0; q < KPL; ++q) {
                    sh[q] = 0.0f;
                    if (sub + q * LPT < a.k && !unsure) sh[q] = share_term(l[q], low, a.sigmoid);
                    sum += sh[q];
                }
                sum = token_sum<LPT>(sum);
                const float f = a.scale / sum;
#pragma unroll
                for (int q = 0; q < KPL; ++q) {
                    const int j = sub + q * LPT;
                    if (j < a.k && !unsure) a.topk_w[(size_t)t * a.k + j] = sh[q] * f;
                }
            }
        }
        uint32_t redo = __ballot_sync(0xffffffffu, alive && unsure && sub == 0);
        if (redo) {
            // (its scratch is both buffers: the copies under way end first and start again)
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            for (; redo; redo &= redo - 1) select_fp64(a, tw + (__ffs(redo) - 1) / LPT, reinterpret_cast<double*>(stage));
            if (PER >= 4 && vec && tw + stride < a.T) {
                clear();
                prefetch(tw + stride, buf);
            }
        } else if (dirty) {
            // empty places are not copied over
            for (int i = n_mine; i < PER; ++i) rows[lane * ROW + i] = -INFINITY;
        }
        __syncwarp();
    }
}

// The gradient of one row.  Lane j < k holds the j-th selected expert; V: float or float4,
// NV of them per lane (V vec = lane + 32 i of the row).  Sparse gradients (sigmoid, or
// renormalised) are zeros and k values; a softmax as it is reads the row once.  Bound by
// the chain of loads, reductions and stores of a row, 64 rows on an SM at a time: 16384 x
// 256 dense 10 us (34 MB, 3.4 TB/s), 4096 x 256 sparse 4.5 us.
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
        const float l = in ? masked_logit(row[e]) : -INFINITY;
        const bool live = l != -INFINITY;
        // (a masked expert's weight is 0 whatever the logits: what its dw holds stays out of the row's sums)
        const float g = live ? dw[(size_t)t * k + lane] : 0.0f;
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

int grid_for(int T, int per_cta = kWarps, int per_sm = 16) {
    const long want = ((long)T + per_cta - 1) / per_cta;
    const long cap = (long)num_sms() * per_sm;
    return (int)(want < cap ? want : cap);
}

template <int LPT, int PER>
cudaError_t launch_scored_per(const RouteArgs& a, int kind, int lpg, int vec, cudaStream_t stream) {
    const size_t smem = (size_t)kWarps * warp_smem(a.E, PER + 4) + LPT * (PER + 4) * sizeof(float);
    auto launch = [&](auto kern) {
        static std::atomic<uint64_t> configured[3];
        const cudaError_t e = configure_once(configured[kind], [&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024);
        });
        if (e != cudaSuccess) return e;
        // four CTAs an SM are resident (registers), each taking several turns: its set-up is paid once
        return launch_pdl(kern, dim3(grid_for(a.T, kWarps * (32 / LPT), 4)), dim3(kWarps * 32), smem, stream, a, lpg, vec);
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
    // Four tokens per warp once every SM has sixteen (65536 x 256, sigmoid and groups: 50
    // against 102 us; 4096: 12.2 against 13.3); below, one ends sooner (512: 6.8 against 5.5).
    const int per8 = a.T >= 16 * num_sms() ? fit(8) : 0;
    if (per8 > 4 && per8 <= 32 && a.k <= 16) {
        if (per8 <= 8) return launch_scored_per<8, 8>(a, kind, lpg, vec, stream);
        if (per8 <= 16) return launch_scored_per<8, 16>(a, kind, lpg, vec, stream);
        return launch_scored_per<8, 32>(a, kind, lpg, vec, stream);
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

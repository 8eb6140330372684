// Matrix products grouped by expert, and their gradients:
//   y[r]  = W_p[s] x[r]                    for the rows r of slot s, parts p side by side (gate, up)
//   dx[r] = sum_p W_p[s]^T dy_p[r],  dW_p[s] = sum over s's rows of dy_p[r] x[r]^T.
// The rows of a slot are consecutive (a dispatch's order), their counts ragged.
#include <cuda_fp8.h>

#include "e4m3.cuh"
#include "operators.cuh"

namespace moe {
namespace {

constexpr int kMaxSlots = 1024;
constexpr int kMaxFeatures = 1 << 24;

struct Args {
    const uint16_t* rows_in;  // x [R][K] | dy [R][P][N]
    const uint16_t* x;
    const uint8_t* x8;
    const float* x8_scale;
    const uint16_t* w[2];
    void* out[2];
    const int32_t* offsets;
    int R, K, N, P, S, type;
    DevStatus st;
};

__device__ __forceinline__ float bf(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }

__device__ __forceinline__ void store(void* out, size_t at, float v, int type) {
    if (type == MOE_OUT_BF16) static_cast<uint16_t*>(out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else if (type == MOE_OUT_F32) static_cast<float*>(out)[at] = v;
    else static_cast<float*>(out)[at] += v;
}

__device__ __forceinline__ float kept(const Args& a, int r, int c) {
    const int nb = (a.K + MOE_PAYLOAD_BLOCK - 1) / MOE_PAYLOAD_BLOCK;
    __nv_fp8_e4m3 v;
    v.__x = a.x8[(size_t)r * a.K + c];
    return (float)v * a.x8_scale[(size_t)r * nb + c / MOE_PAYLOAD_BLOCK];
}

// C [64][64] = sum over l of A(i, l) B(j, l), 256 threads with 4 x 4 each, 16 of l at a time.
template <typename FA, typename FB>
__device__ __forceinline__ void product(int L, FA&& fa, FB&& fb, float (&c)[4][4]) {
    __shared__ float sa[16][65], sb[16][65];
    const int ti = threadIdx.x / 16, tj = threadIdx.x % 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) c[i][j] = 0.0f;
    for (int l0 = 0; l0 < L; l0 += 16) {
        for (int q = threadIdx.x; q < 1024; q += 256) {
            const int l = q & 15, i = q >> 4;
            sa[l][i] = l0 + l < L ? fa(i, l0 + l) : 0.0f;
            sb[l][i] = l0 + l < L ? fb(i, l0 + l) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int l = 0; l < 16; ++l)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i][j] = fmaf(sa[l][ti * 4 + i], sb[l][tj * 4 + j], c[i][j]);
        __syncthreads();
    }
}

// 64 rows of one slot times 64 of the outputs: y, or (DX) dx.
template <bool DX>
__global__ void __launch_bounds__(256) rows_kernel(const Args a) {
    pdl_begin();
    int chunk = blockIdx.y, lo = 0, hi = 0, s = 0;
    for (; s < a.S; ++s) {
        if (!slot_rows(a.offsets, s, a.R, lo, hi) && threadIdx.x == 0) raise_status(a.st, kStatusBadShape);
        const int n = (hi - lo + 63) / 64;
        if (chunk < n) break;
        chunk -= n;
    }
    if (s == a.S) return;
    const int r0 = lo + chunk * 64, O = DX ? a.K : a.P * a.N, o0 = blockIdx.x * 64;
    float c[4][4];
    product(
        DX ? a.P * a.N : a.K,
        [&](int i, int l) { return r0 + i < hi ? bf(a.rows_in[(size_t)(r0 + i) * (DX ? a.P * a.N : a.K) + l]) : 0.0f; },
        [&](int j, int l) {
            if (o0 + j >= O) return 0.0f;
            const int n = DX ? l : o0 + j, k = DX ? o0 + j : l;
            return bf(a.w[n / a.N][((size_t)s * a.N + n % a.N) * a.K + k]);
        },
        c);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + threadIdx.x / 16 * 4 + i, o = o0 + threadIdx.x % 16 * 4 + j;
            if (r < hi && o < O) store(a.out[0], (size_t)r * O + o, c[i][j], a.type);
        }
}

// 64 x 64 of a slot's dW.
__global__ void __launch_bounds__(256) weights_kernel(const Args a) {
    pdl_begin();
    const int s = blockIdx.z, nt = (a.N + 63) / 64, p = blockIdx.y / nt, n0 = blockIdx.y % nt * 64, k0 = blockIdx.x * 64;
    int lo, hi;
    if (!slot_rows(a.offsets, s, a.R, lo, hi) && threadIdx.x == 0) raise_status(a.st, kStatusBadShape);
    float c[4][4];
    product(
        hi - lo, [&](int i, int l) { return n0 + i < a.N ? bf(a.rows_in[((size_t)(lo + l) * a.P + p) * a.N + n0 + i]) : 0.0f; },
        [&](int j, int l) {
            if (k0 + j >= a.K) return 0.0f;
            return a.x ? bf(a.x[(size_t)(lo + l) * a.K + k0 + j]) : kept(a, lo + l, k0 + j);
        },
        c);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + threadIdx.x / 16 * 4 + i, k = k0 + threadIdx.x % 16 * 4 + j;
            if (n < a.N && k < a.K) store(a.out[p], ((size_t)s * a.N + n) * a.K + k, c[i][j], a.type);
        }
}

int check_project(const moe_project_t* p, int rows) {
    if (!p) return api_fail(MOE_ERR_INVALID_ARG, "project is NULL");
    if (rows < 0) return api_fail(MOE_ERR_INVALID_ARG, "rows = %d < 0", rows);
    if (p->in_features <= 0 || p->out_features <= 0 || p->n_slots <= 0)
        return api_fail(MOE_ERR_INVALID_ARG, "non-positive project field");
    if (p->in_features % 8 || p->out_features % 8)
        return api_fail(MOE_ERR_INVALID_ARG, "in_features and out_features must be multiples of 8");
    if (p->n_parts != 1 && p->n_parts != 2) return api_fail(MOE_ERR_INVALID_ARG, "n_parts %d is not 1 or 2", p->n_parts);
    if (p->n_slots > kMaxSlots) return api_fail(MOE_ERR_UNSUPPORTED, "n_slots %d > %d", p->n_slots, kMaxSlots);
    if (p->in_features > kMaxFeatures || p->out_features > kMaxFeatures)
        return api_fail(MOE_ERR_UNSUPPORTED, "more than %d features", kMaxFeatures);
    if (rows > INT32_MAX / 2) return api_fail(MOE_ERR_UNSUPPORTED, "too many rows");
    return MOE_OK;
}

int check_type(int type, const char* name) {
    if (type < MOE_OUT_BF16 || type > MOE_OUT_F32_ADD) return api_fail(MOE_ERR_INVALID_ARG, "%s %d is not a MOE_OUT_* value", name, type);
    return MOE_OK;
}

// Both parts of a pair of pointers, or the first alone.
int need_parts(const moe_project_t* p, const void* a, const void* b, const char* name, const char* name2) {
    int rc = api_need(a, name);
    if (rc) return rc;
    if (p->n_parts == 2) return api_need(b, name2);
    return b ? api_fail(MOE_ERR_INVALID_ARG, "%s is given, but n_parts is 1", name2) : MOE_OK;
}

Args make_args(const moe_project_t* p, int rows, const int32_t* offsets, const void* w, const void* w2) {
    Args a = {};
    a.R = rows;
    a.K = p->in_features;
    a.N = p->out_features;
    a.P = p->n_parts;
    a.S = p->n_slots;
    a.w[0] = static_cast<const uint16_t*>(w);
    a.w[1] = static_cast<const uint16_t*>(w2);
    a.offsets = offsets;
    return a;
}

int launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MOE_OK : api_fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_expert_project(const moe_project_t* project, int rows, const void* x, const int32_t* offsets, const void* w,
                       const void* w2, void* out, int out_type, void* stream) {
    int rc = check_project(project, rows);
    if (rc || (rc = check_type(out_type, "out_type"))) return rc;
    if (rows == 0) return MOE_OK;
    if ((rc = api_need(x, "x")) || (rc = api_need(offsets, "offsets", 4)) || (rc = need_parts(project, w, w2, "w", "w2")) ||
        (rc = api_need(out, "out")))
        return rc;
    PdlScope pdl(rows);
    Args a = make_args(project, rows, offsets, w, w2);
    if ((rc = api_device_status(&a.st))) return rc;
    a.rows_in = static_cast<const uint16_t*>(x);
    a.out[0] = out;
    a.type = out_type;
    return launched(launch_pdl(rows_kernel<false>, dim3((a.P * a.N + 63) / 64, (rows + 63) / 64 + a.S), dim3(256), 0,
                               reinterpret_cast<cudaStream_t>(stream), a),
                    "expert projection launch");
}

int moe_expert_project_backward(const moe_project_t* project, int rows, const void* dy, const void* x, const uint8_t* x8,
                                const float* x8_scale, const int32_t* offsets, const void* w, const void* w2, void* dx,
                                int dx_type, void* dw, void* dw2, int dw_type, void* stream) {
    int rc = check_project(project, rows);
    if (rc || (rc = check_type(dx_type, "dx_type")) || (rc = check_type(dw_type, "dw_type"))) return rc;
    if ((dw || dw2) && (rc = need_parts(project, dw, dw2, "dw", "dw2"))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        const size_t n = (size_t)project->n_slots * project->out_features * project->in_features;
        for (void* g : {dw, dw2})
            if (g && dw_type != MOE_OUT_F32_ADD)
                if ((rc = launched(cudaMemsetAsync(g, 0, n * (dw_type == MOE_OUT_BF16 ? 2 : 4), s), "memset dw"))) return rc;
        return MOE_OK;
    }
    if (!dx && !dw) return MOE_OK;
    if ((rc = api_need(dy, "dy")) || (rc = api_need(offsets, "offsets", 4))) return rc;
    if (dx && ((rc = api_need(dx, "dx")) || (rc = need_parts(project, w, w2, "w", "w2")))) return rc;
    if (dw) {
        if (!x == !x8) return api_fail(MOE_ERR_INVALID_ARG, "dw needs x or x8, and not both");
        if (x && (rc = api_need(x, "x"))) return rc;
        if (x8 && ((rc = api_need(x8, "x8")) || (rc = api_need(x8_scale, "x8_scale", 4)))) return rc;
        if (x8 && project->in_features % 16) return api_fail(MOE_ERR_INVALID_ARG, "x8 needs in_features %% 16 == 0");
    }
    PdlScope pdl(rows);
    Args a = make_args(project, rows, offsets, w, w2);
    if ((rc = api_device_status(&a.st))) return rc;
    a.rows_in = static_cast<const uint16_t*>(dy);
    a.x = static_cast<const uint16_t*>(x);
    a.x8 = x8;
    a.x8_scale = x8_scale;
    if (dx) {
        a.out[0] = dx;
        a.type = dx_type;
        if ((rc = launched(launch_pdl(rows_kernel<true>, dim3((a.K + 63) / 64, (rows + 63) / 64 + a.S), dim3(256), 0, s, a),
                           "expert gradient launch")))
            return rc;
    }
    if (!dw) return MOE_OK;
    a.out[0] = dw;
    a.out[1] = dw2;
    a.type = dw_type;
    return launched(launch_pdl(weights_kernel, dim3((a.K + 63) / 64, (a.N + 63) / 64 * a.P, a.S), dim3(256), 0, s, a),
                    "expert weight gradient launch");
}

}  // extern "C"

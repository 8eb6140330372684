// Activations kept in 8 bits for the backward pass, and SwiGLU with its gradient on them.
//
// Rows are cut into blocks of 128 columns (the last one shorter).  A block's scale is the least
// power of two, from 2^-117 to 2^119, that brings its largest finite value to 448 at most; a code is
// e4m3(x / scale), saturating (448 * 2^119 for the few values above it: 2^120 would round them to an
// infinity).  A power of two divides and multiplies without rounding, so the only error is
// the code's own (2^-4 of a value at most, above 2^-6 of the scale), and code * scale is a bf16
// number again: four significant bits, 2^-117 * 2^-9 the smallest.  The backward pass multiplies
// the very values that were kept.  (A scale of amax / 448 would gain under one bit of range, and
// its products would round a second time.)  Infinities and NaN are kept as NaN, which E4M3 has.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "operators.cuh"

namespace moe {
namespace {

constexpr int kBlock = MOE_PAYLOAD_BLOCK;
constexpr int kThreads = 256;
constexpr int kLanes = 16;                    // lanes that share a block, 8 columns each
constexpr int kGroups = kThreads / kLanes;    // blocks of a CTA side by side

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_two(float lo, float hi) { return pack_bf(__float_as_uint(lo), __float_as_uint(hi)); }

// |x| of two bf16, infinities and NaN as 0
__device__ __forceinline__ uint32_t finite_abs(uint32_t w) {
    w &= 0x7fff7fffu;
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

// infinities as NaN
__device__ __forceinline__ uint32_t no_inf(uint32_t w) {
    if ((w & 0x7fffu) == 0x7f80u) w |= 0x40u;
    if ((w & 0x7fff0000u) == 0x7f800000u) w |= 0x400000u;
    return w;
}

// The largest of 8 bf16 (no signs), as their bits in the lower half.
__device__ __forceinline__ uint32_t top8(uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    const uint32_t m = __vmaxu2(__vmaxu2(x, y), __vmaxu2(z, w));
    return max(m & 0xffffu, m >> 16);
}

// The exponent of a block's scale, from the bits of its largest value: 448 is 1.75 * 2^8.
__device__ __forceinline__ int exponent_of(uint32_t top) {
    return top ? min(max((int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0), -117), 119) : 0;
}

// The exponents of two blocks' scales, from 8 values of each in each of 16 lanes (the whole warp calls):
// their maxima go through the lanes together.  Values that are no numbers leave them, and become NaN.
__device__ __forceinline__ void block_exponents(uint4& v, uint4& w, int& ev, int& ew) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    auto reduce = [](uint32_t m) {
#pragma unroll
        for (int d = kLanes / 2; d > 0; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
        return m;
    };
    uint32_t m = reduce(top8(v.x & kAbs, v.y & kAbs, v.z & kAbs, v.w & kAbs) |
                        (top8(w.x & kAbs, w.y & kAbs, w.z & kAbs, w.w & kAbs) << 16));
    if (__any_sync(0xffffffffu, (m & 0xffffu) >= 0x7f80u || m >= 0x7f800000u)) {
        m = reduce(top8(finite_abs(v.x), finite_abs(v.y), finite_abs(v.z), finite_abs(v.w)) |
                   (top8(finite_abs(w.x), finite_abs(w.y), finite_abs(w.z), finite_abs(w.w)) << 16));
        v = make_uint4(no_inf(v.x), no_inf(v.y), no_inf(v.z), no_inf(v.w));
        w = make_uint4(no_inf(w.x), no_inf(w.y), no_inf(w.z), no_inf(w.w));
    }
    ev = exponent_of(m & 0xffffu);
    ew = exponent_of(m >> 16);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, float inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(lo_of(a) * inv, hi_of(a) * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(lo_of(b) * inv, hi_of(b) * inv), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xffffu) | (hi << 16);
}

__device__ __forceinline__ uint2 encode8(const uint4& v, int e) {
    const float inv = pow2(-e);
    return make_uint2(encode4(v.x, v.y, inv), encode4(v.z, v.w, inv));
}

__device__ __forceinline__ void decode8(uint2 c, float scale, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = (i < 2 ? c.x : c.y) >> (i & 1) * 16;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xffffu), __NV_E4M3);
        const float2 p = __half22float2(__half2(h));
        f[2 * i] = p.x * scale;
        f[2 * i + 1] = p.y * scale;
    }
}

// 1 / (1 + e^-g).  e^-g overflows below -88, where the result is 0 instead of e^g (under 2^-126).
// 1 - sigmoid is taken as a difference: what it loses (2^-24) counts beside 1 where it is used, times g,
// and is 0 from g = 17 on, where the sigmoid is 1.
__device__ __forceinline__ float sigmoid(float g) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// Block u of the CTA's, of `n` a row.  Its row without a division where there are few of them: below
// 4096, at < n + 64 and at * n < 2^32, for which the rounded-up reciprocal gives at / n exactly;
// above, at / n is 0 or 1.
struct Blocks {
    int n;
    uint32_t reciprocal;  // 2^32 / n + 1, 0 from 4096 on
};
struct Place {
    size_t row;
    int block;
};
constexpr int kMostUnits = 64;  // of a CTA
__device__ __forceinline__ Place place_of(uint32_t first, int u, Blocks b) {
    const uint32_t row0 = first / (uint32_t)b.n, at = first - row0 * b.n + u;
    const uint32_t q = b.reciprocal ? (b.n == 1 ? at : __umulhi(at, b.reciprocal)) : at >= (uint32_t)b.n;
    return {(size_t)row0 + q, (int)(at - q * b.n)};
}

// EVEN: rows are whole blocks, which then follow one another whatever the row.
template <int U, bool EVEN>  // U: blocks of a group of lanes
__global__ void __launch_bounds__(kThreads) keep_kernel(const uint16_t* __restrict__ x, size_t rows, int cols, Blocks blocks,
                                                        uint8_t* __restrict__ codes, float* __restrict__ scale) {
    pdl_begin();
    const uint32_t first = blockIdx.x * (kGroups * U);
    const size_t total = rows * blocks.n;
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    uint4 v[U];
    size_t at[U];  // of the lane's columns; ~0: none
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const size_t b = (size_t)first + i * kGroups + group;
        if (EVEN) {
            at[i] = b < total ? b * kBlock + lane * 8 : ~size_t(0);
        } else {
            const Place p = place_of(first, i * kGroups + group, blocks);
            const int c = p.block * kBlock + lane * 8;
            at[i] = b < total && c < cols ? p.row * cols + c : ~size_t(0);
        }
        v[i] = make_uint4(0, 0, 0, 0);
        if (at[i] != ~size_t(0)) v[i] = __ldcs(reinterpret_cast<const uint4*>(x + at[i]));
    }
    static_assert(U % 2 == 0, "blocks in pairs");
    int e[U];
#pragma unroll
    for (int i = 0; i < U; i += 2) block_exponents(v[i], v[i + 1], e[i], e[i + 1]);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (at[i] != ~size_t(0)) *reinterpret_cast<uint2*>(codes + at[i]) = encode8(v[i], e[i]);
        if (lane == 0 && at[i] != ~size_t(0)) scale[(size_t)first + i * kGroups + group] = pow2(e[i]);
    }
}

// Where a lane's gate lies in gate_up and codes (the up `inter` further on), and in h; ~0: none.
struct GatePlace {
    size_t gate, h, scale;
};
__device__ __forceinline__ GatePlace gate_place(uint32_t first, int u, int lane, size_t rows, int inter, Blocks blocks) {
    const Place p = place_of(first, u, blocks);
    const int c = p.block * kBlock + lane * 8;
    if (p.row >= rows || c >= inter) return {~size_t(0), 0, 0};
    return {p.row * 2 * inter + c, p.row * inter + c, p.row * 2 * blocks.n + p.block};
}

// One block of gate and of up for 16 lanes: with two (90 us of 32768 rows of 2048 for the forward pass,
// 84 with one) their registers leave fewer warps to wait with.
__global__ void __launch_bounds__(kThreads) swiglu_keep_kernel(const uint16_t* __restrict__ gate_up, size_t rows, int inter,
                                                               Blocks blocks, uint16_t* __restrict__ h,
                                                               uint8_t* __restrict__ codes, float* __restrict__ scale) {
    pdl_begin();
    const int lane = threadIdx.x % kLanes;
    const GatePlace p = gate_place(blockIdx.x * kGroups, threadIdx.x / kLanes, lane, rows, inter, blocks);
    const bool live = p.gate != ~size_t(0);
    uint4 g = make_uint4(0, 0, 0, 0), u = g;
    if (live) {
        g = __ldcs(reinterpret_cast<const uint4*>(gate_up + p.gate));
        u = __ldcs(reinterpret_cast<const uint4*>(gate_up + p.gate + inter));
    }
    uint32_t out[4];
    const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = lo_of(gw[j]), b = hi_of(gw[j]);
        out[j] = pack_two(a * sigmoid(a) * lo_of(uw[j]), b * sigmoid(b) * hi_of(uw[j]));
    }
    int eg, eu;
    block_exponents(g, u, eg, eu);
    if (!live) return;
    *reinterpret_cast<uint4*>(h + p.h) = make_uint4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<uint2*>(codes + p.gate) = encode8(g, eg);
    *reinterpret_cast<uint2*>(codes + p.gate + inter) = encode8(u, eu);
    if (lane == 0) {
        scale[p.scale] = pow2(eg);
        scale[p.scale + blocks.n] = pow2(eu);
    }
}

__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(const uint8_t* __restrict__ codes,
                                                                   const float* __restrict__ scale,
                                                                   const uint16_t* __restrict__ dh, size_t rows, int inter,
                                                                   Blocks blocks, uint16_t* __restrict__ d_gate_up,
                                                                   uint16_t* __restrict__ h) {
    pdl_begin();
    const GatePlace p = gate_place(blockIdx.x * kGroups, threadIdx.x / kLanes, threadIdx.x % kLanes, rows, inter, blocks);
    if (p.gate == ~size_t(0)) return;
    const uint2 cg = __ldcs(reinterpret_cast<const uint2*>(codes + p.gate));
    const uint2 cu = __ldcs(reinterpret_cast<const uint2*>(codes + p.gate + inter));
    const uint4 d = __ldcs(reinterpret_cast<const uint4*>(dh + p.h));
    float g[8], u[8], act[8], dg[8], du[8];
    decode8(cg, __ldg(scale + p.scale), g);
    decode8(cu, __ldg(scale + p.scale + blocks.n), u);
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float up = j & 1 ? hi_of(dw[j >> 1]) : lo_of(dw[j >> 1]);
        const float s = sigmoid(g[j]), silu = g[j] * s;
        act[j] = silu * u[j];
        du[j] = up * silu;
        // (u times what is 1.1 at most stays below fp32's largest, as a kept u is 448 * 2^119 at most: no product
        // overflows but the result's own)
        dg[j] = up * (u[j] * (s * fmaf(g[j], 1.0f - s, 1.0f)));
    }
    uint16_t* out = d_gate_up + p.gate;
    *reinterpret_cast<uint4*>(out) =
        make_uint4(pack_two(dg[0], dg[1]), pack_two(dg[2], dg[3]), pack_two(dg[4], dg[5]), pack_two(dg[6], dg[7]));
    *reinterpret_cast<uint4*>(out + inter) =
        make_uint4(pack_two(du[0], du[1]), pack_two(du[2], du[3]), pack_two(du[4], du[5]), pack_two(du[6], du[7]));
    if (h)
        *reinterpret_cast<uint4*>(h + p.h) =
            make_uint4(pack_two(act[0], act[1]), pack_two(act[2], act[3]), pack_two(act[4], act[5]), pack_two(act[6], act[7]));
}

int check_rows(int rows, int cols, const char* name) {
    if (rows < 0 || cols <= 0 || cols % 8) return api_fail(MOE_ERR_INVALID_ARG, "rows >= 0 and %s > 0, a multiple of 8, required", name);
    if (cols > 1 << 24) return api_fail(MOE_ERR_UNSUPPORTED, "%s %d > %d", name, cols, 1 << 24);
    // (block numbers are of 32 bits: more of them than that are rows of 500 GB at least)
    if ((long long)rows * ((cols + kBlock - 1) / kBlock) >= UINT32_MAX - kMostUnits) return api_fail(MOE_ERR_UNSUPPORTED, "too many rows");
    return MOE_OK;
}

Blocks blocks_of(int cols) {
    const int n = (cols + kBlock - 1) / kBlock;
    return {n, n < 4096 ? (uint32_t)((1ull << 32) / n + 1) : 0u};
}

template <int U>
dim3 grid_of(int rows, Blocks blocks) {
    static_assert(kGroups * U <= kMostUnits, "place_of's bound");
    return dim3((unsigned)(((size_t)rows * blocks.n + kGroups * U - 1) / (kGroups * U)));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_checkpoint_rows(int rows, int cols, const void* x, uint8_t* codes, float* scale, void* stream) {
    int rc = check_rows(rows, cols, "cols");
    if (rc || rows == 0) return rc;
    if ((rc = api_need(x, "x")) || (rc = api_need(codes, "codes")) || (rc = api_need(scale, "scale", 4))) return rc;
    PdlScope pdl(rows);
    const Blocks blocks = blocks_of(cols);
    return launched(launch_pdl(cols % kBlock ? keep_kernel<4, false> : keep_kernel<4, true>, grid_of<4>(rows, blocks),
                               dim3(kThreads), 0, reinterpret_cast<cudaStream_t>(stream), static_cast<const uint16_t*>(x),
                               (size_t)rows, cols, blocks, codes, scale),
                    "checkpoint launch");
}

int moe_swiglu_checkpoint(int rows, int inter, const void* gate_up, void* h, uint8_t* codes, float* scale, void* stream) {
    int rc = check_rows(rows, inter, "inter");
    if (rc || rows == 0) return rc;
    if ((rc = api_need(gate_up, "gate_up")) || (rc = api_need(h, "h")) || (rc = api_need(codes, "codes")) ||
        (rc = api_need(scale, "scale", 4)))
        return rc;
    PdlScope pdl(rows);
    const Blocks blocks = blocks_of(inter);
    return launched(launch_pdl(swiglu_keep_kernel, grid_of<1>(rows, blocks), dim3(kThreads), 0,
                               reinterpret_cast<cudaStream_t>(stream), static_cast<const uint16_t*>(gate_up), (size_t)rows, inter,
                               blocks, static_cast<uint16_t*>(h), codes, scale),
                    "SwiGLU launch");
}

int moe_swiglu_backward(int rows, int inter, const uint8_t* codes, const float* scale, const void* dh, void* d_gate_up, void* h,
                        void* stream) {
    int rc = check_rows(rows, inter, "inter");
    if (rc || rows == 0) return rc;
    if ((rc = api_need(codes, "codes")) || (rc = api_need(scale, "scale", 4)) || (rc = api_need(dh, "dh")) ||
        (rc = api_need(d_gate_up, "d_gate_up")))
        return rc;
    if (h && (rc = api_need(h, "h"))) return rc;
    PdlScope pdl(rows);
    const Blocks blocks = blocks_of(inter);
    return launched(launch_pdl(swiglu_backward_kernel, grid_of<1>(rows, blocks), dim3(kThreads), 0,
                               reinterpret_cast<cudaStream_t>(stream), codes, scale, static_cast<const uint16_t*>(dh), (size_t)rows,
                               inter, blocks, static_cast<uint16_t*>(d_gate_up), static_cast<uint16_t*>(h)),
                    "SwiGLU gradient launch");
}

}  // extern "C"

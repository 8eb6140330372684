// Low-rank adapters of many requests beside a shared projection:
//   v_t = s_i A_i x_t,  y_t = W x_t + B_i v_t   (i = adapter of token t),
// and the gradients of x, A and B (W is frozen):
//   dv_t = s_i B_i^T dy_t,  dx_t = W^T dy_t + A_i^T dv_t,
//   dA_i = sum dv_t x_t^T,  dB_i = sum dy_t v_t^T.
//
// The projection is a swap-AB tcgen05 GEMM (weight rows are the 128-row UMMA A
// operand, tokens the N operand).  The adapters ride along as extra K chunks of
// the same accumulator: for each adapter i among the tile's tokens and each 64
// of its rank, the A operand is the tile's rows of B_i (TMA) and the B operand
// the tile's v with the rows of other adapters set to zero, written to shared
// memory by the kernel itself.  One pass over W, one rounding of y, and tokens
// in any order.  The backward projection is the same kernel with W and A_i read
// MN-major (the contraction runs over their rows).
#include <algorithm>

#include "kernels.h"

namespace moe {
namespace {

constexpr int kMaxAdapters = 4096;
constexpr int kMaxRank = 256;
constexpr int kMaxExtra = 256 * (kMaxRank / 64);  // adapter chunks of one tile
constexpr int kThreads = 192;  // TMA warp, MMA warp, four warps that write v chunks and drain the accumulator
constexpr int kABytes = 128 * 64 * 2;

__device__ __forceinline__ float bf(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }

__device__ __forceinline__ uint16_t to_bf(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// Two bf16 in a word: is either an infinity or NaN; the word with such elements zero.
__device__ __forceinline__ bool not_finite(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

struct ProjArgs {
    CUtensorMap w;      // forward: box {64 k, 128 n} of W [N][K]; backward: box {64 k, 64 n}
    CUtensorMap lr;     // forward: box {64 r, 128 n} of B [n][N][r]; backward: box {64 k, 64 r} of A [n][r][K]
    CUtensorMap x;      // tokens: box {64, 1, BN} of x [T][K] | dy [T][N]
    const int32_t* adapter_of;
    const uint16_t* v;  // [T][r] v | dv
    const uint16_t* lr_ptr;  // what `lr` maps
    int T, O, C, r, n_adapters;  // O output features, C contracted features
    void* out;          // [T][O]
    int out_fp32;
    DevStatus st;
};

template <int BN>
struct ProjCfg {
    static constexpr int kStageBytes = kABytes + BN * 128;
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 8;
    static constexpr int kTmemCols = BN < 32 ? 32 : BN;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 256 + BN * 8 + kMaxAdapters / 8 + kMaxExtra / 8;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory overflow");
};

// The tile's adapter ids (-1: none) and the list of distinct ones, ascending; returns
// their number.  All threads call it; `bits` holds kMaxAdapters bits.
__device__ __forceinline__ int tile_adapters(const int32_t* adapter_of, int row0, int rows, int n_adapters, int bn,
                                             int* ids, int* list, uint32_t* bits, int* count, const DevStatus& st) {
    const int words = (n_adapters + 31) / 32;
    for (int i = threadIdx.x; i < words; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < bn; i += blockDim.x) {
        int id = -1;
        if (i < rows) {
            id = adapter_of[row0 + i];
            if (id < -1 || id >= n_adapters) {
                raise_status(st, kStatusInvalidExpert);
                id = -1;
            }
        }
        ids[i] = id;
        if (id >= 0) atomicOr(&bits[id >> 5], 1u << (id & 31));
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int base = 0;
        for (int w0 = 0; w0 < words; w0 += 32) {
            const int w = w0 + threadIdx.x;
            uint32_t b = w < words ? bits[w] : 0;
            int incl = __popc(b);
            const int mine = incl;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if ((int)threadIdx.x >= d) incl += o;
            }
            int at = base + incl - mine;
            while (b) {
                list[at++] = w * 32 + __ffs(b) - 1;
                b &= b - 1;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (threadIdx.x == 0) *count = base;
    }
    __syncthreads();
    return *count;
}

template <bool BWD, int BN>
__global__ void __launch_bounds__(kThreads, 1) project_kernel(const __grid_constant__ ProjArgs a) {
    using C = ProjCfg<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
    uint64_t* empty = full + C::kStages;
    uint64_t* landed = empty + C::kStages;  // the adapter tile of a stage, before the v writers are done with it
    uint64_t* done = landed + C::kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* count = reinterpret_cast<int*>(tmem_slot + 2);
    int* ids = reinterpret_cast<int*>(smem + C::kStages * C::kStageBytes + 256);
    int* list = ids + BN;
    uint32_t* bits = reinterpret_cast<uint32_t*>(list + BN);
    uint32_t* odd = bits + kMaxAdapters / 32;  // adapter chunks with an infinity or NaN in this tile

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int m0 = blockIdx.x * 128;
    const int row0 = blockIdx.y * BN;
    const int rows = min(BN, a.T - row0);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < kMaxExtra / 32; i += kThreads) odd[i] = 0;
    pdl_begin();
    tc_fence_before();
    const int n_list =
        tile_adapters(a.adapter_of, row0, rows, a.n_adapters, BN, ids, list, bits, count, a.st);  // syncs the CTA
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const int kc = (a.C + 63) / 64, rc = (a.r + 63) / 64;
    const int total = kc + n_list * rc;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            bool ok = true;
            int armed = 0;
            for (int c = 0; c < total; ++c) {
                const int s = c % C::kStages;
                const uint32_t ph = (c / C::kStages) & 1;
                if (*abort_flag || !mbar_wait(smem_u32(&empty[s]), ph ^ 1, limit)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = smem_u32(smem + s * C::kStageBytes), fb = smem_u32(&full[s]);
                if (c < kc) {
                    mbar_arrive_expect_tx(fb, C::kStageBytes);
                    if (BWD) {
                        tma_load_3d(sa, &a.w, fb, m0, c * 64, 0, pol);
                        tma_load_3d(sa + kABytes / 2, &a.w, fb, m0 + 64, c * 64, 0, pol);
                    } else {
                        tma_load_3d(sa, &a.w, fb, c * 64, m0, 0, pol);
                    }
                    tma_load_3d(sa + kABytes, &a.x, fb, c * 64, 0, row0, pol);
                } else {
                    const int i = list[(c - kc) / rc], j0 = ((c - kc) % rc) * 64;
                    const uint32_t lb = smem_u32(&landed[s]);
                    mbar_arrive_expect_tx(lb, kABytes);
                    if (BWD) {
                        tma_load_3d(sa, &a.lr, lb, m0, j0, i, pol);
                        tma_load_3d(sa + kABytes / 2, &a.lr, lb, m0 + 64, j0, i, pol);
                    } else {
                        tma_load_3d(sa, &a.lr, lb, j0, m0, i, pol);
                    }
                }
                armed = c + 1;
            }
            if (!ok) {
                *abort_flag = 1;
                raise_status(a.st, kStatusWaitTimeout);
            }
            // every copy has landed before the CTA exits
            for (int c = armed > C::kStages ? armed - C::kStages : 0; c < armed; ++c) {
                if (c < kc) mbar_wait(smem_u32(&full[c % C::kStages]), (c / C::kStages) & 1, limit);
                else mbar_wait(smem_u32(&landed[c % C::kStages]), ((c - kc) / C::kStages) & 1, limit);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(128, BN) | (BWD ? kIdescAMnMajor : 0u);
            bool ok = true;
            for (int c = 0; c < total; ++c) {
                const int s = c % C::kStages;
                if (*abort_flag || !mbar_wait(smem_u32(&full[s]), (c / C::kStages) & 1, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * C::kStageBytes);
                const uint64_t ad = BWD ? umma_desc_mn_sw128(sa, kABytes / 2) : umma_desc_sw128(sa);
                const uint64_t bd = umma_desc_sw128(sa + kABytes);
                const int left = c < kc ? a.C - c * 64 : a.r - ((c - kc) % rc) * 64;
                const int steps = min(4, (left + 15) >> 4);
                for (int k = 0; k < steps; ++k)  // 16 of the contraction: 32 bytes along K, or 16 K rows
                    umma_bf16(tbase, ad + (BWD ? 128 : 2) * k, bd + 2 * k, idesc, c > 0 || k > 0);
                umma_commit(smem_u32(&empty[s]));
            }
            if (!ok) {
                *abort_flag = 1;
                raise_status(a.st, kStatusWaitTimeout);
            }
            umma_commit(smem_u32(done));
            mbar_wait(smem_u32(done), 0, limit);
        }
    } else {
        const int tid = threadIdx.x - 64;  // 0..127
        bool ok = true;
        for (int c = kc; c < total; ++c) {
            const int e = c - kc, s = c % C::kStages;
            const int i = list[e / rc], j0 = (e % rc) * 64;
            // the adapter tile has landed: the stage is free of its last use, too
            if (*abort_flag || !mbar_wait(smem_u32(&landed[s]), (e / C::kStages) & 1, limit)) {
                ok = false;
                break;
            }
            uint8_t* st_a = smem + s * C::kStageBytes;
            uint8_t* sb = st_a + kABytes;
            // v of this adapter's tokens, zeros elsewhere
            for (int q = tid; q < BN * 8; q += 128) {
                const int row = q >> 3, seg = q & 7;
                uint4 val = make_uint4(0, 0, 0, 0);
                if (ids[row] == i && j0 + seg * 8 < a.r)
                    val = *reinterpret_cast<const uint4*>(a.v + (size_t)(row0 + row) * a.r + j0 + seg * 8);
                *reinterpret_cast<uint4*>(sb + row * 128 + ((seg ^ (row & 7)) << 4)) = val;
            }
            // Zero times an infinity or NaN of this adapter would reach the other adapters'
            // tokens: such elements leave the tile here and are added to their own
            // tokens in the epilogue.
            bool hit = false;
            for (int q = tid; q < kABytes / 16; q += 128) {
                uint4* at = reinterpret_cast<uint4*>(st_a) + q;
                uint4 val = *at;
                if (not_finite(val.x) | not_finite(val.y) | not_finite(val.z) | not_finite(val.w)) {
                    val.x = finite_part(val.x);
                    val.y = finite_part(val.y);
                    val.z = finite_part(val.z);
                    val.w = finite_part(val.w);
                    *at = val;
                    hit = true;
                }
            }
            if (hit) atomicOr(&odd[e >> 5], 1u << (e & 31));
            fence_async_smem();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (tid == 0) mbar_arrive(smem_u32(&full[s]));
        }
        if (!ok) {
            *abort_flag = 1;
            raise_status(a.st, kStatusWaitTimeout);
        }
        if (ok) ok = mbar_wait(smem_u32(done), 0, limit) && !*abort_flag;
        if (ok) {
            tc_fence_after();
            const int q = warp & 3;
            const int row = m0 + q * 32 + lane;
            const uint32_t tl = tbase + ((uint32_t)(q * 32) << 16);
            // the infinities and NaN that were taken out of the adapter tiles
            auto add_odd = [&](int g, float (&y)[16]) {
                for (int w = 0; w * 32 < total - kc; ++w) {
                    for (uint32_t b = odd[w]; b; b &= b - 1) {
                        const int e = w * 32 + __ffs(b) - 1;
                        const int i = list[e / rc], j0 = (e % rc) * 64;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (ids[g * 16 + j] != i) continue;
                            for (int l = j0; l < min(a.r, j0 + 64); ++l) {
                                const size_t at = BWD ? ((size_t)i * a.r + l) * a.O + row : ((size_t)i * a.O + row) * a.r + l;
                                const float u = bf(a.lr_ptr[at]);
                                if (!isfinite(u)) y[j] += u * bf(a.v[(size_t)(row0 + g * 16 + j) * a.r + l]);
                            }
                        }
                    }
                }
            };
            for (int g = 0; g * 16 < rows; ++g) {
                float v[16];
                tmem_ld16(tl + g * 16, v);
                tmem_ld_wait();
                if (row < a.O) add_odd(g, v);
                if (row >= a.O) {
                } else if (a.out_fp32) {
                    float* dst = reinterpret_cast<float*>(a.out) + row;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (g * 16 + j < rows) dst[(size_t)(row0 + g * 16 + j) * a.O] = v[j];
                } else {
                    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(a.out) + row;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (g * 16 + j < rows) dst[(size_t)(row0 + g * 16 + j) * a.O] = __float2bfloat16_rn(v[j]);
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, C::kTmemCols);
}

// The token's adapter, or -1.
__device__ __forceinline__ int adapter_id(const int32_t* adapter_of, int t, int n_adapters, const DevStatus& st) {
    const int id = adapter_of[t];
    if (id >= -1 && id < n_adapters) return id;
    raise_status(st, kStatusInvalidExpert);
    return -1;
}

// v[t][j] = s_i A_i[j] . x[t]: one warp per (token, j).
__global__ void __launch_bounds__(256) shrink_kernel(const uint16_t* x, const uint16_t* m, const float* scaling,
                                                     const int32_t* adapter_of, int T, int C, int r, int n_adapters,
                                                     uint16_t* v, DevStatus st) {
    pdl_begin();
    const int lane = threadIdx.x & 31;
    for (long w = (long)blockIdx.x * 8 + (threadIdx.x >> 5); w < (long)T * r; w += (long)gridDim.x * 8) {
        const int t = (int)(w / r), j = (int)(w % r);
        const int i = adapter_id(adapter_of, t, n_adapters, st);
        float sum = 0.0f;
        if (i >= 0) {
            const uint16_t* row = m + ((size_t)i * r + j) * C;
            for (int k = lane; k < C; k += 32) sum += bf(x[(size_t)t * C + k]) * bf(row[k]);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == 0) v[(size_t)t * r + j] = to_bf(i >= 0 ? sum * (scaling ? scaling[i] : 1.0f) : 0.0f);
    }
}

// dv[t][j] = s_i sum_n dy[t][n] B_i[n][j]: one CTA per token, a thread per j.
__global__ void __launch_bounds__(256) shrink_back_kernel(const uint16_t* dy, const uint16_t* b, const float* scaling,
                                                          const int32_t* adapter_of, int T, int N, int r,
                                                          int n_adapters, uint16_t* dv, DevStatus st) {
    pdl_begin();
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        const int i = adapter_id(adapter_of, t, n_adapters, st);
        for (int j = threadIdx.x; j < r; j += blockDim.x) {
            float sum = 0.0f;
            if (i >= 0)
                for (int n = 0; n < N; ++n) sum += bf(dy[(size_t)t * N + n]) * bf(b[((size_t)i * N + n) * r + j]);
            dv[(size_t)t * r + j] = to_bf(i >= 0 ? sum * (scaling ? scaling[i] : 1.0f) : 0.0f);
        }
    }
}

// da_i[j][k] = sum over i's tokens of u[t][j] z[t][k] (transposed: db_i[k][j]).
__global__ void __launch_bounds__(256) grad_kernel(const uint16_t* u, const uint16_t* z, const int32_t* adapter_of, int T,
                                                   int C, int r, int n_adapters, int transposed, uint16_t* out) {
    pdl_begin();
    const int k = blockIdx.x * 256 + threadIdx.x;
    const int j = blockIdx.y, i = blockIdx.z;
    if (k >= C) return;
    float sum = 0.0f;
    for (int t = 0; t < T; ++t)
        if (adapter_of[t] == i) sum += bf(u[(size_t)t * r + j]) * bf(z[(size_t)t * C + k]);
    if (transposed) out[((size_t)i * C + k) * r + j] = to_bf(sum);
    else out[((size_t)i * r + j) * C + k] = to_bf(sum);
}

int check_adapter(const moe_adapter_t* p, int T) {
    if (!p) return api_fail(MOE_ERR_INVALID_ARG, "adapter is NULL");
    if (T < 0) return api_fail(MOE_ERR_INVALID_ARG, "T = %d < 0", T);
    if (p->in_features <= 0 || p->out_features <= 0 || p->n_adapters <= 0 || p->rank <= 0)
        return api_fail(MOE_ERR_INVALID_ARG, "non-positive adapter field");
    if (p->in_features % 8 || p->out_features % 8 || p->rank % 8)
        return api_fail(MOE_ERR_INVALID_ARG, "in_features, out_features and rank must be multiples of 8");
    if (p->rank > kMaxRank) return api_fail(MOE_ERR_UNSUPPORTED, "rank %d > %d", p->rank, kMaxRank);
    if (p->n_adapters > kMaxAdapters)
        return api_fail(MOE_ERR_UNSUPPORTED, "n_adapters %d > %d", p->n_adapters, kMaxAdapters);
    return MOE_OK;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

size_t workspace(const moe_adapter_t* p, int T) { return align256((size_t)T * p->rank * 2); }

int check_ws(const moe_adapter_t* p, int T, const void* ws, size_t ws_bytes) {
    const size_t need = workspace(p, T);
    if (!ws || ws_bytes < need)
        return api_fail(MOE_ERR_WORKSPACE, "adapter workspace %zu < %zu bytes", ws_bytes, need);
    return api_need(ws, "workspace");
}

template <bool BWD, int BN>
cudaError_t launch_project_bn(const ProjArgs& a, cudaStream_t stream) {
    auto kern = project_kernel<BWD, BN>;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = configure_once(configured, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ProjCfg<BN>::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3((a.O + 127) / 128, (a.T + BN - 1) / BN), dim3(kThreads), ProjCfg<BN>::kSmemBytes,
                      stream, a);
}

// tokens [T][C] times W (and each token's low-rank matrix times v) into out [T][O]
template <bool BWD>
int project(const moe_adapter_t* p, int T, const void* tokens, const void* w, const void* lr, const int32_t* adapter_of,
            const void* v, void* out, int out_fp32, const DevStatus& st, cudaStream_t stream) {
    const int bn = T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
    const uint64_t K = p->in_features, N = p->out_features, r = p->rank, n = p->n_adapters;
    ProjArgs a;
    a.T = T;
    a.O = BWD ? p->in_features : p->out_features;
    a.C = BWD ? p->out_features : p->in_features;
    a.r = p->rank;
    a.n_adapters = p->n_adapters;
    int rc = make_tmap_3d(&a.w, w, K, N, 1, K * 2, K * N * 2, 64, BWD ? 64 : 128, 1);
    if (rc) return rc;
    if (BWD) rc = make_tmap_3d(&a.lr, lr, K, r, n, K * 2, K * r * 2, 64, 64, 1);
    else rc = make_tmap_3d(&a.lr, lr, r, N, n, r * 2, r * N * 2, 64, 128, 1);
    if (rc) return rc;
    const uint64_t C = a.C;
    if ((rc = make_tmap_3d(&a.x, tokens, C, 1, (uint64_t)T, C * 2, C * 2, 64, 1, bn))) return rc;
    a.lr_ptr = static_cast<const uint16_t*>(lr);
    a.adapter_of = adapter_of;
    a.v = static_cast<const uint16_t*>(v);
    a.out = out;
    a.out_fp32 = out_fp32;
    a.st = st;
    const cudaError_t e = bn == 32 ? launch_project_bn<BWD, 32>(a, stream) : bn == 64 ? launch_project_bn<BWD, 64>(a, stream)
                          : bn == 128 ? launch_project_bn<BWD, 128>(a, stream) : launch_project_bn<BWD, 256>(a, stream);
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "adapter projection launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

#define ADAPTER_CUDA(call, what)                                                                          \
    do {                                                                                                  \
        const cudaError_t e_ = (call);                                                                    \
        if (e_ != cudaSuccess) return api_fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e_));     \
    } while (0)

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adapter_workspace_size(const moe_adapter_t* adapter, int T) {
    return check_adapter(adapter, T) ? 0 : workspace(adapter, T);
}

int moe_adapter_project(const moe_adapter_t* adapter, int T, const void* x, const void* w, const void* a, const void* b,
                        const float* scaling, const int32_t* adapter_of, void* out, int out_fp32, void* v_out, void* ws,
                        size_t ws_bytes, void* stream) {
    int rc = check_adapter(adapter, T);
    if (rc) return rc;
    if (out_fp32 != 0 && out_fp32 != 1) return api_fail(MOE_ERR_INVALID_ARG, "out_fp32 %d is not 0 or 1", out_fp32);
    if (T == 0) return MOE_OK;
    PdlScope pdl(T);
    if ((rc = api_need(x, "x")) || (rc = api_need(w, "w")) || (rc = api_need(a, "a")) || (rc = api_need(b, "b")) ||
        (rc = api_need(adapter_of, "adapter_of", 4)) || (rc = api_need(out, "out")) ||
        (rc = check_ws(adapter, T, ws, ws_bytes)))
        return rc;
    if (scaling && (rc = api_need(scaling, "scaling", 4))) return rc;
    if (v_out && (rc = api_need(v_out, "v_out"))) return rc;
    DevStatus st;
    if ((rc = api_device_status(&st))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint16_t* v = static_cast<uint16_t*>(v_out ? v_out : ws);
    const long warps = (long)T * adapter->rank;
    ADAPTER_CUDA(launch_pdl(shrink_kernel, dim3((unsigned)std::min<long>((warps + 7) / 8, num_sms() * 8L)), dim3(256), 0,
                            s, static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(a), scaling, adapter_of, T,
                            adapter->in_features, adapter->rank, adapter->n_adapters, v, st),
                 "adapter shrink launch");
    return project<false>(adapter, T, x, w, b, adapter_of, v, out, out_fp32, st, s);
}

int moe_adapter_project_backward(const moe_adapter_t* adapter, int T, const void* dy, const void* x, const void* w,
                                 const void* a, const void* b, const float* scaling, const int32_t* adapter_of,
                                 const void* v, void* dx, void* da, void* db, void* ws, size_t ws_bytes, void* stream) {
    int rc = check_adapter(adapter, T);
    if (rc) return rc;
    if (!da != !db) return api_fail(MOE_ERR_INVALID_ARG, "da and db are given together or not at all");
    if (da && ((rc = api_need(da, "da")) || (rc = api_need(db, "db")))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int K = adapter->in_features, N = adapter->out_features, r = adapter->rank, n = adapter->n_adapters;
    if (T == 0) {
        if (da) {
            ADAPTER_CUDA(cudaMemsetAsync(da, 0, (size_t)n * r * K * 2, s), "memset da");
            ADAPTER_CUDA(cudaMemsetAsync(db, 0, (size_t)n * r * N * 2, s), "memset db");
        }
        return MOE_OK;
    }
    PdlScope pdl(T);
    if ((rc = api_need(dy, "dy")) || (rc = api_need(b, "b")) || (rc = api_need(adapter_of, "adapter_of", 4)) ||
        (rc = check_ws(adapter, T, ws, ws_bytes)))
        return rc;
    if (scaling && (rc = api_need(scaling, "scaling", 4))) return rc;
    if (dx && ((rc = api_need(dx, "dx")) || (rc = api_need(w, "w")) || (rc = api_need(a, "a")))) return rc;
    if (da && ((rc = api_need(x, "x")) || (rc = api_need(v, "v")))) return rc;
    if (!dx && !da) return MOE_OK;
    DevStatus st;
    if ((rc = api_device_status(&st))) return rc;
    uint16_t* dv = static_cast<uint16_t*>(ws);
    ADAPTER_CUDA(launch_pdl(shrink_back_kernel, dim3(std::min(T, num_sms() * 8)), dim3(256), 0, s,
                            static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(b), scaling, adapter_of, T, N, r,
                            n, dv, st),
                 "adapter backward shrink launch");
    if (dx && (rc = project<true>(adapter, T, dy, w, a, adapter_of, dv, dx, 0, st, s))) return rc;
    if (da) {
        ADAPTER_CUDA(launch_pdl(grad_kernel, dim3((K + 255) / 256, r, n), dim3(256), 0, s, (const uint16_t*)dv,
                                static_cast<const uint16_t*>(x), adapter_of, T, K, r, n, 0, static_cast<uint16_t*>(da)),
                     "adapter gradient launch");
        ADAPTER_CUDA(launch_pdl(grad_kernel, dim3((N + 255) / 256, r, n), dim3(256), 0, s, static_cast<const uint16_t*>(v),
                                static_cast<const uint16_t*>(dy), adapter_of, T, N, r, n, 1, static_cast<uint16_t*>(db)),
                     "adapter gradient launch");
    }
    return MOE_OK;
}

}  // extern "C"

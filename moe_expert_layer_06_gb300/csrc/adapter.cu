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
constexpr int kMaxTile = 256;                          // tokens of a tile (the UMMA N limit)
constexpr int kMaxExtra = kMaxTile * (kMaxRank / 64);  // adapter chunks of one tile
constexpr int kABytes = 128 * 64 * 2;
constexpr int kThreads = 320;  // TMA warp, MMA warp, four warps that write v chunks, four that drain accumulators

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

__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// fp32 at the same shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ float ld_peer(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// The tile's adapter ids (-1: none) and the list of distinct ones, ascending; *count
// their number.  `n_threads` threads call it (tid 0..), synchronised by barrier `bar`;
// `bits` holds kMaxAdapters bits.
__device__ __forceinline__ void tile_adapters(const int32_t* adapter_of, int row0, int rows, int n_adapters, int bn,
                                              int* ids, int* list, uint32_t* bits, int* count, const DevStatus& st,
                                              int tid, int n_threads, int bar) {
    const int words = (n_adapters + 31) / 32;
    for (int i = tid; i < words; i += n_threads) bits[i] = 0;
    named_sync(bar, n_threads);
    for (int i = tid; i < bn; i += n_threads) {
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
    named_sync(bar, n_threads);
    if (tid < 32) {
        int base = 0;
        for (int w0 = 0; w0 < words; w0 += 32) {
            const int w = w0 + tid;
            uint32_t b = w < words ? bits[w] : 0;
            int incl = __popc(b);
            const int mine = incl;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, d);
                if (tid >= d) incl += o;
            }
            int at = base + incl - mine;
            while (b) {
                list[at++] = w * 32 + __ffs(b) - 1;
                b &= b - 1;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (tid == 0) *count = base;
    }
    named_sync(bar, n_threads);
}

struct ProjArgs {
    CUtensorMap w;      // forward: box {64 k, 128 n} of W [N][K]; backward: box {64 k, 64 n}
    CUtensorMap lr;     // forward: box {64 r, 128 n} of B [n][N][r]; backward: box {64 k, 64 r} of A [n][r][K]
    CUtensorMap x;      // tokens: box {64, 1, bn} of x [T][K] | dy [T][N]
    const int32_t* adapter_of;
    const uint16_t* v;  // [T][r] v | dv
    const uint16_t* lr_ptr;  // what `lr` maps
    int T, O, C, r, n_adapters;  // O output features, C contracted features
    int bn;             // tokens of a tile (a multiple of 16)
    int splits;         // CTAs of a cluster that share one tile's contraction
    void* out;          // [T][O]
    int out_fp32;
    DevStatus st;
};

// What a tile's workers know of its adapters.
struct TileList {
    int count;
    int ids[kMaxTile];   // adapter of each token
    int list[kMaxTile];  // distinct adapters
    uint32_t odd[kMaxExtra / 32];  // adapter chunks with an infinity or NaN in this tile
};

// BN: capacity of the token operand.  Up to 64 tokens two CTAs share an SM.
template <int BN>
struct ProjCfg {
    static constexpr int kStageBytes = kABytes + BN * 128;
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : 4;
    static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int kBarBytes = 256;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBarBytes + 2 * (int)sizeof(TileList) + kMaxAdapters / 8;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory overflow");
    static_assert(kStages * kStageBytes >= BN * 128 * 4, "the split sums fit the stages");
};

// One persistent CTA (or cluster of `splits`) takes tiles of 128 output features x bn
// tokens in turn; the accumulator is double buffered, so a tile's stores run under the
// next tile's products.  A cluster's CTAs take a share of the contraction each and one
// tile only; their fp32 sums meet in distributed shared memory, added in rank order.
// The kernel before this one in the stream writes only v (it waited for its own
// predecessors before it let this one start), so only the readers of v wait for it.
template <bool BWD, int BN>
__global__ void __launch_bounds__(kThreads, BN <= 64 ? 2 : 1) project_kernel(const __grid_constant__ ProjArgs a) {
    using C = ProjCfg<BN>;
    pdl_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
    uint64_t* empty = full + C::kStages;
    uint64_t* landed = empty + C::kStages;  // the adapter tile of a stage, before the v writers are done with it
    uint64_t* tfull = landed + C::kStages;  // accumulator complete / drained
    uint64_t* tempty = tfull + 2;
    uint64_t* listed = tempty + 2;          // a tile's adapter list written / no longer read
    uint64_t* lfree = listed + 2;
    uint64_t* done = lfree + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((3 * 6 + 9) * 8 + 8 <= C::kBarBytes, "barriers");
    TileList* lists = reinterpret_cast<TileList*>(smem + C::kStages * C::kStageBytes + C::kBarBytes);
    uint32_t* bits = reinterpret_cast<uint32_t*>(lists + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int S = a.splits;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int m_tiles = (a.O + 127) / 128;
    const int n_tiles = m_tiles * ((a.T + a.bn - 1) / a.bn);
    const int first = blockIdx.x / S, step = gridDim.x / S;
    const int kc = (a.C + 63) / 64, rc = (a.r + 63) / 64;
    const int c0 = (int)((long)kc * rank / S), c1 = (int)((long)kc * (rank + 1) / S);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&tfull[s]), 1);
            mbar_init(smem_u32(&tempty[s]), 4);
            mbar_init(smem_u32(&listed[s]), 1);
            mbar_init(smem_u32(&lfree[s]), 4);
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.w);
        tma_prefetch_desc(&a.x);
        tma_prefetch_desc(&a.lr);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    auto give_up = [&]() {
        *abort_flag = 1;
        raise_status(a.st, kStatusWaitTimeout);
    };

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0, land_phase = 0;
            uint32_t armed[C::kStages];  // per stage: 0 never, else 1 + parity, + 2 for an adapter tile
            for (int s = 0; s < C::kStages; ++s) armed[s] = 0;
            for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
                const int m0 = (i % m_tiles) * 128, row0 = (i / m_tiles) * a.bn;
                for (int c = c0; c < c1; ++c) {
                    if (*abort_flag || !mbar_wait(smem_u32(&empty[stage]), phase ^ 1, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem_u32(smem + stage * C::kStageBytes), fb = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(fb, kABytes + a.bn * 128);
                    armed[stage] = 1 + phase;
                    if (BWD) {
                        tma_load_3d(sa, &a.w, fb, m0, c * 64, 0, pol);
                        tma_load_3d(sa + kABytes / 2, &a.w, fb, m0 + 64, c * 64, 0, pol);
                    } else {
                        tma_load_3d(sa, &a.w, fb, c * 64, m0, 0, pol);
                    }
                    tma_load_3d(sa + kABytes, &a.x, fb, c * 64, 0, row0, pol);
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok || !(ok = mbar_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, limit))) break;
                const TileList& tl = lists[n & 1];
                for (int e = rank; e < tl.count * rc; e += S) {
                    if (*abort_flag || !mbar_wait(smem_u32(&empty[stage]), phase ^ 1, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = smem_u32(smem + stage * C::kStageBytes), lb = smem_u32(&landed[stage]);
                    const int id = tl.list[e / rc], j0 = (e % rc) * 64;
                    mbar_arrive_expect_tx(lb, kABytes);
                    armed[stage] = 3 + ((land_phase >> stage) & 1u);
                    land_phase ^= 1u << stage;
                    if (BWD) {
                        tma_load_3d(sa, &a.lr, lb, m0, j0, id, pol);
                        tma_load_3d(sa + kABytes / 2, &a.lr, lb, m0 + 64, j0, id, pol);
                    } else {
                        tma_load_3d(sa, &a.lr, lb, j0, m0, id, pol);
                    }
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok) give_up();
            // every copy has landed before the CTA exits
            for (int s = 0; s < C::kStages; ++s)
                if (armed[s]) mbar_wait(smem_u32(armed[s] >= 3 ? &landed[s] : &full[s]), (armed[s] - 1) & 1, limit);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = umma_idesc_bf16(128, a.bn) | (BWD ? kIdescAMnMajor : 0u);
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
                const uint32_t d = tbase + (n & 1) * BN;
                if (*abort_flag || !mbar_wait(smem_u32(&tempty[n & 1]), ((n >> 1) & 1) ^ 1, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t accum = 0;
                auto chunk = [&](int left) {
                    if (*abort_flag || !mbar_wait(smem_u32(&full[stage]), phase, limit)) {
                        ok = false;
                        return;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + stage * C::kStageBytes);
                    const uint64_t ad = BWD ? umma_desc_mn_sw128(sa, kABytes / 2) : umma_desc_sw128(sa);
                    const uint64_t bd = umma_desc_sw128(sa + kABytes);
                    const int steps = min(4, (left + 15) >> 4);
                    for (int k = 0; k < steps; ++k) {  // 16 of the contraction: 32 bytes along K, or 16 K rows
                        umma_bf16(d, ad + (BWD ? 128 : 2) * k, bd + 2 * k, idesc, accum);
                        accum = 1;
                    }
                    umma_commit(smem_u32(&empty[stage]));
                    if (++stage == C::kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                };
                for (int c = c0; c < c1 && ok; ++c) chunk(a.C - c * 64);
                if (!ok || !(ok = mbar_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, limit))) break;
                const int n_ext = lists[n & 1].count * rc;
                for (int e = rank; e < n_ext && ok; e += S) chunk(a.r - (e % rc) * 64);
                umma_commit(smem_u32(&tfull[n & 1]));
            }
            if (!ok) give_up();
            // all MMAs of this thread are complete before TMEM is freed
            umma_commit(smem_u32(done));
            mbar_wait(smem_u32(done), 0, limit);
        }
    } else if (warp < 6) {
        // ---- adapter lists and v chunks
        const int tid = threadIdx.x - 64;  // 0..127
        bool ok = true;
        int stage = 0;
        uint32_t land_phase = 0;
        for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
            const int row0 = (i / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
            TileList& tl = lists[n & 1];
            if (*abort_flag || !mbar_wait(smem_u32(&lfree[n & 1]), ((n >> 1) & 1) ^ 1, limit)) {
                ok = false;
                break;
            }
            for (int q = tid; q < kMaxExtra / 32; q += 128) tl.odd[q] = 0;
            tile_adapters(a.adapter_of, row0, rows, a.n_adapters, a.bn, tl.ids, tl.list, bits, &tl.count, a.st, tid, 128, 1);
            if (tid == 0) mbar_arrive(smem_u32(&listed[n & 1]));
            stage = (stage + c1 - c0) % C::kStages;
            const int n_ext = tl.count * rc;
            if (rank < n_ext) pdl_wait();  // v
            for (int e = rank; e < n_ext; e += S) {
                const int id = tl.list[e / rc], j0 = (e % rc) * 64;
                // the adapter tile has landed: the stage is free of its last use, too
                if (*abort_flag || !mbar_wait(smem_u32(&landed[stage]), (land_phase >> stage) & 1u, limit)) {
                    ok = false;
                    break;
                }
                land_phase ^= 1u << stage;
                uint8_t* st_a = smem + stage * C::kStageBytes;
                uint8_t* sb = st_a + kABytes;
                // v of this adapter's tokens, zeros elsewhere
                for (int q = tid; q < a.bn * 8; q += 128) {
                    const int row = q >> 3, seg = q & 7;
                    uint4 val = make_uint4(0, 0, 0, 0);
                    if (tl.ids[row] == id && j0 + seg * 8 < a.r)
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
                if (hit) atomicOr(&tl.odd[e >> 5], 1u << (e & 31));
                fence_async_smem();
                named_sync(1, 128);
                if (tid == 0) mbar_arrive(smem_u32(&full[stage]));
                if (++stage == C::kStages) stage = 0;
            }
        }
        if (!ok) give_up();
    } else {
        // ---- epilogue: TMEM lane = output feature, column = token
        const int q = warp & 3;
        bool ok = true;
        for (int i = first, n = 0; i < n_tiles; i += step, ++n) {
            const int m0 = (i % m_tiles) * 128, row0 = (i / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
            const TileList& tl = lists[n & 1];
            if (*abort_flag || !mbar_wait(smem_u32(&tfull[n & 1]), (n >> 1) & 1, limit)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // (the MMA warp read the list before its last commit)
            const int feat = m0 + q * 32 + lane;
            const int n_ext = tl.count * rc;
            const uint32_t tmem = tbase + (n & 1) * BN + ((uint32_t)(q * 32) << 16);
            bool any_odd = false;
            for (int w = 0; w * 32 < n_ext; ++w) any_odd |= tl.odd[w] != 0;
            if (any_odd) pdl_wait();  // reads v
            // the infinities and NaN that were taken out of the adapter tiles
            auto add_odd = [&](int g, float (&y)[16]) {
                for (int w = 0; w * 32 < n_ext; ++w) {
                    for (uint32_t b = tl.odd[w]; b; b &= b - 1) {
                        const int e = w * 32 + __ffs(b) - 1;
                        const int id = tl.list[e / rc], j0 = (e % rc) * 64;
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (tl.ids[g * 16 + j] != id) continue;
                            for (int l = j0; l < min(a.r, j0 + 64); ++l) {
                                const size_t at = BWD ? ((size_t)id * a.r + l) * a.O + feat : ((size_t)id * a.O + feat) * a.r + l;
                                const float u = bf(a.lr_ptr[at]);
                                if (!isfinite(u)) y[j] += u * bf(a.v[(size_t)(row0 + g * 16 + j) * a.r + l]);
                            }
                        }
                    }
                }
            };
            for (int g = 0; g * 16 < rows; ++g) {
                float v[16];
                tmem_ld16(tmem + g * 16, v);
                tmem_ld_wait();
                if (any_odd && feat < a.O) add_odd(g, v);
                __syncwarp();
                if (S > 1) {
                    // this CTA's share of the sum, [token][feature]
                    float* part = reinterpret_cast<float*>(smem) + (size_t)g * 16 * 128 + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[j * 128] = v[j];
                } else if (a.out_fp32) {
                    float* dst = reinterpret_cast<float*>(a.out) + feat;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (feat < a.O && g * 16 + j < rows) dst[(size_t)(row0 + g * 16 + j) * a.O] = v[j];
                } else {
                    // words of two features: lanes 2m and 2m+1 swap half their tokens, so the even
                    // lane holds the even tokens of features (2m, 2m+1) and the odd lane the odd
                    // ones (O % 8 == 0: both features of a pair are valid together)
                    const bool odd = lane & 1;
                    uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + (feat & ~1));
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const __nv_bfloat162 p2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                        const uint32_t p = *reinterpret_cast<const uint32_t*>(&p2);
                        const uint32_t o = __shfl_xor_sync(0xffffffffu, p, 1);
                        const uint32_t w = __byte_perm(p, o, odd ? 0x3276 : 0x5410);
                        const int col = g * 16 + 2 * j + (odd ? 1 : 0);
                        if (feat < a.O && col < rows) dst[(size_t)(row0 + col) * (a.O >> 1)] = w;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&tempty[n & 1]));
                mbar_arrive(smem_u32(&lfree[n & 1]));
            }
        }
        if (!ok && lane == 0) give_up();
    }
    if (S > 1) {
        // every share is in its CTA's shared memory; each CTA adds up a part of the tile
        __syncwarp();
        cluster_sync();
        const int m0 = (first % m_tiles) * 128, row0 = (first / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
        const int pairs = rows * 64;  // words of two features
        const int p0 = (int)((long)pairs * rank / S), p1 = (int)((long)pairs * (rank + 1) / S);
        if (!*abort_flag)
            for (int p = p0 + threadIdx.x; p < p1; p += kThreads) {
                const uint32_t addr = smem_u32(smem) + p * 8;
                float u = 0.0f, w = 0.0f;
                for (int s = 0; s < S; ++s) {
                    u += ld_peer(addr, s);
                    w += ld_peer(addr + 4, s);
                }
                const int feat = m0 + (p & 63) * 2;
                const size_t at = (size_t)(row0 + (p >> 6)) * a.O + feat;
                if (feat >= a.O) continue;
                if (a.out_fp32) {
                    *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at) = make_float2(u, w);
                } else {
                    const __nv_bfloat162 p2 = __floats2bfloat162_rn(u, w);
                    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + at) = *reinterpret_cast<const uint32_t*>(&p2);
                }
            }
        cluster_sync();  // no CTA leaves while another reads its shared memory
    }
    pdl_wait();  // the grid is complete only when the v kernel is
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
    pdl_wait();
    pdl_launch_dependents();
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
    pdl_wait();
    pdl_launch_dependents();
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
cudaError_t launch_project_bn(const ProjArgs& a, int grid, cudaStream_t stream) {
    auto kern = project_kernel<BWD, BN>;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = configure_once(configured, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ProjCfg<BN>::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kern, dim3(grid), dim3(kThreads), ProjCfg<BN>::kSmemBytes, stream, a.splits, a);
}

// How a projection of T tokens to O features is cut: tokens per tile, CTAs per tile, grid.
struct ProjPlan {
    int cap, bn, splits, grid;
};

ProjPlan project_plan(int T, int O, int C) {
    ProjPlan p;
    const int sms = num_sms(), m_tiles = (O + 127) / 128, kc = (C + 63) / 64;
    p.cap = T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
    p.bn = p.cap;
    p.splits = 1;
    if (T > 256) {
        // the tile height whose rounds over the SMs cost least: rounds x (tokens + a
        // fixed 16 for the accumulator's hand-over)
        long best = -1;
        for (int bn = 256; bn >= 128; bn -= 16) {
            const long tiles = (long)m_tiles * ((T + bn - 1) / bn);
            const long cost = (tiles + sms - 1) / sms * (bn + 16);
            if (best < 0 || cost < best) {
                best = cost;
                p.bn = bn;
            }
        }
    }
    const long tiles = (long)m_tiles * ((T + p.bn - 1) / p.bn);
    const int resident = p.cap <= 64 ? 2 : 1;
    // few tiles: clusters share a tile's contraction, four chunks of it per CTA at least
    while (p.splits < 8 && tiles * (p.splits + 1) <= (long)sms * resident && (p.splits + 1) * 4 <= kc) ++p.splits;
    p.grid = p.splits > 1 ? (int)tiles * p.splits : (int)std::min<long>(tiles, sms);
    return p;
}

// tokens [T][C] times W (and each token's low-rank matrix times v) into out [T][O]
template <bool BWD>
int project(const moe_adapter_t* p, int T, const void* tokens, const void* w, const void* lr, const int32_t* adapter_of,
            const void* v, void* out, int out_fp32, const DevStatus& st, cudaStream_t stream) {
    const uint64_t K = p->in_features, N = p->out_features, r = p->rank, n = p->n_adapters;
    ProjArgs a;
    a.T = T;
    a.O = BWD ? p->in_features : p->out_features;
    a.C = BWD ? p->out_features : p->in_features;
    a.r = p->rank;
    a.n_adapters = p->n_adapters;
    const ProjPlan plan = project_plan(T, a.O, a.C);
    a.bn = plan.bn;
    a.splits = plan.splits;
    int rc = make_tmap_3d(&a.w, w, K, N, 1, K * 2, K * N * 2, 64, BWD ? 64 : 128, 1);
    if (rc) return rc;
    if (BWD) rc = make_tmap_3d(&a.lr, lr, K, r, n, K * 2, K * r * 2, 64, 64, 1);
    else rc = make_tmap_3d(&a.lr, lr, r, N, n, r * 2, r * N * 2, 64, 128, 1);
    if (rc) return rc;
    const uint64_t C = a.C;
    if ((rc = make_tmap_3d(&a.x, tokens, C, 1, (uint64_t)T, C * 2, C * 2, 64, 1, plan.bn))) return rc;
    a.lr_ptr = static_cast<const uint16_t*>(lr);
    a.adapter_of = adapter_of;
    a.v = static_cast<const uint16_t*>(v);
    a.out = out;
    a.out_fp32 = out_fp32;
    a.st = st;
    const cudaError_t e = plan.cap == 32    ? launch_project_bn<BWD, 32>(a, plan.grid, stream)
                          : plan.cap == 64  ? launch_project_bn<BWD, 64>(a, plan.grid, stream)
                          : plan.cap == 128 ? launch_project_bn<BWD, 128>(a, plan.grid, stream)
                                            : launch_project_bn<BWD, 256>(a, plan.grid, stream);
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

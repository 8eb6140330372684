// Low-rank adapters of many requests beside a shared projection:
//   v_t = s_i A_i x_t,  y_t = W x_t + B_i v_t   (i = adapter of token t),
// and the gradients of x, A and B (W is frozen):
//   dv_t = s_i B_i^T dy_t,  dx_t = W^T dy_t + A_i^T dv_t,
//   dA_i = sum dv_t x_t^T,  dB_i = sum dy_t v_t^T.
// v and dv are summed in fp32 and rounded to bf16 once, as they are tensor-core operands beside
// bf16 A and B: 2^-8 of a value at most, which takes the error of y against 64 bits from 1.7e-3
// (its own rounding) to 1.8e-3 - 2.2e-3 where the adapter adds half as much as W does, and that of
// the gradients to 2.3e-3.
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

#include "operators.cuh"

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

// Two bf16 in a word, infinities and NaN among them replaced by 1 of their sign: beside the
// infinity that is added later it is lost, and times an infinite v it is that infinity already.
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w = (w & 0xffff8000u) | 0x3f80u;
    if ((w & 0x7f800000u) == 0x7f800000u) w = (w & 0x8000ffffu) | 0x3f800000u;
    return w;
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
// `bits` holds kMaxAdapters bits.  False on all of them, and nothing written, if one is not `ready`.
__device__ __forceinline__ bool tile_adapters(const int32_t* adapter_of, int row0, int rows, int n_adapters, int bn,
                                              int* ids, int* list, uint32_t* bits, int* count, const DevStatus& st,
                                              int tid, int n_threads, int bar, bool ready = true) {
    const int words = (n_adapters + 31) / 32;
    for (int i = tid; i < words; i += n_threads) bits[i] = 0;
    if (!named_and(bar, n_threads, ready)) return false;
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
    return true;
}

struct ProjArgs {
    CUtensorMap w;      // forward: box {64 k, 128 n} of W [N][K]; backward: box {64 k, 64 n}
    CUtensorMap lr;     // forward: box {64 r, 128 n} of B [n][N][r]; backward: box {64 k, 64 r} of A [n][r][K]
    CUtensorMap x;      // tokens: box {64, 1, tokens of one CTA} of x [T][K] | dy [T][N]
    CUtensorMap y;      // box {64, 1, 16} of a bf16 output
    const int32_t* adapter_of;
    const uint16_t* v;  // [T][r] v | dv
    const uint16_t* lr_ptr;  // what `lr` maps
    int T, O, C, r, n_adapters;  // O output features, C contracted features
    int bn;             // tokens of a tile (a multiple of 16)
    int splits;         // CTAs of a cluster that share one tile's contraction
    int v_ready;        // v was complete before this kernel could start
    void* out;          // [T][O]
    int out_fp32;
    DevStatus st;
};

// How adapters fill the 64-wide chunks: small ranks share one, `per` adapters of `seg`
// columns each (a rank up to 16 four, up to 32 two), larger ones take several.
struct Packing {
    int r, per, seg;
    __device__ __forceinline__ explicit Packing(int rank)
        : r(rank), per(rank <= 16 ? 4 : rank <= 32 ? 2 : 1), seg(64 / per) {}
    __device__ __forceinline__ int chunks(int count) const {
        return per > 1 ? (count + per - 1) / per : count * ((r + 63) / 64);
    }
    // adapters of chunk e: list[first .. first + n)
    __device__ __forceinline__ int first(int e, int count) const { return per > 1 ? e * per : e % count; }
    __device__ __forceinline__ int n(int e, int count) const { return per > 1 ? min(per, count - e * per) : 1; }
    __device__ __forceinline__ int j0(int e, int count) const { return per > 1 ? 0 : e / count * 64; }
    // 16-wide steps of chunk e, of which step q is used if it lies in an adapter's rank
    __device__ __forceinline__ bool step(int q, int e, int count) const {
        return per > 1 ? q * 16 / seg < n(e, count) && q * 16 % seg < r : j0(e, count) + q * 16 < r;
    }
};

// What a tile's workers know of its adapters.
struct TileList {
    int count;
    int ids[kMaxTile];   // adapter of each token
    int list[kMaxTile];  // distinct adapters
    uint32_t odd[kMaxExtra / 32];  // adapter chunks with an infinity or NaN in this tile
};

// The v rows of a thread's tokens, 64 of their rank, held in registers while the tile's
// adapters pass: the thread of 128 with index tid has the tokens tid and (RPT = 2) tid + 128.
template <int RPT>
struct VRows {
    int id[RPT];
    int pos[RPT];  // of its adapter in the list
    uint4 v[RPT][8];

    __device__ __forceinline__ void ids(const int* of, int n, const int* list, int count, int tid) {
#pragma unroll
        for (int q = 0; q < RPT; ++q) {
            id[q] = tid + q * 128 < n ? of[tid + q * 128] : -1;
            int lo = 0, hi = count - 1;  // the list ascends
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] < id[q]) lo = mid + 1;
                else hi = mid;
            }
            pos[q] = id[q] >= 0 ? lo : -1;
        }
    }
    __device__ __forceinline__ void load(const ProjArgs& a, int row0, int j0, int tid) {
#pragma unroll
        for (int q = 0; q < RPT; ++q)
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                v[q][g] = make_uint4(0, 0, 0, 0);
                if (id[q] >= 0 && j0 + g * 8 < a.r)
                    v[q][g] = *reinterpret_cast<const uint4*>(a.v + (size_t)(row0 + tid + q * 128) * a.r + j0 + g * 8);
            }
    }
    // sb: the rows of the PER adapters from `first` of the list, each in its own columns,
    // zeros elsewhere (n rows, swizzled as TMA would)
    template <int PER>
    __device__ __forceinline__ void store_per(uint8_t* sb, int n, int first, int tid) const {
#pragma unroll
        for (int q = 0; q < RPT; ++q) {
            const int row = tid + q * 128;
            if (row >= n) continue;
            const int p = pos[q] < 0 ? -1 : pos[q] - first;
#pragma unroll
            for (int g = 0; g < 8; ++g)
                *reinterpret_cast<uint4*>(sb + row * 128 + ((g ^ (row & 7)) << 4)) =
                    p == g / (8 / PER) ? v[q][g % (8 / PER)] : make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void store(uint8_t* sb, int n, int first, int per, int tid) const {
        if (per == 4) store_per<4>(sb, n, first, tid);
        else if (per == 2) store_per<2>(sb, n, first, tid);
        else store_per<1>(sb, n, first, tid);
    }
};

// The copies of adapter chunk e: rows of B_i (features, then rank) or A_i (rank, then
// features) of each of its adapters.
template <bool BWD>
__device__ __forceinline__ void load_adapters(const ProjArgs& a, const Packing& pk, const TileList& tl, int e, uint32_t sa,
                                              uint32_t bar, int m0, uint64_t pol) {
    const int first = pk.first(e, tl.count), n = pk.n(e, tl.count), j0 = pk.j0(e, tl.count);
    mbar_arrive_expect_tx(bar, n * pk.seg * 256);
    for (int p = 0; p < n; ++p) {
        const int id = tl.list[first + p];
        if (BWD) {
            tma_load_3d(sa + p * pk.seg * 128, &a.lr, bar, m0, j0, id, pol);
            tma_load_3d(sa + kABytes / 2 + p * pk.seg * 128, &a.lr, bar, m0 + 64, j0, id, pol);
        } else {
            tma_load_3d(sa + p * pk.seg * 256, &a.lr, bar, j0, m0, id, pol);
        }
    }
}

// The A operand of adapter chunks (forward): each adapter's 128 rows of `seg` columns, swizzled
// over their own width (layout codes 2, 4, 6: 128, 64, 32 bytes).
__device__ __forceinline__ uint64_t adapter_desc(uint32_t smem_addr, const Packing& pk) {
    uint64_t d = (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)1u << 16;
    d |= (uint64_t)(pk.seg * 16 >> 4) << 32;  // 8 rows
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)(pk.per == 1 ? 2u : pk.per == 2 ? 4u : 6u) << 61;
    return d;
}

// Offset of step q in it, in 16 bytes.
__device__ __forceinline__ int adapter_step(int q, const Packing& pk) {
    return pk.per == 4 ? q * 256 : pk.per == 2 ? (q >> 1) * 512 + (q & 1) * 2 : q * 2;
}

// Zero times an infinity or NaN of an adapter would reach the other adapters' tokens: ones take
// the places of such elements in its tile here (true: there were some), and what they are is
// added to their own tokens in the epilogue.  Only the columns that were copied are looked at: the rest of a stage,
// which no product reads, holds what was there before.
template <bool BWD>
__device__ __forceinline__ bool take_odd(uint8_t* st_a, int columns, int tid) {
    // (backward: features along the rows, in two halves)
    const int used = columns * (BWD ? 8 : 16);
    auto in = [&](int q) { return (BWD ? tid + (q & 3) * 128 : tid + q * 128) < used; };
    uint4* at = reinterpret_cast<uint4*>(st_a) + tid;
    uint32_t most = 0;  // largest magnitudes, as pairs of 16-bit numbers
#pragma unroll
    for (int q = 0; q < kABytes / 16 / 128; ++q) {
        const uint4 val = in(q) ? at[q * 128] : make_uint4(0, 0, 0, 0);
        most = __vmaxu2(__vmaxu2(most, val.x & 0x7fff7fffu), val.y & 0x7fff7fffu);
        most = __vmaxu2(__vmaxu2(most, val.z & 0x7fff7fffu), val.w & 0x7fff7fffu);
    }
    if ((most & 0xffffu) < 0x7f80u && (most >> 16) < 0x7f80u) return false;
    for (int q = 0; q < kABytes / 16 / 128; ++q) {
        if (!in(q)) continue;
        uint4 val = at[q * 128];
        val.x = finite_part(val.x);
        val.y = finite_part(val.y);
        val.z = finite_part(val.z);
        val.w = finite_part(val.w);
        at[q * 128] = val;
    }
    return true;
}

__device__ __forceinline__ bool has_odd(const TileList& tl, int n_ext) {
    bool any = false;
    for (int w = 0; w * 32 < n_ext; ++w) any |= tl.odd[w] != 0;
    return any;
}

// The infinities and NaN that were taken out of the adapter tiles, for 16 tokens from t0
// (position at in the tile) and one feature.
template <bool BWD>
__device__ __noinline__ void add_odd(const ProjArgs& a, const TileList& tl, int n_ext, int t0, int at, int feat,
                                     float (&y)[16]) {
    pdl_wait();  // v
    const Packing pk(a.r);
    for (int w = 0; w * 32 < n_ext; ++w) {
        for (uint32_t b = tl.odd[w]; b; b &= b - 1) {
            const int e = w * 32 + __ffs(b) - 1;
            const int first = pk.first(e, tl.count), last = first + pk.n(e, tl.count) - 1, j0 = pk.j0(e, tl.count);
            for (int j = 0; j < 16; ++j) {
                const int id = tl.ids[at + j];
                if (id < tl.list[first] || id > tl.list[last]) continue;  // (the list ascends)
                for (int l = j0; l < min(a.r, j0 + 64); ++l) {
                    const size_t el = BWD ? ((size_t)id * a.r + l) * a.O + feat : ((size_t)id * a.O + feat) * a.r + l;
                    const float u = bf(a.lr_ptr[el]);
                    if (!isfinite(u)) y[j] += u * bf(a.v[(size_t)(t0 + j) * a.r + l]);
                }
            }
        }
    }
}

// Feature `feat` (this lane's) of up to 16 tokens from t0, `n` of them valid.
__device__ __forceinline__ void store_group(const ProjArgs& a, int t0, int n, int feat, const float (&v)[16]) {
    if (a.out_fp32) {
        float* dst = reinterpret_cast<float*>(a.out) + (size_t)t0 * a.O + feat;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (feat < a.O && j < n) dst[(size_t)j * a.O] = v[j];
        return;
    }
    // words of two features: lanes 2m and 2m+1 swap half their tokens, so the even lane
    // holds the even tokens of features (2m, 2m+1) and the odd lane the odd ones
    // (O % 8 == 0: both features of a pair are valid together)
    const bool odd = threadIdx.x & 1;
    uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out) + (size_t)t0 * a.O + (feat & ~1));
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 p2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        const uint32_t p = *reinterpret_cast<const uint32_t*>(&p2);
        const uint32_t o = __shfl_xor_sync(0xffffffffu, p, 1);
        const uint32_t w = __byte_perm(p, o, odd ? 0x3276 : 0x5410);
        const int col = 2 * j + (odd ? 1 : 0);
        if (feat < a.O && col < n) dst[(size_t)col * (a.O >> 1)] = w;
    }
}

// ---- a tile's bf16 outputs through shared memory
// A lane that holds one feature of 16 tokens writes 64 bytes of a row with its warp: 450 ns
// for 16 tokens, 7 us for the 256 of a tile, more than its products take below 1700 of the
// contraction.  Here the accumulator comes as 8 x 8 fragments, which stmatrix turns to rows
// of features, and copies of 16 tokens x 64 features take them out.
constexpr int kOutBlock = 4096;           // 32 tokens x 64 features
constexpr int kOutBytes = 2 * 2 * kOutBlock;  // two of each pair of warps

// Warp q's quarter of the accumulator at `tmem`: `rows` tokens from row0, of the 128
// features from m0.  Warps 2 p and 2 p + 1 share 64 features, two blocks at `out` and the
// copies, which the first one's lane 0 issues; `blocks` counts the blocks so far.
__device__ __forceinline__ void drain_tile(const ProjArgs& a, uint32_t tmem, uint32_t out, int row0, int rows, int m0, int q,
                                           int lane, int& blocks) {
    const int pair = q >> 1, f0 = m0 + pair * 64;
    const bool issuer = !(q & 1) && lane == 0;
    // this lane's address of a row of 8 features: token lane % 8, features 8 (lane / 8) of the warp's 32 (swizzled as the copy reads)
    const uint32_t at = (lane & 7) * 128 + ((((q & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
    for (int t = 0; t < rows; t += 32, ++blocks) {
        uint32_t lo[16], hi[16];
        tmem_ld_16x256(tmem + t, lo);
        tmem_ld_16x256(tmem + t + (16u << 16), hi);
        tmem_ld_wait();
        const uint32_t block = out + (pair * 2 + (blocks & 1)) * kOutBlock;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            stmatrix_trans(block + i * 1024 + at, pack_bf(lo[4 * i], lo[4 * i + 1]), pack_bf(lo[4 * i + 2], lo[4 * i + 3]),
                           pack_bf(hi[4 * i], hi[4 * i + 1]), pack_bf(hi[4 * i + 2], hi[4 * i + 3]));
        fence_async_smem();
        if (issuer) bulk_wait_read();  // the other block is free, which the next round writes
        __syncwarp();
        named_sync(2 + pair, 64);
        if (issuer) {
            // (a tile's tokens are a multiple of 16 but at the end of the batch, where the copy ends too)
            if (f0 < a.O) {
                tma_store_3d(&a.y, block, f0, 0, row0 + t);
                if (t + 16 < rows) tma_store_3d(&a.y, block + kOutBlock / 2, f0, 0, row0 + t + 16);
            }
            bulk_commit();
        }
        __syncwarp();
    }
}

// BN: capacity of the token operand.  Up to 64 tokens two CTAs share an SM.
template <int BN>
struct ProjCfg {
    static constexpr int kStageBytes = kABytes + BN * 128;
    // Up to 64 tokens two CTAs fit an SM, if only the next launch's beside the last one's:
    // nine stages and one CTA took 17.5 us a call at one token, where this takes 13.
    static constexpr int kStages = BN == 256 ? 4 : BN == 128 ? 6 : BN == 64 ? 4 : 5;
    static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int kBarBytes = 512;
    static constexpr bool kCopyOut = BN > 64;  // (the shared memory of two CTAs has no room for it)
    static constexpr int kRingBytes = kStages * kStageBytes + (kCopyOut ? kOutBytes : 0);
    static constexpr int kSmemBytes = 1024 + kRingBytes + kBarBytes + 2 * (int)sizeof(TileList) + kMaxAdapters / 8;
    static_assert(kSmemBytes <= (BN <= 64 ? 113 : 227) * 1024, "shared memory overflow");
    static_assert(kStages * kStageBytes >= BN * 128 * 4, "the split sums fit the stages");
};

// One persistent CTA (or cluster of `splits`) takes tiles of 128 output features x bn
// tokens in turn; the accumulator is double buffered, so a tile's stores run under the
// next tile's products.  A cluster's CTAs take a share of the contraction each and one
// tile only; their fp32 sums meet in distributed shared memory, added in rank order.  (The
// plan counts the chunks of as many adapters as the tile may hold, so a short contraction
// may have more CTAs than chunks: a CTA without any adds zeros.)
// Measured: one token, 7168 to 2048 features, 11 us a call with v's kernel (29 MB of W at
// 6.5 TB/s in the middle 4.5 us; the rest is the start, the cluster's sum and the launches);
// 192 tokens, 2048 to 7168, 18 us without adapters (each feature tile reads the tokens
// again) and 28 with 23 of them.
// The kernel before this one in the stream writes only v (it waited for its own
// predecessors before it let this one start), so only the readers of v wait for it.
template <bool BWD, int BN>
__global__ void __launch_bounds__(kThreads, BN <= 64 ? 2 : 1) project_kernel(const __grid_constant__ ProjArgs a) {
    using C = ProjCfg<BN>;
    constexpr int stages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRingBytes);
    uint64_t* empty = full + stages;
    uint64_t* landed = empty + stages;  // the adapter tile of a stage, before the v writers are done with it
    uint64_t* tfull = landed + stages;  // accumulator complete / drained
    uint64_t* tempty = tfull + 2;
    uint64_t* listed = tempty + 2;          // a tile's adapter list written / no longer read
    uint64_t* lfree = listed + 2;
    uint64_t* done = lfree + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((3 * C::kStages + 9) * 8 + 8 <= C::kBarBytes, "barriers");
    TileList* lists = reinterpret_cast<TileList*>(smem + C::kRingBytes + C::kBarBytes);
    uint32_t* bits = reinterpret_cast<uint32_t*>(lists + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int S = a.splits;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int m_tiles = (a.O + 127) / 128;
    const int n_tiles = m_tiles * ((a.T + a.bn - 1) / a.bn);
    const int first = blockIdx.x / S, step = gridDim.x / S;
    const int kc = (a.C + 63) / 64;
    const Packing pk(a.r);
    const int c0 = (int)((long)kc * rank / S), c1 = (int)((long)kc * (rank + 1) / S);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&tfull[s]), 1);
            mbar_init(smem_u32(&tempty[s]), 4);
            mbar_init(smem_u32(&listed[s]), 1);
            mbar_init(smem_u32(&lfree[s]), 5);  // the epilogue and the loads
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.w);
        tma_prefetch_desc(&a.x);
        tma_prefetch_desc(&a.lr);
        if (!a.out_fp32) tma_prefetch_desc(&a.y);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();  // (not before the tensor memory is this CTA's: see shrink_kernel)
    const uint32_t tbase = *tmem_slot;
    auto give_up = [&]() {
        *abort_flag = 1;
        raise_status(a.st, kStatusWaitTimeout);
    };

    const uint32_t full_u = smem_u32(full), empty_u = smem_u32(empty), landed_u = smem_u32(landed);
    const uint32_t stage_u = smem_u32(smem);
    if (warp == 0) {
        const uint64_t pol = policy_evict_normal();
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0, land_phase = 0;
        uint32_t used = 0, used_land = 0, used_phase = 0;  // stages filled, whether by an adapter tile, parity
        auto advance = [&](bool land) {
            const uint32_t bit = 1u << stage, par = land ? (land_phase >> stage) & 1u : phase;
            used |= bit;
            used_land = land ? used_land | bit : used_land & ~bit;
            used_phase = par ? used_phase | bit : used_phase & ~bit;
            if (land) land_phase ^= bit;
            if (++stage == stages) {
                stage = 0;
                phase ^= 1;
            }
        };
        for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
            const int m0 = (i % m_tiles) * 128, row0 = (i / m_tiles) * a.bn;
            for (int c = c0; c < c1; ++c) {
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                if (elect_one()) {
                    const uint32_t sa = stage_u + stage * C::kStageBytes, fb = full_u + stage * 8;
                    mbar_arrive_expect_tx(fb, kABytes + a.bn * 128);
                    if (BWD) {
                        tma_load_3d(sa, &a.w, fb, m0, c * 64, 0, pol);
                        tma_load_3d(sa + kABytes / 2, &a.w, fb, m0 + 64, c * 64, 0, pol);
                    } else {
                        tma_load_3d(sa, &a.w, fb, c * 64, m0, 0, pol);
                    }
                    tma_load_3d(sa + kABytes, &a.x, fb, c * 64, 0, row0, pol);
                }
                __syncwarp();
                advance(false);
            }
            if (!ok || !(ok = warp_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, abort_flag, limit))) break;
            const TileList& tl = lists[n & 1];
            const int n_ext = pk.chunks(tl.count);
            for (int e = rank; e < n_ext; e += S) {
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                if (elect_one())
                    load_adapters<BWD>(a, pk, tl, e, stage_u + stage * C::kStageBytes, landed_u + stage * 8, m0, pol);
                __syncwarp();
                advance(true);
            }
            if (lane == 0) mbar_arrive(smem_u32(&lfree[n & 1]));  // the list has been read
        }
        if (!ok && lane == 0) give_up();
        // every copy has landed before the CTA exits
        for (int s = 0; s < stages; ++s)
            if ((used >> s) & 1u)
                mbar_wait(((used_land >> s) & 1u ? landed_u : full_u) + s * 8, (used_phase >> s) & 1u, limit);
    } else if (warp == 1) {
        const uint32_t idesc = umma_idesc_bf16(128, a.bn) | (BWD ? kIdescAMnMajor : 0u);
        const uint64_t ad0 = BWD ? umma_desc_mn_sw128(stage_u, kABytes / 2) : umma_desc_sw128(stage_u);
        const uint64_t bd0 = umma_desc_sw128(stage_u + kABytes);
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
            const uint32_t d = tbase + (n & 1) * BN;
            if (!(ok = warp_wait(smem_u32(&tempty[n & 1]), ((n >> 1) & 1) ^ 1, abort_flag, limit))) break;
            tc_fence_after();
            uint32_t accum = 0;
            // 64 of the contraction (`left` of them), or adapter chunk e >= 0
            auto chunk = [&](int left, int e, int count) {
                if (!(ok = warp_wait(full_u + stage * 8, phase, abort_flag, limit))) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = ad0 + stage * (C::kStageBytes >> 4), bd = bd0 + stage * (C::kStageBytes >> 4);
                    // 16 of the contraction per instruction: 32 bytes along K, or 16 K rows
                    constexpr int kAStep = BWD ? 128 : 2;
                    if (e < 0) {
                        umma_bf16(d, ad, bd, idesc, accum);
                        if (left > 16) umma_bf16(d, ad + kAStep, bd + 2, idesc, 1);
                        if (left > 32) umma_bf16(d, ad + 2 * kAStep, bd + 4, idesc, 1);
                        if (left > 48) umma_bf16(d, ad + 3 * kAStep, bd + 6, idesc, 1);
                    } else {
                        const uint64_t ed = BWD ? ad : adapter_desc(stage_u, pk) + stage * (C::kStageBytes >> 4);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (pk.step(q, e, count))
                                umma_bf16(d, ed + (BWD ? kAStep * q : adapter_step(q, pk)), bd + 2 * q, idesc, accum || q > 0);
                    }
                    umma_commit(empty_u + stage * 8);
                }
                __syncwarp();
                accum = 1;
                if (++stage == stages) {
                    stage = 0;
                    phase ^= 1;
                }
            };
            for (int c = c0; c < c1 && ok; ++c) chunk(a.C - c * 64, -1, 0);
            if (!ok || !(ok = warp_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, abort_flag, limit))) break;
            const int count = lists[n & 1].count, n_ext = pk.chunks(count);
            for (int e = rank; e < n_ext && ok; e += S) chunk(0, e, count);
            if (elect_one()) umma_commit(smem_u32(&tfull[n & 1]));
            __syncwarp();
        }
        if (!ok && lane == 0) give_up();
        // all MMAs of this warp are complete before TMEM is freed
        if (elect_one()) umma_commit(smem_u32(done));
        __syncwarp();
        mbar_wait(smem_u32(done), 0, limit);
    } else if (warp < 6) {
        // ---- adapter lists and v chunks (one verdict on each wait: the four warps leave together)
        const int tid = threadIdx.x - 64;  // 0..127
        bool ok = true;
        int stage = 0;
        uint32_t land_phase = 0;
        for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
            const int row0 = (i / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
            TileList& tl = lists[n & 1];
            const bool ready = !*abort_flag && mbar_wait(smem_u32(&lfree[n & 1]), ((n >> 1) & 1) ^ 1, limit);
            for (int q = tid; q < kMaxExtra / 32 && ready; q += 128) tl.odd[q] = 0;
            if (!(ok = tile_adapters(a.adapter_of, row0, rows, a.n_adapters, a.bn, tl.ids, tl.list, bits, &tl.count, a.st,
                                     tid, 128, 1, ready)))
                break;
            if (tid == 0) mbar_arrive(smem_u32(&listed[n & 1]));
            stage = (stage + c1 - c0) % stages;
            const int n_ext = pk.chunks(tl.count);
            if (rank < n_ext && !a.v_ready) pdl_wait();
            VRows<BN == 256 ? 2 : 1> vr;
            vr.ids(tl.ids, a.bn, tl.list, tl.count, tid);
            int held = -1;
            for (int e = rank; e < n_ext; e += S) {
                const int first_of = pk.first(e, tl.count), j0 = pk.j0(e, tl.count);
                if (j0 != held) vr.load(a, row0, held = j0, tid);
                // the adapter tile has landed: the stage is free of its last use, too
                const bool here = !*abort_flag && mbar_wait(smem_u32(&landed[stage]), (land_phase >> stage) & 1u, limit);
                land_phase ^= 1u << stage;
                if (here) {
                    uint8_t* st_a = smem + stage * C::kStageBytes;
                    vr.store(st_a + kABytes, a.bn, first_of, pk.per, tid);
                    if (take_odd<BWD>(st_a, pk.n(e, tl.count) * pk.seg, tid)) atomicOr(&tl.odd[e >> 5], 1u << (e & 31));
                    fence_async_smem();
                }
                if (!(ok = named_and(1, 128, here))) break;
                if (tid == 0) mbar_arrive(smem_u32(&full[stage]));
                if (++stage == stages) stage = 0;
            }
        }
        if (!ok) give_up();
    } else {
        // ---- epilogue: TMEM lane = output feature, column = token
        const int q = warp & 3;
        bool ok = true;
        int blocks = 0;
        for (int i = first, n = 0; i < n_tiles; i += step, ++n) {
            const int m0 = (i % m_tiles) * 128, row0 = (i / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
            const TileList& tl = lists[n & 1];
            ok = warp_wait(smem_u32(&tfull[n & 1]), (n >> 1) & 1, abort_flag, limit);
            if (C::kCopyOut) ok = named_and(2 + (q >> 1), 64, ok);  // (the two warps that share drain_tile's barrier)
            if (!ok) break;
            tc_fence_after();
            // (the MMA warp read the list before its last commit)
            const int feat = m0 + q * 32 + lane;
            const int n_ext = pk.chunks(tl.count);
            const uint32_t tmem = tbase + (n & 1) * BN + ((uint32_t)(q * 32) << 16);
            const bool any_odd = has_odd(tl, n_ext);
            const bool copy_out = C::kCopyOut && S == 1 && !a.out_fp32 && !any_odd;
            // A short contraction may leave a CTA of the cluster without a chunk of it, and the tile
            // without an adapter chunk for it: its accumulator was never written.
            const bool no_share = c0 == c1 && rank >= n_ext;
            if (copy_out) drain_tile(a, tmem, stage_u + stages * C::kStageBytes, row0, rows, m0, q, lane, blocks);
            for (int g = 0; g * 16 < rows && !copy_out; ++g) {
                float v[16];
                tmem_ld16(tmem + g * 16, v);
                tmem_ld_wait();
                if (no_share) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
                }
                if (any_odd && feat < a.O) add_odd<BWD>(a, tl, n_ext, row0 + g * 16, g * 16, feat, v);
                __syncwarp();
                if (S > 1) {
                    // this CTA's share of the sum, [token][feature]
                    float* part = reinterpret_cast<float*>(smem) + (size_t)g * 16 * 128 + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[j * 128] = v[j];
                } else {
                    store_group(a, row0 + g * 16, rows - g * 16, feat, v);
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
        if (C::kCopyOut && lane == 0) bulk_wait();
    }
    if (S > 1) {
        // every share is in its CTA's shared memory; each CTA adds up a part of the tile
        __syncwarp();
        cluster_sync();
        const int m0 = (first % m_tiles) * 128, row0 = (first / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
        const int quads = rows * 32;  // four features of a token
        const int p0 = (int)((long)quads * rank / S), p1 = (int)((long)quads * (rank + 1) / S);
        if (!*abort_flag)
            for (int p = p0 + threadIdx.x; p < p1; p += kThreads) {
                const int feat = m0 + (p & 31) * 4;
                if (feat >= a.O) continue;  // (O % 8 == 0: the four are valid together)
                const uint32_t addr = stage_u + p * 16;
                float4 f[8];
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < S) f[s] = ld_peer4(addr, s);
                float4 y = f[0];
#pragma unroll
                for (int s = 1; s < 8; ++s)
                    if (s < S) {
                        y.x += f[s].x;
                        y.y += f[s].y;
                        y.z += f[s].z;
                        y.w += f[s].w;
                    }
                const size_t at = (size_t)(row0 + (p >> 5)) * a.O + feat;
                if (a.out_fp32) {
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = y;
                } else {
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + at) =
                        make_uint2((uint32_t)to_bf(y.x) | ((uint32_t)to_bf(y.y) << 16),
                                   (uint32_t)to_bf(y.z) | ((uint32_t)to_bf(y.w) << 16));
                }
            }
        cluster_sync_read();  // no CTA leaves while another reads its shared memory
    }
    pdl_wait();  // the grid is complete only when the v kernel is
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, C::kTmemCols);
}

// Many tiles: a pair of CTAs computes 256 features x bn tokens with one product per 16 of
// the contraction (cta_group::2).  Each CTA holds 128 rows of W and half of the tokens,
// 32 KB per 64 of the contraction, so six stages (6 x 512 cycles of products) fit where a CTA
// on its own has four of 48 KB (4 x 512, less than the round trip of a stage).
// The leader (rank 0) issues the products; both load, write v and drain their own half.
// Bound by the tensor cores: 4096 tokens, 7168 to 4096 features, 140 us (1.71 PFLOP/s, 89%
// of the measured burst; 550 cycles a stage of 512 cycles of products).
constexpr int kPairStages = 6;
constexpr int kPairStageBytes = kABytes + 128 * 128;
constexpr int kPairRing = kPairStages * kPairStageBytes + kOutBytes;
constexpr int kPairSmem = 1024 + kPairRing + 512 + 2 * (int)sizeof(TileList) + kMaxAdapters / 8;
static_assert(kPairSmem <= 227 * 1024, "shared memory overflow");

template <bool BWD>
__global__ void __launch_bounds__(kThreads, 1) project_pair_kernel(const __grid_constant__ ProjArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairRing);  // (beside the leader: of adapter chunks only)
    uint64_t* empty = full + kPairStages;
    uint64_t* landed = empty + kPairStages;
    uint64_t* other = landed + kPairStages;  // (the leader's) the other CTA's half of an adapter chunk is in place
    uint64_t* tfull = other + kPairStages;
    uint64_t* tempty = tfull + 2;  // (the leader's)
    uint64_t* listed = tempty + 2;
    uint64_t* lfree = listed + 2;
    uint64_t* done = lfree + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((4 * kPairStages + 9) * 8 + 8 <= 512, "barriers");
    TileList* lists = reinterpret_cast<TileList*>(smem + kPairRing + 512);
    uint32_t* bits = reinterpret_cast<uint32_t*>(lists + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int rank = (int)cluster_rank();
    const int half = a.bn / 2;
    const int m_tiles = (a.O + 255) / 256;
    const int n_tiles = m_tiles * ((a.T + a.bn - 1) / a.bn);
    const int first = blockIdx.x / 2, step = gridDim.x / 2;
    const int kc = (a.C + 63) / 64;
    const Packing pk(a.r);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&other[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&tfull[s]), 1);
            mbar_init(smem_u32(&tempty[s]), 8);
            mbar_init(smem_u32(&listed[s]), 1);
            mbar_init(smem_u32(&lfree[s]), 5 + rank);  // the epilogue, the loads and, beside the leader, the signals
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.w);
        tma_prefetch_desc(&a.x);
        tma_prefetch_desc(&a.lr);
        if (!a.out_fp32) tma_prefetch_desc(&a.y);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the barriers of both CTAs exist before either is signalled
    tc_fence_after();
    pdl_launch_dependents();  // (not before the tensor memory is this pair's: see shrink_kernel)
    const uint32_t tbase = *tmem_slot;
    auto give_up = [&]() {
        *abort_flag = 1;
        raise_status(a.st, kStatusWaitTimeout);
    };
    const uint32_t full_u = smem_u32(full), empty_u = smem_u32(empty), landed_u = smem_u32(landed);
    const uint32_t stage_u = smem_u32(smem);
    const uint32_t lead_full = leader_addr(full_u), lead_tempty = leader_addr(smem_u32(tempty));
    const uint32_t lead_other = leader_addr(smem_u32(other));

    if (warp == 0) {
        const uint64_t pol = policy_evict_normal();
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0, land_phase = 0, used = 0, used_land = 0;
        auto advance = [&](bool land) {
            const uint32_t bit = 1u << stage;
            used |= bit;
            used_land = land ? used_land | bit : used_land & ~bit;
            if (land) land_phase ^= bit;
            if (++stage == kPairStages) {
                stage = 0;
                phase ^= 1;
            }
        };
        for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
            const int m0 = (i % m_tiles) * 256 + rank * 128, row0 = (i / m_tiles) * a.bn + rank * half;
            for (int c = 0; c < kc; ++c) {
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                if (elect_one()) {
                    const uint32_t sa = stage_u + stage * kPairStageBytes, fb = lead_full + stage * 8;
                    // the leader expects the bytes of both (an arrival from the other CTA takes it 500 cycles)
                    if (rank == 0) mbar_arrive_expect_tx(full_u + stage * 8, 2 * kABytes + a.bn * 128);
                    if (BWD) {
                        tma_load_3d_pair(sa, &a.w, fb, m0, c * 64, 0, pol);
                        tma_load_3d_pair(sa + kABytes / 2, &a.w, fb, m0 + 64, c * 64, 0, pol);
                    } else {
                        tma_load_3d_pair(sa, &a.w, fb, c * 64, m0, 0, pol);
                    }
                    tma_load_3d_pair(sa + kABytes, &a.x, fb, c * 64, 0, row0, pol);
                }
                __syncwarp();
                advance(false);
            }
            if (!ok || !(ok = warp_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, abort_flag, limit))) break;
            const TileList& tl = lists[n & 1];
            const int n_ext = pk.chunks(tl.count);
            for (int e = 0; e < n_ext; ++e) {
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                if (elect_one())
                    load_adapters<BWD>(a, pk, tl, e, stage_u + stage * kPairStageBytes, landed_u + stage * 8, m0, pol);
                __syncwarp();
                advance(true);
            }
            if (lane == 0) mbar_arrive(smem_u32(&lfree[n & 1]));  // the list has been read
        }
        if (!ok && lane == 0) give_up();
        // every stage's last products are done, so its copies have landed
        for (int s = 0; s < kPairStages; ++s) {
            const int bit = stage;
            if ((used >> bit) & 1u) {
                if (!ok && ((used_land >> bit) & 1u)) mbar_wait(landed_u + bit * 8, ((land_phase >> bit) & 1u) ^ 1, limit);
                mbar_wait(empty_u + bit * 8, phase ^ 1, limit);
            }
            if (++stage == kPairStages) {
                stage = 0;
                phase ^= 1;
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = umma_idesc_bf16(256, a.bn) | (BWD ? kIdescAMnMajor : 0u);
            const uint64_t ad0 = BWD ? umma_desc_mn_sw128(stage_u, kABytes / 2) : umma_desc_sw128(stage_u);
            const uint64_t bd0 = umma_desc_sw128(stage_u + kABytes);
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0, other_phase = 0;
            // what the other CTA wrote and signalled is read: the waits acquire for the cluster
            auto wait_cluster = [&](uint32_t bar, uint32_t parity) {
                bool done_ = mbar_try_wait_cluster(bar, parity);
                if (!__all_sync(0xffffffffu, done_)) {
                    const uint64_t t0 = globaltimer_ns();
                    while (!done_ && !*abort_flag && globaltimer_ns() - t0 <= limit) done_ = mbar_try_wait_cluster(bar, parity);
                    done_ = __all_sync(0xffffffffu, done_);
                }
                return done_;
            };
            for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
                const uint32_t d = tbase + (n & 1) * 256;
                if (!(ok = wait_cluster(smem_u32(&tempty[n & 1]), ((n >> 1) & 1) ^ 1))) break;
                tc_fence_after();
                uint32_t accum = 0;
                auto chunk = [&](int left, int e, int count) {
                    if (!(ok = wait_cluster(full_u + stage * 8, phase))) return;
                    if (e >= 0) {
                        if (!(ok = wait_cluster(smem_u32(&other[stage]), (other_phase >> stage) & 1u))) return;
                        other_phase ^= 1u << stage;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = ad0 + stage * (kPairStageBytes >> 4), bd = bd0 + stage * (kPairStageBytes >> 4);
                        constexpr int kAStep = BWD ? 128 : 2;
                        if (e < 0) {
                            umma_bf16_pair(d, ad, bd, idesc, accum);
                            if (left > 16) umma_bf16_pair(d, ad + kAStep, bd + 2, idesc, 1);
                            if (left > 32) umma_bf16_pair(d, ad + 2 * kAStep, bd + 4, idesc, 1);
                            if (left > 48) umma_bf16_pair(d, ad + 3 * kAStep, bd + 6, idesc, 1);
                        } else {
                            const uint64_t ed = BWD ? ad : adapter_desc(stage_u, pk) + stage * (kPairStageBytes >> 4);
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (pk.step(q, e, count))
                                    umma_bf16_pair(d, ed + (BWD ? kAStep * q : adapter_step(q, pk)), bd + 2 * q, idesc,
                                                   accum || q > 0);
                        }
                        umma_commit_pair(empty_u + stage * 8);
                    }
                    __syncwarp();
                    accum = 1;
                    if (++stage == kPairStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                };
                for (int c = 0; c < kc && ok; ++c) chunk(a.C - c * 64, -1, 0);
                if (!ok || !(ok = warp_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, abort_flag, limit))) break;
                const int count = lists[n & 1].count, n_ext = pk.chunks(count);
                for (int e = 0; e < n_ext && ok; ++e) chunk(0, e, count);
                if (elect_one()) umma_commit_pair(smem_u32(&tfull[n & 1]));
                __syncwarp();
            }
            if (!ok && lane == 0) give_up();
            // all products are complete before TMEM is freed
            if (elect_one()) umma_commit_pair(smem_u32(done));
            __syncwarp();
        } else {
            // the other CTA's workers signal here, and the leader hears of it from this warp: the
            // arrival there takes 500 cycles, which kept them from their next chunk
            bool ok = true;
            int at = 0;
            uint32_t ext_phase = 0;
            for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
                if (!(ok = warp_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, abort_flag, limit))) break;
                const int n_ext = pk.chunks(lists[n & 1].count);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&lfree[n & 1]));
                at += kc;
                for (int e = 0; e < n_ext; ++e, ++at) {
                    const int stage = at % kPairStages;
                    if (!(ok = warp_wait(full_u + stage * 8, (ext_phase >> stage) & 1u, abort_flag, limit))) break;
                    ext_phase ^= 1u << stage;
                    if (lane == 0) mbar_arrive_cluster(lead_other + stage * 8);
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) give_up();
        }
        mbar_wait(smem_u32(done), 0, limit);
    } else if (warp < 6) {
        const int tid = threadIdx.x - 64;
        bool ok = true;
        int stage = 0;
        uint32_t land_phase = 0;
        for (int i = first, n = 0; i < n_tiles && ok; i += step, ++n) {
            const int row0 = (i / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
            TileList& tl = lists[n & 1];
            const bool ready = !*abort_flag && mbar_wait(smem_u32(&lfree[n & 1]), ((n >> 1) & 1) ^ 1, limit);
            for (int q = tid; q < kMaxExtra / 32 && ready; q += 128) tl.odd[q] = 0;
            if (!(ok = tile_adapters(a.adapter_of, row0, rows, a.n_adapters, a.bn, tl.ids, tl.list, bits, &tl.count, a.st,
                                     tid, 128, 1, ready)))
                break;
            if (tid == 0) mbar_arrive(smem_u32(&listed[n & 1]));
            stage = (stage + kc) % kPairStages;
            const int n_ext = pk.chunks(tl.count);
            if (n_ext && !a.v_ready) pdl_wait();
            VRows<1> vr;
            vr.ids(tl.ids + rank * half, half, tl.list, tl.count, tid);
            int held = -1;
            for (int e = 0; e < n_ext; ++e) {
                const int first_of = pk.first(e, tl.count), j0 = pk.j0(e, tl.count);
                if (j0 != held) vr.load(a, row0 + rank * half, held = j0, tid);
                const bool here = !*abort_flag && mbar_wait(landed_u + stage * 8, (land_phase >> stage) & 1u, limit);
                land_phase ^= 1u << stage;
                if (here) {
                    uint8_t* st_a = smem + stage * kPairStageBytes;
                    vr.store(st_a + kABytes, half, first_of, pk.per, tid);
                    if (take_odd<BWD>(st_a, pk.n(e, tl.count) * pk.seg, tid)) atomicOr(&tl.odd[e >> 5], 1u << (e & 31));
                    fence_async_smem();
                }
                if (!(ok = named_and(1, 128, here))) break;
                if (tid == 0) mbar_arrive(full_u + stage * 8);
                if (++stage == kPairStages) stage = 0;
            }
        }
        if (!ok) give_up();
    } else {
        const int q = warp & 3;
        bool ok = true;
        int blocks = 0;
        for (int i = first, n = 0; i < n_tiles; i += step, ++n) {
            const int m0 = (i % m_tiles) * 256 + rank * 128, row0 = (i / m_tiles) * a.bn, rows = min(a.bn, a.T - row0);
            const TileList& tl = lists[n & 1];
            // (in the leader the product warp has read the list before its last commit)
            ok = warp_wait(smem_u32(&listed[n & 1]), (n >> 1) & 1, abort_flag, limit) &&
                 warp_wait(smem_u32(&tfull[n & 1]), (n >> 1) & 1, abort_flag, limit);
            if (!(ok = named_and(2 + (q >> 1), 64, ok))) break;  // (the two warps that share drain_tile's barrier)
            tc_fence_after();
            const int feat = m0 + q * 32 + lane;
            const int n_ext = pk.chunks(tl.count);
            const uint32_t tmem = tbase + (n & 1) * 256 + ((uint32_t)(q * 32) << 16);
            const bool any_odd = has_odd(tl, n_ext);
            const bool copy_out = !a.out_fp32 && !any_odd;
            if (copy_out) drain_tile(a, tmem, stage_u + kPairStages * kPairStageBytes, row0, rows, m0, q, lane, blocks);
            for (int g = 0; g * 16 < rows && !copy_out; ++g) {
                float v[16];
                tmem_ld16(tmem + g * 16, v);
                tmem_ld_wait();
                if (any_odd && feat < a.O) add_odd<BWD>(a, tl, n_ext, row0 + g * 16, g * 16, feat, v);
                __syncwarp();
                store_group(a, row0 + g * 16, rows - g * 16, feat, v);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_cluster(lead_tempty + (n & 1) * 8);
                mbar_arrive(smem_u32(&lfree[n & 1]));
            }
        }
        if (!ok && lane == 0) give_up();
        if (lane == 0) bulk_wait();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) settle_after_timeout();  // (a stage's copies signal the leader, whatever their own CTA has seen)
    __syncwarp();
    cluster_sync();  // neither CTA leaves while the other may signal it or read its memory
    pdl_wait();      // the grid is complete only when the v kernel is
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tbase, 512);
}

// ---------------------------------------------------------------- v = s A x, few tokens
// One CTA per adapter (or, with fewer tokens than adapters, per first token of an adapter),
// JR of its rows and a share of its tokens: the rows stream from memory once for up to NT
// tokens at a time, the eight warps share the contraction.  The rows are what there is to
// read, so many small CTAs keep them coming.  It ends sooner than the tensor-core kernel,
// whose 128-token tiles multiply every token with every adapter of the tile, while tokens
// x rank is small (32 tokens, rank 16: 4 against 13 us; 192 tokens, rank 32: 5 against 12).
constexpr int kFewTokens = 64;
constexpr int kFewProducts = 8192;  // tokens x rank
constexpr int kFewShares = 4;       // of an adapter's tokens at most, one for 16 tokens of the batch
constexpr int JR = 2, NT = 8;

__device__ __forceinline__ void dot8(float& acc, const uint4& p, const uint4& q) {
    const uint32_t* x = &p.x;
    const uint32_t* y = &q.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), acc);
        acc = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), acc);
    }
}

template <int N>
__device__ __forceinline__ void few_dots(const uint4* const (&xr)[NT], const uint4* const (&ar)[JR], int nv, int tid,
                                         float (&acc)[NT][JR]) {
#pragma unroll 2
    for (int k = tid; k < nv; k += 256) {
        uint4 av[JR], xv[N];
#pragma unroll
        for (int j = 0; j < JR; ++j) av[j] = __ldg(ar[j] + k);
#pragma unroll
        for (int n = 0; n < N; ++n) xv[n] = __ldg(xr[n] + k);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int j = 0; j < JR; ++j) dot8(acc[n][j], xv[n], av[j]);
    }
}

__global__ void __launch_bounds__(256, 3) shrink_few_kernel(const uint16_t* x, const uint16_t* m, const float* scaling,
                                                         const int32_t* adapter_of, int T, int C, int r, int n_adapters,
                                                         uint16_t* v, DevStatus st) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float part[8][NT][JR];
    __shared__ uint16_t mine[kFewTokens];  // the adapter's tokens, ascending
    __shared__ int counts[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool by_token = T < n_adapters;
    const int of = tid < T ? adapter_of[tid] : -2;
    const int id = by_token ? adapter_of[blockIdx.x] : (int)blockIdx.x;
    if (blockIdx.y == 0 && blockIdx.z == 0 && tid < T && (of < 0 || of >= n_adapters) &&
        (by_token ? tid == (int)blockIdx.x : blockIdx.x == 0)) {
        // a token without adapter: v = 0
        if (of != -1) raise_status(st, kStatusInvalidExpert);
        for (int j = 0; j < r; j += 8) *reinterpret_cast<uint4*>(v + (size_t)tid * r + j) = make_uint4(0, 0, 0, 0);
    }
    if (id < 0 || id >= n_adapters) return;
    const uint32_t here = __ballot_sync(0xffffffffu, of == id);
    if (lane == 0) counts[warp] = __popc(here);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        before += w < warp ? counts[w] : 0;
        total += counts[w];
    }
    if (of == id) mine[before + __popc(here & ((1u << lane) - 1u))] = (uint16_t)tid;
    __syncthreads();
    // (with fewer tokens than adapters, an earlier token of the same adapter does the work)
    if ((int)blockIdx.z * NT >= total || (by_token && mine[0] != blockIdx.x)) return;
    const int j0 = blockIdx.y * JR;
    const uint4* ar[JR];
#pragma unroll
    for (int j = 0; j < JR; ++j) ar[j] = reinterpret_cast<const uint4*>(m + ((size_t)id * r + j0 + j) * C);
    const float scale = scaling ? scaling[id] : 1.0f;
    for (int q0 = blockIdx.z * NT; q0 < total; q0 += gridDim.z * NT) {
        const int n = min(NT, total - q0);
        const uint4* xr[NT];
#pragma unroll
        for (int q = 0; q < NT; ++q) xr[q] = reinterpret_cast<const uint4*>(x + (size_t)mine[q0 + min(q, n - 1)] * C);
        float acc[NT][JR] = {};
        if (n == 1) few_dots<1>(xr, ar, C / 8, tid, acc);
        else if (n == 2) few_dots<2>(xr, ar, C / 8, tid, acc);
        else if (n <= 4) few_dots<4>(xr, ar, C / 8, tid, acc);
        else few_dots<NT>(xr, ar, C / 8, tid, acc);
        __syncthreads();  // part is free
#pragma unroll
        for (int q = 0; q < NT; ++q) {
            if (q >= n) break;
#pragma unroll
            for (int j = 0; j < JR; ++j) {
                float f = acc[q][j];
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) f += __shfl_xor_sync(0xffffffffu, f, d);
                if (lane == 0) part[warp][q][j] = f;
            }
        }
        __syncthreads();
        if (tid < n * JR) {
            const int q = tid / JR, j = tid % JR;
            float f = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) f += part[w][q][j];
            v[(size_t)mine[q0 + q] * r + j0 + j] = to_bf(f * scale);  // (the one rounding of v)
        }
    }
}

// ---------------------------------------------------------------- v and dv, many tokens
// D[128 tokens][columns] = X tile . [A_i of the tile's adapters, stacked]^T on the tensor
// cores: every token is multiplied with every adapter of its tile and keeps its own
// columns, so the tokens are read once whatever their order.  Bound by reading them: 4096 x
// 7168 (58 MB) at rank 64 takes 12 us in a stream of calls.  Up to 256 columns at a time
// (`per_pass` adapters); clusters share the contraction.  Backward: dY . B_i, with B_i
// read MN-major.
struct ShrinkArgs {
    CUtensorMap x;   // box {64, 1, 128} of x [T][K] | dy [T][N]
    CUtensorMap m;   // forward: box {64 k, cols} of A [n][r][K]; backward: box {64 r, 64 n} of B [n][N][r]
    const float* scaling;
    const int32_t* adapter_of;
    int T, C, r, n_adapters;
    int cols;        // columns of one adapter: r rounded up to 16 (forward) or 64 (backward)
    int per_pass;    // adapters of a pass: 256 / cols at most
    int splits, passes;  // CTAs per cluster; passes that run at the same time
    int ring;        // bytes of the stages
    uint16_t* v;     // [T][r]
    DevStatus st;
};
// A stage is the tokens' 16 KB and as much of A as the pass needs: as many as fit, up to 12.
constexpr int kShrinkRing = 192 * 1024;
constexpr int kShrinkStages = 12;
constexpr int kShrinkThreads = 192;
constexpr int kShrinkExtra = 1024 + 256 + 128 * 8 + kMaxAdapters / 8;
// An allocation of tensor memory waits until the columns are free.  It must not wait for a
// kernel that waits for its own, nor for a CTA that waits for this one's cluster, so
// whatever shares an SM fits its 512 columns at the same time:
//  - the rank product, the first kernel of a call, takes its columns when the kernel before has
//    ended, whatever that was (the layer's GEMM starts the next kernel before it has its own);
//  - the kernels of a call let the next one start only when their CTAs have their columns;
//  - at most two of these CTAs (256 columns each) are on an SM, none beside one that holds
//    all 512: a short ring is filled up to a third of an SM's shared memory and more.
constexpr int kShrinkLeast = 77 * 1024;
constexpr int kSmShared = 228 * 1024;
static_assert(3 * kShrinkLeast > kSmShared, "a third CTA would wait for columns");
static_assert(kShrinkLeast + kPairSmem > kSmShared && kShrinkLeast + ProjCfg<256>::kSmemBytes > kSmShared,
              "a projection would wait for columns");
static_assert(2 * kShrinkLeast + ProjCfg<32>::kSmemBytes > kSmShared && ProjCfg<128>::kTmemCols <= 256,
              "a projection beside one of these CTAs has the columns that it needs");

template <bool BWD>
__global__ void __launch_bounds__(kShrinkThreads, 1) shrink_kernel(const __grid_constant__ ShrinkArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + a.ring);
    uint64_t* empty = full + kShrinkStages;
    uint64_t* tfull = empty + kShrinkStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* count = reinterpret_cast<int*>(tmem_slot + 2);
    int* ids = reinterpret_cast<int*>(smem + a.ring + 256);
    int* list = ids + 128;
    uint32_t* bits = reinterpret_cast<uint32_t*>(list + 128);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int S = a.splits;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int pass0 = (blockIdx.x / S) % a.passes;
    const int row0 = (blockIdx.x / S / a.passes) * 128, rows = min(128, a.T - row0);
    const int kc = (a.C + 63) / 64;
    const int c0 = (int)((long)kc * rank / S), c1 = (int)((long)kc * (rank + 1) / S);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kShrinkStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.x);
        tma_prefetch_desc(&a.m);
    }
    pdl_wait();
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tbase = *tmem_slot;
    tile_adapters(a.adapter_of, row0, rows, a.n_adapters, 128, ids, list, bits, count, a.st, threadIdx.x, kShrinkThreads, 1);
    const int n_list = *count;
    if (pass0 == 0 && rank == 0)
        for (int q = threadIdx.x; q < rows * (a.r / 8); q += kShrinkThreads)
            if (ids[q / (a.r / 8)] < 0)
                *reinterpret_cast<uint4*>(a.v + (size_t)row0 * a.r + (size_t)q * 8) = make_uint4(0, 0, 0, 0);

    uint32_t phase = 0, acc_phase = 0;  // phase: parity of each stage's next use
    uint32_t armed = 0;                 // stages ever filled
    const uint32_t full_u = smem_u32(full), empty_u = smem_u32(empty), ring_u = smem_u32(smem);
    bool ok = true;
    for (int pass = pass0; pass * a.per_pass < n_list; pass += a.passes) {
        const int cnt = min(a.per_pass, n_list - pass * a.per_pass);
        const int* mine = list + pass * a.per_pass;
        const int stage_bytes = 16384 + cnt * a.cols * 128;
        const int stages = min(kShrinkStages, a.ring / stage_bytes);
        int stage = 0;
        if (warp == 0) {
            const uint64_t pol = policy_evict_normal();
            for (int c = c0; c < c1 && ok; ++c) {
                if (!(ok = warp_wait(empty_u + stage * 8, ((phase >> stage) & 1u) ^ 1, abort_flag, limit))) break;
                if (elect_one()) {
                    const uint32_t sx = ring_u + stage * stage_bytes, sm = sx + 16384, fb = full_u + stage * 8;
                    mbar_arrive_expect_tx(fb, stage_bytes);
                    tma_load_3d(sx, &a.x, fb, c * 64, 0, row0, pol);
                    for (int p = 0; p < cnt; ++p) {
                        if (BWD) {
                            for (int j0 = 0; j0 < a.cols; j0 += 64)
                                tma_load_3d(sm + (p * a.cols + j0) * 128, &a.m, fb, j0, c * 64, mine[p], pol);
                        } else {
                            tma_load_3d(sm + p * a.cols * 128, &a.m, fb, c * 64, 0, mine[p], pol);
                        }
                    }
                }
                __syncwarp();
                armed |= 1u << stage;
                phase ^= 1u << stage;
                if (++stage == stages) stage = 0;
            }
        } else if (warp == 1) {
            const uint32_t idesc = umma_idesc_bf16(128, cnt * a.cols) | (BWD ? kIdescBMnMajor : 0u);
            const uint64_t ad0 = umma_desc_sw128(ring_u);
            const uint64_t bd0 = BWD ? umma_desc_mn_sw128(ring_u + 16384, 8192) : umma_desc_sw128(ring_u + 16384);
            for (int c = c0; c < c1 && ok; ++c) {
                if (!(ok = warp_wait(full_u + stage * 8, (phase >> stage) & 1u, abort_flag, limit))) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = ad0 + stage * (stage_bytes >> 4), bd = bd0 + stage * (stage_bytes >> 4);
                    constexpr int kBStep = BWD ? 128 : 2;
                    const int left = a.C - c * 64;
                    umma_bf16(tbase, ad, bd, idesc, c > c0);
                    if (left > 16) umma_bf16(tbase, ad + 2, bd + kBStep, idesc, 1);
                    if (left > 32) umma_bf16(tbase, ad + 4, bd + 2 * kBStep, idesc, 1);
                    if (left > 48) umma_bf16(tbase, ad + 6, bd + 3 * kBStep, idesc, 1);
                    umma_commit(empty_u + stage * 8);
                }
                __syncwarp();
                phase ^= 1u << stage;
                if (++stage == stages) stage = 0;
            }
            if (elect_one()) umma_commit(smem_u32(tfull));  // on a failure too: the products issued so far end
            __syncwarp();
        } else {
            // each token's own columns into this CTA's share, [column][token]
            if (ok) ok = __all_sync(0xffffffffu, warp_wait(smem_u32(tfull), acc_phase, abort_flag, limit) && !*abort_flag);
            if (ok) {
                tc_fence_after();
                const int q = warp & 3, row = q * 32 + lane;
                float* part = reinterpret_cast<float*>(smem) + row;
                for (int p = 0; p < cnt; ++p) {
                    const bool own = ids[row] == mine[p];
                    if (!__any_sync(0xffffffffu, own)) continue;
                    for (int g = 0; g * 16 < a.r; ++g) {
                        float f[16];
                        tmem_ld16(tbase + ((uint32_t)(q * 32) << 16) + p * a.cols + g * 16, f);
                        tmem_ld_wait();
                        if (own) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) part[(g * 16 + j) * 128] = f[j];
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
            }
        }
        acc_phase ^= 1;
        if (!ok) {
            *abort_flag = 1;
            raise_status(a.st, kStatusWaitTimeout);
        }
        __syncwarp();
        if (S > 1) cluster_sync();
        else __syncthreads();
        tc_fence_after();
        const int items = 128 * (a.r / 8);
        const int i0 = (int)((long)items * rank / S), i1 = (int)((long)items * (rank + 1) / S);
        for (int i = i0 + threadIdx.x; i < i1 && !*abort_flag; i += kShrinkThreads) {
            const int row = i & 127, j0 = (i >> 7) * 8;
            const int id = ids[row];
            if (row >= rows || id < mine[0] || id > mine[cnt - 1]) continue;  // (the list ascends)
            const float scale = a.scaling ? a.scaling[id] : 1.0f;
            float f[8];
            const uint32_t addr = smem_u32(smem) + (j0 * 128 + row) * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
#pragma unroll 4
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] += S > 1 ? ld_peer(addr + j * 512, s) : reinterpret_cast<const float*>(smem)[(j0 + j) * 128 + row];
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)  // (the one rounding of v or dv)
                w[j] = (uint32_t)to_bf(f[2 * j] * scale) | ((uint32_t)to_bf(f[2 * j + 1] * scale) << 16);
            *reinterpret_cast<uint4*>(a.v + (size_t)(row0 + row) * a.r + j0) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // the shares have been read before the next pass writes the stages
        fence_async_smem();
        if (S > 1) cluster_sync_read();
        else __syncthreads();
    }
    if (warp == 0)
        for (int s = 0; s < kShrinkStages; ++s)
            if ((armed >> s) & 1u) mbar_wait(full_u + s * 8, ((phase >> s) & 1u) ^ 1, limit);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, 256);
}

// ---------------------------------------------------------------- dA and dB
// dA_i^T [features][r] = sum over i's tokens of x[t] dv[t]^T (dB_i: dy[t] v[t]^T): one CTA
// (or cluster, splitting the tokens) per adapter and 256 features walks the 64-token chunks
// that hold tokens of its adapter, and reads nothing else.  Both operands are MN-major (the
// contraction runs over tokens).  In a chunk with other tokens too, their rows are set to
// zero in shared memory, in both operands, so whatever they hold stays out.  What bounds
// it is reading the tokens (40 KB a chunk at rank 64, five in flight) and the adapter with
// the most of them: 4096 tokens of 4 adapters, 7168 and 2048 features, 25 us, where the 75 MB
// take 11.
struct GradArgs {
    CUtensorMap z[2];  // box {64 features, 64 tokens} of x [T][K], dy [T][N]
    CUtensorMap u[2];  // box {64 r, 64 tokens} of dv, v [T][r]
    const int32_t* adapter_of;
    int T, r;
    int F[2];          // K, N
    int splits;        // CTAs of a cluster
    uint16_t* out[2];  // da [n][r][K], db [n][N][r]
    DevStatus st;
};
constexpr int kGradThreads = 192;
constexpr int kGradSegment = 4096;  // chunks whose list is held at a time

template <int RB>  // 64-column blocks of the rank
struct GradCfg {
    static constexpr int kStageBytes = 32768 + RB * 8192;
    // (two CTAs of two stages on an SM took 37 us where one of five takes 26)
    static constexpr int kStages = RB == 1 ? 5 : RB == 2 ? 4 : 3;
    static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 256 + kGradSegment * 2;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory overflow");
};

template <int RB>
__global__ void __launch_bounds__(kGradThreads, 1) grad_kernel(const __grid_constant__ GradArgs a) {
    using C = GradCfg<RB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* landed = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
    uint64_t* full = landed + C::kStages;
    uint64_t* empty = full + C::kStages;
    uint64_t* done = empty + C::kStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* count = reinterpret_cast<volatile int*>(tmem_slot + 2);
    // chunks of the segment with tokens of the adapter, + 0x8000 where there are others too
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + C::kStages * C::kStageBytes + 256);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int id = blockIdx.y;
    const int S = a.splits;
    const int rank = S > 1 ? (int)cluster_rank() : 0;
    const int blocks0 = (a.F[0] + 255) / 256;
    const int block = blockIdx.x / S;
    const int side = block >= blocks0;
    const int f0 = (block - (side ? blocks0 : 0)) * 256;
    const int F = a.F[side];
    const int chunks = (a.T + 63) / 64;
    constexpr int kTmemCols = 2 * RB * 64;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(smem_u32(&landed[s]), 1);
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.z[side]);
        tma_prefetch_desc(&a.u[side]);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const uint32_t landed_u = smem_u32(landed), full_u = smem_u32(full), empty_u = smem_u32(empty), stage_u = smem_u32(smem);
    pdl_wait();
    pdl_launch_dependents();  // (dx's projection, which needs nothing of this kernel)

    int stage = 0;
    uint32_t phase = 0, accum = 0, armed = 0, armed_phase = 0;
    bool ok = true, none = true;
    int ordinal = 0;  // of the segment's first listed chunk among all
    for (int seg = 0; seg < chunks; seg += kGradSegment) {
        const int n = min(kGradSegment, chunks - seg);
        // marks, eight chunks of a warp at a time: 0 no token of the adapter, 1 some, 2 all
        for (int c0 = warp * 8; c0 < n; c0 += kGradThreads / 32 * 8) {
            int of[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const long t = (long)(seg + c0) * 64 + q * 32 + lane;
                of[q] = t < a.T ? a.adapter_of[t] : -2;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const bool any = __any_sync(0xffffffffu, of[2 * q] == id || of[2 * q + 1] == id);
                const bool all = __all_sync(0xffffffffu, (of[2 * q] == id || of[2 * q] == -2) &&
                                                             (of[2 * q + 1] == id || of[2 * q + 1] == -2));
                if (lane == 0 && c0 + q < n) list[c0 + q] = any ? (all ? 2 : 1) : 0;
            }
        }
        __syncthreads();
        if (warp == 0) {  // compacted in place, in order
            int at = 0;
            for (int c = lane; c - lane < n; c += 32) {
                const int mark = c < n ? list[c] : 0;
                const uint32_t b = __ballot_sync(0xffffffffu, mark != 0);
                __syncwarp();
                if (mark) list[at + __popc(b & ((1u << lane) - 1u))] = (uint16_t)(c | (mark == 1 ? 0x8000 : 0));
                at += __popc(b);
                __syncwarp();
            }
            if (lane == 0) *count = at;
        }
        __syncthreads();
        const int cnt = *count;
        if (cnt) none = false;
        const int q0 = (rank - ordinal % S + S) % S;  // every S-th listed chunk is this CTA's
        ordinal += cnt;
        if (warp == 0) {
            const uint64_t pol = policy_evict_normal();
            for (int q = q0; q < cnt && ok; q += S) {
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                if (elect_one()) {
                    const uint32_t sz = stage_u + stage * C::kStageBytes, lb = landed_u + stage * 8;
                    const int t0 = (seg + (list[q] & 0x7fff)) * 64;
                    mbar_arrive_expect_tx(lb, C::kStageBytes);
#pragma unroll
                    for (int b = 0; b < 4; ++b) tma_load_3d(sz + b * 8192, &a.z[side], lb, f0 + b * 64, t0, 0, pol);
#pragma unroll
                    for (int b = 0; b < RB; ++b) tma_load_3d(sz + 32768 + b * 8192, &a.u[side], lb, b * 64, t0, 0, pol);
                }
                __syncwarp();
                armed |= 1u << stage;
                armed_phase = (armed_phase & ~(1u << stage)) | (phase << stage);
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        } else if (warp == 1) {
            const uint32_t idesc = umma_idesc_bf16(128, (a.r + 15) & ~15) | kIdescAMnMajor | kIdescBMnMajor;
            const uint64_t ad0 = umma_desc_mn_sw128(stage_u, 8192), bd0 = umma_desc_mn_sw128(stage_u + 32768, 8192);
            for (int q = q0; q < cnt && ok; q += S) {
                if (!(ok = warp_wait(full_u + stage * 8, phase, abort_flag, limit))) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = ad0 + stage * (C::kStageBytes >> 4), bd = bd0 + stage * (C::kStageBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        umma_bf16(tbase, ad + 128 * k, bd + 128 * k, idesc, k > 0 ? 1 : accum);
                        umma_bf16(tbase + RB * 64, ad + 1024 + 128 * k, bd + 128 * k, idesc, k > 0 ? 1 : accum);
                    }
                    umma_commit(empty_u + stage * 8);
                }
                __syncwarp();
                accum = 1;
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        } else {
            const int tid = threadIdx.x - 64;
            // (to the end of the list whatever happens: the barrier is for all four warps)
            for (int q = q0; q < cnt; q += S) {
                if (ok && !(ok = warp_wait(landed_u + stage * 8, phase, abort_flag, limit))) *abort_flag = 1;
                if (list[q] & 0x8000) {
                    const int t0 = (seg + (list[q] & 0x7fff)) * 64;
                    uint8_t* sz = smem + stage * C::kStageBytes;
                    // 8 threads per token row; the 128-byte rows of all blocks
                    for (int row = tid >> 3; row < 64 && ok; row += 16) {
                        if (t0 + row < a.T && a.adapter_of[t0 + row] == id) continue;
#pragma unroll
                        for (int b = 0; b < 4 + RB; ++b)
                            *reinterpret_cast<uint4*>(sz + b * 8192 + row * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    named_sync(1, 128);
                }
                if (tid == 0 && ok) mbar_arrive(full_u + stage * 8);
                if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            *abort_flag = 1;
            raise_status(a.st, kStatusWaitTimeout);
        }
        __syncthreads();  // the list is rewritten
    }
    // this CTA's share of the chunks may be empty: its accumulators were then never written
    const bool empty_share = none || ordinal <= rank;
    if (warp == 0) {
        for (int s = 0; s < C::kStages; ++s)
            if ((armed >> s) & 1u) mbar_wait(landed_u + s * 8, (armed_phase >> s) & 1u, limit);
    } else if (warp == 1) {
        if (elect_one()) umma_commit(smem_u32(done));
        __syncwarp();
        mbar_wait(smem_u32(done), 0, limit);
    } else {
        // (the same for every lane, with its warp's loads and shuffles below)
        ok = __all_sync(0xffffffffu, warp_wait(smem_u32(done), 0, abort_flag, limit) && !*abort_flag);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();  // also: the drained stages may hold the shares of a split sum
    tc_fence_after();
    const int q = warp & 3;
    uint16_t* out = a.out[side];
    // 16 columns of this lane's feature, in words of two columns
    auto store16 = [&](int feat, int j0, const float (&f)[16]) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = (uint32_t)to_bf(f[2 * j]) | ((uint32_t)to_bf(f[2 * j + 1]) << 16);
        if (side) {  // db_i [feature][r]
            if (feat < F) {
                uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)id * F + feat) * a.r + j0);
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                if (j0 + 8 < a.r) dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            return;
        }
        // da_i [r][feature], words of two features (as in the projection)
        const bool odd = lane & 1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, w[j], 1);
            const uint32_t p = __byte_perm(w[j], o, odd ? 0x3276 : 0x5410);
            const int col = j0 + 2 * j + (odd ? 1 : 0);
            if (feat < F && col < a.r)
                *reinterpret_cast<uint32_t*>(out + ((size_t)id * a.r + col) * F + (feat & ~1)) = p;
        }
    };
    float* part = reinterpret_cast<float*>(smem);  // split sums: [column][256 features]
    if (warp >= 2 && ok) {
        for (int h = 0; h < 2; ++h)
            for (int g = 0; g * 16 < a.r; ++g) {
                float f[16];
                tmem_ld16(tbase + h * RB * 64 + ((uint32_t)(q * 32) << 16) + g * 16, f);
                tmem_ld_wait();
                if (empty_share) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) f[j] = 0.0f;
                }
                const int feat = h * 128 + q * 32 + lane;
                if (S > 1) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) part[(g * 16 + j) * 256 + feat] = f[j];
                } else {
                    store16(f0 + feat, g * 16, f);
                }
            }
        tc_fence_before();
    }
    if (S > 1) {
        __syncwarp();
        cluster_sync();
        // (16 columns, 32 features) at a time, the warps of the cluster in turn
        const int groups = (a.r + 15) / 16 * 8;
        for (int w = rank * (kGradThreads / 32) + warp; w < groups && !*abort_flag; w += S * (kGradThreads / 32)) {
            const int g = w >> 3, feat = (w & 7) * 32 + lane;
            float f[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] = 0.0f;
            // (only what is stored is read: see cluster_sync_read)
            for (int s = 0; s < S && f0 + feat < F; ++s)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (g * 16 + j < a.r) f[j] += ld_peer(stage_u + ((g * 16 + j) * 256 + feat) * 4, s);
            store16(f0 + feat, g * 16, f);
        }
        cluster_sync_read();
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tbase, kTmemCols);
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

template <typename Kern>
cudaError_t launch_project(Kern kern, std::atomic<uint64_t>& configured, int smem, int grid, int cluster,
                           cudaStream_t stream, const ProjArgs& a) {
    const cudaError_t e = configure_once(
        configured, [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kern, dim3(grid), dim3(kThreads), smem, stream, cluster, a);
}

template <bool BWD, int BN>
cudaError_t launch_project_bn(const ProjArgs& a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    return launch_project(project_kernel<BWD, BN>, configured, ProjCfg<BN>::kSmemBytes, grid, a.splits, stream, a);
}

template <bool BWD>
cudaError_t launch_project_pair(const ProjArgs& a, int grid, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    return launch_project(project_pair_kernel<BWD>, configured, kPairSmem, grid, 2, stream, a);
}

// Clusters of `size` CTAs that are resident at a time, where a CTA fills an SM (or `two` fit
// one): processors come in groups that a cluster does not cross (15 clusters of 8 and 36 of 4
// of 152 SMs).  Asked once per device.
int active_clusters(int size, bool two) {
    if (size == 1) return num_sms() * (two ? 2 : 1);
    static std::atomic<int> known[64][2][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms() / (2 * size);
    int n = known[dev][two][size].load(std::memory_order_relaxed);
    if (n) return n;
    auto kern = two ? project_kernel<false, 32> : project_kernel<false, 256>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = two ? ProjCfg<32>::kSmemBytes : ProjCfg<256>::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        n = std::max(1, num_sms() / (2 * size));
    }
    known[dev][two][size].store(n, std::memory_order_relaxed);
    return n;
}

// CTAs per cluster, up to `most`, that share `chunks` of contraction of each of `tiles`: the
// least of rounds x (a CTA's chunks + 8 for its start and end), at least four chunks each.
int split_of(long tiles, int chunks, int most, bool two) {
    int at = 1;
    long best = -1;
    for (int s = 1; s <= most && (s == 1 || s * 4 <= chunks); ++s) {
        const long slots = active_clusters(s, two);
        const long cost = (tiles + slots - 1) / slots * ((chunks + s - 1) / s + 8 + (s > 1 ? 1 : 0));
        if (best < 0 || cost < best) {
            best = cost;
            at = s;
        }
    }
    return at;
}

// How a projection of T tokens to O features is cut: token capacity and tokens per tile,
// CTAs that share a tile's contraction, or pairs of CTAs; grid.
struct ProjPlan {
    int cap, bn, splits, pair, grid;
};

// The tile height, a multiple of `by` in [128, 256], whose rounds over `slots` cost least:
// rounds x (tokens + 16 for the accumulator's hand-over).
int tile_height(int T, int units, int slots, int by) {
    int at = 256;
    long best = -1;
    for (int bn = 256; bn >= 128; bn -= by) {
        const long tiles = (long)units * ((T + bn - 1) / bn);
        const long cost = (tiles + slots - 1) / slots * (bn + 16);
        if (best < 0 || cost < best) {
            best = cost;
            at = bn;
        }
    }
    return at;
}

ProjPlan project_plan(int T, int O, int C, int r, int n_adapters) {
    ProjPlan p;
    const int sms = num_sms(), m_tiles = (O + 127) / 128, kc = (C + 63) / 64;
    p.cap = T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
    p.bn = T > 256 ? tile_height(T, m_tiles, sms, 16) : (T + 15) / 16 * 16;
    const long tiles = (long)m_tiles * ((T + p.bn - 1) / p.bn);
    // (a small batch may hold as many adapters as tokens, and each adds a chunk per 64 of its rank)
    const int held = T <= 256 ? std::min(T, n_adapters) : 2;
    const int extra = r <= 16 ? (held + 3) / 4 : r <= 32 ? (held + 1) / 2 : held * ((r + 63) / 64);
    const bool many = T > 128 && (long)m_tiles * ((T + 255) / 256) >= sms;
    p.splits = !many && tiles < 2 * sms ? split_of(tiles, kc + extra, 8, p.cap <= 64) : 1;
    // As many tiles as SMs, or a long contraction that no cluster shares: pairs of CTAs.  (4096
    // tokens, 4608 to 1024 features, a backward pass without gradients: 64 pairs 39 us, 128 CTAs
    // on their own 44; 2933 tokens, 1992 to 400: 25 and 27.  A pair begins later: 2048 tokens,
    // 1024 to 1024, 16 and 15 us.)
    p.pair = many || (T > 128 && p.splits == 1 && kc >= 31);
    if (p.pair) {
        const int units = (O + 255) / 256, slots = sms / 2;
        p.cap = 256;
        p.bn = tile_height(T, units, slots, 32);
        p.grid = 2 * (int)std::min<long>((long)units * ((T + p.bn - 1) / p.bn), slots);
        return p;
    }
    p.grid = p.splits > 1 ? (int)tiles * p.splits : (int)std::min<long>(tiles, sms);
    return p;
}

// tokens [T][C] times W (and each token's low-rank matrix times v) into out [T][O]
template <bool BWD>
int project(const moe_adapter_t* p, int T, const void* tokens, const void* w, const void* lr, const int32_t* adapter_of,
            const void* v, bool v_ready, void* out, int out_fp32, const DevStatus& st, cudaStream_t stream) {
    const uint64_t K = p->in_features, N = p->out_features, r = p->rank, n = p->n_adapters;
    ProjArgs a;
    a.T = T;
    a.O = BWD ? p->in_features : p->out_features;
    a.C = BWD ? p->out_features : p->in_features;
    a.r = p->rank;
    a.n_adapters = p->n_adapters;
    const ProjPlan plan = project_plan(T, a.O, a.C, a.r, a.n_adapters);
    a.bn = plan.bn;
    a.splits = plan.splits;
    a.v_ready = v_ready;
    int rc = make_tmap_rows(&a.w, w, K, N, 1, K * 2, K * N * 2, 64, BWD ? 64 : 128, 1);
    if (rc) return rc;
    const uint32_t seg = a.r <= 16 ? 16 : a.r <= 32 ? 32 : 64;  // (as Packing)
    if (BWD) rc = make_tmap_rows(&a.lr, lr, K, r, n, K * 2, K * r * 2, 64, seg, 1);
    else rc = make_tmap_rows(&a.lr, lr, r, N, n, r * 2, r * N * 2, seg, 128, 1, seg * 2);
    if (rc) return rc;
    const uint64_t C = a.C;
    if ((rc = make_tmap_rows(&a.x, tokens, C, 1, (uint64_t)T, C * 2, C * 2, 64, 1, plan.pair ? plan.bn / 2 : plan.bn))) return rc;
    const uint64_t O = a.O;
    if (!out_fp32 && (rc = make_tmap_rows(&a.y, out, O, 1, (uint64_t)T, O * 2, O * 2, 64, 1, 16))) return rc;
    a.lr_ptr = static_cast<const uint16_t*>(lr);
    a.adapter_of = adapter_of;
    a.v = static_cast<const uint16_t*>(v);
    a.out = out;
    a.out_fp32 = out_fp32;
    a.st = st;
    const cudaError_t e = plan.pair         ? launch_project_pair<BWD>(a, plan.grid, stream)
                          : plan.cap == 32  ? launch_project_bn<BWD, 32>(a, plan.grid, stream)
                          : plan.cap == 64  ? launch_project_bn<BWD, 64>(a, plan.grid, stream)
                          : plan.cap == 128 ? launch_project_bn<BWD, 128>(a, plan.grid, stream)
                                            : launch_project_bn<BWD, 256>(a, plan.grid, stream);
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "adapter projection launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

// v = scaling * (the token's A) . x, or dv = scaling * (the token's B)^T . dy
template <bool BWD>
int shrink(const moe_adapter_t* p, int T, const void* tokens, const void* m, const float* scaling,
           const int32_t* adapter_of, void* v, const DevStatus& st, cudaStream_t stream) {
    const int C = BWD ? p->out_features : p->in_features;
    cudaError_t e;
    if (!BWD && T <= kFewTokens && (long)T * p->rank <= kFewProducts) {
        e = launch_pdl(shrink_few_kernel, dim3(std::min(T, p->n_adapters), p->rank / JR, std::min((T + 15) / 16, kFewShares)), dim3(256),
                       0, stream,
                       static_cast<const uint16_t*>(tokens), static_cast<const uint16_t*>(m), scaling, adapter_of, T, C,
                       (int)p->rank, (int)p->n_adapters, static_cast<uint16_t*>(v), st);
    } else {
        ShrinkArgs a;
        const uint64_t c = C, r = p->rank, n = p->n_adapters;
        int rc = make_tmap_rows(&a.x, tokens, c, 1, (uint64_t)T, c * 2, c * 2, 64, 1, 128);
        if (rc) return rc;
        a.cols = BWD ? (p->rank + 63) / 64 * 64 : (p->rank + 15) / 16 * 16;
        a.per_pass = 256 / a.cols;
        if (BWD) rc = make_tmap_rows(&a.m, m, r, c, n, r * 2, r * c * 2, 64, 64, 1);
        else rc = make_tmap_rows(&a.m, m, c, r, n, c * 2, c * r * 2, 64, a.cols, 1);
        if (rc) return rc;
        a.scaling = scaling;
        a.adapter_of = adapter_of;
        a.T = T;
        a.C = C;
        a.r = p->rank;
        a.n_adapters = p->n_adapters;
        a.v = static_cast<uint16_t*>(v);
        a.st = st;
        // clusters share the contraction
        const int tiles = (T + 127) / 128, kc = (C + 63) / 64;
        a.splits = split_of(tiles, kc, 8, false);
        // A tile's adapters in as many passes side by side as clusters are resident, so narrower
        // ones than 256 columns where there are few tiles.
        const int most = std::min(std::min(T, 128), p->n_adapters), beside = std::max(1, active_clusters(a.splits, false) / tiles);
        a.per_pass = std::min(a.per_pass, (most + beside - 1) / beside);
        a.passes = std::min((most + a.per_pass - 1) / a.per_pass, beside);
        // a stage per chunk of the CTA's share at most (and room for its sums)
        const int pass_cols = std::min(a.per_pass, p->n_adapters) * a.cols, share = (kc + a.splits - 1) / a.splits;
        a.ring = (int)std::min<long>(kShrinkRing, std::max((long)share * (16384 + pass_cols * 128), (p->rank + 15L) / 16 * 16 * 512));
        a.ring = (a.ring + 1023) / 1024 * 1024;
        auto kern = shrink_kernel<BWD>;
        static std::atomic<uint64_t> configured{0};
        e = configure_once(configured, [&] {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kShrinkRing + kShrinkExtra);
        });
        if (e == cudaSuccess)
            e = launch_pdl_cluster(kern, dim3(tiles * a.passes * a.splits), dim3(kShrinkThreads),
                                   std::max(a.ring + kShrinkExtra, kShrinkLeast), stream, a.splits, a);
    }
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "adapter rank-product launch: %s", cudaGetErrorString(e));
    return MOE_OK;
}

template <int RB>
cudaError_t launch_grad_rb(const GradArgs& a, int n_adapters, cudaStream_t stream) {
    auto kern = grad_kernel<RB>;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = configure_once(configured, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, GradCfg<RB>::kSmemBytes);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kern, dim3(((a.F[0] + 255) / 256 + (a.F[1] + 255) / 256) * a.splits, n_adapters),
                              dim3(kGradThreads), GradCfg<RB>::kSmemBytes, stream, a.splits, a);
}

int gradients(const moe_adapter_t* p, int T, const void* dy, const void* x, const void* dv, const void* v,
              const int32_t* adapter_of, void* da, void* db, const DevStatus& st, cudaStream_t stream) {
    GradArgs a;
    const uint64_t K = p->in_features, N = p->out_features, r = p->rank, t = T;
    int rc;
    if ((rc = make_tmap_rows(&a.z[0], x, K, t, 1, K * 2, K * t * 2, 64, 64, 1)) ||
        (rc = make_tmap_rows(&a.z[1], dy, N, t, 1, N * 2, N * t * 2, 64, 64, 1)) ||
        (rc = make_tmap_rows(&a.u[0], dv, r, t, 1, r * 2, r * t * 2, 64, 64, 1)) ||
        (rc = make_tmap_rows(&a.u[1], v, r, t, 1, r * 2, r * t * 2, 64, 64, 1)))
        return rc;
    a.adapter_of = adapter_of;
    a.T = T;
    a.r = p->rank;
    a.F[0] = p->in_features;
    a.F[1] = p->out_features;
    a.out[0] = static_cast<uint16_t*>(da);
    a.out[1] = static_cast<uint16_t*>(db);
    a.st = st;
    const int rb = (p->rank + 63) / 64;
    // few adapters: clusters split the tokens (the shares of ranks above 128 do not fit shared memory)
    const int ctas = ((a.F[0] + 255) / 256 + (a.F[1] + 255) / 256) * p->n_adapters;
    a.splits = rb <= 2 ? split_of(ctas, (T + 63) / 64 / p->n_adapters, 4, false) : 1;
    const cudaError_t e = rb == 1   ? launch_grad_rb<1>(a, p->n_adapters, stream)
                          : rb == 2 ? launch_grad_rb<2>(a, p->n_adapters, stream)
                                    : launch_grad_rb<4>(a, p->n_adapters, stream);
    if (e != cudaSuccess) return api_fail(MOE_ERR_CUDA, "adapter gradient launch: %s", cudaGetErrorString(e));
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
    if ((rc = shrink<false>(adapter, T, x, a, scaling, adapter_of, v, st, s))) return rc;
    return project<false>(adapter, T, x, w, b, adapter_of, v, false, out, out_fp32, st, s);
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
    void* dv = ws;
    if ((rc = shrink<true>(adapter, T, dy, b, scaling, adapter_of, dv, st, s))) return rc;
    // the gradients first: the projection starts while they end (it waits for no predecessor
    // before it reads dv, and each of them started after dv's kernel had ended)
    if (da && (rc = gradients(adapter, T, dy, x, dv, v, adapter_of, da, db, st, s))) return rc;
    if (dx) return project<true>(adapter, T, dy, w, a, adapter_of, dv, da != nullptr, dx, 0, st, s);
    return MOE_OK;
}

}  // extern "C"

// Matrix products grouped by expert, and their gradients:
//   y[r]  = W_p[s] x[r]                    for the rows r of slot s, parts p side by side (gate, up)
//   dx[r] = sum_p W_p[s]^T dy_p[r],  dW_p[s] = sum over s's rows of dy_p[r] x[r]^T.
// The rows of a slot are consecutive (a dispatch's order), their counts ragged.
//
// All three are tcgen05 products of CTA pairs (cta_group::2), 256 outputs of one operand times up to
// 256 of the other, fp32 sums in tensor memory, double buffered so that a tile's stores run under the
// next tile's products.  Persistent pairs take tiles in turn; what there is of them follows from the
// offsets on the device.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "operators.cuh"

namespace moe {
namespace {

constexpr int kMaxSlots = 1024;
constexpr int kMaxFeatures = 1 << 24;
constexpr int kHalf = 128 * 64 * 2;  // one CTA's 128 rows or features of an operand's 64-wide chunk
constexpr int kRing = 12 * kHalf;

__device__ __forceinline__ uint32_t to_u(float f) { return __float_as_uint(f); }

__device__ __forceinline__ void tma_reduce_add_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// A block of outputs in shared memory into (or added to) the tensor.
__device__ __forceinline__ void put(const CUtensorMap* map, int type, uint32_t src, int c0, int c1, int c2) {
    if (type == MOE_OUT_F32_ADD) tma_reduce_add_3d(map, src, c0, c1, c2);
    else tma_store_3d(map, src, c0, c1, c2);
}

template <int N>
__device__ __forceinline__ void bulk_wait_read_but() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); }
__device__ __forceinline__ void st_shared4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

// 16 lanes x 64 columns: as tmem_ld_16x256, i up to 7
__device__ __forceinline__ void tmem_ld_16x256_64(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void stmatrix(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 32 lanes x 32 bits, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
          "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
          "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// An accumulator has been read (its loads are complete): nothing written before is read after this
// arrival by the other CTA, so it releases nothing.  (A release waits for the stores on their way out:
// 1600 to 3400 cycles of a tile of dW that takes 5500 with it.)
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// An arrival that releases what was written to this CTA's shared memory, and a wait for such arrivals: fences
// at cluster scope that are restricted to shared memory, and so wait for no store to global memory.  (A full
// release holds a thread for 1400 to 2000 cycles: one for each chunk, and codes took 3087 us of 4096 tokens, 8
// experts each, gate and up, where rows in bf16 took 1170; handed on by one warp of the CTA, 1376 against 1127 us.)
__device__ __forceinline__ void mbar_arrive_shared_cluster(uint32_t bar) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    mbar_arrive_relaxed_cluster(bar);
}
__device__ __forceinline__ bool mbar_try_wait_relaxed_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool warp_wait_shared_cluster(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                                         unsigned long long limit) {
    bool ok = mbar_try_wait_relaxed_cluster(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = globaltimer_ns();
        while (!ok && !*abort_flag && globaltimer_ns() - t0 <= limit) ok = mbar_try_wait_relaxed_cluster(bar, parity);
        ok = __all_sync(0xffffffffu, ok);
    }
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
    return ok;
}

// Four outputs of a sum that pairs shared.
__device__ __forceinline__ void put4(void* out, int type, size_t at, float4 v) {
    if (type == MOE_OUT_BF16) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf(to_u(v.x), to_u(v.y)), pack_bf(to_u(v.z), to_u(v.w)));
        return;
    }
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    if (type == MOE_OUT_F32_ADD) {
        const float4 old = *p;
        v.x += old.x, v.y += old.y, v.z += old.z, v.w += old.w;
    }
    *p = v;
}

// What `splits` pairs hold of four sums, from the CTA of rank `first` on, added in the pairs' order.  The
// loads are on their way together.
__device__ __forceinline__ float4 sum_of_pairs(uint32_t addr, uint32_t first, int splits) {
    float4 v[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = s < splits ? ld_peer4(addr, first + 2 * s) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = 1; s < 4; ++s) v[0].x += v[s].x, v[0].y += v[s].y, v[0].z += v[s].z, v[0].w += v[s].w;
    return v[0];
}

// How the pair's kernels end; `owner`: the warp that took the tensor memory, and has waited on `done` for the last
// products (`complete`: they were).  On the way out nobody signals the other CTA any more (who waits for
// signals has waited for all of them), so the barrier need not see them through; after a wait that
// expired it does, when everything has had the time to land.
__device__ __forceinline__ void leave_pair(const volatile int* abort_flag, const DevStatus& st, bool owner, bool complete, uint32_t done,
                                           uint32_t tmem) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // (In the CTA that issues no products this warp has waited since the kernel began, which may take longer than a
    // wait's limit.  The other warps are through by now, and the issuing one is or gives up.)
    if (owner && !complete && !mbar_wait(done, 0, max(st.limit_ns, kSettleNs))) {
        raise_status(st, kStatusWaitTimeout);
        settle_after_timeout();
    }
    __syncwarp();
    if (*abort_flag) {
        settle_after_timeout();
        __syncwarp();
        cluster_sync();
    } else {
        cluster_arrive_relaxed();
        cluster_wait();
    }
    tc_fence_after();
    if (owner) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------- y and dx
// One pair's tile: 256 outputs (128 rows of W, or for dx columns, in each CTA) times the rows of
// a slot in chunks of equal height, a multiple of 32 up to `cap` (half of them in each CTA).
// dx's W is read MN-major, as its contraction runs over W's rows.
// Few tiles with a long contraction: the pairs of a cluster take a share of it each, and their sums meet
// in distributed shared memory, added in the pairs' order.  The launch has pairs for as many tiles as
// offsets in order give; offsets that run backwards may name rows again and give more, which the pairs
// then take whole and in turn.
struct RowsArgs {
    CUtensorMap w[2];  // box {64, 128} of [S][N][K], dx: {64, 64}
    CUtensorMap in[4]; // box {64, 1, 16 << j} of x [R][1][K], dx: dy [R][P][N]
    CUtensorMap out;   // box {64, 1, 16} bf16, {32, 1, 16} fp32 of y [R][P][N], dx: [R][1][K]
    const int32_t* offsets;
    void* out_ptr;
    int R, K, N, P, S, type;
    int cap, stages;   // rows of a chunk at most (64, 128, 256); stages of the ring that then fit
    int splits;        // pairs of a cluster, which share a tile's contraction (1, 2, 4); above 1, pairs for every tile
    DevStatus st;
};
constexpr int kMostStages = 9;
__host__ __device__ constexpr int stage_bytes(int cap) { return kHalf + cap / 2 * 128; }
static_assert(kMostStages * stage_bytes(64) <= kRing && 8 * stage_bytes(128) <= kRing && 6 * stage_bytes(256) <= kRing, "rings");
constexpr int kRowsThreads = 192;  // copies, products, four warps that drain accumulators
constexpr int kOutBlocks = 3;
constexpr int kOutBytes = 2 * kOutBlocks * 4096;  // of 32 rows x 64 features each, for two pairs of warps
constexpr int kRowsSmem = 1024 + kRing + kOutBytes + 256 + 2 * (kMaxSlots + 1) * 4;
static_assert(kRowsSmem <= 227 * 1024, "shared memory overflow");

// cap is a power of two
__device__ __forceinline__ int chunks_of(int count, int cap) { return (int)((unsigned)(count + cap - 1) / (unsigned)cap); }

struct RowsTile {
    int s, part, m0;   // slot; part and first output of it
    int row0, rows, bn;
    bool shared_w;     // other tiles read the same of W
};

template <bool DX>
__device__ __forceinline__ RowsTile rows_tile(const RowsArgs& a, const int* pre, const int* start, int i) {
    // the last slot with pre[s] <= i, which the warp looks for together: among the first slots of 32
    // stretches, then in one of them
    const int lane = threadIdx.x & 31, per = (a.S + 31) / 32;
    const int at = (__popc(__ballot_sync(0xffffffffu, lane * per < a.S && pre[min(lane * per, a.S)] <= i)) - 1) * per;
    RowsTile t;
    t.s = per == 1 ? at : at + __popc(__ballot_sync(0xffffffffu, lane < per && at + lane < a.S && pre[min(at + lane, a.S)] <= i)) - 1;
    const int r0 = start[t.s], r1 = max(r0, start[t.s + 1]);
    const int n = chunks_of(r1 - r0, a.cap), l = i - pre[t.s], m = n > 1 ? l / n : l, c = l - m * n;
    // (heights within 32 of each other: a chunk of few rows reads as much of W as a high one)
    const int units = (r1 - r0 + 31) / 32, h = n > 1 ? units / n : units, more = units - h * n;
    const int tiles = ((DX ? a.K : a.N) + 255) / 256;
    t.part = m >= tiles;
    t.m0 = (m - t.part * tiles) * 256;
    t.row0 = r0 + 32 * (c * h + min(c, more));
    t.bn = 32 * (h + (c < more ? 1 : 0));
    t.rows = min(t.bn, r1 - t.row0);
    t.shared_w = n > 1;
    return t;
}

// Warps 2 p and 2 p + 1 share 64 features and three blocks at `out`, the copies of which the first
// one's lane 0 issues (with two, the drain waited for its copies: 640 cycles for 32 rows).  Copies take
// 16 rows at a time; the rows after a slot's last full 16 are stored by the threads, as what follows
// belongs to another slot.
__device__ __forceinline__ void drain_bf16(const RowsArgs& a, const RowsTile& t, int O, int P, uint32_t tmem, uint32_t out, int m0,
                                           int q, int lane, int& blocks) {
    const int pair = q >> 1, f0 = m0 + pair * 64;
    const bool issuer = !(q & 1) && lane == 0;
    const uint32_t at = (lane & 7) * 128 + ((((q & 1) * 4 + (lane >> 3)) ^ (lane & 7)) << 4);
    for (int r = 0; r < t.rows; r += 32, ++blocks) {
        uint32_t lo[16], hi[16];
        tmem_ld_16x256(tmem + r, lo);
        tmem_ld_16x256(tmem + r + (16u << 16), hi);
        tmem_ld_wait();
        const uint32_t block = out + (pair * kOutBlocks + blocks % kOutBlocks) * 4096;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            stmatrix_trans(block + i * 1024 + at, pack_bf(lo[4 * i], lo[4 * i + 1]), pack_bf(lo[4 * i + 2], lo[4 * i + 3]),
                           pack_bf(hi[4 * i], hi[4 * i + 1]), pack_bf(hi[4 * i + 2], hi[4 * i + 3]));
        fence_async_smem();
        if (issuer) bulk_wait_read_but<kOutBlocks - 2>();  // the block is free that the next round writes
        __syncwarp();
        named_sync(2 + pair, 64);
        if (issuer) {
            if (f0 < O) {
                if (r + 16 <= t.rows) tma_store_3d(&a.out, block, f0, t.part, t.row0 + r);
                if (r + 32 <= t.rows) tma_store_3d(&a.out, block + 2048, f0, t.part, t.row0 + r + 16);
            }
            bulk_commit();
        }
        __syncwarp();
        // the rest: 8 rows at a time, 8 threads a row
        const int piece = lane & 7;
        for (int k = max(r, t.rows & ~15) - r + (q & 1) * 4 + (lane >> 3); k < min(32, t.rows - r); k += 8)
            if (f0 + piece * 8 < O)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out_ptr) + ((size_t)(t.row0 + r + k) * P + t.part) * O + f0 + piece * 8) =
                    ld_shared4(block + k * 128 + ((piece ^ (k & 7)) << 4));
        __syncwarp();
    }
}

// fp32: a warp's 32 features of 16 rows at a time.
__device__ __forceinline__ void drain_f32(const RowsArgs& a, const RowsTile& t, int O, int P, uint32_t tmem, uint32_t out, int m0,
                                          int q, int lane, int& blocks) {
    const int f0 = m0 + q * 32;
    for (int r = 0; r < t.rows; r += 16, ++blocks) {
        float v[16];
        tmem_ld16(tmem + r, v);
        tmem_ld_wait();
        if (r + 16 > t.rows) {
            float* dst = static_cast<float*>(a.out_ptr) + ((size_t)(t.row0 + r) * P + t.part) * O + f0 + lane;
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (r + k < t.rows && f0 + lane < O) {
                    float* d = dst + (size_t)k * P * O;
                    *d = a.type == MOE_OUT_F32_ADD ? *d + v[k] : v[k];
                }
            __syncwarp();
            break;
        }
        const uint32_t block = out + (q * 2 + (blocks & 1)) * 2048;
        if (lane == 0) bulk_wait_read_but<1>();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 16; ++k) st_shared(block + k * 128 + (((lane >> 2) ^ (k & 7)) << 4) + (lane & 3) * 4, to_u(v[k]));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (f0 < O) put(&a.out, a.type, block, f0, t.part, t.row0 + r);
            bulk_commit();
        }
        __syncwarp();
    }
}

// Pair `pair` of `pairs`, which share the tiles.
template <bool DX>
__device__ __forceinline__ void rows_pair(const RowsArgs& a, const int pair, const int pairs) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing + kOutBytes);  // (the leader's)
    uint64_t* empty = full + kMostStages;
    uint64_t* tfull = empty + kMostStages;
    uint64_t* tempty = tfull + 2;  // (the leader's)
    uint64_t* done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * kMostStages + 5) * 8 + 8 <= 256, "barriers");
    int* pre = reinterpret_cast<int*>(smem + kRing + kOutBytes + 256);  // tiles before each slot
    int* start = pre + kMaxSlots + 1;                                   // its first row

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int place = (int)cluster_rank(), rank = place & 1;
    const uint32_t lead = place & ~1, both = 3u << lead;
    const int O = DX ? a.K : a.N, out_parts = DX ? 1 : a.P;
    const int m_tiles = (O + 255) / 256 * out_parts;
    const int kc1 = ((DX ? a.N : a.K) + 63) / 64, kc = kc1 * (DX ? a.P : 1);  // chunks of a part, of a tile
    const int kStages = a.stages, kStageBytes = stage_bytes(a.cap);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&tfull[s]), 1);
            mbar_init(smem_u32(&tempty[s]), 8);
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.w[0]);
        tma_prefetch_desc(&a.in[3]);
        tma_prefetch_desc(&a.out);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    __syncwarp();
    cluster_arrive_relaxed();
    pdl_wait();
    if (warp == 0) {
        const int per = (a.S + 31) / 32, s0 = min(a.S, lane * per), s1 = min(a.S, s0 + per);
        int sum = 0;
        bool fits = true;
        for (int s = s0; s < s1; ++s) {
            int r0, r1;
            fits &= slot_rows(a.offsets, s, a.R, r0, r1);
            start[s] = r0;
            if (s == a.S - 1) start[a.S] = r1;
            pre[s] = sum;
            sum += chunks_of(r1 - r0, a.cap) * m_tiles;
        }
        if (!fits && pair < a.splits) raise_status(a.st, kStatusBadShape);
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        for (int s = s0; s < s1; ++s) pre[s] += incl - sum;
        if (lane == 31) pre[a.S] = incl;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    // (1, 2 or 4: without divisions, which cost a call of few tiles 0.3 us here)
    const int n_tiles = pre[a.S], splits = n_tiles <= pairs >> (a.splits >> 1) ? a.splits : 1, bits = splits >> 1;
    const int first = pair >> bits, step = splits > 1 ? max(1, n_tiles) : pairs;
    const int share = (place >> 1) & (splits - 1), c0 = kc * share >> bits, c1 = kc * (share + 1) >> bits;  // of the contraction
    RowsTile t = {};
    if (first < n_tiles) t = rows_tile<DX>(a, pre, start, first);
    auto next_tile = [&](int i) {
        if (i + step < n_tiles) t = rows_tile<DX>(a, pre, start, i + step);
    };
    cluster_wait();  // the barriers and tensor memory of both CTAs are there before either is used
    pdl_launch_dependents();  // (not before the tensor memory is this pair's: the next kernel takes its own)
    auto give_up = [&]() {
        *abort_flag = 1;
        raise_status(a.st, kStatusWaitTimeout);
    };
    bool complete = true;  // (warp 1: the products are)
    const uint32_t full_u = smem_u32(full), empty_u = smem_u32(empty), stage_u = smem_u32(smem);
    const uint32_t lead_full = leader_addr(full_u, lead), lead_tempty = leader_addr(smem_u32(tempty), lead);

    if (warp == 0) {
        const uint64_t pol_once = policy_evict_first(), pol = policy_evict_normal();
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0, used = 0;
        for (int i = first; i < n_tiles && ok; next_tile(i), i += step) {
            const int m0 = t.m0 + rank * 128, n16 = t.bn / 32, row0 = t.row0 + rank * n16 * 16;
            const uint64_t pol_w = t.shared_w ? pol : pol_once;
            // y: a box of W wholly past the last output, which reaches only what is not stored, is left out, as
            // boxes of nothing are slow (23840 rows, 448 features to 128, 24 us with them and 13 without; for dx
            // and dW, with more and smaller boxes, the conditions cost as much as they gave)
            const bool w_there = DX || m0 < O, both_there = DX || t.m0 + 128 < O;
            for (int c = c0; c < c1; ++c) {
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                const int part = DX ? (c >= kc1) : t.part, at = (DX && part ? c - kc1 : c) * 64;
                if (elect_one()) {
                    const uint32_t sa = stage_u + stage * kStageBytes, fb = lead_full + stage * 8;
                    // the leader expects the bytes of both
                    if (rank == 0) mbar_arrive_expect_tx(full_u + stage * 8, (both_there ? 2 * kHalf : kHalf) + t.bn * 128);
                    if (DX) {
                        tma_load_3d_pair(sa, &a.w[part], fb, m0, at, t.s, pol_w);
                        tma_load_3d_pair(sa + kHalf / 2, &a.w[part], fb, m0 + 64, at, t.s, pol_w);
                    } else if (w_there) {
                        tma_load_3d_pair(sa, &a.w[part], fb, at, m0, t.s, pol_w);
                    }
                    for (int bit = 3, off = 0; bit >= 0; --bit)
                        if (n16 & (1 << bit)) {
                            tma_load_3d_pair(sa + kHalf + off * 2048, &a.in[bit], fb, at, DX ? part : 0, row0 + off * 16, pol);
                            off += 1 << bit;
                        }
                }
                __syncwarp();
                used |= 1u << stage;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // every stage's last products are done, so its copies have landed
        for (int s = 0; s < kStages && ok; ++s) {
            if ((used >> stage) & 1u) ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok && lane == 0) give_up();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint64_t ad0 = DX ? umma_desc_mn_sw128(stage_u, kHalf / 2) : umma_desc_sw128(stage_u);
            const uint64_t bd0 = umma_desc_sw128(stage_u + kHalf);
            constexpr int kAStep = DX ? 128 : 2;  // 16 of the contraction, in 16 bytes
            const int last = (DX ? a.N : a.K) - (kc1 - 1) * 64;  // width of a part's last chunk
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            for (int i = first, n = 0; i < n_tiles && ok; next_tile(i), i += step, ++n) {
                const uint32_t idesc = umma_idesc_bf16(256, t.bn) | (DX ? kIdescAMnMajor : 0u);
                const uint32_t d = tbase + (n & 1) * 256;
                if (!(ok = warp_wait(smem_u32(&tempty[n & 1]), ((n >> 1) & 1) ^ 1, abort_flag, limit))) break;
                tc_fence_after();
                for (int c = c0; c < c1; ++c) {
                    if (!(ok = warp_wait(full_u + stage * 8, phase, abort_flag, limit))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = ad0 + stage * (kStageBytes >> 4), bd = bd0 + stage * (kStageBytes >> 4);
                        const int left = c == kc1 - 1 || c == kc - 1 ? last : 64;
                        umma_bf16_pair(d, ad, bd, idesc, c > c0);
                        if (left > 16) umma_bf16_pair(d, ad + kAStep, bd + 2, idesc, 1);
                        if (left > 32) umma_bf16_pair(d, ad + 2 * kAStep, bd + 4, idesc, 1);
                        if (left > 48) umma_bf16_pair(d, ad + 3 * kAStep, bd + 6, idesc, 1);
                        umma_commit_pair(empty_u + stage * 8, both);
                    }
                    __syncwarp();
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (elect_one()) umma_commit_pair(smem_u32(&tfull[n & 1]), both);
                __syncwarp();
            }
            if (!ok && lane == 0) give_up();
            // all products are complete before the tensor memory is freed
            if (elect_one()) umma_commit_pair(smem_u32(done), both);
            __syncwarp();
        }
        complete = mbar_wait(smem_u32(done), 0, limit);
    } else if (warp < 6) {  // (a launch for dW too has more)
        const int q = warp & 3;
        bool ok = true;
        int blocks = 0;
        for (int i = first, n = 0; i < n_tiles; next_tile(i), i += step, ++n) {
            ok = warp_wait(smem_u32(&tfull[n & 1]), (n >> 1) & 1, abort_flag, limit);
            if (!(ok = named_and(2 + (q >> 1), 64, ok))) break;  // (the two warps that share drain_bf16's barrier)
            tc_fence_after();
            const uint32_t tmem = tbase + (n & 1) * 256 + ((uint32_t)(q * 32) << 16), out = stage_u + kRing;
            if (splits > 1) {
                // [row][128 outputs] where the ring was: all its products are done
                for (int r = 0; r < t.rows; r += 16) {
                    float v[16];
                    tmem_ld16(tmem + r, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) st_shared(stage_u + ((r + k) * 128 + q * 32 + lane) * 4, to_u(v[k]));
                }
            } else if (a.type == MOE_OUT_BF16) drain_bf16(a, t, O, out_parts, tmem, out, t.m0 + rank * 128, q, lane, blocks);
            else drain_f32(a, t, O, out_parts, tmem, out, t.m0 + rank * 128, q, lane, blocks);
            tc_fence_before();
            __syncwarp();
            // (not where nobody waits for it any more: no signal is on its way at the end)
            if (lane == 0 && i + 2 * step < n_tiles) mbar_arrive_relaxed_cluster(lead_tempty + (n & 1) * 8);
        }
        if (!ok && lane == 0) give_up();
        if (lane == 0) bulk_wait();
    }
    if (splits > 1) {
        __syncwarp();
        tc_fence_before();
        cluster_sync();
        // every pair's CTA of this rank holds the same 128 outputs: the rows in turn, 4 outputs a lane
        const int f = t.m0 + rank * 128 + lane * 4;
        const uint32_t base = (place >> 1) - share;
        if (first < n_tiles && f < O && !*abort_flag)
            for (int r = share + splits * warp; r < t.rows; r += splits * (blockDim.x / 32)) {
                const float4 sum = sum_of_pairs(stage_u + (r * 128 + lane * 4) * 4, 2 * base + rank, splits);
                put4(a.out_ptr, a.type, ((size_t)(t.row0 + r) * out_parts + t.part) * O + f, sum);
            }
    }
    leave_pair(abort_flag, a.st, warp == 1, complete, smem_u32(done), tbase);
}

template <bool DX>
__global__ void __launch_bounds__(kRowsThreads, 1) rows_kernel(const __grid_constant__ RowsArgs a) {
    rows_pair<DX>(a, blockIdx.x / 2, gridDim.x / 2);
}

// ---------------------------------------------------------------- dW
// One pair's tile: 256 of N, or twice that (128 of dy's columns in each CTA), times 256 of K (128 of x's columns in
// each), summed over the slot's rows, 64 at a time; both operands are MN-major.  Of a slot's last
// chunk as many 16 rows are copied and multiplied as it has; the rows of the next slot among them are
// set to zero in shared memory, in both operands, so whatever they hold stays out.
// Rows in 8 bits are copied as codes into the lower half of their operand's place, taken from there
// into registers and written back as bf16 over the whole of it.
struct WeightArgs {
    CUtensorMap dy[3];   // box {64, 1, 16 << j} of dy [R][P][N]
    CUtensorMap x[3];    // of x [R][1][K]; codes: box {128, 1, 16 << j}
    void* out_ptr[2];
    CUtensorMap out[2];  // box {64, 16, 1} bf16, {32, 32, 1} fp32 of dw [S][N][K]
    const float* scale;  // [R][n_blk]
    const int32_t* offsets;
    int R, K, N, P, S, type, n_blk, n_tiles;
    int splits;          // pairs of a cluster that share a tile's rows, as for y and dx
    DevStatus st;
};
template <bool M2>
struct WeightRing {
    static constexpr int kA = M2 ? 2 * kHalf : kHalf;  // dy's; then x's
    static constexpr int kStageBytes = kA + kHalf;
    static constexpr int kStages = M2 ? 4 : 6;
};
static_assert(kRing == WeightRing<false>::kStages * WeightRing<false>::kStageBytes &&
                  kRing == WeightRing<true>::kStages * WeightRing<true>::kStageBytes,
              "rings of one size");

// The products of one tile's chunks, issued by a warp that waits for chunk c by `ready(c)` and for an
// accumulator by `free(slot, phase)`; `issue(half, stage, c, slot)` multiplies, and `release(stage)`
// and `full(slot)` commit.  `u` counts accumulators.  With two halves the first runs ahead over the
// stages in flight until the second one's accumulator is free; a stage is released by the second.
template <int STAGES, typename Ready, typename Free, typename TestFree, typename Issue, typename Release, typename Full>
__device__ __forceinline__ bool tile_products(bool two, int chunks, int& stage, int& u, Ready&& ready, Free&& free, TestFree&& test_free,
                                              Issue&& issue, Release&& release, Full&& full) {
    const int u0 = u;
    u += two ? 2 : 1;
    if (!free(u0)) return false;
    if (!two) {
        for (int c = 0; c < chunks; ++c) {
            if (!ready(c)) return false;
            issue(0, stage, c, u0);
            release(stage);
            if (++stage == STAGES) stage = 0;
        }
        full(u0);
        return true;
    }
    int k0 = 0, k1 = 0, st1 = stage;
    bool second = false;
    while (k1 < chunks) {
        if (!second) second = test_free(u0 + 1);
        if (second && k1 < k0) {
            issue(1, st1, k1, u0 + 1);
            release(st1);
            if (++st1 == STAGES) st1 = 0;
            ++k1;
        } else if (k0 < chunks && k0 - k1 < STAGES) {
            if (!ready(k0)) return false;
            issue(0, stage, k0, u0);
            if (++stage == STAGES) stage = 0;
            if (++k0 == chunks) full(u0);
        } else {
            if (!free(u0 + 1)) return false;
            second = true;
        }
    }
    full(u0 + 1);
    return true;
}

// Four warps work on the rows of a chunk, 16 rows each, where the last one of a slot needs it.  Codes
// all need it, and take them longer than the chunk's products: several such groups take chunks in turn.
// A stage's chunks are all one group's (the groups divide the stages): a group that waited for a chunk
// of a stage whose last chunk another group had not seen land would take that one's phase for its own.
constexpr int kWork = 4;
constexpr int kDrainWarps = 8;
constexpr int kWeightOut = kDrainWarps * 4096;  // a block of 32 x 128 bytes of each draining warp
constexpr int work_groups(bool x8, bool m2) { return !x8 ? 1 : m2 ? 2 : 3; }
constexpr int weight_threads(bool x8, bool m2) { return 64 + 32 * kWork * work_groups(x8, m2) + 32 * kDrainWarps; }
constexpr int kWeightSmem = 1024 + kRing + kWeightOut + 512;
static_assert(kWeightSmem <= 227 * 1024, "shared memory overflow");

struct WeightTile {
    int s, part, n0, k0;
    int row0, rows;
    int r0, r1;  // this pair's share of the rows
    bool two;    // halves (M2)
};

template <bool M2, bool SHARED>
__device__ __forceinline__ WeightTile weight_tile(const WeightArgs& a, int i, int share) {
    constexpr int kM = M2 ? 512 : 256;
    const int kt = (a.K + 255) / 256, nt = (a.N + kM - 1) / kM;
    WeightTile t;
    t.k0 = i % kt * 256;
    i /= kt;
    t.n0 = i % nt * kM;
    t.two = M2 && t.n0 + 256 < a.N;
    i /= nt;
    t.part = i % a.P;
    t.s = i / a.P;
    int r1;
    slot_rows(a.offsets, t.s, a.R, t.row0, r1);
    t.rows = r1 - t.row0;
    t.r0 = 0;
    t.r1 = t.rows;
    if (SHARED) {  // whole chunks, none perhaps
        const long chunks = (t.rows + 63) / 64;
        t.r0 = (int)min((long)t.rows, chunks * share / a.splits * 64);
        t.r1 = (int)min((long)t.rows, chunks * (share + 1) / a.splits * 64);
    }
    return t;
}

// 16 codes times their scale as bf16: both steps are exact (the header of checkpoint.cu says why).
__device__ __forceinline__ void decode16(const uint4& c, float scale, uint32_t (&w)[8]) {
    const uint32_t v[4] = {c.x, c.y, c.z, c.w};
    const __nv_bfloat162 by = __float2bfloat162_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((v[i >> 1] >> (i & 1) * 16) & 0xffffu), __NV_E4M3);
        const __nv_bfloat162 p = __hmul2(__float22bfloat162_rn(__half22float2(__half2(h))), by);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
}

template <bool X8, bool M2, bool SHARED>
__device__ __forceinline__ void weights_pair(const WeightArgs& a, const int pair, const int pairs) {
    constexpr int kStages = WeightRing<M2>::kStages, kStageBytes = WeightRing<M2>::kStageBytes, kA = WeightRing<M2>::kA;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing + kWeightOut);  // (the leader's) copies that need no work, of both
    uint64_t* empty = full + kStages;
    uint64_t* landed = empty + kStages;  // this CTA's copies that need work
    uint64_t* ready = landed + kStages;  // (the leader's) ... which have had it, in both
    uint64_t* tfull = ready + kStages;
    uint64_t* tempty = tfull + 2;        // (the leader's)
    uint64_t* done = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((4 * kStages + 5) * 8 + 8 <= 512, "barriers");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned long long limit = a.st.limit_ns;
    const int place = (int)cluster_rank(), rank = place & 1, share = SHARED ? (place >> 1) % a.splits : 0;
    const int first = SHARED ? pair / a.splits : pair, step = SHARED ? a.n_tiles : pairs;
    const uint32_t lead = place & ~1, both = 3u << lead;
    constexpr int kGroups = work_groups(X8, M2);
    static_assert(kStages % kGroups == 0, "a stage is one group's");

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&landed[s]), 1);
            mbar_init(smem_u32(&ready[s]), 2 * kWork);  // the workers of both
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&tfull[s]), 1);
            mbar_init(smem_u32(&tempty[s]), 2 * kDrainWarps);
        }
        mbar_init(smem_u32(done), 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.dy[2]);
        tma_prefetch_desc(&a.x[2]);
        tma_prefetch_desc(&a.out[0]);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
    __syncwarp();
    cluster_arrive_relaxed();
    pdl_wait();
    WeightTile t = {};
    if (first < a.n_tiles) t = weight_tile<M2, SHARED>(a, first, share);
    auto next_tile = [&](int i) {
        if (i + step < a.n_tiles) t = weight_tile<M2, SHARED>(a, i + step, share);
    };
    if (warp == 0 && first == 0)
        for (int s = lane; s < a.S; s += 32) {
            int r0, r1;
            if (!slot_rows(a.offsets, s, a.R, r0, r1)) raise_status(a.st, kStatusBadShape);
        }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_wait();  // the barriers and tensor memory of both CTAs are there before either is used
    pdl_launch_dependents();  // (not before the tensor memory is this pair's)
    const uint32_t tbase = *tmem_slot;
    auto give_up = [&]() {
        *abort_flag = 1;
        raise_status(a.st, kStatusWaitTimeout);
    };
    bool complete = true;  // (warp 1: the products are)
    const uint32_t full_u = smem_u32(full), empty_u = smem_u32(empty), landed_u = smem_u32(landed), ready_u = smem_u32(ready);
    const uint32_t stage_u = smem_u32(smem);
    const uint32_t lead_full = leader_addr(full_u, lead), lead_tempty = leader_addr(smem_u32(tempty), lead), lead_ready = leader_addr(ready_u, lead);

    if (warp == 0) {
        const uint64_t pol = policy_evict_normal();
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0, used = 0;
        for (int i = first; i < a.n_tiles && ok; next_tile(i), i += step) {
            const int n0 = t.n0 + rank * 128, k0 = t.k0 + rank * 128;
            for (int r = t.r0; r < t.r1; r += 64) {
                const int left = min(64, t.r1 - r), n16 = (left + 15) / 16;
                const bool work = X8 || (left & 15);
                if (!(ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit))) break;
                if (elect_one()) {
                    const uint32_t sa = stage_u + stage * kStageBytes, sb = sa + kA;
                    const uint32_t fb = lead_full + stage * 8, lb = landed_u + stage * 8;
                    const uint32_t dy_bytes = (t.two ? 2 : 1) * n16 * 4096, x_bytes = X8 ? n16 * 2048 : n16 * 4096;
                    if (!work && rank == 0) mbar_arrive_expect_tx(full_u + stage * 8, 2 * (dy_bytes + x_bytes));
                    if (work) mbar_arrive_expect_tx(lb, dy_bytes + x_bytes);
                    for (int bit = 2, off = 0; bit >= 0; --bit)
                        if (n16 & (1 << bit)) {
                            const int row = t.row0 + r + off * 16;
                            const uint32_t o = off * 2048;
#pragma unroll
                            for (int h = 0; h < (M2 ? 2 : 1); ++h) {
                                if (h && !t.two) break;
                                const uint32_t to = sa + h * kHalf + o;
                                const int n = n0 + h * 256;
                                if (work) {
                                    tma_load_3d(to, &a.dy[bit], lb, n, t.part, row, pol);
                                    tma_load_3d(to + kHalf / 2, &a.dy[bit], lb, n + 64, t.part, row, pol);
                                } else {
                                    tma_load_3d_pair(to, &a.dy[bit], fb, n, t.part, row, pol);
                                    tma_load_3d_pair(to + kHalf / 2, &a.dy[bit], fb, n + 64, t.part, row, pol);
                                }
                            }
                            if (X8) {
                                tma_load_3d(sb + o, &a.x[bit], lb, k0, 0, row, pol);
                            } else if (work) {
                                tma_load_3d(sb + o, &a.x[bit], lb, k0, 0, row, pol);
                                tma_load_3d(sb + o + kHalf / 2, &a.x[bit], lb, k0 + 64, 0, row, pol);
                            } else {
                                tma_load_3d_pair(sb + o, &a.x[bit], fb, k0, 0, row, pol);
                                tma_load_3d_pair(sb + o + kHalf / 2, &a.x[bit], fb, k0 + 64, 0, row, pol);
                            }
                            off += 1 << bit;
                        }
                }
                __syncwarp();
                used |= 1u << stage;
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        // every stage's last products are done, so its copies have landed
        for (int s = 0; s < kStages && ok; ++s) {
            if ((used >> stage) & 1u) ok = warp_wait(empty_u + stage * 8, phase ^ 1, abort_flag, limit);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        if (!ok && lane == 0) give_up();
    } else if (warp == 1) {
        // What it waits for is read by the tensor cores alone, each CTA's half in its own shared
        // memory.  Rows that threads stored are acquired from both CTAs, by fences restricted to shared memory;
        // the waits for copies alone do not acquire for the cluster (100 to 200 ns each where unrestricted).
        bool ok = true;
        int stage = 0, at = 0, u = 0;
        uint32_t full_phase = 0, work_phase = 0;  // (of each stage: not every chunk uses both)
        if (rank == 0) {
            const uint32_t idesc = umma_idesc_bf16(256, 256) | kIdescAMnMajor | kIdescBMnMajor;
            const uint64_t ad0 = umma_desc_mn_sw128(stage_u, kHalf / 2), bd0 = umma_desc_mn_sw128(stage_u + kA, kHalf / 2);
            for (int i = first; i < a.n_tiles && ok; next_tile(i), i += step) {
                if (t.r0 >= t.r1) continue;
                ok = tile_products<kStages>(
                    t.two, (t.r1 - t.r0 + 63) / 64, stage, u,
                    [&](int c) {
                        // one wait a chunk: two or three of 180 cycles each held up the products of codes
                        bool got;
                        if (X8 || (min(64, t.r1 - t.r0 - c * 64) & 15)) {
                            got = warp_wait_shared_cluster(ready_u + at * 8, (work_phase >> at) & 1u, abort_flag, limit);
                            work_phase ^= 1u << at;
                        } else {
                            got = warp_wait(full_u + at * 8, (full_phase >> at) & 1u, abort_flag, limit);
                            full_phase ^= 1u << at;
                        }
                        if (++at == kStages) at = 0;
                        tc_fence_after();
                        return got;
                    },
                    [&](int v) {
                        const bool got = warp_wait(smem_u32(&tempty[v & 1]), ((v >> 1) & 1) ^ 1, abort_flag, limit);
                        tc_fence_after();
                        return got;
                    },
                    [&](int v) {
                        const bool got = __all_sync(0xffffffffu, mbar_test_wait(smem_u32(&tempty[v & 1]), ((v >> 1) & 1) ^ 1));
                        tc_fence_after();
                        return got;
                    },
                    [&](int half, int st, int c, int v) {
                        if (elect_one()) {
                            const uint64_t ad = ad0 + st * (kStageBytes >> 4) + half * (kHalf >> 4), bd = bd0 + st * (kStageBytes >> 4);
                            const uint32_t d = tbase + (v & 1) * 256;
                            const int left = min(64, t.r1 - t.r0 - c * 64);
                            umma_bf16_pair(d, ad, bd, idesc, c > 0);
                            if (left > 16) umma_bf16_pair(d, ad + 128, bd + 128, idesc, 1);
                            if (left > 32) umma_bf16_pair(d, ad + 256, bd + 256, idesc, 1);
                            if (left > 48) umma_bf16_pair(d, ad + 384, bd + 384, idesc, 1);
                        }
                        __syncwarp();
                    },
                    [&](int st) {
                        if (elect_one()) umma_commit_pair(empty_u + st * 8, both);
                        __syncwarp();
                    },
                    [&](int v) {
                        if (elect_one()) umma_commit_pair(smem_u32(&tfull[v & 1]), both);
                        __syncwarp();
                    });
            }
            // (the last accumulators have been handed back: no signal is on its way at the end)
            for (int v = max(0, u - 2); v < u && ok; ++v) ok = warp_wait(smem_u32(&tempty[v & 1]), (v >> 1) & 1, abort_flag, limit);
            if (!ok && lane == 0) give_up();
            // all products are complete before the tensor memory is freed
            if (elect_one()) umma_commit_pair(smem_u32(done), both);
            __syncwarp();
        }
        complete = mbar_wait(smem_u32(done), 0, limit);
    } else if (warp < 2 + kWork * kGroups) {
        const int group = (warp - 2) / kWork, sub = (warp - 2) % kWork;
        bool ok = true;
        int stage = 0, turn = 0;  // of the chunks that need work
        uint32_t land_phase = 0;
        for (int i = first; i < a.n_tiles && ok; next_tile(i), i += step) {
            const int blk = (t.k0 + rank * 128) / MOE_PAYLOAD_BLOCK;
            for (int r = t.r0; r < t.r1; r += 64) {
                const int left = min(64, t.r1 - r), rows16 = (left + 15) & ~15;
                const bool work = X8 || (left & 15), mine = work && turn == group;
                if (work && ++turn == kGroups) turn = 0;
                if (mine) {
                    const uint32_t sa = stage_u + stage * kStageBytes, sb = sa + kA;
                    // codes: four threads a row, 32 columns each, 8 rows at a time
                    const int row0 = sub * 16 + (lane >> 2), part = lane & 3, flip = part >> 1;
                    float scale[2] = {0.0f, 0.0f};
                    if (X8 && blk < a.n_blk)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            if (row0 + k * 8 < left) scale[k] = __ldg(a.scale + (size_t)(t.row0 + r + row0 + k * 8) * a.n_blk + blk);
                    if (!(ok = warp_wait(landed_u + stage * 8, (land_phase >> stage) & 1u, abort_flag, limit))) break;
                    if (X8 && sub * 16 < rows16) {
                        // pieces of 16 bytes in the order of the swizzle, those of the second 64 columns
                        // in another, so that all find their banks free.  A row's codes lie where the
                        // first 64 columns of the same row go: its four threads are of one warp.
                        uint4 c[2][2];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                c[k][i] = ld_shared4(sb + (row0 + k * 8) * 128 + (((part * 2 + (i ^ flip)) ^ (row0 & 7)) << 4));
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t to = sb + flip * (kHalf / 2) + (row0 + k * 8) * 128;
                            const bool live = row0 + k * 8 < left;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                uint32_t w[8];
                                decode16(c[k][i], scale[k], w);
                                const int piece = (part & 1) * 4 + (i ^ flip) * 2;
                                st_shared4(to + ((piece ^ (row0 & 7)) << 4), live ? w[0] : 0u, live ? w[1] : 0u, live ? w[2] : 0u, live ? w[3] : 0u);
                                st_shared4(to + (((piece + 1) ^ (row0 & 7)) << 4), live ? w[4] : 0u, live ? w[5] : 0u, live ? w[6] : 0u,
                                           live ? w[7] : 0u);
                            }
                        }
                    }
                    if (left & 15) {
                        // the rows of the last 16 that are not the slot's, 8 threads a row
                        const int row = rows16 - 16 + sub * 4 + (lane >> 3);
                        if (row >= left) {
                            const uint32_t o = row * 128 + (lane & 7) * 16;
                            st_shared4(sa + o, 0, 0, 0, 0);
                            st_shared4(sa + o + kHalf / 2, 0, 0, 0, 0);
                            if (t.two) {
                                st_shared4(sa + o + kHalf, 0, 0, 0, 0);
                                st_shared4(sa + o + kHalf + kHalf / 2, 0, 0, 0, 0);
                            }
                            if (!X8) {
                                st_shared4(sb + o, 0, 0, 0, 0);
                                st_shared4(sb + o + kHalf / 2, 0, 0, 0, 0);
                            }
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive(ready_u + stage * 8);
                        else mbar_arrive_shared_cluster(lead_ready + stage * 8);
                    }
                    __syncwarp();
                }
                if (work) land_phase ^= 1u << stage;
                if (++stage == kStages) stage = 0;
            }
        }
        if (!ok && lane == 0) give_up();
    } else {
        // two warps for each quarter of the accumulators, half of the columns each
        const int q = warp & 3, part = (warp - 2 - kWork * kGroups) >> 2;
        const uint32_t block = stage_u + kRing + (part * 4 + q) * 4096;
        bool ok = true;
        int u = 0;
        for (int i = first; i < a.n_tiles && ok; next_tile(i), i += step) {
            const bool some = t.r0 < t.r1;  // products to drain
            if (SHARED) {
                // [N][K] where the ring was (all its products are done), 16 bytes in the order of a swizzle
                if (some && !(ok = warp_wait(smem_u32(&tfull[u & 1]), (u >> 1) & 1, abort_flag, limit))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = part * 128; c < part * 128 + 128; c += 32) {
                    uint32_t v[32];
                    if (some) {
                        tmem_ld32(tbase + (u & 1) * 256 + ((uint32_t)(q * 32) << 16) + c, v);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st_shared4(stage_u + (q * 32 + lane) * 1024 + (((c >> 2) + (k ^ (lane & 7))) << 4), v[4 * k], v[4 * k + 1],
                                   v[4 * k + 2], v[4 * k + 3]);
                }
                if (some) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed_cluster(lead_tempty + (u & 1) * 8);
                    ++u;
                }
                continue;
            }
            if (!some && a.type == MOE_OUT_F32_ADD) continue;
            for (int half = 0; half < (t.two ? 2 : 1); ++half) {
                if (some) {
                    if (!(ok = warp_wait(smem_u32(&tfull[u & 1]), (u >> 1) & 1, abort_flag, limit))) break;
                    tc_fence_after();
                }
                const uint32_t tmem = tbase + (u & 1) * 256 + ((uint32_t)(q * 32) << 16);
                const int row = t.n0 + half * 256 + rank * 128 + q * 32;
                const int c_end = min(part * 128 + 128, a.K - t.k0);
                if (a.type == MOE_OUT_BF16) {
                    // 16 rows x 64 columns at a time, as 8 x 8 fragments that stmatrix puts in rows, in two
                    // blocks in turn (32 rows in one waited for each copy: 2200 cycles an accumulator)
                    for (int c = part * 128; c < c_end; c += 64)
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[32];
                            if (some) {
                                tmem_ld_16x256_64(tmem + c + ((uint32_t)(h * 16) << 16), v);
                                tmem_ld_wait();
                            } else {
#pragma unroll
                                for (int k = 0; k < 32; ++k) v[k] = 0;
                            }
                            if (lane == 0) bulk_wait_read_but<1>();  // the copy before the last has read this block
                            __syncwarp();
                            // this lane's address of 8 columns of a row: matrix lane / 8 is columns 8 (lane / 16), rows 8 (lane / 8 % 2)
                            const int row8 = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                            for (int k = 0; k < 8; k += 2)
                                stmatrix(block + h * 2048 + row8 * 128 + (((k + (lane >> 4)) ^ (lane & 7)) << 4), pack_bf(v[4 * k], v[4 * k + 1]),
                                         pack_bf(v[4 * k + 2], v[4 * k + 3]), pack_bf(v[4 * k + 4], v[4 * k + 5]),
                                         pack_bf(v[4 * k + 6], v[4 * k + 7]));
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                if (row + h * 16 < a.N) tma_store_3d(&a.out[t.part], block + h * 2048, t.k0 + c, row + h * 16, t.s);
                                bulk_commit();
                            }
                            __syncwarp();
                        }
                } else {
                    for (int c = part * 128; c < c_end; c += 32) {
                        uint32_t v[32];
                        if (some) {
                            tmem_ld32(tmem + c, v);
                            tmem_ld_wait();
                        } else {
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = 0;
                        }
                        if (lane == 0) bulk_wait_read();  // the block's last copy has read it
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            st_shared4(block + lane * 128 + ((k ^ (lane & 7)) << 4), v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (row < a.N) put(&a.out[t.part], a.type, block, t.k0 + c, row, t.s);
                            bulk_commit();
                        }
                        __syncwarp();
                    }
                }
                if (some) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed_cluster(lead_tempty + (u & 1) * 8);
                    ++u;
                }
            }
        }
        if (!ok && lane == 0) give_up();
        if (lane == 0) bulk_wait();
    }
    if (SHARED) {
        __syncwarp();
        tc_fence_before();
        cluster_sync();
        // every pair's CTA of this rank holds the same 128 x 256: the rows of them in turn, 4 columns a lane
        const uint32_t base = (place >> 1) - share;
        if (first < a.n_tiles && !*abort_flag && (t.rows || a.type != MOE_OUT_F32_ADD))
            for (int n = share + a.splits * warp; n < min(128, a.N - t.n0 - rank * 128); n += a.splits * (blockDim.x / 32)) {
                const int k = lane * 4, most = a.K - t.k0;
                const uint32_t row = stage_u + n * 1024, at = (lane ^ (n & 7)) << 4;
                float4 low = make_float4(0.0f, 0.0f, 0.0f, 0.0f), high = low;
                if (t.rows && k < most) low = sum_of_pairs(row + at, 2 * base + rank, a.splits);
                if (t.rows && k + 128 < most) high = sum_of_pairs(row + at + 512, 2 * base + rank, a.splits);
                const size_t out = ((size_t)t.s * a.N + t.n0 + rank * 128 + n) * a.K + t.k0 + k;
                if (k < most) put4(a.out_ptr[t.part], a.type, out, low);
                if (k + 128 < most) put4(a.out_ptr[t.part], a.type, out + 128, high);
            }
    }
    leave_pair(abort_flag, a.st, warp == 1, complete, smem_u32(done), tbase);
}

// (SHARED: with it in every kernel dW of 38 rows, 1856 to 264 features of 16 slots, took 15.8 us, not 14.8)
template <bool X8, bool M2, bool SHARED>
__global__ void __launch_bounds__(weight_threads(X8, M2), 1) weights_kernel(const __grid_constant__ WeightArgs a) {
    weights_pair<X8, M2, SHARED>(a, blockIdx.x / 2, gridDim.x / 2);
}

// dx and dW in one launch, `dx_pairs` of its pairs for dx: where neither fills the device for long, one
// runs beside the other instead of after it.
struct BothArgs {
    RowsArgs dx;
    WeightArgs dw;
    int dx_pairs;
};
constexpr int kBothSmem = kRowsSmem > kWeightSmem ? kRowsSmem : kWeightSmem;
template <bool X8, bool SHARED>
__global__ void __launch_bounds__(weight_threads(X8, false), 1) gradients_kernel(const __grid_constant__ BothArgs a) {
    const int pair = blockIdx.x / 2;
    if (pair < a.dx_pairs) rows_pair<true>(a.dx, pair, a.dx_pairs);
    else weights_pair<X8, false, SHARED>(a.dw, pair - a.dx_pairs, gridDim.x / 2 - a.dx_pairs);
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
    if ((double)p->in_features * p->out_features * p->n_slots * p->n_parts > 0x1p46)
        return api_fail(MOE_ERR_UNSUPPORTED, "weights of more than 2^46 elements");
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

template <typename Kern, typename A>
int launch_pairs(Kern kern, std::atomic<uint64_t>& configured, int threads, int smem, long pairs, int splits, cudaStream_t stream,
                 const A& a, const char* what) {
    const int rc = launched(configure_once(configured,
                                           [&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); }),
                            what);
    return rc ? rc : launched(launch_pdl_cluster(kern, dim3(2 * (unsigned)pairs), dim3(threads), smem, stream, 2 * splits, a), what);
}

constexpr long kBothTiles = 16;  // of a pair
long most_pairs() { return std::max(1, num_sms() / 2); }

// A tensor that is written: box of 128 bytes.
int out_map(CUtensorMap* map, void* out, uint64_t d0, uint64_t d1, uint64_t d2, int type, uint32_t box1, uint32_t box2) {
    const uint64_t size = type == MOE_OUT_BF16 ? 2 : 4;
    return type == MOE_OUT_BF16 ? make_tmap_3d(map, out, d0, d1, d2, d0 * size, d0 * d1 * size, 64, box1, box2)
                                : make_tmap_f32(map, out, d0, d1, d2, 32, box1, box2);
}

// Tiles of y or dx (as many as there may be), the rows of a chunk at most, 64-wide chunks of a sum.
struct RowsPlan {
    long tiles;
    int cap, chunks;
};
template <bool DX>
RowsPlan rows_plan(const moe_project_t* p, int rows) {
    // Where there is about a tile for each pair, what counts is how soon its chunks are there: lower ones,
    // of which more fit the ring, where slots have few rows (400 rows of 16 slots, gate and up of 600 to
    // 328: 6.8 us with 256 rows, 6.5 with 64).
    const long m_tiles = ((DX ? p->in_features : p->out_features) + 255L) / 256 * (DX ? 1 : p->n_parts), used = std::min(rows, p->n_slots);
    const int cap = m_tiles * used > most_pairs() ? 256 : rows <= 48 * used ? 64 : rows <= 96 * used ? 128 : 256;
    return {m_tiles * (rows / cap + used), cap, DX ? (p->out_features + 63) / 64 * p->n_parts : (p->in_features + 63) / 64};
}

template <bool DX>
int rows_args(const moe_project_t* p, int rows, const void* in, const int32_t* offsets, const void* w, const void* w2, void* out, int type,
              const DevStatus& st, int cap, int splits, RowsArgs& a) {
    const uint64_t K = p->in_features, N = p->out_features, S = p->n_slots, P = p->n_parts, R = rows;
    int rc = make_tmap_3d(&a.w[0], w, K, N, S, K * 2, K * N * 2, 64, DX ? 64 : 128, 1);
    if (rc) return rc;
    a.w[1] = a.w[0];
    if (w2 && (rc = make_tmap_3d(&a.w[1], w2, K, N, S, K * 2, K * N * 2, 64, DX ? 64 : 128, 1))) return rc;
    const uint64_t C = DX ? N : K, CP = DX ? P : 1, O = DX ? K : N, OP = DX ? 1 : P;
    for (int j = 0; j < 4; ++j)
        if ((rc = make_tmap_3d(&a.in[j], in, C, CP, R, C * 2, C * CP * 2, 64, 1, 16u << j))) return rc;
    if ((rc = out_map(&a.out, out, O, OP, R, type, 1, 16))) return rc;
    a.offsets = offsets;
    a.out_ptr = out;
    a.R = rows;
    a.K = p->in_features;
    a.N = p->out_features;
    a.P = p->n_parts;
    a.S = p->n_slots;
    a.type = type;
    a.st = st;
    a.cap = cap;
    a.stages = a.cap == 64 ? kMostStages : a.cap == 128 ? 8 : 6;
    a.splits = splits;
    return MOE_OK;
}

// Clusters of two or four pairs that are resident: they do not cross the device's groups of processors
// (36 and 15 of 152).
long resident(int pairs) { return (long)num_sms() * (pairs == 2 ? 36 : 15) / 152; }

// Pairs that share a tile's contraction, where clusters for all tiles are resident: four from 16 chunks
// on, else two from 16 (y and dx) or 24 (dW, whose sums are larger).  (One pair, two and four, us: y of 64
// rows, 1024 to 256 (16 chunks), 6.9, 6.7 and 5.6, of 2048 features 10.2, 8.4 and 6.4, of 512 5.3 and 5.8
// with two; dW of 1024 rows, 256 by 256, 8.6, 9.3 and 8.6, in 8 bits 10.1, 9.9 and 9.3, of 2048 rows 12.8,
// 11.5 and 9.7, of 512 6.5 and 8.2 with two.)
int splits_of(int chunks, long tiles, int two) {
    if (chunks >= 16 && tiles <= resident(4)) return 4;
    return chunks >= two && tiles <= resident(2) ? 2 : 1;
}

// Chunks of 64 rows of a slot, of slots of equal counts.
int chunks_of_slot(int rows, int slots) {
    const int used = std::min(rows, slots);
    return ((rows + used - 1) / used + 63) / 64;
}

template <bool DX>
int launch_rows(const RowsArgs& a, long tiles, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    return launch_pairs(rows_kernel<DX>, configured, kRowsThreads, kRowsSmem, a.splits > 1 ? tiles * a.splits : std::min(tiles, most_pairs()),
                        a.splits, stream, a, DX ? "expert gradient" : "expert projection");
}

template <bool X8>
int weight_args(const moe_project_t* p, int rows, const void* dy, const void* x, const float* scale, const int32_t* offsets, void* dw,
                void* dw2, int type, const DevStatus& st, int n_tiles, int splits, WeightArgs& a) {
    const uint64_t K = p->in_features, N = p->out_features, S = p->n_slots, P = p->n_parts, R = rows;
    int rc;
    for (int j = 0; j < 3; ++j)
        if ((rc = make_tmap_3d(&a.dy[j], dy, N, P, R, N * 2, N * P * 2, 64, 1, 16u << j)) ||
            (rc = X8 ? make_tmap_3d(&a.x[j], x, K, 1, R, K, K, 128, 1, 16u << j, true)
                     : make_tmap_3d(&a.x[j], x, K, 1, R, K * 2, K * 2, 64, 1, 16u << j)))
            return rc;
    const uint32_t box = type == MOE_OUT_BF16 ? 16 : 32;
    if ((rc = out_map(&a.out[0], dw, K, N, S, type, box, 1))) return rc;
    a.out[1] = a.out[0];
    if (dw2 && (rc = out_map(&a.out[1], dw2, K, N, S, type, box, 1))) return rc;
    a.scale = scale;
    a.offsets = offsets;
    a.R = rows;
    a.K = p->in_features;
    a.N = p->out_features;
    a.P = p->n_parts;
    a.S = p->n_slots;
    a.type = type;
    a.n_blk = (p->in_features + MOE_PAYLOAD_BLOCK - 1) / MOE_PAYLOAD_BLOCK;
    a.st = st;
    a.out_ptr[0] = dw;
    a.out_ptr[1] = dw2;
    a.n_tiles = n_tiles;
    a.splits = splits;
    return MOE_OK;
}

template <bool X8, bool M2, bool SHARED>
int launch_weights(const WeightArgs& a, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    return launch_pairs(weights_kernel<X8, M2, SHARED>, configured, weight_threads(X8, M2), kWeightSmem,
                        SHARED ? (long)a.n_tiles * a.splits : std::min<long>(a.n_tiles, most_pairs()), a.splits, stream, a,
                        "expert weight gradient");
}

// How dx and dW share the pairs of one launch: what they cost, in cycles, is 600 a tile and, for each chunk of its
// sum, of dx 2 for each row and 400 at least, of dW 512, or the turning of its codes, and a tile's drain at least,
// of dx 10 for each row, of dW 2400; sharing a sum costs 2300 and 5500.  Slots are not equal, so the pairs' last
// tiles count by half.  The plan is the one that ends first, and of those that end together the one that does the
// other part sooner.  (In place of pairs by the sums of the costs, and dW never shared: 10062 rows, 144 to 248
// features of 3 slots, gate and up, codes, 52 us and 21 so; 56 rows, 424 to 2856 of 7 slots, 27 and 16; 26 rows,
// 112 to 6064 of 29 slots, 52 both; 2771 rows, 504 to 3672 of 2 slots, 57 and 61.)
struct Work {
    int tiles, chunks, chunk, least, join;
    int64_t time(int pairs, int splits) const {
        const int64_t sum = std::max<int64_t>(least, (int64_t)((chunks + splits - 1) / splits) * chunk);
        const int64_t tile = 600 + sum + (splits > 1 ? join : 0), at_once = pairs / splits;
        return ((tiles + at_once - 1) / at_once * tile + std::max(tile, tiles * tile / at_once)) / 2;
    }
};
struct Plan {
    int x_pairs, w_pairs, x_splits, w_splits;
    int64_t time;
};
Plan best_plan(const Work& x, const Work& w) {
    Plan best{0, 0, 1, 1, INT64_MAX};
    auto offer = [&](int x_pairs, int w_pairs, int xs, int ws) {
        const int64_t xt = x.time(x_pairs, xs), wt = w.time(w_pairs, ws), time = std::max(xt, wt) + std::min(xt, wt) / 8;
        if (time < best.time) best = {x_pairs, w_pairs, xs, ws, time};
    };
    for (int xs = 1; xs <= 4; xs *= 2)
        for (int ws = 1; ws <= 4; ws *= 2) {
            const int group = std::max(xs, ws), there = group == 1 ? (int)most_pairs() : (int)resident(group) * group;
            if ((xs > 1 && x.chunks < 16) || (ws > 1 && w.chunks < 16)) continue;
            auto whole = [&](int pairs) { return (pairs + group - 1) / group * group; };  // of whole clusters
            const long x_need = (long)x.tiles * xs, w_need = (long)w.tiles * ws;
            if ((xs > 1 && x_need > there - group) || (ws > 1 && w_need > there - group)) continue;
            const int x_pairs = whole((int)std::min<long>(x_need, there)), w_pairs = whole((int)std::min<long>(w_need, there));
            if (xs > 1 && ws > 1) {
                if (x_pairs + w_pairs <= there) offer(x_pairs, w_pairs, xs, ws);
            } else if (xs > 1) {
                if (x_pairs < there) offer(x_pairs, std::min(w_pairs, there - x_pairs), xs, ws);
            } else if (ws > 1) {
                if (w_pairs < there) offer(std::min(x_pairs, there - w_pairs), w_pairs, xs, ws);
            } else {
                for (int n = 1; n < there && n <= x_pairs; ++n) offer(n, std::min(w_pairs, there - n), 1, 1);
            }
        }
    return best;
}

// How a backward pass runs: dx and dW in one launch (`one`), dW in tiles of twice 256 of N (`tall`), how many pairs
// share a sum.
struct BackwardPlan {
    RowsPlan rows;
    int w_tiles;
    bool one, tall;
    Plan plan;
};
BackwardPlan backward_plan(const moe_project_t* p, int rows, bool dx, bool dw, bool x8) {
    BackwardPlan b{rows_plan<true>(p, rows), 0, false, false, {0, 0, 1, 1, 0}};
    auto tiles = [&](int height) { return (p->in_features + 255L) / 256 * ((p->out_features + height - 1) / height) * p->n_parts * p->n_slots; };
    b.w_tiles = (int)tiles(256);
    const int w_chunks = chunks_of_slot(rows, p->n_slots);
    // Both in one launch up to a few tiles a pair.  (100 rows, 328 to 600 features of 16 slots, a tile or
    // two a pair, 12.2 us one after the other and 8.3 beside each other; 8000 rows, 2048 to 1024 of 16
    // slots, 12 tiles, 65 and 55; 4096 rows, 2048 to 7168 of 32 slots, a hundred, 332 and 383: there one
    // reads memory and the other writes it, and each takes all the pairs.)
    if (dx && dw && b.rows.tiles + b.w_tiles <= kBothTiles * most_pairs() && most_pairs() > 1) {
        const int used = std::min(rows, p->n_slots), each = (rows + used - 1) / used, height = std::min(b.rows.cap, each);
        // (dx's tiles: as many as there may be; chunks of dW: of equal slots)
        Work x{(int)b.rows.tiles, b.rows.chunks, std::max(400, 2 * height), 10 * height, 2300};
        Work w{b.w_tiles, w_chunks, x8 ? 900 : 512, 2400, 5500};
        b.one = true;
        b.plan = best_plan(x, w);
        return b;
    }
    if (dx) b.plan.x_splits = splits_of(b.rows.chunks, b.rows.tiles, 16);
    if (!dw) return b;
    // Twice 256 of N where that leaves every pair several tiles and, rows in bf16, where a slot has many
    // rows: the products of a tile hide the drain of one accumulator, not of the first of two (16 slots,
    // gate and up of 7168 to 2048: 128 rows a slot 163 us with 256 and 167 with twice that, 256 both 226,
    // 512 396 and 329; codes, which are turned half as often, 187 and 171, 266 and 244, 447 and 428.  16
    // slots of 1024 to 1024, 512 rows each: 19.1 and 21.1).
    b.tall = tiles(512) >= 4 * most_pairs() && (x8 || rows >= 384L * p->n_slots);
    if (b.tall) b.w_tiles = (int)tiles(512);
    else b.plan.w_splits = splits_of(w_chunks, b.w_tiles, 24);
    return b;
}

template <bool X8, bool SHARED>
int launch_both(const BothArgs& a, const Plan& plan, cudaStream_t stream) {
    static std::atomic<uint64_t> configured{0};
    return launch_pairs(gradients_kernel<X8, SHARED>, configured, weight_threads(X8, false), kBothSmem, plan.x_pairs + plan.w_pairs,
                        std::max(plan.x_splits, plan.w_splits), stream, a, "expert gradients");
}

template <bool X8>
int gradients(const moe_project_t* p, int rows, const void* dy, const void* x, const float* scale, const int32_t* offsets, const void* w,
              const void* w2, void* dx, int dx_type, void* dw, void* dw2, int dw_type, const DevStatus& st, cudaStream_t stream) {
    const BackwardPlan b = backward_plan(p, rows, dx, dw, X8);
    BothArgs a;
    int rc;
    if (dx && (rc = rows_args<true>(p, rows, dy, offsets, w, w2, dx, dx_type, st, b.rows.cap, b.plan.x_splits, a.dx))) return rc;
    if (dw && (rc = weight_args<X8>(p, rows, dy, x, scale, offsets, dw, dw2, dw_type, st, b.w_tiles, b.plan.w_splits, a.dw))) return rc;
    if (b.one) {
        a.dx_pairs = b.plan.x_pairs;
        return b.plan.w_splits > 1 ? launch_both<X8, true>(a, b.plan, stream) : launch_both<X8, false>(a, b.plan, stream);
    }
    if (dx && (rc = launch_rows<true>(a.dx, b.rows.tiles, stream))) return rc;
    if (!dw) return MOE_OK;
    if (b.tall) return launch_weights<X8, true, false>(a.dw, stream);
    return b.plan.w_splits > 1 ? launch_weights<X8, false, true>(a.dw, stream) : launch_weights<X8, false, false>(a.dw, stream);
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
    DevStatus st;
    if ((rc = api_device_status(&st))) return rc;
    const RowsPlan plan = rows_plan<false>(project, rows);
    RowsArgs a;
    if ((rc = rows_args<false>(project, rows, x, offsets, w, w2, out, out_type, st, plan.cap, splits_of(plan.chunks, plan.tiles, 16), a)))
        return rc;
    return launch_rows<false>(a, plan.tiles, reinterpret_cast<cudaStream_t>(stream));
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
    DevStatus st;
    if ((rc = api_device_status(&st))) return rc;
    return x8 ? gradients<true>(project, rows, dy, x8, x8_scale, offsets, w, w2, dx, dx_type, dw, dw2, dw_type, st, s)
              : gradients<false>(project, rows, dy, x, nullptr, offsets, w, w2, dx, dx_type, dw, dw2, dw_type, st, s);
}

int moe_debug_project_plan(const moe_project_t* project, int rows, int outputs, int32_t* plan) {
    const int rc = check_project(project, rows);
    if (rc) return rc;
    if (rows == 0 || outputs < 0 || outputs > 7 || outputs == MOE_PLAN_ROWS8 || !plan)
        return api_fail(MOE_ERR_INVALID_ARG, "rows > 0, MOE_PLAN_* of an output, and plan required");
    if (outputs == 0) {
        const RowsPlan y = rows_plan<false>(project, rows);
        plan[0] = splits_of(y.chunks, y.tiles, 16);
        plan[1] = plan[2] = plan[3] = 0;
        return MOE_OK;
    }
    const BackwardPlan b = backward_plan(project, rows, outputs & MOE_PLAN_DX, outputs & MOE_PLAN_DW, outputs & MOE_PLAN_ROWS8);
    plan[0] = outputs & MOE_PLAN_DX ? b.plan.x_splits : 0;
    plan[1] = outputs & MOE_PLAN_DW ? b.plan.w_splits : 0;
    plan[2] = b.one;
    plan[3] = b.tall;
    return MOE_OK;
}

}  // extern "C"

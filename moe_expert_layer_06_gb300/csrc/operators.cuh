// What the operators around the layer (scored_route.cu, adapter.cu, expert_project.cu, checkpoint.cu) share.
#pragma once

#include "kernels.h"

namespace moe {

// ---------------------------------------------------------------- launches
// launch_pdl in clusters of `cluster` CTAs along x (1: none).
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl_cluster(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                                      int cluster, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// ---------------------------------------------------------------- device
// Order this thread's shared-memory writes before later reads by the async proxy (TMA, UMMA).
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Barrier `id` of `threads` threads (whole warps).
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The same with a verdict of each thread: true on all of them if it was on every one.  Threads
// that share a barrier and wait for something with a limit decide this way whether they go on:
// one that left on its own would keep the others in their next barrier, which has no limit.
__device__ __forceinline__ bool named_and(int id, int threads, bool ok) {
    uint32_t all;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)ok), "r"(id), "r"(threads)
        : "memory");
    return all != 0;
}

// Shared-memory matrix descriptor of an MN-major operand tile written by TMA with
// 128-byte swizzle: K rows of 128 B (64 bf16 of M or N), 8-row groups 1024 B apart,
// blocks of 64 of M or N `block_bytes` apart.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(block_bytes >> 4) << 16;        // leading byte offset: next 64 of M or N
    d |= (uint64_t)(1024u >> 4) << 32;              // stride byte offset: next 8 of K
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
constexpr uint32_t kIdescAMnMajor = 1u << 15;  // A / B transposed (MN-major) in an instruction descriptor
constexpr uint32_t kIdescBMnMajor = 1u << 16;

// One lane of the (converged) warp.  TMA and UMMA operands have to sit in uniform
// registers: where the whole warp runs a loop and only the issue is guarded this way, they
// stay there (a loop inside `if (lane == 0)` took 540 cycles more per K chunk).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
    return p != 0;
}

// The whole warp waits for the phase: false on a timeout, or when another warp gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                          unsigned long long limit) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        if (!ok) ok = !*abort_flag && mbar_wait(bar, parity, limit);
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// After a wait that expired, before a CTA of a pair leaves: what is still on its way to shared memory (copies
// that signal the other CTA's barrier, signals, commits) cannot all be waited for by itself, as some of it is
// counted by barriers that the one who gave up no longer completes.  10 ms is a thousand times what any of it takes,
// however short the waits' own limit.
constexpr unsigned long long kSettleNs = 10000000;
__device__ __forceinline__ void settle_after_timeout() {
    for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < kSettleNs;) {}
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same where nothing written before it is read after it by another CTA: what it holds
// back is the reuse or the end of shared memory that has been read.  Every load from a peer
// before it has to be used before it, too (here: stored), as only that says that the load is
// over: none is issued whose value is then dropped.  (A release waits for the stores to
// global memory, 1.4 us at the end of a rank product.)
__device__ __forceinline__ void cluster_sync_read() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The two halves of a cluster's barrier, releasing nothing: barriers initialised before it (and
// fenced) are there for the others after it.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Four fp32 at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_peer4(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// ---- CTA pairs (cta_group::2): one product over the shared memory and tensor memory of both
// The address of `addr` in the pair's leader, CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr, uint32_t rank = 0) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

// Tiled load into this CTA, completing on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// D (+)= A B^T over the pair: 128 rows of A and half the rows of B in each CTA.
__device__ __forceinline__ void umma_bf16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the mbarrier at this offset of both CTAs (of the cluster, by their bits) when this thread's
// products are done.
__device__ __forceinline__ void umma_commit_pair(uint32_t bar, uint32_t ctas = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)ctas)
        : "memory");
}

// ---- a tile's bf16 outputs through shared memory
// 16 lanes x 32 columns: r[4 i + 0, 1] columns 8 i + 2 (lane % 4) + 0, 1 of row lane / 4, r[4 i + 2, 3] of row lane / 4 + 8
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ uint32_t pack_bf(uint32_t lo, uint32_t hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
    return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void stmatrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// The rows of slot s: offsets[s] to offsets[s + 1], within [0, rows] whatever they hold (false: they
// did not lie there, or ran backwards).
__device__ __forceinline__ bool slot_rows(const int32_t* offsets, int s, int rows, int& lo, int& hi) {
    const int a = __ldg(offsets + s), b = __ldg(offsets + s + 1);
    lo = min(max(a, 0), rows);
    hi = min(max(b, lo), rows);
    return a == lo && b == hi;
}

// ---------------------------------------------------------------- moe_api.cu
// make_tmap_3d for bf16 rows along dimension 1 (or 2 where dimension 1 is 1), with a swizzle of 128,
// 64 or 32 bytes, the box's inner extent at least.  Parts of rows that do not start on 128-byte lines
// are fetched 128 bytes at a time instead of 256: a wider fetch brings in more that the box does not
// read (4096 tokens, 840 to 4472 features: 48 us with wide fetches of W and the adapters, 46.8 with
// narrow ones; its gradients 71 and 67.5).
int make_tmap_rows(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1_bytes,
                   uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2, int swizzle_bytes = 128);
// Dense fp32 [d2][d1][d0], 128-byte swizzle.
int make_tmap_f32(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box0, uint32_t box1,
                  uint32_t box2);
int api_device_status(DevStatus* st);
// The router GEMM into ws (checked against moe_route_workspace_size): *ksplit partial
// logits [ksplit][T][E], to be added in order.
int api_router_gemm(const moe_shape_t* shape, int T, const void* x, const void* w_router, void* ws, size_t ws_bytes,
                    int* ksplit, cudaStream_t stream);
// Pointer checks: 0, or the error code with its text set.
int api_need(const void* p, const char* name, unsigned align = 16);
inline int launched(cudaError_t e, const char* what) {
    return e == cudaSuccess ? MOE_OK : api_fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace moe

// What the operators around the layer (scored_route.cu, adapter.cu) share.
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

// ---------------------------------------------------------------- moe_api.cu
// make_tmap_3d for bf16 rows along dimension 1 (or 2 where dimension 1 is 1), with a swizzle of 128,
// 64 or 32 bytes, the box's inner extent at least.  Parts of rows that do not start on 128-byte lines
// are fetched 128 bytes at a time instead of 256: a wider fetch brings in more that the box does not
// read (4096 tokens, 840 to 4472 features: 48 us with wide fetches of W and the adapters, 46.8 with
// narrow ones; its gradients 71 and 67.5).
int make_tmap_rows(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1_bytes,
                   uint64_t stride2_bytes, uint32_t box0, uint32_t box1, uint32_t box2, int swizzle_bytes = 128);
int api_device_status(DevStatus* st);
// The router GEMM into ws (checked against moe_route_workspace_size): *ksplit partial
// logits [ksplit][T][E], to be added in order.
int api_router_gemm(const moe_shape_t* shape, int T, const void* x, const void* w_router, void* ws, size_t ws_bytes,
                    int* ksplit, cudaStream_t stream);
// Pointer checks: 0, or the error code with its text set.
int api_need(const void* p, const char* name, unsigned align = 16);

}  // namespace moe

// What the attention kernels share: launches, the log-sum-exp they hand on, and their entry
// points for the dispatch in kv_attend.cu.
#pragma once

#include <atomic>

#include "kv_split.cuh"

namespace ftmoe {
namespace kv {

constexpr int kStepRows = 16;  // rows a (sequence, key head) of the single-token kernel

__device__ __forceinline__ void put_lse(const AttendParams &p, int64_t token, int h, float lse2) {
    if (p.lse) p.lse[token * p.q_heads + h] = lse2 * 0.6931471805599453f;
    if (p.lse2) p.lse2[token * p.q_heads + h] = lse2;
}

// 16 bytes to shared memory, zeros past the first `bytes` (0 or 16) of them; and all of them.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Clusters: this CTA's rank, a barrier of all, a read of another rank's shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();  // the barrier's instructions want converged warps
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_rank(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
        "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}
__device__ __forceinline__ float ld_rank1(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
        "ld.shared::cluster.f32 %0, [a];\n\t}"
        : "=f"(v)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// Dynamic shared memory of a kernel, allowed once a device (the call costs as much as a launch's
// other host work).
template <auto Kern>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Clusters of `size` (at most 8) CTAs of a kernel that the device holds at once, asked once a device.
template <auto Kern>
int most_clusters(int size, int threads, int smem) {
    static std::atomic<int> known[64][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    int n = dev < 64 ? known[dev][size].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, Kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (dev < 64) known[dev][size].store(n, std::memory_order_relaxed);
    return n;
}

// Launch in clusters of `size` CTAs along x.
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*kern)(P...), dim3 grid, int size, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr, cfg.numAttrs = size > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Launch that may start while the kernel before it still runs; it waits (griddepcontrol.wait)
// before it reads what that kernel wrote.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

int step_ctas(const AttendParams &p, int num_sms);
bool step_parts(const AttendParams &p, int num_sms);  // whether CTAs may leave parts to join
cudaError_t launch_step(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);
int chunk_ctas(const AttendParams &p, int num_sms);
bool chunk_parts(const AttendParams &p, int num_sms);
size_t chunk_rows();  // rows of an item of the chunk kernel
cudaError_t launch_chunk(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);
int mass_split(const AttendParams &p, int num_sms);
cudaError_t launch_mass(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace kv
}  // namespace ftmoe

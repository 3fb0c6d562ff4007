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

template <typename... P, typename... A>
cudaError_t launch_plain(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
    kern<<<grid, threads, smem, st>>>(args...);
    return cudaGetLastError();
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
cudaError_t launch_step(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);
int chunk_ctas(const AttendParams &p, int num_sms);
size_t chunk_rows();  // rows of an item of the chunk kernel
cudaError_t launch_chunk(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);
cudaError_t launch_mass(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace kv
}  // namespace ftmoe

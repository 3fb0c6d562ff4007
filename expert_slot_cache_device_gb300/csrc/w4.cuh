// Decoding of packed 4-bit codes, for both product kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.cuh"

namespace ftmoe {
namespace w4 {

// (128 + z, 128 + z) in bf16 or (1024 + z, 1024 + z) in f16.
template <bool BF>
__device__ __forceinline__ uint32_t offset2(uint32_t z) {
    return (BF ? 0x43004300u : 0x64006400u) | z | z << 16;
}
template <bool BF>
__device__ __forceinline__ uint32_t decode2(uint32_t w, uint32_t off) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "r"(0x000f000fu), "r"(BF ? 0x43004300u : 0x64006400u));
    if (BF) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&off));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// The product kernel of w4_tc05.cu.
cudaError_t launch_tc05(const MatvecParams &p, bool bf16, cudaStream_t st);

}  // namespace w4
}  // namespace ftmoe

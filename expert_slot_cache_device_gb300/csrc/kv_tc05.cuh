// tcgen05 pieces of the attention kernels: shared-memory descriptors, matrix instructions with
// the A operand in shared memory or in tensor memory, tensor-memory loads and stores, bounded
// barrier waits and the tensor maps of the pages.
#pragma once

#include <cuda.h>

#include "kv_attend.cuh"
#include "pipeline.cuh"

namespace ftmoe {
namespace kv {

using pipe::bar_arrive;
using pipe::bar_expect;
using pipe::bar_init;
using pipe::su32;

// Wait for the phase with the given parity, for at most two seconds (false then). The clock is
// read only once the barrier has not come at the first tries.
__device__ __forceinline__ bool try_bar(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(su32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_bar(uint64_t *b, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 16; i++)
        if (try_bar(b, parity)) return true;
    return pipe::bar_wait(b, parity);
}
// The same for a whole warp, which is converged afterwards.
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity) { return __all_sync(~0u, wait_bar(b, parity)); }

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(su32(bar)) : "memory");
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B of one 16-bit type, M = 128;
// b_mn: B stored with N (not K) consecutive.
template <bool BF, int N, bool B_MN>
constexpr uint32_t kInstr = (1u << 4) | ((BF ? 1u : 0u) << 7) | ((BF ? 1u : 0u) << 10) | ((B_MN ? 1u : 0u) << 16) |
                            ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);

// Operand of 128-byte rows with the 128-byte swizzle, groups of eight rows 1024 bytes apart
// (stride offset). K-major: rows are M or N, a K = 16 step 32 bytes further in the row. MN-major:
// rows are K, the next 64 elements of N `lead` bytes further (leading offset).
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <uint32_t I>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(I), "r"(acc)
        : "memory");
}
template <uint32_t I>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(I), "r"(acc)
        : "memory");
}

#define FTMOE_R4(x, i) "=r"((x)[i]), "=r"((x)[i + 1]), "=r"((x)[i + 2]), "=r"((x)[i + 3])
#define FTMOE_R32(x) FTMOE_R4(x, 0), FTMOE_R4(x, 4), FTMOE_R4(x, 8), FTMOE_R4(x, 12), FTMOE_R4(x, 16), FTMOE_R4(x, 20), FTMOE_R4(x, 24), FTMOE_R4(x, 28)
#define FTMOE_I4(x, i) "r"((x)[i]), "r"((x)[i + 1]), "r"((x)[i + 2]), "r"((x)[i + 3])
#define FTMOE_I32(x) FTMOE_I4(x, 0), FTMOE_I4(x, 4), FTMOE_I4(x, 8), FTMOE_I4(x, 12), FTMOE_I4(x, 16), FTMOE_I4(x, 20), FTMOE_I4(x, 24), FTMOE_I4(x, 28)

// 32 consecutive 32-bit columns of this thread's lane; the loaded registers are valid after the wait,
// which is in the same statement so that no use can move before it.
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : FTMOE_R32(x)
        : "r"(a)
        : "memory");
}
// 64 columns, one wait.
__device__ __forceinline__ void tm_ld64(uint32_t a, uint32_t *x) {
    uint32_t *y = x + 32;
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
        "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : FTMOE_R32(x), FTMOE_R32(y)
        : "r"(a), "r"(a + 32)
        : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
        FTMOE_I32(x)
        : "memory");
}
__device__ __forceinline__ void tm_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Packed fp32 pairs.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar))
        : "memory");
}

// Rows of an item of the tiled kernels: kTileRows consecutive (token, query head of the key
// head) rows, row r token r / group; an item's visible slots, lo cut down to a multiple of 128.
constexpr int kTileRows = 256, kTileSlots = 128;

struct Item {
    int lo, hi, seen_lo, tiles;
};

__device__ __forceinline__ int row_tiles(const Seq &s, int group) {
    return (int)(((int64_t)s.q_len * group + kTileRows - 1) / kTileRows);
}
__device__ __forceinline__ Item item_of(const AttendParams &p, const Seq &s, int qt) {
    const int64_t rows = (int64_t)s.q_len * p.group, r0 = (int64_t)qt * kTileRows;
    const int64_t r1 = r0 + kTileRows < rows ? r0 + kTileRows : rows;
    const Range v = visible(s, (int)(r0 / p.group), (int)((r1 - 1) / p.group) + 1, p.window, p.causal);
    Item it;
    it.seen_lo = v.lo, it.hi = v.hi, it.lo = v.lo & ~(kTileSlots - 1);
    it.tiles = (it.hi - it.lo + kTileSlots - 1) / kTileSlots;
    if (it.tiles < 1) it.tiles = 1;
    return it;
}
// Steps of one (sequence, key head) over all its row tiles; the whole warp calls.
__device__ __forceinline__ int seq_tiles(const AttendParams &p, const Seq &s, int end_qt) {
    int n = 0;
    for (int qt = threadIdx.x & 31; qt < end_qt; qt += 32) n += item_of(p, s, qt).tiles;
    return __reduce_add_sync(~0u, n);
}

// Tensor map of pages: [page][head][slot][element], boxes of 64 elements x box_slots slots.
bool page_map(CUtensorMap &m, const View &c, bool keys, bool bf16, int box_slots);

}  // namespace kv
}  // namespace ftmoe

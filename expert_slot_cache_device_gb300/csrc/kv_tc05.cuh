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

// Wait for the phase with the given parity: one test, which is all that a phase that is there
// costs, then at most 2^21 tries that suspend the thread for up to a microsecond each (false after
// the last).
__device__ __forceinline__ bool test_bar(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_bar(uint64_t *b, uint32_t parity) {
    const uint32_t bar = su32(b);
    if (test_bar(bar, parity)) return true;
#pragma unroll 1
    for (uint32_t i = 0; i < (1u << 21); i++) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return false;
}
// The same for a whole warp, which is converged afterwards.
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity) { return __all_sync(~0u, wait_bar(b, parity)); }

__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t elected, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(su32(bar)),
        "r"(elected)
        : "memory");
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B of one 16-bit type, M = 128;
// b_mn: B stored with N (not K) consecutive.
template <bool BF, int N, bool B_MN>
constexpr uint32_t kInstr = (1u << 4) | ((BF ? 1u : 0u) << 7) | ((BF ? 1u : 0u) << 10) | ((B_MN ? 1u : 0u) << 16) |
                            ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);

// Operand of 128-byte rows with the 128-byte swizzle, groups of eight rows 1024 bytes apart
// (stride offset), as the low word of its descriptor; the high word is kDescHi. K-major: rows are M
// or N, a K = 16 step 32 bytes further in the row. MN-major: rows are K, the next 64 elements of
// N `lead` bytes further (leading offset). Shared addresses fit the field, so a step of n bytes
// adds n / 16.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}

// The products are issued by a whole warp with one lane elected inside the statement, so that
// descriptors and addresses stay in uniform registers: issued under a lane's own branch, each
// instruction took 100 to 140 cycles to set up, longer than the 64 that it runs.
template <uint32_t I>
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(I), "r"(acc), "r"(elected), "r"(kDescHi)
        : "memory");
}
template <uint32_t I>
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b64 y, {%2, %6};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(I), "r"(acc), "r"(elected), "r"(kDescHi)
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
// 64 columns without a wait: the registers are valid after tm_ld_wait of the same registers.
__device__ __forceinline__ void tm_ld64(uint32_t a, uint32_t *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
        "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : FTMOE_R32(x), FTMOE_R32(x + 32)
        : "r"(a)
        : "memory");
}
#define FTMOE_U4(x, i) "+r"((x)[i]), "+r"((x)[i + 1]), "+r"((x)[i + 2]), "+r"((x)[i + 3])
#define FTMOE_U32(x) FTMOE_U4(x, 0), FTMOE_U4(x, 4), FTMOE_U4(x, 8), FTMOE_U4(x, 12), FTMOE_U4(x, 16), FTMOE_U4(x, 20), FTMOE_U4(x, 24), FTMOE_U4(x, 28)
__device__ __forceinline__ void tm_ld_wait(uint32_t *x) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : FTMOE_U32(x), FTMOE_U32(x + 32)::"memory");
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
        FTMOE_I4(x, 0), FTMOE_I4(x, 4), FTMOE_I4(x, 8), FTMOE_I4(x, 12)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
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

__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(su32(bar))
        : "memory");
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(su32(bar))
        : "memory");
}

// An item of the tiled kernels: two row tiles of 128 / group whole tokens each, row r of a tile
// (token r / group, query head r % group of the key head), so that a tile of queries is one box of
// a tensor map; the rows past the last whole token are not used. A step is 128 slots; an
// item's visible slots start at lo, cut down to a multiple of 128.
constexpr int kTileRows = 256, kTileSlots = 128;

struct Item {
    int lo, hi, seen_lo, tiles;
};

__device__ __forceinline__ int row_tiles(const AttendParams &p, const Seq &s) {
    return (int)((uint32_t)(s.q_len + p.item_tokens - 1) / (uint32_t)p.item_tokens);
}
__device__ __forceinline__ Item item_of(const AttendParams &p, const Seq &s, int qt) {
    const int i0 = qt * p.item_tokens, i1 = i0 + p.item_tokens < s.q_len ? i0 + p.item_tokens : s.q_len;
    const Range v = visible(s, i0, i1, p.window, p.causal);
    Item it;
    it.seen_lo = v.lo, it.hi = v.hi, it.lo = v.lo & ~(kTileSlots - 1);
    it.tiles = (it.hi - it.lo + kTileSlots - 1) / kTileSlots;
    if (it.tiles < 1) it.tiles = 1;
    return it;
}
// What an item adds to the line of work besides its steps: its start and end take about as long.
constexpr int kItemCost = 2;

// Units of one (sequence, key head) over its first end_qt items; the whole warp calls. They are counted
// in 64 bits: a prompt of a million tokens whose 128 query heads share a key head has 2^31. (The warp's 32-bit sums
// take the low 16 bits and the rest apart, which lanes below 2^43 fit.)
__device__ __forceinline__ long long seq_units(const AttendParams &p, const Seq &s, int end_qt) {
    long long n = 0;
    for (int qt = threadIdx.x & 31; qt < end_qt; qt += 32) n += item_of(p, s, qt).tiles + kItemCost;
    return ((long long)__reduce_add_sync(~0u, (uint32_t)(n >> 16)) << 16) + __reduce_add_sync(~0u, (uint32_t)n & 0xffffu);
}

// Where unit `at` of a sequence lies, whose key heads have `per` units each: key head, item, units into the item. The
// whole warp calls.
struct Place {
    int hk, qt, at;
};
__device__ __forceinline__ Place place_of(const AttendParams &p, const Seq &s, int n_qt, long long per, long long at) {
    const int lane = threadIdx.x & 31;
    // (a 64-bit division takes longer than the rest)
    const int hk = (at | per) >> 32 ? (int)(at / per) : (int)((uint32_t)at / (uint32_t)per);
    const long long rem = at - hk * per;
    long long before = 0;
    Place w{hk, -1, 0};
    for (int q0 = 0; q0 < n_qt && w.qt < 0; q0 += 32) {
        const int n = q0 + lane < n_qt ? item_of(p, s, q0 + lane).tiles + kItemCost : 0;  // 32 of them: below 2^30
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        const long long r = rem - before;
        const unsigned hit = __ballot_sync(~0u, n > 0 && r >= x - n && r < x);
        if (hit) {
            const int l = __ffs(hit) - 1;
            w.qt = q0 + l;
            w.at = (int)(r - __shfl_sync(~0u, x - n, l));
        }
        before += __shfl_sync(~0u, x, 31);
    }
    return w;
}

// Tensor map of pages: [page][head][slot][element], boxes of 64 elements x box_slots slots.
bool page_map(CUtensorMap &m, const View &c, bool keys, bool bf16, int box_slots);
// Tensor map of query rows: [token][head][element], boxes of 64 elements x group heads x 128 / group tokens.
bool query_map(CUtensorMap &m, const AttendParams &p, bool bf16);
// Tensor map of rows: [row][column], boxes of 64 columns x box_rows rows; zeros past the ends.
bool row_map(CUtensorMap &m, const void *x, int cols, int rows, int64_t stride, int box_rows, bool bf16);

}  // namespace kv
}  // namespace ftmoe

// How the attention kernels cut their work: an item is (sequence, key head, tile of rows) and takes
// as many units as its visible slots have steps of kUnit. The items' units stand in one line,
// sequence by sequence, head by head, tile by tile; CTA c of C takes units [c W / C, (c + 1) W / C) of
// the W in all. Lengths are on the device, so every CTA forms W and finds its own start. An item
// that one CTA covers is finished there. Of an item that several cover, each leaves the running
// maximum, sum and output rows of its part: in slot 2c + 1 if the part starts the item, else in
// slot 2c (a CTA has at most one part of each kind), and the combine kernel joins them in
// order: one CTA for each item that CTA c starts and does not end. Nothing depends on which
// runs first.
#pragma once

#include "kv.cuh"

namespace ftmoe {
namespace kv {

// What CTA c tells the joining kernel: x rows (or tokens) left of the item that its last part starts
// without ending (0: none), y key head, z first token row; w: its first part goes on with an item
// that an earlier CTA started (1), and ends it (2), or neither (0).
enum { kJoinNone = 0, kJoinOn = 1, kJoinEnd = 2 };

struct Range {
    int lo, hi;  // slots [lo, hi) that at least one row sees
};

// Visible slots of rows [i0, i1) (tokens) of a sequence: each token i, in slot kv_len - q_len + i,
// sees (slot - window, slot], or all slots when not causal.
__device__ __forceinline__ Range visible(const Seq &s, int i0, int i1, int window, int causal) {
    Range r;
    const int first = s.kv_len - s.q_len;
    r.hi = causal ? first + i1 : (first + i1 > 0 ? s.kv_len : 0);
    r.lo = window ? first + i0 - window + 1 : 0;
    if (r.hi < 0) r.hi = 0;
    if (r.lo < 0) r.lo = 0;
    if (r.lo > r.hi) r.lo = r.hi;
    return r;
}

// No CTA is left without a unit: of a grid wider than the line the first W take one each.
__device__ __forceinline__ int used_ctas(int grid, long long W) { return W < grid ? (int)W : grid; }
__device__ __forceinline__ long long unit_start(int c, int C, long long W) {
    if ((uint64_t)c * (uint64_t)W < (1ull << 32)) return (uint32_t)(c * (uint32_t)W) / (uint32_t)C;  // (a 64-bit division takes longer than the rest)
    return (long long)c * W / C;
}

// Parts of the item that CTA c starts: its own and those of the CTAs after it, up to the one that ends it.
__device__ __forceinline__ int count_parts(const int4 *join, int c, int grid) {
    const int lane = threadIdx.x & 31;
    for (int n = 1;; n += 32) {
        const int at = c + n + lane;
        const unsigned end = __ballot_sync(~0u, at >= grid || join[at].w == kJoinEnd);
        if (end) return n + __ffs(end);
    }
}

// Sum of v over the CTA's NT threads, and over the threads before this one.
template <int NT>
__device__ __forceinline__ long long block_scan(long long v, long long &total, long long *s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; w++) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    __syncthreads();
    return before + x - v;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// Factor that turns an unnormalised output row (maximum m in powers of two, sum l) into the
// result, and the row's log-sum-exp in powers of two, with the head's sink logit joined in.
__device__ __forceinline__ float finish_row(float m, float l, const float *sinks, int h, float &lse2) {
    float a = 1.f;
    if (sinks) {
        const float x = sinks[h] * kLog2e, n = fmaxf(m, x);
        a = m == -INFINITY ? 0.f : ex2(m - n);
        l = l * a + (x == -INFINITY ? 0.f : ex2(x - n));
        m = n;
    }
    lse2 = l == 0.f ? -INFINITY : m + log2f(l);
    return l == 0.f ? 0.f : a / l;
}

}  // namespace kv
}  // namespace ftmoe

// Eviction by accumulated attention weight: which slots of a (sequence, key head) stay, and the
// move of their rows to new pages.
//
// Select (one CTA a (sequence, key head)): masses become 32-bit keys in the floats' order (NaN
// lowest, -0 as 0). Four passes of eight bits from the top find the key T that the
// (budget - recent)-th largest has: a pass counts, among the keys that agree with T's known
// bits, each value of the next eight. Then one pass in slot order keeps keys above T and, of those
// equal to T, the first ones that fill the budget; positions come from block-wide prefix counts.
//
// Move: a kept row of K and of V is read and written once, 16 bytes a thread.
#include "kv.cuh"

namespace ftmoe {
namespace kv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

__device__ __forceinline__ uint32_t mass_key(float m) {
    if (m != m) return 0u;
    const uint32_t u = m == 0.f ? 0u : __float_as_uint(m);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sums of two 16-bit counts packed in v over the threads before this one, and over all.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t &total, uint32_t *s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        uint32_t w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(~0u, w, o);
            if (lane >= o) w += y;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    total = s_warp[31];
    const uint32_t r = x - v + (warp ? s_warp[warp - 1] : 0u);
    __syncthreads();
    return r;
}

__global__ void __launch_bounds__(kSelThreads) evict_select(const EvictParams p) {
    __shared__ uint32_t s_hist[256], s_warp[32];
    __shared__ uint32_t s_pick[2];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const int n = seq_kv_len(p.bt, b, p.c.status);
    const int m = n < p.budget ? n : p.budget;
    const int old = n <= p.budget ? n : n - p.recent;        // candidates: slots [0, old)
    const int need = m - (n - old);                          // of which this many stay
    const float *mass = p.mass + b * p.mass_seq + h * p.mass_head;
    int32_t *kept = p.kept + ((int64_t)b * p.c.kv_heads + h) * p.budget;
    float *out = p.new_mass + ((int64_t)b * p.c.kv_heads + h) * p.budget;
    if (h == 0 && tid == 0) p.new_lens[b] = m;

    uint32_t top = 0, mask = 0, left = need;  // T's known bits; how many of the keys that have them stay
    if (need < old && need > 0)
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) s_hist[tid] = 0;
            __syncthreads();
            for (int j = tid; j < old; j += kSelThreads) {
                const uint32_t k = mass_key(mass[j]);
                if ((k & mask) == top) atomicAdd(&s_hist[(k >> shift) & 255], 1u);
            }
            __syncthreads();
            if (tid == 0) {
                uint32_t c = 0;
                int d = 255;
                while (c + s_hist[d] < left) c += s_hist[d--];
                s_pick[0] = d;
                s_pick[1] = left - c;
            }
            __syncthreads();
            top |= s_pick[0] << shift;
            mask |= 255u << shift;
            left = s_pick[1];
            __syncthreads();
        }
    // slot order: above T, and the first `left` of those equal to it
    const bool all = need >= old;
    int base = 0, eq_before = 0;
    if (need > 0)
        for (int j0 = 0; j0 < old; j0 += kSelThreads) {
            const int j = j0 + tid;
            const float v = j < old ? mass[j] : 0.f;
            const uint32_t k = mass_key(v);
            const bool gt = j < old && (all || k > top), eq = j < old && !all && k == top;
            uint32_t total;
            const uint32_t pre = block_prefix((gt ? 1u : 0u) | (eq ? 1u << 16 : 0u), total, s_warp);
            const int e = eq_before + (int)(pre >> 16), used = e < (int)left ? e : (int)left;
            const int used0 = eq_before < (int)left ? eq_before : (int)left;
            const int at = base + (int)(pre & 0xffffu) + used - used0;
            if (gt || (eq && e < (int)left)) {
                kept[at] = j;
                out[at] = v;
            }
            eq_before += total >> 16;
            const int used1 = eq_before < (int)left ? eq_before : (int)left;
            base += (int)(total & 0xffffu) + used1 - used0;
        }
    for (int i = need + tid; i < p.budget; i += kSelThreads) {
        const int j = old + (i - need);
        kept[i] = i < m ? j : -1;
        out[i] = i < m ? mass[j] : 0.f;
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(const EvictParams p) {
    const int chunks = p.c.dim >> 3, heads = p.c.kv_heads, b = blockIdx.y;
    const int n = seq_kv_len(p.bt, b, p.c.status);
    const int m = n < p.budget ? n : p.budget;
    const int64_t items = (int64_t)m * heads * chunks;
    for (int64_t it = blockIdx.x * (int64_t)kMoveThreads + threadIdx.x; it < items; it += (int64_t)gridDim.x * kMoveThreads) {
        const int c = (int)(it % chunks), h = (int)(it / chunks % heads), i = (int)(it / chunks / heads);
        const int j = p.kept[((int64_t)b * heads + h) * p.budget + i];
        const int from = page_of(p.c, p.bt, b, j);
        const int to = p.new_table[b * p.new_stride + (i >> p.c.page_shift)];
        const int mask = (1 << p.c.page_shift) - 1;
        if (from < 0) continue;
        if ((uint32_t)to >= (uint32_t)p.c.num_pages) {
            flag(p.c.status, FTMOE_ERR_ID_RANGE);
            continue;
        }
        const uint4 k = *reinterpret_cast<const uint4 *>(p.c.k + k_at(p.c, from, j & mask, h) + 8 * c);
        const uint4 v = *reinterpret_cast<const uint4 *>(p.c.v + v_at(p.c, from, j & mask, h) + 8 * c);
        *reinterpret_cast<uint4 *>(p.c.k + k_at(p.c, to, i & mask, h) + 8 * c) = k;
        *reinterpret_cast<uint4 *>(p.c.v + v_at(p.c, to, i & mask, h) + 8 * c) = v;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t st) {
    evict_select<<<dim3(p.c.kv_heads, p.bt.batch), kSelThreads, 0, st>>>(p);
    const int most = p.budget < p.bt.max_kv ? p.budget : p.bt.max_kv;
    int64_t blocks = ((int64_t)most * p.c.kv_heads * (p.c.dim >> 3) + kMoveThreads - 1) / kMoveThreads;
    const int64_t cap = ((int64_t)num_sms * 8 + p.bt.batch - 1) / p.bt.batch;
    if (blocks > cap) blocks = cap;
    if (blocks > 0) evict_move<<<dim3((unsigned)blocks, p.bt.batch), kMoveThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kv
}  // namespace ftmoe

// Eviction by accumulated attention weight: which slots of a (sequence, key head) stay, and the
// move of their rows to new pages.
//
// Select (one CTA a (sequence, key head)): masses become 32-bit keys in the floats' order (NaN
// lowest, -0 as 0) in registers, warp w's keys consecutive in slots. The key T of the
// (budget - recent)-th largest is found two bits at a time from the top: the CTA counts the keys at or
// above three candidates, sixteen times. (Counting digits in shared memory took four times as
// long: most masses share their top bits, and atomics on one address wait for each other.) The search
// ends as soon as a candidate has exactly as many keys as are wanted.
// Keys above T stay and, of those equal to T, the first ones that fill the budget; their places
// come from ballots within a warp and one prefix over the warps.
//
// Move: a kept row of K and of V is read and written once, 16 bytes a thread.
//
// 16 sequences of up to 16384 slots, 8 key heads of 128, 4096 kept: 105 us, 25 for the selection (16 counts over a
// CTA, latency) and 78 for the move (0.52 GB, 6.7 TB/s, a plain copy's rate); 2 of 1013 slots, 500 kept: 8 us.
#include "kv_attend.cuh"

namespace ftmoe {
namespace kv {
namespace {

constexpr int kMoveThreads = 256;

__device__ __forceinline__ uint32_t mass_key(float m) {
    if (m != m) return 0u;
    const uint32_t u = m == 0.f ? 0u : __float_as_uint(m);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// NT threads hold KPT keys each at once; longer rows take several rounds, read again each time.
template <int NT, int KPT>
__global__ void __launch_bounds__(NT) evict_select(const EvictParams p) {
    constexpr int ROUND = NT * KPT;
    __shared__ int s_count[2][3][32];  // per warp, two iterations' in turn
    __shared__ int s_gt[32], s_eq[32];
    const int b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" :::);
    const int n = seq_kv_len(p.bt, b, p.c.status);
    const int m = n < p.budget ? n : p.budget;
    const int old = n <= p.budget ? n : n - p.recent;  // candidates: slots [0, old)
    const int need = m - (n - old);                    // of which this many stay
    const float *mass = p.mass + b * p.mass_seq + h * p.mass_head;
    int32_t *kept = p.kept + ((int64_t)b * p.c.kv_heads + h) * p.budget;
    float *out = p.new_mass + ((int64_t)b * p.c.kv_heads + h) * p.budget;
    if (h == 0 && tid == 0) p.new_lens[b] = m;
    if (tid < 32) {
        s_gt[tid] = s_eq[tid] = 0;
#pragma unroll
        for (int q = 0; q < 3; q++) s_count[0][q][tid] = s_count[1][q][tid] = 0;
    }

    const int rounds = (old + ROUND - 1) / ROUND;
    uint32_t key[KPT];
    float val[KPT];
    auto slot = [&](int r, int k) { return r * ROUND + (warp * KPT + k) * 32 + lane; };
    auto load = [&](int r) {
#pragma unroll
        for (int k = 0; k < KPT; k++) {
            const int j = slot(r, k);
            val[k] = j < old ? mass[j] : 0.f;
            key[k] = j < old ? mass_key(val[k]) : 0u;  // below every candidate threshold
        }
    };
    if (rounds > 0) load(0);
    __syncthreads();
    uint32_t T = 0;  // at least `need` keys are at or above it
    if (need < old && need > 0) {
        for (int it = 0; it < 16; it++) {
            const int shift = 30 - 2 * it;
            int c[3] = {0, 0, 0};
            for (int r = 0; r < rounds; r++) {
                if (rounds > 1) load(r);
#pragma unroll
                for (int k = 0; k < KPT; k++)
#pragma unroll
                    for (int q = 0; q < 3; q++) c[q] += key[k] >= (T | (uint32_t)(q + 1) << shift);
            }
#pragma unroll
            for (int q = 0; q < 3; q++) {
                c[q] = __reduce_add_sync(~0u, c[q]);
                if (lane == 0) s_count[it & 1][q][warp] = c[q];
            }
            __syncthreads();
            int at = 0, has = 0;
#pragma unroll
            for (int q = 2; q >= 0; q--) {
                const int sum = __reduce_add_sync(~0u, s_count[it & 1][q][lane]);
                if (at == 0 && sum >= need) at = q + 1, has = sum;
            }
            T |= (uint32_t)at << shift;
            if (has == need) {  // exactly the keys at or above T stay
                T--;
                break;
            }
        }
    }
    const bool all = need >= old;
    int gt_before = 0, eq_before = 0, above = 0;
    if (!all && need > 0) {  // keys above T: the rest of `need` are equal to it
        int c = 0;
        for (int r = 0; r < rounds; r++) {
            if (rounds > 1) load(r);
#pragma unroll
            for (int k = 0; k < KPT; k++) c += key[k] > T;
        }
        c = __reduce_add_sync(~0u, c);
        if (lane == 0) s_gt[warp] = c;
        __syncthreads();
        above = __reduce_add_sync(~0u, s_gt[lane]);
        __syncthreads();
    }
    const int quota = all ? 0 : need - above;  // keys equal to T that stay
    if (need > 0)
        for (int r = 0; r < rounds; r++) {
            if (rounds > 1) load(r);
            int gt = 0, eq = 0;
#pragma unroll
            for (int k = 0; k < KPT; k++) {
                const bool in = slot(r, k) < old;
                gt += __popc(__ballot_sync(~0u, in && (all || key[k] > T)));
                eq += __popc(__ballot_sync(~0u, in && !all && key[k] == T));
            }
            if (lane == 0) s_gt[warp] = gt, s_eq[warp] = eq;
            __syncthreads();
            int g0 = gt_before + __reduce_add_sync(~0u, lane < warp ? s_gt[lane] : 0);
            int e0 = eq_before + __reduce_add_sync(~0u, lane < warp ? s_eq[lane] : 0);
            gt_before += __reduce_add_sync(~0u, s_gt[lane]);
            eq_before += __reduce_add_sync(~0u, s_eq[lane]);
            const uint32_t lt = (1u << lane) - 1;
#pragma unroll
            for (int k = 0; k < KPT; k++) {
                const int j = slot(r, k);
                const bool isgt = j < old && (all || key[k] > T), iseq = j < old && !all && key[k] == T;
                const uint32_t bg = __ballot_sync(~0u, isgt), be = __ballot_sync(~0u, iseq);
                const int g = g0 + __popc(bg & lt), e = e0 + __popc(be & lt);
                if (isgt || (iseq && e < quota)) {
                    const int at = g + (e < quota ? e : quota);
                    kept[at] = j;
                    out[at] = val[k];
                }
                g0 += __popc(bg), e0 += __popc(be);
            }
            __syncthreads();
        }
    for (int i = need + tid; i < p.budget; i += NT) {
        const int j = old + (i - need);
        kept[i] = i < m ? j : -1;
        out[i] = i < m ? mass[j] : 0.f;
    }
}

__global__ void __launch_bounds__(kMoveThreads) evict_move(const EvictParams p) {
    const int chunks = p.c.dim >> 3, heads = p.c.kv_heads, b = blockIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    const dim3 grid(p.c.kv_heads, p.bt.batch);
    // the fewest threads that hold the longest row at once: every count waits for all of them (two sequences of 1013
    // slots: 256 threads 7.7 us, 1024 threads 12.2; of 8000 slots: 512 threads 16.7, 1024 threads 24.6)
    if (p.bt.max_kv <= 256 * 8)
        evict_select<256, 8><<<grid, 256, 0, st>>>(p);
    else if (p.bt.max_kv <= 512 * 16)
        evict_select<512, 16><<<grid, 512, 0, st>>>(p);
    else
        evict_select<1024, 16><<<grid, 1024, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int most = p.budget < p.bt.max_kv ? p.budget : p.bt.max_kv;
    int64_t blocks = ((int64_t)most * p.c.kv_heads * (p.c.dim >> 3) + kMoveThreads - 1) / kMoveThreads;
    const int64_t cap = ((int64_t)num_sms * 8 + p.bt.batch - 1) / p.bt.batch;
    if (blocks > cap) blocks = cap;
    if (blocks == 0) return cudaSuccess;
    return launch_after(evict_move, dim3((unsigned)blocks, p.bt.batch), kMoveThreads, 0, st, p);
}

}  // namespace kv
}  // namespace ftmoe

// Attention of at most 16 rows a (sequence, key head): the decode step, where the query heads of a
// key head (and the few new tokens) are the M = 16 rows of mma.sync m16n8k16. Bound by reading
// K and V once, 4 dim bytes a slot and key head.
//
// A CTA is four warps that share nothing while they read: warp w takes tiles w, w + 4, ... of 16
// slots (4 KiB of K and of V of 128 elements a head, 2 KiB of 64) through its own ring of kStages
// tiles filled by 16-byte cp.async, two CTAs an SM (four for 64), so up to 192 KiB are in flight on an SM. Rows
// past the visible range are zero-filled by the copy itself, so what such slots hold never
// reaches a product. Rows are stored with 16-byte chunk c of row r at c ^ (r % 8), which makes the
// eight rows of an ldmatrix distinct banks. Scores S = Q K^T and O += P V per tile; the softmax keeps
// a running maximum that O is rescaled to only when it grew by more than 2^8 (the sum and P use
// the same stale maximum, so the result is the same). P is rounded to the cache's type for P V, the type in which the tensor
// cores take it beside V (errors against 64 bits of 2.0e-3 in place of 1.6e-3 in bf16, where the output's own rounding is most of
// either); the sum, the log-sum-exp and the mass are of P in fp32.
//
// Work is cut by kv_split.cuh: one line of units of 64 slots over all (sequence, key head)s, an equal
// part for each CTA; a cut inside an item of at most kSnap units moves to its start, since joining
// parts costs more than the imbalance. Calls with few items and short caches, where latency is
// all, give each item to the eight CTAs of a cluster instead, which join through distributed shared
// memory: one launch, and no line of work to walk. With mass, the scaled scores are kept (fp32, powers of two) and the
// mass kernel adds 2^(x - lse) once the log-sum-exp is known, reading 4 bytes a (row, slot)
// instead of K again.
//
// 24 sequences of up to 16300 tokens, 4 key heads of 128, 16 query heads each (373 MB of K and V): 77 us, of which the
// first kernel takes 70 (5.3 TB/s, 0.79 of a plain copy) and the joining one the rest; with mass 95. SMs finish 10 us apart;
// 160 such sequences reach 6.5 TB/s. One sequence of 777 tokens: 5.4 us, 64 with a window of 128: 9.4, both latency.
#include "kv_split.cuh"
#include "kv_attend.cuh"
#include "pipeline.cuh"

namespace ftmoe {
namespace kv {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kStages = 3, kRows = kStepRows;
constexpr int kTile = 16, kUnit = kWarps * kTile, kSnap = 4, kCluster = 8;
template <int D>
struct Shape {
    static constexpr int kTileBytes = kTile * D * 2;  // K or V of one tile
    static constexpr int kStageBytes = 2 * kTileBytes, kRingBytes = kStages * kStageBytes, kSmem = kWarps * kRingBytes;
    static constexpr int kCtas = D == 64 ? 4 : 2;     // an SM
};
constexpr float kSlack = 8.f;  // the maximum may lag by 2^8

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a));
}
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        pipe::mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        pipe::mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Units of one (sequence, key head); a sequence with rows has at least one, which writes the
// result of rows that see nothing.
__device__ __forceinline__ int units_of(const Seq &s, const AttendParams &p, Range &r) {
    r = visible(s, 0, s.q_len, p.window, p.causal);
    r.lo &= ~(kTile - 1);
    const int u = (r.hi - r.lo + kUnit - 1) / kUnit;
    return s.q_len == 0 ? 0 : (u > 0 ? u : 1);
}

// A place on the line of units: sequence, key head, units into the item.
struct Spot {
    int b, hk, first;
};

// This CTA's units [u0, u1) and where u0 lies; false if there are none. s_cut: two entries.
__device__ __forceinline__ bool plan(const AttendParams &p, long long &u0, long long &u1, Spot &spot, long long *s_warp, Spot *s_spot,
                                     long long *s_cut) {
    const int tid = threadIdx.x;
    int32_t *status = blockIdx.x == 0 ? p.c.status : nullptr;
    long long mine = 0, total, at = 0;
    for (int b = tid; b < p.bt.batch; b += kThreads) {
        Range r;
        mine += units_of(seq_info(p.bt, b, status), p, r);
    }
    const bool once = p.bt.batch <= kThreads;  // then `mine` is sequence tid's, and one scan is all
    at = block_scan<kThreads>(mine, total, s_warp);
    const long long W = total * p.c.kv_heads;
    const int C = used_ctas(gridDim.x, W);
    if (blockIdx.x >= C) return false;
    u0 = unit_start(blockIdx.x, C, W), u1 = unit_start(blockIdx.x + 1, C, W);
    if (tid == 0) s_cut[0] = u0, s_cut[1] = u1;
    __syncthreads();
    long long base = 0;
    for (int b0 = 0; b0 < p.bt.batch; b0 += kThreads) {
        const int b = b0 + tid;
        if (!once) {
            Range r;
            mine = b < p.bt.batch ? units_of(seq_info(p.bt, b, nullptr), p, r) : 0;
            at = block_scan<kThreads>(mine, total, s_warp);
        }
        const long long from = base + at * p.c.kv_heads, to = from + mine * p.c.kv_heads;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const long long u = e ? u1 : u0;
            if (u >= from && u < to) {
                const int n = (int)mine;
                int first = (int)((u - from) % n);
                if (n <= kSnap) s_cut[e] = u - first, first = 0;
                if (e == 0) s_spot->b = b, s_spot->hk = (int)((u - from) / n), s_spot->first = first;
            }
        }
        base += total * p.c.kv_heads;
        if (once || base > u1) break;
    }
    __syncthreads();
    u0 = s_cut[0], u1 = s_cut[1], spot = *s_spot;
    return u0 < u1;
}

template <bool BF, int D, bool LOGITS, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, Shape<D>::kCtas) step_kernel(const AttendParams p) {
    constexpr int kTileBytes = Shape<D>::kTileBytes, kStageBytes = Shape<D>::kStageBytes, kRingBytes = Shape<D>::kRingBytes;
    constexpr int T = kTile, NT = T / 8, KT = T / 16, KS = D / 16, CH = D / 8, RPI = 32 / CH;
    extern __shared__ __align__(1024) unsigned char sm[];
    __shared__ long long s_warp[kWarps], s_cut[2];
    __shared__ Spot s_spot;
    __shared__ float s_ml[kWarps][kRows][2];
    __shared__ __align__(16) float s_out[CLUSTER ? kRows : 1][D + 4];  // joined across the cluster
    __shared__ __align__(16) float s_sum[CLUSTER ? kRows : 1][4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = pipe::su32(sm) + warp * kRingBytes;

    int b, hk, first, n_units;
    long long u = 0, u1 = 0;
    int4 join = make_int4(0, 0, 0, kJoinNone);
    Seq sq;
    Range vis;
    if (CLUSTER) {
        const int item = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
        b = item / p.c.kv_heads, hk = item % p.c.kv_heads;
        sq = seq_info(p.bt, b, p.c.status);
        n_units = units_of(sq, p, vis);
        asm volatile("griddepcontrol.launch_dependents;" :::);
        if (n_units == 0) return;  // the whole cluster
        first = rank * n_units / kCluster, u1 = (rank + 1) * n_units / kCluster - first;
    } else {
        Spot spot;
        const bool any = plan(p, u, u1, spot, s_warp, &s_spot, s_cut);
        asm volatile("griddepcontrol.launch_dependents;" :::);
        if (!any) {
            if (tid == 0 && p.join) p.join[blockIdx.x] = join;
            return;
        }
        b = spot.b, hk = spot.hk, first = spot.first;
        sq = seq_info(p.bt, b, nullptr);
        n_units = units_of(sq, p, vis);
    }

    const float c2 = p.scale * kLog2e;
    // this lane's chunk of a copied row, and its swizzled place in the RPI rows of one copy
    const int crow = lane / CH, cch = lane % CH;

    do {
        const int last = (int)(u1 - u < n_units - first ? first + (u1 - u) : n_units);  // units [first, last)
        const int rows = sq.q_len * p.group;
        const int lo_q = visible(sq, 0, sq.q_len, p.window, p.causal).lo;
        const int t0 = vis.lo / T + first * kWarps + warp;             // this warp's tiles: t0, t0 + 4, ...
        const int tiles = last - first;
        const uint16_t *kb = p.c.k + hk * p.c.k_head + 8 * cch, *vb = p.c.v + hk * p.c.v_head + 8 * cch;
        const int32_t *tab = p.bt.table + (int64_t)b * p.bt.table_stride;
        const int pmask = (1 << p.c.page_shift) - 1;

        // page of each 16 slots of tile i, one tile ahead of its copy; -1: nothing there to read
        auto pages = [&](int i, int (&pg)[KT]) {
#pragma unroll
            for (int k = 0; k < KT; k++) {
                const int slot = (t0 + i * kWarps) * T + 16 * k;
                pg[k] = -1;
                if (i < tiles && slot < vis.hi && slot + 16 > lo_q) {
                    pg[k] = tab[slot >> p.c.page_shift];
                    if ((uint32_t)pg[k] >= (uint32_t)p.c.num_pages) {
                        flag(p.c.status, FTMOE_ERR_ID_RANGE);
                        pg[k] = -1;
                    }
                }
            }
        };
        auto copy = [&](int i, const int (&pg)[KT]) {
            if (i < tiles) {
                const int slot0 = (t0 + i * kWarps) * T;
                const uint32_t st = ring + (i % kStages) * kStageBytes;
#pragma unroll
                for (int n = 0; n < T / RPI; n++) {
                    const int r = n * RPI + crow, slot = slot0 + r, page = pg[n * RPI / 16];
                    const bool ok = page >= 0 && slot >= lo_q && slot < vis.hi;
                    const uint32_t at = st + r * (2 * D) + (((cch & ~7) | ((cch ^ r) & 7)) << 4);
                    const int64_t pr = ok ? page : 0, row = ok ? slot & pmask : 0;
                    cp16(at, kb + pr * p.c.k_page + row * p.c.k_slot, ok ? 16 : 0);
                    cp16(at + kTileBytes, vb + pr * p.c.v_page + row * p.c.v_slot, ok ? 16 : 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        int pg[KT];
#pragma unroll
        for (int i = 0; i < kStages; i++) {
            pages(i, pg);
            copy(i, pg);
        }

        // the rows' queries as A fragments: rows g and g + 8
        uint32_t qf[KS][4];
        int end[2], beg[2];
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const int r = g + 8 * e, i = r / p.group, h = hk * p.group + r % p.group;
            const bool live = r < rows;
            const Range v = visible(sq, i, i + 1, p.window, p.causal);
            beg[e] = live ? v.lo : 0, end[e] = live ? v.hi : 0;
            const uint16_t *q = p.q.d + (int64_t)(sq.q0 + i) * p.q.token + h * p.q.head + 2 * t;
#pragma unroll
            for (int k = 0; k < KS; k++) {
                qf[k][e] = live ? *reinterpret_cast<const uint32_t *>(q + 16 * k) : 0;
                qf[k][2 + e] = live ? *reinterpret_cast<const uint32_t *>(q + 16 * k + 8) : 0;
            }
        }
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
        for (int n = 0; n < D / 8; n++) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

        for (int i = 0; i < tiles; i++) {
            pages(i + kStages, pg);
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint32_t st = ring + (i % kStages) * kStageBytes;
            const int slot0 = (t0 + i * kWarps) * T;

            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            // matrices of an ldmatrix: (slots 0-7, d 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
            const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    const int r = kr + 8 * n, ch = 2 * k + kc;
                    uint32_t f[4];
                    ldsm4(f, st + r * (2 * D) + (((ch & ~7) | ((ch ^ r) & 7)) << 4));
                    mma<BF>(s[n], qf[k], f[0], f[1]);
                    mma<BF>(s[n + 1], qf[k], f[2], f[3]);
                }
            // visible slots, in powers of two
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int slot = slot0 + 8 * n + 2 * t + (e & 1), r = e >> 1;
                    s[n][e] = slot >= beg[r] && slot < end[r] ? s[n][e] * c2 : -INFINITY;
                    mx[r] = fmaxf(mx[r], s[n][e]);
                }
            if (LOGITS) {
#pragma unroll
                for (int r = 0; r < 2; r++)
                    if (g + 8 * r < rows) {
                        float *x = p.logits + ((int64_t)(b * p.c.kv_heads + hk) * p.logit_rows + g + 8 * r) * p.logit_stride;
#pragma unroll
                        for (int n = 0; n < NT; n++)
                            if (slot0 + 8 * n < vis.hi)
                                *reinterpret_cast<float2 *>(x + slot0 + 8 * n + 2 * t) = make_float2(s[n][2 * r], s[n][2 * r + 1]);
                    }
            }
#pragma unroll
            for (int r = 0; r < 2; r++) {
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
            }
            if (__any_sync(~0u, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const float n = fmaxf(m[r], mx[r]), a = m[r] == -INFINITY ? 0.f : ex2(m[r] - n);
                    m[r] = n;
                    l[r] *= a;
#pragma unroll
                    for (int k = 0; k < D / 8; k++) o[k][2 * r] *= a, o[k][2 * r + 1] *= a;
                }
            }
            const float z[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
            uint32_t pf[KT][4];
#pragma unroll
            for (int n = 0; n < NT; n++) {
                const float p0 = ex2(s[n][0] - z[0]), p1 = ex2(s[n][1] - z[0]);
                const float p2 = ex2(s[n][2] - z[1]), p3 = ex2(s[n][3] - z[1]);
                l[0] += p0 + p1;
                l[1] += p2 + p3;
                pf[n / 2][2 * (n & 1)] = from_f2<BF>(p0, p1);
                pf[n / 2][2 * (n & 1) + 1] = from_f2<BF>(p2, p3);
            }
            // matrices: (slots 0-7, d 0-7), (slots 8-15, d 0-7), (0-7, 8-15), (8-15, 8-15)
#pragma unroll
            for (int k = 0; k < KT; k++)
#pragma unroll
                for (int n = 0; n < D / 8; n += 2) {
                    const int r = 16 * k + (lane & 15), ch = n + (lane >> 4);
                    uint32_t f[4];
                    ldsm4t(f, st + kTileBytes + r * (2 * D) + (((ch & ~7) | ((ch ^ r) & 7)) << 4));
                    mma<BF>(o[n], pf[k], f[0], f[1]);
                    mma<BF>(o[n + 1], pf[k], f[2], f[3]);
                }
            __syncwarp();
            copy(i + kStages, pg);  // into the stage just read, before the next wait: kStages tiles are in flight then
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        // ---- join the four warps: a common maximum, then the sums in warp order
#pragma unroll
        for (int r = 0; r < 2; r++) {
            l[r] += __shfl_xor_sync(~0u, l[r], 1);
            l[r] += __shfl_xor_sync(~0u, l[r], 2);
            if (t == 0) s_ml[warp][g + 8 * r][0] = m[r], s_ml[warp][g + 8 * r][1] = l[r];
        }
        __syncthreads();
        constexpr int OS = D + 4;  // row stride of the exchanged rows (fp32), off the banks' period
        float *mine = reinterpret_cast<float *>(sm + warp * kRingBytes);
#pragma unroll
        for (int r = 0; r < 2; r++) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; w++) M = fmaxf(M, s_ml[w][g + 8 * r][0]);
            const float a = m[r] == -INFINITY ? 0.f : ex2(m[r] - M);
#pragma unroll
            for (int n = 0; n < D / 8; n++)
                *reinterpret_cast<float2 *>(mine + (g + 8 * r) * OS + 8 * n + 2 * t) = make_float2(o[n][2 * r] * a, o[n][2 * r + 1] * a);
        }
        __syncthreads();
        const bool whole = !CLUSTER && first == 0 && last == n_units;
        constexpr int PER = kRows * D / kThreads;  // consecutive elements of one row a thread
        const int row = tid / (D / PER), d0 = tid % (D / PER) * PER;
        if (row < rows) {
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) M = fmaxf(M, s_ml[w][row][0]);
#pragma unroll
            for (int w = 0; w < kWarps; w++) L += s_ml[w][row][1] * (s_ml[w][row][0] == -INFINITY ? 0.f : ex2(s_ml[w][row][0] - M));  // (a NaN stays)
            float x[PER];
#pragma unroll
            for (int e = 0; e < PER; e += 4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; w++) {
                    const float4 y = *reinterpret_cast<const float4 *>(sm + w * kRingBytes + (row * OS + d0 + e) * 4);
                    v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                }
                x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
            }
            if (CLUSTER) {
#pragma unroll
                for (int e = 0; e < PER; e += 4) *reinterpret_cast<float4 *>(&s_out[row][d0 + e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                if (d0 == 0) *reinterpret_cast<float4 *>(s_sum[row]) = make_float4(M, L, 0.f, 0.f);
            } else if (whole) {
                const int i = row / p.group, h = hk * p.group + row % p.group;
                float lse2;
                const float f = finish_row(M, L, p.sinks, h, lse2);
                uint16_t *out = p.out.d + (int64_t)(sq.q0 + i) * p.out.token + h * p.out.head + d0;
#pragma unroll
                for (int e = 0; e < PER; e += 8)
                    *reinterpret_cast<uint4 *>(out + e) =
                        make_uint4(from_f2<BF>(x[e] * f, x[e + 1] * f), from_f2<BF>(x[e + 2] * f, x[e + 3] * f),
                                   from_f2<BF>(x[e + 4] * f, x[e + 5] * f), from_f2<BF>(x[e + 6] * f, x[e + 7] * f));
                if (d0 == 0) put_lse(p, sq.q0 + i, h, lse2);
            } else {
                const int slot = 2 * blockIdx.x + (first == 0 ? 1 : 0);
                float *po = p.part_o + ((int64_t)slot * kRows + row) * D + d0;
#pragma unroll
                for (int e = 0; e < PER; e += 4) *reinterpret_cast<float4 *>(po + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                if (d0 == 0) p.part_ml[slot * kRows + row] = make_float2(M, L);
            }
        }
        if (CLUSTER) {
            cluster_sync();
            // rank r joins rows 2r and 2r + 1: half the threads a row
            constexpr int EP = kRows * D / kCluster / kThreads;
            const int jr = (blockIdx.x % kCluster) * (kRows / kCluster) + tid / (D / EP), d = tid % (D / EP) * EP;
            float M = -INFINITY, L = 0.f, x[2] = {0.f, 0.f};
            if (jr < rows) {
                float4 ml[kCluster];
#pragma unroll
                for (int k = 0; k < kCluster; k++) ml[k] = ld_rank(pipe::su32(s_sum[jr]), k);
#pragma unroll
                for (int k = 0; k < kCluster; k++) M = fmaxf(M, ml[k].x);
#pragma unroll
                for (int k = 0; k < kCluster; k++) {
                    const float a = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
                    L += ml[k].y * a;
#pragma unroll
                    for (int e = 0; e < EP; e++) x[e] += ld_rank1(pipe::su32(&s_out[jr][d + e]), k) * a;
                }
                const int i = jr / (uint32_t)p.group, h = hk * p.group + jr - i * p.group;
                float lse2;
                const float f = finish_row(M, L, p.sinks, h, lse2);
                uint16_t *out = p.out.d + (int64_t)(sq.q0 + i) * p.out.token + h * p.out.head + d;
                if (EP == 2)
                    *reinterpret_cast<uint32_t *>(out) = from_f2<BF>(x[0] * f, x[1] * f);
                else
                    *out = from_f<BF>(x[0] * f);
                if (d == 0) put_lse(p, sq.q0 + i, h, lse2);
            }
            cluster_sync();  // no rank leaves while its rows are read
            return;
        }
        if (!whole) {
            if (first == 0)
                join.x = rows, join.y = hk, join.z = sq.q0;
            else
                join.w = last == n_units ? kJoinEnd : kJoinOn;
        }
        __syncthreads();  // the rings are written again
        // ---- the next item
        u += last - first;
        first = 0;
        if (u < u1 && ++hk == p.c.kv_heads) {
            hk = 0;
            do {
                sq = seq_info(p.bt, ++b, nullptr);
                n_units = units_of(sq, p, vis);
            } while (n_units == 0);
        }
    } while (u < u1);
    if (tid == 0 && p.join) p.join[blockIdx.x] = join;  // (null where no item is cut)
}

// Joins the parts of the item that CTA c of the step kernel started: one warp a row, lanes over the
// elements, the parts' weights first.
template <bool BF, int D>
__global__ void __launch_bounds__(32 * kRows) step_combine(const AttendParams p) {
    constexpr int E = D / 32;
    const int c = blockIdx.x, row = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" :::);
    // the first 32 CTAs' entries and this row's sums of their parts come together
    auto slot = [&](int i) { return (2 * (c + i) + (i == 0)) * kRows + row; };
    const bool in = c + lane < gridDim.x;
    const int4 mine = in ? p.join[c + lane] : make_int4(0, 0, 0, kJoinEnd);
    float2 ml = in ? p.part_ml[slot(lane)] : make_float2(-INFINITY, 0.f);
    const int4 join = make_int4(__shfl_sync(~0u, mine.x, 0), __shfl_sync(~0u, mine.y, 0), __shfl_sync(~0u, mine.z, 0), 0);
    if (row >= join.x) return;
    const unsigned end = __ballot_sync(~0u, lane > 0 && mine.w == kJoinEnd);
    const int n = end ? __ffs(end) : count_parts(p.join, c, gridDim.x);
    float M = -INFINITY, L = 0.f, x[E];
#pragma unroll
    for (int e = 0; e < E; e++) x[e] = 0.f;
    if (lane < n) M = ml.x;
    for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    for (int i0 = 0; i0 < n; i0 += 32) {
        float a = 0.f;
        if (i0 + lane < n) {
            if (i0) ml = p.part_ml[slot(i0 + lane)];
            a = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            L += ml.y * a;
        }
        const int m = n - i0 < 32 ? n - i0 : 32;
#pragma unroll 16
        for (int i = 0; i < m; i++) {
            const float w = __shfl_sync(~0u, a, i);
            const float *po = p.part_o + (int64_t)slot(i0 + i) * D + lane * E;
            float v[E];
            if (E == 4)
                *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(po);
            else
                *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(po);
#pragma unroll
            for (int e = 0; e < E; e++) x[e] += v[e] * w;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(~0u, L, o);
    const int i = row / (uint32_t)p.group, h = join.y * p.group + row - i * p.group;
    float lse2;
    const float f = finish_row(M, L, p.sinks, h, lse2);
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out.d + (int64_t)(join.z + i) * p.out.token + h * p.out.head + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = from_f2<BF>(x[e] * f, x[e + 1] * f);
    if (lane == 0) put_lse(p, join.z + i, h, lse2);
}

// mass += sum over rows of 2^(x - lse2), x the kept scores: one thread a slot, rows in order.
__global__ void __launch_bounds__(256) step_mass(const AttendParams p) {
    __shared__ float s_lse[kRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int hk = blockIdx.y, b = blockIdx.z;
    const Seq sq = seq_info(p.bt, b, nullptr);
    const int rows = sq.q_len * p.group;
    const Range vis = visible(sq, 0, sq.q_len, p.window, p.causal);
    const int j0 = blockIdx.x * 1024;
    if (rows == 0 || j0 >= vis.hi || j0 + 1024 <= vis.lo) return;
    if (threadIdx.x < rows) {
        const int i = threadIdx.x / p.group, h = hk * p.group + threadIdx.x % p.group;
        s_lse[threadIdx.x] = p.lse2[(int64_t)(sq.q0 + i) * p.q_heads + h];
    }
    __syncthreads();
    const int j = j0 + threadIdx.x * 4;
    if (j >= vis.hi || j + 4 <= vis.lo) return;
    const float *x = p.logits + (int64_t)(b * p.c.kv_heads + hk) * p.logit_rows * p.logit_stride + j;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int r = 0; r < rows; r++) {
        const float4 v = *reinterpret_cast<const float4 *>(x + r * p.logit_stride);
        const float z = s_lse[r];
        if (z == -INFINITY) continue;
        s[0] += ex2(v.x - z), s[1] += ex2(v.y - z), s[2] += ex2(v.z - z), s[3] += ex2(v.w - z);
    }
    float *m = p.mass + b * p.mass_seq + hk * p.mass_head + j;
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (j + e >= vis.lo && j + e < vis.hi) m[e] += s[e];
}

// The most units that an item of this call can have.
int most_units(const AttendParams &p) {
    int64_t slots = p.bt.max_kv;
    if (p.window && (int64_t)p.window + p.bt.max_q + kTile < slots) slots = p.window + p.bt.max_q + kTile;
    return (int)((slots + kUnit - 1) / kUnit);
}

// Clusters while all of them fit at once and a rank has at most eight units (one sequence of 777
// tokens, four key heads: 6 us against 12 with a second kernel; beyond, the line of work
// uses every SM).
bool in_clusters(const AttendParams &p, int num_sms) {
    const int fit = num_sms * (p.c.dim == 64 ? Shape<64>::kCtas : Shape<128>::kCtas);
    return (int64_t)p.bt.batch * p.c.kv_heads * kCluster <= fit && most_units(p) <= 8 * kCluster;
}

template <bool BF, int D, bool LOGITS>
cudaError_t launch_kernels(const AttendParams &p, int num_sms, cudaStream_t st) {
    constexpr int smem = Shape<D>::kSmem;
    const int C = step_ctas(p, num_sms);
    const int64_t items = (int64_t)p.bt.batch * p.c.kv_heads;
    cudaError_t e;
    if (in_clusters(p, num_sms)) {
        if ((e = allow_smem<step_kernel<BF, D, LOGITS, true>>(smem)) != cudaSuccess) return e;
        e = launch_clusters(step_kernel<BF, D, LOGITS, true>, dim3((unsigned)items * kCluster), kCluster, kThreads, smem, st, p);
    } else {
        if ((e = allow_smem<step_kernel<BF, D, LOGITS, false>>(smem)) != cudaSuccess) return e;
        step_kernel<BF, D, LOGITS, false><<<C, kThreads, smem, st>>>(p);
        e = cudaGetLastError();
        if (e == cudaSuccess && step_parts(p, num_sms)) e = launch_after(step_combine<BF, D>, dim3(C), 32 * kRows, 0, st, p);
    }
    if (e == cudaSuccess && LOGITS && p.bt.max_kv > 0) e = launch_after(step_mass, dim3((p.bt.max_kv + 1023) / 1024, p.c.kv_heads, p.bt.batch), 256, 0, st, p);
    return e;
}

template <bool BF, int D>
cudaError_t launch(const AttendParams &p, int num_sms, cudaStream_t st) {
    return p.logits ? launch_kernels<BF, D, true>(p, num_sms, st) : launch_kernels<BF, D, false>(p, num_sms, st);
}

}  // namespace

// No joining kernel where no item is long enough to be cut.
bool step_parts(const AttendParams &p, int num_sms) { return !in_clusters(p, num_sms) && most_units(p) > kSnap; }

int step_ctas(const AttendParams &p, int num_sms) {
    const long long most = (long long)p.bt.batch * p.c.kv_heads * ((p.bt.max_kv + kUnit - 1) / kUnit + 1);
    const int fit = num_sms * (p.c.dim == 64 ? Shape<64>::kCtas : Shape<128>::kCtas);
    return (int)(most < fit ? (most > 0 ? most : 1) : fit);
}

cudaError_t launch_step(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    if (p.c.dim == 64) return bf16 ? launch<true, 64>(p, num_sms, st) : launch<false, 64>(p, num_sms, st);
    return bf16 ? launch<true, 128>(p, num_sms, st) : launch<false, 128>(p, num_sms, st);
}

}  // namespace kv
}  // namespace ftmoe

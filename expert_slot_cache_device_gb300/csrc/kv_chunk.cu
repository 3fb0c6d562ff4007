// Attention of chunks of new tokens on the 5th-generation tensor cores. An item is 256 consecutive
// (token, query head) rows of one (sequence, key head), as two tiles of M = 128: the query heads that
// share a key head read K and V from shared memory once. Bound by the tensor cores: 4 dim flops a
// (row, slot) against one exponential.
//
// Persistent, one CTA an SM, work cut by kv_split.cuh in steps of 128 slots. Roles:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: a thread holds one row. S comes from tensor
//                   memory; the row's maximum, P = 2^(s scale log2 e - m) in fp32, the row's sum; P
//                   goes back as 16-bit pairs. O is rescaled (in tensor memory) only when the
//                   maximum grew by more than 2^8; P and the sum share the stale maximum.
//   warp 8          tensor copies of K and V tiles (a box a page and 64 elements, 128-byte swizzle)
//                   into a ring of stages; pages outside the visible range are not touched.
//   warp 9          issues tcgen05.mma: S_t = Q_t K^T (both from shared memory) and O_t += P_t V (P
//                   from tensor memory, V with its elements consecutive). While the softmax of one
//                   tile runs, the other tile's products do.
//   warps 10, 11    copy Q of the next item as soon as the last S product has read the present
//                   one, and zero the V rows of slots that no row sees in the tiles at the ends
//                   of the visible range (what such slots hold must not reach 0 * V).
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (dim each). P_t lies over S_t for 128
// elements a head: S_t of the next step is issued after the product that reads P_t, and products
// of one shape run in order. For 64 the shapes differ, and P_0, P_1 have columns of their own.
// Every wait is bounded; one that runs out is recorded and ends the role.
#include "kv_tc05.cuh"

namespace ftmoe {
namespace kv {
namespace {

constexpr int kWarps = 12, kThreads = kWarps * 32;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kHelpWarp = 10;
constexpr float kSlack = 8.f;
constexpr int kMaxStages = 8;

template <int D>
struct Shape {
    static constexpr int kStage = kTileSlots * D * 2;         // K or V of one step
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kHalf = kTileSlots * 128;            // 64 elements of 128 rows
    static constexpr int kQ = kTileRows * D * 2;
    static constexpr int kSmem = 1024 + kStages * kStage + kQ;
    static constexpr uint32_t kO = 256, kP = D == 128 ? 0 : 384;  // columns of O_0 and P_0
    static constexpr uint32_t kPStep = D == 128 ? 128 : 64;       // from P_0 to P_1
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t qfull, qempty, s[2], p[2], o[2], clean, done;
};

// A part of an item that this CTA works on, and the walk from part to part. Every role walks on
// its own.
struct Part {
    int b, hk, qt, first, last;  // steps [first, last) of the item
    Item it;
    Seq sq;
};

struct Walk {
    long long left;
    int b, hk, qt, n_qt, first;
    Seq sq;
    __device__ __forceinline__ bool next(const AttendParams &p, Part &w) {
        if (left <= 0) return false;
        w.it = item_of(p, sq, qt);
        w.b = b, w.hk = hk, w.qt = qt, w.sq = sq, w.first = first;
        w.last = left < w.it.tiles - first ? first + (int)left : w.it.tiles;
        left -= w.last - first;
        first = 0;
        if (left > 0 && ++qt == n_qt) {
            qt = 0;
            if (++hk == p.c.kv_heads) {
                hk = 0;
                do {
                    sq = seq_info(p.bt, ++b, nullptr);
                    n_qt = row_tiles(sq, p.group);
                } while (n_qt == 0);
            }
        }
        return true;
    }
};

// Total steps and this CTA's start. s_sum: kThreads entries.
__device__ __forceinline__ bool plan(const AttendParams &p, Walk &w, long long *s_warp, int *s_sum, Walk *s_walk) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    long long sum = 0, total;
    for (int b0 = 0; b0 < p.bt.batch; b0 += kThreads) {
        for (int i = warp; i < kThreads; i += kWarps) {
            int n = 0;
            if (b0 + i < p.bt.batch) {
                const Seq s = seq_info(p.bt, b0 + i, blockIdx.x == 0 && lane == 0 ? p.c.status : nullptr);
                n = seq_tiles(p, s, row_tiles(s, p.group));
            }
            if (lane == 0) s_sum[i] = n;
            if (b0 + i >= p.bt.batch) break;
        }
        __syncthreads();
        if (b0 + tid < p.bt.batch) sum += s_sum[tid];
        if (b0 + kThreads < p.bt.batch) __syncthreads();
    }
    block_scan<kThreads>(sum, total, s_warp);
    const long long W = total * p.c.kv_heads;
    const int C = used_ctas(gridDim.x, W);
    if (blockIdx.x >= C) return false;
    const long long u0 = unit_start(blockIdx.x, C, W), u1 = unit_start(blockIdx.x + 1, C, W);
    long long base = 0;
    for (int b0 = 0; b0 < p.bt.batch; b0 += kThreads) {
        if (p.bt.batch > kThreads) {  // the sums of the last round are not these
            __syncthreads();
            for (int i = warp; i < kThreads; i += kWarps) {
                if (b0 + i >= p.bt.batch) break;
                const Seq s = seq_info(p.bt, b0 + i, nullptr);
                const int n = seq_tiles(p, s, row_tiles(s, p.group));
                if (lane == 0) s_sum[i] = n;
            }
            __syncthreads();
        }
        const long long n = b0 + tid < p.bt.batch ? (long long)s_sum[tid] * p.c.kv_heads : 0;
        const long long at = base + block_scan<kThreads>(n, total, s_warp);
        if (u0 >= at && u0 < at + n) {
            s_walk->b = b0 + tid;
            s_walk->left = u0 - at;  // for now: the start within the sequence
        }
        base += total;
        if (base > u0) break;
    }
    __syncthreads();
    if (warp == 0) {
        const int b = s_walk->b;
        const Seq s = seq_info(p.bt, b, nullptr);
        const int n_qt = row_tiles(s, p.group), per = seq_tiles(p, s, n_qt);
        long long at = s_walk->left;
        const int hk = (int)(at / per);
        int rem = (int)(at % per), found = -1, first = 0, before = 0;
        for (int q0 = 0; q0 < n_qt && found < 0; q0 += 32) {
            const int n = q0 + lane < n_qt ? item_of(p, s, q0 + lane).tiles : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            const unsigned hit = __ballot_sync(~0u, n > 0 && rem >= before + x - n && rem < before + x);
            if (hit) {
                const int l = __ffs(hit) - 1;
                found = q0 + l;
                first = rem - (before + __shfl_sync(~0u, x - n, l));
            }
            before += __shfl_sync(~0u, x, 31);
        }
        __syncwarp();
        if (lane == 0) {
            s_walk->hk = hk, s_walk->qt = found, s_walk->n_qt = n_qt, s_walk->first = first, s_walk->sq = s;
            s_walk->left = u1 - u0;
        }
    }
    __syncthreads();
    w = *s_walk;
    return true;
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const AttendParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D>;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ Bars bar;
    __shared__ uint32_t s_tmem;
    __shared__ long long s_warp[kWarps];
    __shared__ int s_sum[kThreads];
    __shared__ Walk s_walk;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (su32(sm_raw) + 1023u) & ~1023u, qs = ring + S::kStages * S::kStage;

    Walk walk;
    const bool any = plan(p, walk, s_warp, s_sum, &s_walk);
    asm volatile("griddepcontrol.launch_dependents;" :::);
    if (!any) return;

    if (tid == 0) {
        for (int i = 0; i < S::kStages; i++) bar_init(&bar.full[i], 1), bar_init(&bar.empty[i], 1);
        bar_init(&bar.qfull, 64), bar_init(&bar.qempty, 1), bar_init(&bar.clean, 64), bar_init(&bar.done, 1);
        for (int t = 0; t < 2; t++) bar_init(&bar.s[t], 1), bar_init(&bar.p[t], 4), bar_init(&bar.o[t], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = *reinterpret_cast<volatile uint32_t *>(&s_tmem);
    bool ok = true;
    Part w;

    // registers: 384 threads x 168 at launch = 256 x 208 + 128 x 88
    if (warp < 8) {  // ---------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tm + lanes + 128 * t, tO = tm + lanes + S::kO + D * t, tP = tm + lanes + S::kP + S::kPStep * t;
        const float c2 = p.scale * kLog2e;
        uint32_t ns = 0, no = 0;
        while (ok && walk.next(p, w)) {
            const int64_t rows = (int64_t)w.sq.q_len * p.group;
            const int64_t r = (int64_t)w.qt * kTileRows + tid;  // tid: 128 t + row of the tile
            if (rows - (int64_t)w.qt * kTileRows <= 128 * t) continue;  // the second tile has no rows
            const bool live = r < rows;
            const int i = live ? (int)(r / p.group) : 0, h = w.hk * p.group + (live ? (int)(r % p.group) : 0);
            const Range v = visible(w.sq, i, i + 1, p.window, p.causal);
            const int beg = live ? v.lo : 0, end = live ? v.hi : 0;
            float m = -INFINITY, l = 0.f;
            for (int j = w.first; j < w.last && ok; j++, ns++) {
                const int s0 = w.it.lo + j * kTileSlots;
                if (!warp_wait(&bar.s[t], ns & 1)) {
                    ok = false;
                    break;
                }
                fence_after();
                uint32_t x[128];
                tm_ld64(tS, x);
                tm_ld64(tS + 64, x + 64);
                if (__any_sync(~0u, beg > s0 || end < s0 + kTileSlots)) {
                    const int a = beg - s0, e = end - s0;
#pragma unroll
                    for (int k = 0; k < 128; k++)
                        if (k < a || k >= e) x[k] = 0xff800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 128; k++) mx[k & 3] = fmaxf(mx[k & 3], __uint_as_float(x[k]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
                if (__any_sync(~0u, top > m + kSlack)) {
                    const float n = fmaxf(m, top), a = m == -INFINITY ? 0.f : ex2(m - n);
                    m = n;
                    l *= a;
                    if (j > w.first) {  // O's last product ended before this step's S did
#pragma unroll
                        for (int k = 0; k < D; k += 32) {
                            uint32_t y[32];
                            tm_ld32(tO + k, y);
#pragma unroll
                            for (int e = 0; e < 32; e++) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
                            tm_st32(tO + k, y);
                        }
                    }
                }
                const float z = m == -INFINITY ? 0.f : -m;
                const uint64_t cc = pack2(c2, c2), zz = pack2(z, z);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    uint32_t y[32];
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        const int e = 64 * q + 2 * k;
                        const float2 f = unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), cc, zz));
                        const float a = ex2(f.x), b = ex2(f.y);
                        sum[k & 1] = add2(sum[k & 1], pack2(a, b));
                        y[k] = from_f2<BF>(a, b);
                    }
                    tm_st32(tP + 32 * q, y);
                }
                const float2 f = unpack2(add2(sum[0], sum[1]));
                l += f.x + f.y;
                tm_st_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bar.p[t]);
            }
            if (!ok) break;
            if (!warp_wait(&bar.o[t], no & 1)) {
                ok = false;
                break;
            }
            no++;
            fence_after();
            const bool whole = w.first == 0 && w.last == w.it.tiles;
            const int64_t token = w.sq.q0 + i;
            const int part = 2 * blockIdx.x + (w.first == 0 ? 1 : 0);
            float f = 1.f, lse2 = 0.f;
            if (whole && live) f = finish_row(m, l, p.sinks, h, lse2);
            uint16_t *out = p.out.d + token * p.out.token + h * p.out.head;
            float *po = p.part_o + ((int64_t)part * kTileRows + tid) * D;
#pragma unroll
            for (int k = 0; k < D; k += 32) {
                uint32_t y[32];
                tm_ld32(tO + k, y);
                if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float z[8];
#pragma unroll
                        for (int q = 0; q < 8; q++) z[q] = __uint_as_float(y[e + q]) * f;
                        if (whole) {
                            *reinterpret_cast<uint4 *>(out + k + e) = make_uint4(from_f2<BF>(z[0], z[1]), from_f2<BF>(z[2], z[3]),
                                                                                 from_f2<BF>(z[4], z[5]), from_f2<BF>(z[6], z[7]));
                        } else {
                            *reinterpret_cast<float4 *>(po + k + e) = make_float4(z[0], z[1], z[2], z[3]);
                            *reinterpret_cast<float4 *>(po + k + e + 4) = make_float4(z[4], z[5], z[6], z[7]);
                        }
                    }
                }
                __syncwarp();
            }
            if (live) {
                if (whole)
                    put_lse(p, token, h, lse2);
                else
                    p.part_ml[part * kTileRows + tid] = make_float2(m, l);
            }
            fence_before();  // O is read before the next item's first P is announced
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }
    if (warp == kCopyWarp) {  // -------------------------------------------- K and V
        const int box = 1 << (p.c.page_shift < 7 ? p.c.page_shift : 7), boxes = kTileSlots / box, halves = D / 64;
        const int mine = lane % boxes, half = lane / boxes;  // one box a lane (8 pages x 2 halves at most)
        uint32_t cnt = 0;
        while (ok && walk.next(p, w)) {
            const int32_t *tab = p.bt.table + (int64_t)w.b * p.bt.table_stride;
            for (int j = w.first; j < w.last && ok; j++) {
                const int slot = w.it.lo + j * kTileSlots + mine * box;
                int page = -1;
                if (half < halves && slot < w.it.hi && slot + box > w.it.seen_lo) {
                    page = tab[slot >> p.c.page_shift];
                    if ((uint32_t)page >= (uint32_t)p.c.num_pages) {
                        flag(p.c.status, FTMOE_ERR_ID_RANGE);
                        page = -1;
                    }
                }
                const uint32_t bytes = __popc(__ballot_sync(~0u, page >= 0)) * box * 128;
                const int row = slot & ((1 << p.c.page_shift) - 1);
#pragma unroll
                for (int kv = 0; kv < 2; kv++, cnt++) {
                    const int st = cnt % S::kStages;
                    if (!warp_wait(&bar.empty[st], ((cnt / S::kStages) & 1) ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) bar_expect(&bar.full[st], bytes);
                    __syncwarp();
                    if (page >= 0)
                        tma4(ring + st * S::kStage + half * S::kHalf + mine * box * 128, kv ? &vmap : &kmap, 64 * half, row, w.hk, page,
                             &bar.full[st]);
                }
            }
        }
        if (!ok)  // wait (bounded) until the copies already issued have landed
            for (uint32_t c = cnt < S::kStages ? 0 : cnt - S::kStages; c < cnt; c++) wait_bar(&bar.full[c % S::kStages], (c / S::kStages) & 1);
    } else if (warp == kMmaWarp) {  // -------------------------------------- products
        if (lane == 0) {
            constexpr uint32_t IS = kInstr<BF, kTileSlots, false>, IO = kInstr<BF, D, true>;
            uint32_t cnt = 0, np[2] = {0, 0}, ni = 0, nc = 0;
            auto scores = [&](int t, uint32_t st) {
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t off = (k >> 2) * S::kHalf + (k & 3) * 32;
                    mma_ss<IS>(tm + 128 * t, desc128(qs + t * (128 * D * 2) + off, 16), desc128(ring + st * S::kStage + off, 16), k > 0);
                }
                commit(&bar.s[t]);
            };
            while (ok && walk.next(p, w)) {
                const int n = w.last - w.first;
                const int tiles = (int64_t)w.sq.q_len * p.group - (int64_t)w.qt * kTileRows > 128 ? 2 : 1;
                if (!wait_bar(&bar.qfull, ni & 1)) ok = false;
                ni++;
                if (ok && !wait_bar(&bar.full[cnt % S::kStages], (cnt / S::kStages) & 1)) ok = false;
                if (!ok) break;
                fence_after();
                for (int t = 0; t < tiles; t++) scores(t, cnt % S::kStages);
                commit(&bar.empty[cnt % S::kStages]);
                if (n == 1) commit(&bar.qempty);
                cnt++;
                for (int j = 0; j < n && ok; j++) {
                    const uint32_t sv = cnt % S::kStages, pv = (cnt / S::kStages) & 1;
                    const uint32_t sk = (cnt + 1) % S::kStages, pk = ((cnt + 1) / S::kStages) & 1;
                    const int s0 = w.it.lo + (w.first + j) * kTileSlots;
                    ok = wait_bar(&bar.full[sv], pv);
                    if (ok && (s0 < w.it.seen_lo || s0 + kTileSlots > w.it.hi)) ok = wait_bar(&bar.clean, nc++ & 1);
                    for (int t = 0; t < tiles && ok; t++) {
                        ok = wait_bar(&bar.p[t], np[t]++ & 1);
                        if (!ok) break;
                        fence_after();
#pragma unroll
                        for (int k = 0; k < kTileSlots / 16; k++)
                            mma_ts<IO>(tm + S::kO + D * t, tm + S::kP + S::kPStep * t + 8 * k,
                                       desc128(ring + sv * S::kStage + k * 2048, S::kHalf), j > 0 || k > 0);
                        if (j + 1 < n) {
                            if (t == 0) ok = wait_bar(&bar.full[sk], pk);
                            if (!ok) break;
                            fence_after();
                            scores(t, sk);
                        } else {
                            commit(&bar.o[t]);
                        }
                    }
                    if (!ok) break;
                    commit(&bar.empty[sv]);
                    cnt++;
                    if (j + 1 < n) {
                        commit(&bar.empty[sk]);
                        cnt++;
                        if (j + 2 == n) commit(&bar.qempty);
                    }
                }
            }
            commit(&bar.done);  // every product is done when this arrives
            wait_bar(&bar.done, 0);
        }
        __syncwarp();
    } else if (warp >= kHelpWarp) {  // ------------------------------------- queries, ends of V
        const int half = warp - kHelpWarp;
        constexpr int CH = D / 8, RPI = 32 / CH;
        uint32_t cnt = 0, nq = 0;
        while (ok && walk.next(p, w)) {
            if (nq > 0 && !warp_wait(&bar.qempty, (nq - 1) & 1)) {
                ok = false;
                break;
            }
            nq++;
            const int64_t rows = (int64_t)w.sq.q_len * p.group, r0 = (int64_t)w.qt * kTileRows;
            const int ch = lane % CH;
            for (int n = 0; n < 128; n += RPI) {  // half h copies tile h
                const int row = n + lane / CH;
                const int64_t r = r0 + 128 * half + row;
                const bool live = r < rows;
                const int64_t i = live ? r / p.group : 0;
                const int h = w.hk * p.group + (live ? (int)(r % p.group) : 0);
                const uint16_t *src = p.q.d + (w.sq.q0 + i) * p.q.token + h * p.q.head + 8 * ch;
                const uint32_t dst = qs + half * (128 * D * 2) + (ch >> 3) * S::kHalf + row * 128 + (((ch ^ row) & 7) << 4);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
            }
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
            fence_async();
            bar_arrive(&bar.qfull);
            for (int j = w.first; j < w.last && ok; j++, cnt += 2) {
                const int s0 = w.it.lo + j * kTileSlots;
                if (s0 >= w.it.seen_lo && s0 + kTileSlots <= w.it.hi) continue;
                const uint32_t st = (cnt + 1) % S::kStages;
                if (!warp_wait(&bar.full[st], ((cnt + 1) / S::kStages) & 1)) {
                    ok = false;
                    break;
                }
                for (int c = half * 32 + lane; c < kTileSlots * CH; c += 64) {
                    const int row = c / CH, k = c % CH;
                    if (s0 + row < w.it.seen_lo || s0 + row >= w.it.hi)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring + st * S::kStage + (k >> 3) * S::kHalf + row * 128 + ((k & 7) << 4)),
                                     "r"(0)
                                     : "memory");
                }
                fence_async();
                bar_arrive(&bar.clean);
            }
        }
    }
    if (!ok && lane == 0) flag(p.c.status, FTMOE_ERR_STATE);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
}

// Joins the parts of an item that several CTAs covered, in order. One CTA takes 32 rows of an item, a
// warp four of them.
constexpr int kJoinThreads = 256, kJoinRows = 32;

template <bool BF, int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_combine(const AttendParams p, int grid) {
    __shared__ long long s_warp[kJoinThreads / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int qt = blockIdx.x / (kTileRows / kJoinRows), sub = blockIdx.x % (kTileRows / kJoinRows);
    const int hk = blockIdx.y, b = blockIdx.z;
    const Seq sq = seq_info(p.bt, b, nullptr);
    const int n_qt = row_tiles(sq, p.group);
    long long all = 0, less = 0, total, before;
    for (int i = warp; i < p.bt.batch; i += kJoinThreads / 32) {
        const Seq s = seq_info(p.bt, i, nullptr);
        const int n = seq_tiles(p, s, row_tiles(s, p.group));
        all += n;
        if (i < b) less += n;
    }
    block_scan<kJoinThreads>(lane == 0 ? all : 0, total, s_warp);
    block_scan<kJoinThreads>(lane == 0 ? less : 0, before, s_warp);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // on every path: this grid ends after the one before it
    if (qt >= n_qt) return;
    const int per = seq_tiles(p, sq, n_qt), ahead = seq_tiles(p, sq, qt), n = item_of(p, sq, qt).tiles;
    const long long W = total * p.c.kv_heads, u = before * p.c.kv_heads + (long long)hk * per + ahead;
    const int C = used_ctas(grid, W), c0 = unit_owner(u, C, W), c1 = unit_owner(u + n - 1, C, W);
    if (c0 == c1) return;
    constexpr int E = D / 32;
    for (int k = 0; k < kJoinRows / 8; k++) {
        const int row = sub * kJoinRows + 8 * k + warp;
        const int64_t r = (int64_t)qt * kTileRows + row;
        if (r >= (int64_t)sq.q_len * p.group) break;
        float M = -INFINITY, L = 0.f, x[E];
#pragma unroll
        for (int e = 0; e < E; e++) x[e] = 0.f;
        for (int c = c0; c <= c1; c++) M = fmaxf(M, p.part_ml[(2 * c + (c == c0)) * kTileRows + row].x);
        for (int c = c0; c <= c1; c++) {
            const int64_t at = (int64_t)(2 * c + (c == c0)) * kTileRows + row;
            const float2 ml = p.part_ml[at];
            const float a = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            L += ml.y * a;
            const float *po = p.part_o + at * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(po + e);
                x[e] += v.x * a, x[e + 1] += v.y * a;
            }
        }
        const int64_t token = sq.q0 + r / p.group;
        const int h = hk * p.group + (int)(r % p.group);
        float lse2;
        const float f = finish_row(M, L, p.sinks, h, lse2);
        uint32_t *out = reinterpret_cast<uint32_t *>(p.out.d + token * p.out.token + h * p.out.head + lane * E);
#pragma unroll
        for (int e = 0; e < E; e += 2) out[e / 2] = from_f2<BF>(x[e] * f, x[e + 1] * f);
        if (lane == 0) put_lse(p, token, h, lse2);
    }
}

template <bool BF, int D>
cudaError_t launch(const AttendParams &p, int C, cudaStream_t st) {
    using S = Shape<D>;
    CUtensorMap km, vm;
    const int box = p.c.page_shift < 7 ? 1 << p.c.page_shift : 128;
    if (!page_map(km, p.c, true, BF, box) || !page_map(vm, p.c, false, BF, box)) return cudaErrorInvalidValue;
    auto kern = chunk_kernel<BF, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    kern<<<C, kThreads, S::kSmem, st>>>(p, km, vm);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int n_qt = (int)(((int64_t)p.bt.max_q * p.group + kTileRows - 1) / kTileRows);
    return launch_after(chunk_combine<BF, D>, dim3(n_qt * (kTileRows / kJoinRows), p.c.kv_heads, p.bt.batch), kJoinThreads, 0, st, p, C);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(f);
        cudaGetLastError();
        return static_cast<EncodeFn>(nullptr);
    }();
    return fn;
}

}  // namespace

bool page_map(CUtensorMap &m, const View &c, bool keys, bool bf16, int box_slots) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const int64_t sp = keys ? c.k_page : c.v_page, ss = keys ? c.k_slot : c.v_slot, sh = keys ? c.k_head : c.v_head;
    const cuuint64_t dims[4] = {(cuuint64_t)c.dim, (cuuint64_t)1 << c.page_shift, (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)ss * 2, (cuuint64_t)sh * 2, (cuuint64_t)sp * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_slots, 1, 1}, es[4] = {1, 1, 1, 1};
    return fn(&m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, keys ? c.k : c.v, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int chunk_ctas(const AttendParams &p, int num_sms) {
    const int64_t n_qt = ((int64_t)p.bt.max_q * p.group + kTileRows - 1) / kTileRows;
    const int64_t most = n_qt * p.bt.batch * p.c.kv_heads * (p.bt.max_kv / kTileSlots + 2);
    return (int)(most < num_sms ? (most > 0 ? most : 1) : num_sms);
}

size_t chunk_part_rows(const AttendParams &p, int num_sms) { return 2 * (size_t)chunk_ctas(p, num_sms) * kTileRows; }

cudaError_t launch_chunk(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    const int C = chunk_ctas(p, num_sms);
    if (p.c.dim == 64) return bf16 ? launch<true, 64>(p, C, st) : launch<false, 64>(p, C, st);
    return bf16 ? launch<true, 128>(p, C, st) : launch<false, 128>(p, C, st);
}

}  // namespace kv
}  // namespace ftmoe

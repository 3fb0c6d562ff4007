// Attention of chunks of new tokens on the 5th-generation tensor cores. An item is 256 consecutive
// (token, query head) rows of one (sequence, key head), as two tiles of M = 128: the query heads that
// share a key head read K and V from shared memory once. Bound by the tensor cores: 4 dim flops a
// (row, slot) against one exponential.
//
// Persistent, one CTA an SM, work cut by kv_split.cuh in steps of 128 slots. Roles:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: a thread holds one row. S comes from tensor
//                   memory; P = 2^(s scale log2 e - m) in fp32 with the maximum m of the steps
//                   before, so that the row's own maximum is off the path from S to P; P goes back
//                   as 16-bit pairs, the first 64 slots as soon as they are formed. The maximum is
//                   taken after that; one more than 2^8 above m raises m for the next step, which
//                   first rescales O (in tensor memory). A half whose sum is too large for P's type (and
//                   a row's first step) raises m at once. P, the sum and O always share one m. P is rounded to
//                   the cache's type because the tensor cores take it beside V in that type; the sum is
//                   of P in fp32.
//   warps 8, 10     tensor copies: K and V tiles (a box a page and 64 elements, 128-byte swizzle)
//                   into a ring of stages, pages outside the visible range untouched; warp 8 also
//                   the queries of the next item once the last S product has read the present ones.
//   warp 9          issues tcgen05.mma, tile 0's and tile 1's in turn: O_t += P_t V (P from tensor
//                   memory, V with its elements consecutive), S_t = Q_t K^T of the next step
//                   (both from shared memory). While the softmax of one tile runs, the products of
//                   the other do. (A warp for each tile fell into step and left no overlap.)
//   warp 11         walks the work and hands the parts out through a small ring (done by each
//                   role, a walk step cost 3000 to 5000 cycles of cold code between items); and zeroes
//                   the V rows of slots that no row sees in the tiles at the ends of the visible
//                   range (what such slots hold must not reach 0 * V).
// Tensor memory: S_0, S_1 (128 columns each), O_0, O_1 (dim each). P_t lies over S_t for 128
// elements a head: S_t of the next step is issued after the product that reads P_t, and products
// of one shape run in order. For 64 the shapes differ, and P_0, P_1 have columns of their own.
// Every wait is bounded; one that runs out is recorded and ends the role.
//
// 2048 tokens over 31000, 32 query heads of 128 on 8: 654 us, 1.54 PFLOP/s (0.82 of a large bf16 product). What is left is
// mostly the S products, which read both operands from shared memory and take 98 cycles instead of 64. A whole
// prompt of 4096 tokens, 32 heads on 4: 119 us, 1.16 PFLOP/s, where an item has 17 steps on average and its start and end cost
// two more. Seven sequences of up to 97 new tokens over 1500: 24 us, the cold starts of two kernels.
#include "kv_tc05.cuh"

namespace ftmoe {
namespace kv {
namespace {

constexpr int kWarps = 12, kThreads = kWarps * 32;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kCopyWarp2 = 10, kHelpWarp = 11;
constexpr int kParts = 4;  // entries of the ring of parts
constexpr float kSlack = 8.f;
// The largest sum of 64 P that is let through: P below it is finite in its type, sums in fp32.
template <bool BF>
constexpr float kMost = BF ? 18446744073709551616.f : 16384.f;
constexpr int kMaxStages = 8;

template <int D>
struct Shape {
    static constexpr int kStage = kTileSlots * D * 2;         // K or V of one step
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kHalf = kTileSlots * 128;            // 64 elements of 128 rows
    static constexpr int kQ = kTileRows * D * 2;
    static constexpr int kOut = 8 * 32 * 64;                  // a warp's 32 output rows, 32 elements at a time
    static constexpr int kSmem = 1024 + kStages * kStage + kQ + kOut;
    static constexpr uint32_t kO = 256, kP = D == 128 ? 0 : 384;  // columns of O_0 and P_0
    static constexpr uint32_t kPStep = D == 128 ? 128 : 64;       // from P_0 to P_1
};

// A part of an item that this CTA works on, as the roles take it from the ring.
struct Part {
    int b, hk;
    int token, left;        // first token row of the item; new tokens from there to the sequence's end
    int slot, kv_len;       // the first token's slot
    int lo, hi, seen_lo;    // Item
    int first, last, tiles; // steps [first, last) of the item's tiles; tiles = 0: no more parts
};

struct Bars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t clean[kMaxStages];  // the stage's unseen V rows are zero (every use of a stage, K or V)
    uint64_t qfull, qempty, s[2], p[2][2], half[2], o[2], done;
    uint64_t part_full[kParts], part_empty[kParts];
};

// The walk along the line of work.
struct Walk {
    long long left;
    int b, hk, qt, n_qt, at;  // at: units into the item (its kItemCost first)
    Seq sq;
    __device__ __forceinline__ bool next(const AttendParams &p, Part &w) {
        while (left > 0) {
            const Item it = item_of(p, sq, qt);
            const int n = it.tiles + kItemCost, end = left < n - at && p.join ? at + (int)left : n;
            w.b = b, w.hk = hk;
            w.token = sq.q0 + qt * p.item_tokens, w.left = sq.q_len - qt * p.item_tokens;
            w.slot = sq.kv_len - sq.q_len + qt * p.item_tokens, w.kv_len = sq.kv_len;
            w.lo = it.lo, w.hi = it.hi, w.seen_lo = it.seen_lo, w.tiles = it.tiles;
            w.first = at > kItemCost ? at - kItemCost : 0, w.last = end - kItemCost;
            left = p.join ? left - (end - at) : 0;  // (no join array: a CTA has one item, whole)
            at = 0;
            if (left > 0 && ++qt == n_qt) {
                qt = 0;
                if (++hk == p.c.kv_heads) {
                    hk = 0;
                    do {
                        sq = seq_info(p.bt, ++b, nullptr);
                        n_qt = row_tiles(p, sq);
                    } while (n_qt == 0);
                }
            }
            if (w.last > w.first) return true;
        }
        w.tiles = 0;
        return false;
    }
};

// Takes the next part; the whole warp calls. False at the end (or when the wait ran out: ok).
__device__ __forceinline__ bool take(Bars &bar, const Part *ring, uint32_t &n, Part &w, bool &ok) {
    const uint32_t e = n % kParts;
    ok = warp_wait(&bar.part_full[e], (n / kParts) & 1);
    if (!ok) return false;
    w = ring[e];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(&bar.part_empty[e]);
    n++;
    return w.tiles > 0;
}

// Total steps and this CTA's start. s_sum: kThreads entries.
__device__ __forceinline__ bool plan(const AttendParams &p, Walk &w, long long *s_warp, long long *s_sum, Walk *s_walk) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!p.join) {  // a CTA an item that there can be, and no line to walk
        const int most = (p.bt.max_q + p.item_tokens - 1) / p.item_tokens, head = blockIdx.x / most;
        w.qt = blockIdx.x - head * most, w.b = head / p.c.kv_heads, w.hk = head - w.b * p.c.kv_heads;
        w.sq = seq_info(p.bt, w.b, w.qt == 0 && w.hk == 0 && tid == 0 ? p.c.status : nullptr);
        w.n_qt = row_tiles(p, w.sq), w.at = 0, w.left = 1;
        return w.qt < w.n_qt;
    }
    long long sum = 0, total;
    for (int b0 = 0; b0 < p.bt.batch; b0 += kThreads) {
        for (int i = warp; i < kThreads; i += kWarps) {
            long long n = 0;
            if (b0 + i < p.bt.batch) {
                const Seq s = seq_info(p.bt, b0 + i, blockIdx.x == 0 && lane == 0 ? p.c.status : nullptr);
                n = seq_units(p, s, row_tiles(p, s));
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
                const long long n = seq_units(p, s, row_tiles(p, s));
                if (lane == 0) s_sum[i] = n;
            }
            __syncthreads();
        }
        const long long n = b0 + tid < p.bt.batch ? s_sum[tid] * p.c.kv_heads : 0;
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
        const int n_qt = row_tiles(p, s);
        const long long per = seq_units(p, s, n_qt);
        const Place at = place_of(p, s, n_qt, per, s_walk->left);
        __syncwarp();
        if (lane == 0) {
            s_walk->hk = at.hk, s_walk->qt = at.qt, s_walk->n_qt = n_qt, s_walk->at = at.at, s_walk->sq = s;
            s_walk->left = u1 - u0;
        }
    }
    __syncthreads();
    w = *s_walk;
    return true;
}

// O *= a, a row's D columns of tensor memory. The whole warp calls.
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t tO, float a) {
#pragma unroll 1
    for (int k = 0; k < D; k += 32) {
        uint32_t y[32];
        tm_ld32(tO + k, y);
#pragma unroll
        for (int e = 0; e < 32; e++) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
        tm_st32(tO + k, y);
    }
    tm_st_wait();
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const AttendParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
    using S = Shape<D>;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ Bars bar;
    __shared__ uint32_t s_tmem;
    __shared__ long long s_warp[kWarps];
    __shared__ long long s_sum[kThreads];  // (not over the ring: tensor copies are not ordered after plain stores to the same bytes)
    __shared__ Walk s_walk;
    __shared__ Part s_part[kParts];
    __shared__ int64_t s_row[128];  // offset of a tile's row from its first token and head, -1 past the last
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ring = (su32(sm_raw) + 1023u) & ~1023u, qs = ring + S::kStages * S::kStage, stage_out = qs + S::kQ;

    if (tid == 0) {
        for (int i = 0; i < S::kStages; i++) bar_init(&bar.full[i], 1), bar_init(&bar.empty[i], 2), bar_init(&bar.clean[i], 1);
        for (int i = 0; i < kParts; i++) bar_init(&bar.part_full[i], 1), bar_init(&bar.part_empty[i], 11);  // softmax, copies, products
        bar_init(&bar.qfull, 1), bar_init(&bar.qempty, 1), bar_init(&bar.done, 1);
        for (int t = 0; t < 2; t++) {
            bar_init(&bar.s[t], 1), bar_init(&bar.p[t][0], 4), bar_init(&bar.p[t][1], 4);
            bar_init(&bar.o[t], 1), bar_init(&bar.half[t], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid < 128) {
        const int i = tid / (uint32_t)p.group, g = tid - i * p.group;
        s_row[tid] = i < p.item_tokens >> 1 ? i * p.out.token + g * p.out.head : -1;
    }
    Walk walk;
    const bool any = plan(p, walk, s_warp, s_sum, &s_walk);
    asm volatile("griddepcontrol.launch_dependents;" :::);
    fence_before();
    __syncthreads();
    fence_after();
    if (!any) {  // the whole CTA
        if (tid == 0 && p.join) p.join[blockIdx.x] = make_int4(0, 0, 0, kJoinNone);
        if (warp == kMmaWarp)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*reinterpret_cast<volatile uint32_t *>(&s_tmem)) : "memory");
        return;
    }
    const uint32_t tm = *reinterpret_cast<volatile uint32_t *>(&s_tmem);
    bool ok = true;
    Part w;
    uint32_t n_part = 0;

    // registers: 384 threads x 168 at launch = 256 x 208 + 128 x 88
    if (warp < 8) {  // ---------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tm + lanes + 128 * t, tO = tm + lanes + S::kO + D * t, tP = tm + lanes + S::kP + S::kPStep * t;
        const float c2 = p.scale * kLog2e;
        // this thread's row of the tile: token and query head
        const int row_l = (tid & 127) / (uint32_t)p.group, row_g = (tid & 127) - row_l * p.group;
        const int row_i = t * (p.item_tokens >> 1) + row_l;
        const bool row_used = row_l < (p.item_tokens >> 1);
        uint32_t ns = 0, no = 0;
        while (take(bar, s_part, n_part, w, ok)) {
            if (w.left <= t * (p.item_tokens >> 1)) continue;  // the second tile has no rows
            const bool live = row_used && row_i < w.left;
            const int h = w.hk * p.group + row_g, at = w.slot + row_i;
            const int end = !live || at < 0 ? 0 : (p.causal ? at + 1 : w.kv_len);
            const int beg = live && p.window && at >= p.window ? at - p.window + 1 : 0;
            float m = live ? -INFINITY : 0.f, l = 0.f, up = 1.f;  // rows that are none stay at P = 0
            bool raise = false;  // O is to be multiplied by up
            for (int j = w.first; j < w.last && ok; j++, ns++) {
                const int s0 = w.lo + j * kTileSlots;
                if (!warp_wait(&bar.s[t], ns & 1)) {
                    ok = false;
                    break;
                }
                fence_after();
                uint32_t x[128];
                tm_ld64(tS, x);
                tm_ld_wait(x);
                tm_ld64(tS + 64, x + 64);  // in flight while the first half of P is formed
                if (raise) {               // O's last product ended before this step's S did
                    rescale_o<D>(tO, up);
                    raise = false;
                }
                const bool cut = __any_sync(~0u, beg > s0 || end < s0 + kTileSlots);
                // slots that the row does not see, in the groups of 32 that some row of the warp does not see whole
                auto hide = [&](int q) {
#pragma unroll
                    for (int g = 64 * q; g < 64 * q + 64; g += 32) {
                        const int a = beg - s0 - g, e = end - s0 - g;
                        if (__any_sync(~0u, a > 0 || e < 32)) {
#pragma unroll
                            for (int k = 0; k < 32; k++)
                                if (k < a || k >= e) x[g + k] = 0xff800000u;
                        }
                    }
                };
                const uint64_t cc = pack2(c2, c2);
                // P of 64 slots, and their sum
                auto form = [&](int q) {
                    const float z = m == -INFINITY ? 0.f : -m;
                    const uint64_t zz = pack2(z, z);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int c = 2 * q; c < 2 * q + 2; c++) {
                        uint32_t y[16];
#pragma unroll
                        for (int k = 0; k < 16; k++) {
                            const int e = 32 * c + 2 * k;
                            const float2 f = unpack2(fma2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), cc, zz));
                            const float a = ex2(f.x), b = ex2(f.y);
                            sum[k & 1] = add2(sum[k & 1], pack2(a, b));
                            y[k] = from_f2<BF>(a, b);
                        }
                        tm_st16(tP + 16 * c, y);
                    }
                    const float2 f = unpack2(add2(sum[0], sum[1]));
                    return f.x + f.y;
                };
                auto announce = [&](int q) {
                    tm_st_wait();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(&bar.p[t][q]);
                };
                auto top_of = [&] {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 128; k += 2)
                        mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
                };
                // m to at least the row's maximum; returns the factor of what was summed before
                auto raised = [&](float top) {
                    const float n = fmaxf(m, top), a = m == -INFINITY ? 0.f : ex2(m - n);
                    m = n;
                    l *= a;
                    return a;
                };
                if (cut) hide(0);
                const bool fresh = __any_sync(~0u, m == -INFINITY);
                float part;
                if (!fresh) part = form(0);
                tm_ld_wait(x + 64);
                if (cut) hide(1);
                if (fresh || __any_sync(~0u, part > kMost<BF>)) {
                    const float a = raised(top_of());
                    if (j > w.first) rescale_o<D>(tO, a);
                    part = form(0);
                }
                announce(0);
                l += part;
                part = form(1);
                if (__any_sync(~0u, part > kMost<BF>)) {  // the first half's product has m as it was
                    if (!warp_wait(&bar.half[t], ns & 1)) ok = false;
                    fence_after();
                    rescale_o<D>(tO, raised(top_of()));
                    part = form(1);
                }
                announce(1);
                l += part;
                const float top = top_of();
                if (__any_sync(~0u, top > m + kSlack)) {
                    up = raised(top);
                    raise = true;
                }
            }
            if (!ok) break;
            if (!warp_wait(&bar.o[t], no & 1)) {
                ok = false;
                break;
            }
            no++;
            fence_after();
            const bool whole = w.first == 0 && w.last == w.tiles;
            const int64_t token = w.token + row_i;
            const int part = 2 * blockIdx.x + (w.first == 0 ? 1 : 0);
            float f = raise ? up : 1.f, lse2 = 0.f;
            if (whole) f *= finish_row(m, l, p.sinks, h, lse2);
            // 32 elements of the warp's rows at a time, in a loop: run once an item, unrolled code took most of its
            // time to be fetched
            const uint32_t st = stage_out + warp * 2048;
            uint16_t *out = p.out.d + (int64_t)(w.token + t * (p.item_tokens >> 1)) * p.out.token + w.hk * p.group * p.out.head;
            const int here = w.left < p.item_tokens ? w.left : p.item_tokens;
            const int rows = (here - t * (p.item_tokens >> 1)) * p.group - 32 * (warp & 3);  // of this warp's 32
            float *po = p.part_o + (int64_t)part * kTileRows * D + tid;
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
                uint32_t y[32];
                tm_ld32(tO + k, y);
                if (whole) {
                    // through shared memory, 16-byte chunk c of row r at c ^ (r / 2 % 4), so that four lanes write a
                    // row's 64 bytes together
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        uint32_t z[4];
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            z[e] = from_f2<BF>(__uint_as_float(y[8 * c + 2 * e]) * f, __uint_as_float(y[8 * c + 2 * e + 1]) * f);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(st + lane * 64 + ((c ^ (lane >> 1 & 3)) << 4)), "r"(z[0]),
                                     "r"(z[1]), "r"(z[2]), "r"(z[3])
                                     : "memory");
                    }
                    __syncwarp();
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const int r = 8 * c + (lane >> 2);
                        const int64_t off = s_row[32 * (warp & 3) + r];
                        uint4 z;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(z.x), "=r"(z.y), "=r"(z.z), "=r"(z.w)
                                     : "r"(st + r * 64 + (((lane ^ (r >> 1)) & 3) << 4))
                                     : "memory");
                        if (off >= 0 && r < rows) *reinterpret_cast<uint4 *>(out + off + k + 8 * (lane & 3)) = z;
                    }
                    __syncwarp();
                } else {  // parts are kept element by element, rows consecutive: a warp's store is one line
#pragma unroll
                    for (int e = 0; e < 32; e++) po[(k + e) * kTileRows] = __uint_as_float(y[e]) * f;
                }
            }
            if (!whole)
                p.part_ml[part * kTileRows + tid] = make_float2(m, l);
            else if (live)
                put_lse(p, token, h, lse2);
            fence_before();  // O is read before the next item's first P is announced
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }
    if (warp == kCopyWarp || warp == kCopyWarp2) {  // ------------------------- K and the queries; V
        const int kv = warp == kCopyWarp2;
        const int box = 1 << (p.c.page_shift < 7 ? p.c.page_shift : 7), boxes = kTileSlots / box, halves = D / 64;
        const int mine = lane % boxes, half = lane / boxes;  // one box a lane (8 pages x 2 halves at most)
        uint32_t cnt = kv, nq = 0;                           // stages alternate: K, V
        while (ok && take(bar, s_part, n_part, w, ok)) {
            const int32_t *tab = p.bt.table + (int64_t)w.b * p.bt.table_stride;
            auto wanted = [&](int j) {  // whether this lane has a box of step j to read
                const int slot = w.lo + j * kTileSlots + mine * box;
                return half < halves && j < w.last && slot < w.hi && slot + box > w.seen_lo;
            };
            auto page_at = [&](int j) { return wanted(j) ? tab[(w.lo + j * kTileSlots + mine * box) >> p.c.page_shift] : -1; };
            int next = page_at(w.first);
            for (int j = w.first; j < w.last && ok; j++, cnt += 2) {
                int page = next;
                next = page_at(j + 1);  // on its way while this step waits for its stage
                if ((uint32_t)page >= (uint32_t)p.c.num_pages) {
                    if (wanted(j)) flag(p.c.status, FTMOE_ERR_ID_RANGE);
                    page = -1;
                }
                const uint32_t bytes = __popc(__ballot_sync(~0u, page >= 0)) * box * 128;
                const int slot = w.lo + j * kTileSlots + mine * box, row = slot & ((1 << p.c.page_shift) - 1);
                const int st = cnt % S::kStages;
                if (!warp_wait(&bar.empty[st], ((cnt / S::kStages) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) bar_expect(&bar.full[st], bytes);
                __syncwarp();
                if (page >= 0)
                    tma4(ring + st * S::kStage + half * S::kHalf + mine * box * 128, kv ? &vmap : &kmap, 64 * half, row, w.hk, page, &bar.full[st]);
                if (kv == 0 && j == w.first) {  // the item's queries, after its first K
                    if (nq > 0 && !warp_wait(&bar.qempty, (nq - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    nq++;
                    if (lane == 0) {
                        const int per = p.item_tokens >> 1, tiles = w.left > per ? 2 : 1;
                        bar_expect(&bar.qfull, tiles * (D / 64) * per * p.group * 128);
                        for (int t = 0; t < tiles; t++)
                            for (int e = 0; e < D / 64; e++)
                                tma3(qs + t * (128 * D * 2) + e * S::kHalf, &qmap, 64 * e, w.hk * p.group, w.token + t * per, &bar.qfull);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) {  // wait (bounded) until the copies already issued have landed
            for (uint32_t c = cnt < S::kStages ? kv : cnt - S::kStages; c < cnt; c += 2) wait_bar(&bar.full[c % S::kStages], (c / S::kStages) & 1);
            if (nq > 0) wait_bar(&bar.qfull, (nq - 1) & 1);
        }
    } else if (warp == kMmaWarp) {  // -------------------------------------- products
        constexpr uint32_t IS = kInstr<BF, kTileSlots, false>, IO = kInstr<BF, D, true>;
        const uint32_t one = elect_one();
        const uint32_t qd = desc_lo(qs, 16), kd = desc_lo(ring, 16), vd = desc_lo(ring, S::kHalf);
        uint32_t st = 0, ph = 0, np = 0, ni = 0;  // the stage in turn and its phase; bit t of np: the phase of tile t's P
        auto next_stage = [&] {
            if (++st == S::kStages) st = 0, ph ^= 1;
        };
        // Loops, not unrolled code: the warp runs this once a step between the softmax's long code, and
        // fetching instructions took longer than the products.
        auto scores = [&](int t, uint32_t sk) {
            uint32_t a = qd + t * (128 * D * 2 / 16), b = kd + sk * (S::kStage / 16), acc = 0;
#pragma unroll 1
            for (int e = 0; e < D / 64; e++) {
#pragma unroll
                for (int k = 0; k < 4; k++, acc = 1) mma_ss<IS>(one, tm + 128 * t, a + 2 * k, b + 2 * k, acc);
                a += S::kHalf / 16, b += S::kHalf / 16;
            }
            commit(one, &bar.s[t]);
        };
        auto values = [&](int t, uint32_t sv, uint32_t acc) {
            uint32_t v = vd + sv * (S::kStage / 16), a = tm + S::kP + S::kPStep * t;
#pragma unroll 1
            for (int q = 0; q < 2; q++) {
                ok = ok && warp_wait(&bar.p[t][q], (np >> t) & 1);
                if (!ok) return;
                fence_after();
#pragma unroll
                for (int k = 0; k < 4; k++, acc = 1) mma_ts<IO>(one, tm + S::kO + D * t, a + 8 * k, v + k * (2048 / 16), acc);
                if (q == 0) commit(one, &bar.half[t]);
                a += 32, v += 4 * 2048 / 16;
            }
            np ^= 1 << t;
        };
        while (ok && take(bar, s_part, n_part, w, ok)) {
            // uniform values keep the loop's addresses in uniform registers
            const int n = __shfl_sync(~0u, w.last - w.first, 0), two = __shfl_sync(~0u, w.left > (p.item_tokens >> 1) ? 1 : 0, 0);
            const int s0 = __shfl_sync(~0u, w.lo + w.first * kTileSlots, 0), lo = __shfl_sync(~0u, w.seen_lo, 0), hi = __shfl_sync(~0u, w.hi, 0);
            ok = warp_wait(&bar.qfull, ni++ & 1) && warp_wait(&bar.full[st], ph);
            if (!ok) break;
            fence_after();
#pragma unroll 1
            for (int t = 0; t <= two; t++) scores(t, st);
            commit(one, &bar.empty[st]);
            if (n == 1) commit(one, &bar.qempty);
            next_stage();
#pragma unroll 1
            for (int j = 0; j < n && ok; j++) {  // O_t += P_t V_j, S_t = Q_t K_{j+1}
                const uint32_t sv = st, pv = ph;
                ok = warp_wait(&bar.full[sv], pv);
                if (s0 + j * kTileSlots < lo || s0 + (j + 1) * kTileSlots > hi) ok = ok && warp_wait(&bar.clean[sv], pv);
                next_stage();
                const bool more = j + 1 < n;
                if (more) ok = ok && warp_wait(&bar.full[st], ph);
#pragma unroll 1
                for (int t = 0; t <= two && ok; t++) {
                    values(t, sv, j > 0);
                    if (!ok) break;
                    if (t == two) commit(one, &bar.empty[sv]);
                    if (more)
                        scores(t, st);
                    else
                        commit(one, &bar.o[t]);
                }
                if (more) {
                    commit(one, &bar.empty[st]);
                    if (j + 2 == n) commit(one, &bar.qempty);
                    next_stage();
                }
            }
        }
        commit(one, &bar.done);  // every product is done when this arrives
        warp_wait(&bar.done, 0);
    } else if (warp == kHelpWarp) {  // ------------------------------------------ parts, ends of V
        constexpr int CH = D / 8;
        uint32_t cnt = 0, put = 0;
        bool more = true;
        int4 join = make_int4(0, 0, 0, kJoinNone);
        auto hand_out = [&] {
            if (!more) return;
            if (put >= kParts && !warp_wait(&bar.part_empty[put % kParts], (put / kParts - 1) & 1)) {
                ok = more = false;
                return;
            }
            Part n;
            more = walk.next(p, n);
            if (more && (n.first > 0 || n.last < n.tiles)) {
                if (n.first == 0)
                    join.x = n.left, join.y = n.hk, join.z = n.token;
                else
                    join.w = n.last == n.tiles ? kJoinEnd : kJoinOn;
            }
            __syncwarp();
            if (lane == 0) {
                s_part[put % kParts] = n;
                bar_arrive(&bar.part_full[put % kParts]);
            }
            __syncwarp();
            put++;
        };
        for (int i = 0; i < kParts - 1; i++) hand_out();
        for (uint32_t n = 0; ok; n++) {
            w = s_part[n % kParts];  // handed out by this warp and not yet overwritten
            if (w.tiles == 0) break;
            for (int j = 2 * w.first; j < 2 * w.last; j++, cnt++) {  // K and V of each step
                const uint32_t st = cnt % S::kStages;
                if (!warp_wait(&bar.full[st], (cnt / S::kStages) & 1)) {
                    ok = false;
                    break;
                }
                const int s0 = w.lo + (j >> 1) * kTileSlots;
                if ((j & 1) && (s0 < w.seen_lo || s0 + kTileSlots > w.hi)) {
                    const int r0 = w.seen_lo - s0, r1 = w.hi - s0 > 0 ? w.hi - s0 : 0;
                    const uint32_t at = ring + st * S::kStage;
                    auto zero = [&](int c) {
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + ((c % CH) >> 3) * S::kHalf + (c / CH) * 128 + ((c & 7) << 4)),
                                     "r"(0)
                                     : "memory");
                    };
                    for (int c = lane; c < r0 * CH; c += 32) zero(c);
                    for (int c = r1 * CH + lane; c < kTileSlots * CH; c += 32) zero(c);
                    fence_async();
                    __syncwarp();
                }
                // the stage is not filled again before this warp has seen it, so that no wait meets a barrier two phases on
                if (lane == 0) bar_arrive(&bar.clean[st]), bar_arrive(&bar.empty[st]);
            }
            hand_out();
        }
        if (lane == 0 && p.join) p.join[blockIdx.x] = join;
    }
    if (!ok && lane == 0) flag(p.c.status, FTMOE_ERR_STATE);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
}

// Joins the parts of the item that CTA c of the chunk kernel started. A CTA takes 32 rows, a lane a row
// and a warp an eighth of the elements; rows go out through shared memory.
constexpr int kJoinThreads = 256, kJoinRows = 32;

template <bool BF, int D>
__global__ void __launch_bounds__(kJoinThreads) chunk_combine(const AttendParams p) {
    constexpr int E = D / 8;  // elements a thread
    __shared__ __align__(16) uint16_t s_out[kJoinRows][D + 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the first 32 CTAs' entries come together
    const int4 mine = c + lane < gridDim.x ? p.join[c + lane] : make_int4(0, 0, 0, kJoinEnd);
    const int4 join = make_int4(__shfl_sync(~0u, mine.x, 0), __shfl_sync(~0u, mine.y, 0), __shfl_sync(~0u, mine.z, 0), 0);
    const int row = blockIdx.y * kJoinRows + lane, half = p.item_tokens >> 1;
    const int li = (row & 127) / (uint32_t)p.group, g = (row & 127) - li * p.group;
    const int i = (row >> 7) * half + li, h = join.y * p.group + g;
    const bool live = li < half && i < join.x;
    if (!__any_sync(~0u, live)) return;  // the same rows in every warp
    const unsigned end = __ballot_sync(~0u, lane > 0 && mine.w == kJoinEnd);
    const int n = end ? __ffs(end) : count_parts(p.join, c, gridDim.x);
    // the first four parts, which are mostly all, load at once
    constexpr int K = 4;
    auto slot = [&](int k) { return 2 * (c + k) + (k == 0); };
    auto part = [&](int k) { return p.part_o + ((int64_t)slot(k) * D + warp * E) * kTileRows + row; };
    float2 ml[K];
    float v[K][E], M = -INFINITY, L = 0.f, x[E];
#pragma unroll
    for (int k = 0; k < K; k++) {
        ml[k] = k < n ? p.part_ml[slot(k) * kTileRows + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; e++) v[k][e] = k < n ? part(k)[e * kTileRows] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; k++) M = fmaxf(M, ml[k].x);
    for (int k = K; k < n; k++) M = fmaxf(M, p.part_ml[slot(k) * kTileRows + row].x);
#pragma unroll
    for (int e = 0; e < E; e++) x[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; k++) {
        const float a = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
        L += ml[k].y * a;
#pragma unroll
        for (int e = 0; e < E; e++) x[e] += v[k][e] * a;
    }
    for (int k = K; k < n; k++) {
        const float2 y = p.part_ml[slot(k) * kTileRows + row];
        const float a = y.x == -INFINITY ? 0.f : ex2(y.x - M);
        L += y.y * a;
#pragma unroll
        for (int e = 0; e < E; e++) x[e] += part(k)[e * kTileRows] * a;
    }
    float lse2;
    const float f = finish_row(M, L, p.sinks, live ? h : 0, lse2);
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(&s_out[lane][warp * E + e]) = from_f2<BF>(x[e] * f, x[e + 1] * f);
    if (warp == 0 && live) put_lse(p, join.z + i, h, lse2);
    __syncthreads();
    for (int k = threadIdx.x; k < kJoinRows * D / 8; k += kJoinThreads) {
        const int r = k / (D / 8), ch = k % (D / 8), rr = blockIdx.y * kJoinRows + r;
        const int ri = (rr & 127) / (uint32_t)p.group, rg = (rr & 127) - ri * p.group, rt = (rr >> 7) * half + ri;
        if (ri < half && rt < join.x)
            *reinterpret_cast<uint4 *>(p.out.d + (int64_t)(join.z + rt) * p.out.token + (join.y * p.group + rg) * p.out.head + 8 * ch) =
                *reinterpret_cast<const uint4 *>(&s_out[r][8 * ch]);
    }
}

template <bool BF, int D>
cudaError_t launch(const AttendParams &p, int C, cudaStream_t st) {
    using S = Shape<D>;
    CUtensorMap qm, km, vm;
    const int box = p.c.page_shift < 7 ? 1 << p.c.page_shift : 128;
    if (!query_map(qm, p, BF) || !page_map(km, p.c, true, BF, box) || !page_map(vm, p.c, false, BF, box)) return cudaErrorInvalidValue;
    cudaError_t e = allow_smem<chunk_kernel<BF, D>>(S::kSmem);
    if (e != cudaSuccess) return e;
    chunk_kernel<BF, D><<<C, kThreads, S::kSmem, st>>>(p, qm, km, vm);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return !p.join ? e : launch_after(chunk_combine<BF, D>, dim3(C, kTileRows / kJoinRows), kJoinThreads, 0, st, p);
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

bool query_map(CUtensorMap &m, const AttendParams &p, bool bf16) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)p.c.dim, (cuuint64_t)p.q_heads, (cuuint64_t)p.bt.tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)p.q.head * 2, (cuuint64_t)p.q.token * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(p.item_tokens / 2)}, es[3] = {1, 1, 1};
    return fn(&m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p.q.d, dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool row_map(CUtensorMap &m, const void *x, int cols, int rows, int64_t stride, int box_rows, bool bf16) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, 1}, strides[2] = {(cuuint64_t)stride * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
    return fn(&m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(x), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool box_map(CUtensorMap &m, bool bf16, const void *x, const int64_t (&dims)[3], int64_t stride1, int64_t stride2, const int (&box)[3],
             bool swizzle) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t d[3] = {(cuuint64_t)dims[0], (cuuint64_t)dims[1], (cuuint64_t)dims[2]}, st[2] = {(cuuint64_t)stride1, (cuuint64_t)stride2};
    const cuuint32_t b[3] = {(cuuint32_t)box[0], (cuuint32_t)box[1], (cuuint32_t)box[2]}, es[3] = {1, 1, 1};
    const CUtensorMapSwizzle sw = swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
    return fn(&m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(x), d, st, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the call's items are cut. Not if there is an SM for each, and the longest has few steps and hardly more than an
// even share of all steps: that saves the walk along the line (2 us) and the joining kernel (112 items, heads of 64, one
// step: 8.9 us whole, 12.6 cut; three steps: 13.9 and 18.8; six: 20.0 and 21.5; eight: 24 and 21.6. Heads of 128, three
// steps: 16.1 and 22.9, eight: 27 and 26.7; 32 items of three steps, whose share is two: 16 and 17).
bool chunk_parts(const AttendParams &p, int num_sms) {
    const int64_t items = (int64_t)((p.bt.max_q + p.item_tokens - 1) / p.item_tokens) * p.bt.batch * p.c.kv_heads;
    int64_t slots = p.bt.max_kv;
    if (p.window && (int64_t)p.window + p.item_tokens + kTileSlots < slots) slots = p.window + p.item_tokens + kTileSlots;
    const int64_t steps = (slots + kTileSlots - 1) / kTileSlots;
    return items > num_sms || steps > 6 || steps > (items * (steps + kItemCost) + num_sms - 1) / num_sms + 1;
}

int chunk_ctas(const AttendParams &p, int num_sms) {
    const int64_t n_qt = (p.bt.max_q + p.item_tokens - 1) / p.item_tokens;
    if (!chunk_parts(p, num_sms)) return (int)(n_qt * p.bt.batch * p.c.kv_heads);
    const int64_t most = n_qt * p.bt.batch * p.c.kv_heads * (p.bt.max_kv / kTileSlots + 2);
    return (int)(most < num_sms ? (most > 0 ? most : 1) : num_sms);
}

size_t chunk_rows() { return kTileRows; }

cudaError_t launch_chunk(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    const int C = chunk_ctas(p, num_sms);
    if (p.c.dim == 64) return bf16 ? launch<true, 64>(p, C, st) : launch<false, 64>(p, C, st);
    return bf16 ? launch<true, 128>(p, C, st) : launch<false, 128>(p, C, st);
}

}  // namespace kv
}  // namespace ftmoe

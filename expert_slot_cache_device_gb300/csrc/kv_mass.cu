// The mass pass of chunks: mass[j] += sum over the rows that see slot j of 2^(s scale log2 e - lse), on
// the 5th-generation tensor cores. An item is 128 slots of one (sequence, key head): K is the A
// operand (M = 128 slots), the queries of 128 / group tokens at a time are B, so a thread of the
// epilogue holds one slot and adds over the columns (rows) in order: one writer and one order for each
// mass element. Bound by the exponentials and the products alike: 2 dim flops and one exponential a
// (row, slot).
//
// Persistent, one CTA an SM, items dealt round-robin with the slots that most rows see first. Where there are too few
// items for an even share, each is cut by rows into mass_split pieces, whose sums a second kernel adds
// in order. Roles:
//   warps 0-11      sums: three groups of four warps take the row tiles in turn and join at an item's end. The
//                   first four move the next item's K from shared to tensor memory: read from
//                   there, a product needs only its queries from shared memory and runs at 64
//                   cycles instead of 98;
//   warp 12         tensor copies of K and the query tiles (a ring);
//   warp 13         issues S = K Q^T into three tensor-memory buffers of 128 columns;
//   warps 14, 15    the rows' negated log-sum-exps (powers of two) of each tile.
// Slots outside the visible range may hold anything: they only meet their own lane, whose sum
// is not written. Every wait is bounded.
//
// 2048 tokens over 31000, 32 query heads of 128 on 8: 378 us, 1.33 PFLOP/s in the products (0.71 of a large bf16 one) and
// 5.2 exponentials a nanosecond. (A share of the exponentials as polynomials on the FMA pipe, a quarter to a
// half, made it 444 to 604 us.)
#include "kv_tc05.cuh"

namespace ftmoe {
namespace kv {
namespace {

// Three groups of four warps sum: with two, every pipe was below half (exponentials 49 %, products 48 %)
// for want of warps to cover the loads of the others.
constexpr int kGroups = 3, kSums = 4 * kGroups, kWarps = kSums + 4, kThreads = kWarps * 32;
constexpr int kCopyWarp = kSums, kMmaWarp = kSums + 1, kLseWarp = kSums + 2;
constexpr int kBufs = 3;
constexpr int kLse = 2 * kGroups;  // buffers of log-sum-exps: each belongs to one group and one loading warp
static_assert(kBufs == kGroups && kLse % 2 == 0, "a barrier's waiter sees its every phase");
constexpr uint32_t kKCol = 384;  // two buffers of K in tensor memory, 64 columns each

template <int D>
struct Shape {
    static constexpr int kTile = 128 * D * 2, kHalf = 128 * 128;
    static constexpr int kStages = 4;
    static constexpr int kSmem = 1024 + (1 + kStages) * kTile;
};

struct Bars {
    uint64_t kfull, kread, ktm[2], kempty[2], qfull[4], qempty[4], s[kBufs], free[kBufs], lse[kLse], lfree[kLse], joined, read, done;
};

// Piece `n` of the line: slot tile, sequence, key head, piece of the rows; its row tiles [first, last) that see some
// of the slots.
struct Slots {
    int b, hk, piece, s0, first, last;
    Seq sq;
    Range vis;  // slots that some row sees
};

__device__ __forceinline__ bool slots_of(const AttendParams &p, int n, Slots &w) {
    const int per = p.bt.batch * p.c.kv_heads;
    w.piece = n % p.mass_split, n /= p.mass_split;
    w.s0 = n / per * kTileSlots;
    w.b = n % per / p.c.kv_heads, w.hk = n % p.c.kv_heads;
    w.sq = seq_info(p.bt, w.b, nullptr);
    w.vis = visible(w.sq, 0, w.sq.q_len, p.window, p.causal);
    if (w.s0 >= w.vis.hi || w.s0 + kTileSlots <= w.vis.lo) return false;
    const int before = w.sq.kv_len - w.sq.q_len, tok = p.item_tokens >> 1;
    // tokens i in [i0, i1) see a slot of the tile: slot before + i >= s0, and before + i - window < s0 + 127
    int i0 = p.causal ? w.s0 - before : -before, i1 = p.window ? w.s0 + kTileSlots - 1 + p.window - before : w.sq.q_len;
    if (i0 < 0) i0 = 0;
    if (i1 > w.sq.q_len) i1 = w.sq.q_len;
    w.first = i0 / tok, w.last = (i1 + tok - 1) / tok;
    if (p.mass_split > 1) {
        const int tiles = (w.sq.q_len + tok - 1) / tok;
        const int lo = (int)((int64_t)w.piece * tiles / p.mass_split), hi = (int)((int64_t)(w.piece + 1) * tiles / p.mass_split);
        w.first = w.first > lo ? w.first : lo, w.last = w.last < hi ? w.last : hi;
    }
    return w.first < w.last;
}

// The first of items n, n + gridDim.x, ... that has rows.
__device__ __forceinline__ int next_item(const AttendParams &p, int items, int n, Slots &w) {
    while (n < items && !slots_of(p, n, w)) n += gridDim.x;
    return n;
}

template <bool BF, int D>
__global__ void __launch_bounds__(kThreads, 1)
    mass_kernel(const AttendParams p, const int items, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap) {
    using S = Shape<D>;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ Bars bar;
    __shared__ uint32_t s_tmem;
    __shared__ __align__(16) float s_lse[kLse][128];
    __shared__ float s_part[kGroups - 1][128];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t ks = (su32(sm_raw) + 1023u) & ~1023u, qs = ks + S::kTile;
    const int tok = p.item_tokens >> 1;

    if (tid == 0) {
        bar_init(&bar.kfull, 1), bar_init(&bar.kread, 4);
        for (int i = 0; i < 2; i++) bar_init(&bar.ktm[i], 4), bar_init(&bar.kempty[i], 1);
        for (int i = 0; i < S::kStages; i++) bar_init(&bar.qfull[i], 1), bar_init(&bar.qempty[i], 1);
        for (int i = 0; i < kBufs; i++) bar_init(&bar.s[i], 1), bar_init(&bar.free[i], 4);
        for (int i = 0; i < kLse; i++) bar_init(&bar.lse[i], 1), bar_init(&bar.lfree[i], 4);
        bar_init(&bar.done, 1), bar_init(&bar.joined, 4 * (kGroups - 1)), bar_init(&bar.read, 4);
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
    Slots w;

    if (warp < kSums) {  // ---------------------------------------------------- sums
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const float c2 = p.scale * kLog2e;
        const uint64_t cc = pack2(c2, c2);
        uint32_t cnt = 0, ni = 0;
        // K of the item that is `m`-th here, from shared memory to its tensor-memory buffer
        auto move_k = [&](uint32_t m) {
            const uint32_t to = tm + lanes + kKCol + 64 * (m & 1), row = tid & 127;
            if (!warp_wait(&bar.kfull, m & 1) || !warp_wait(&bar.kempty[m & 1], ((m >> 1) & 1) ^ 1)) return false;
            fence_after();  // the products that read the buffer are done
#pragma unroll
            for (int e = 0; e < D / 64; e++) {
                uint32_t x[32];
#pragma unroll
                for (int c = 0; c < 8; c++)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(x[4 * c]), "=r"(x[4 * c + 1]), "=r"(x[4 * c + 2]), "=r"(x[4 * c + 3])
                                 : "r"(ks + e * S::kHalf + row * 128 + ((c ^ (row & 7)) << 4))
                                 : "memory");
                tm_st32(to + 32 * e, x);
            }
            tm_st_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&bar.ktm[m & 1]), bar_arrive(&bar.kread);
            return true;
        };
        Slots v;
        int n = next_item(p, items, blockIdx.x, w);
        if (t == 0 && n < items) ok = move_k(0);
        while (n < items && ok) {
            const int nn = next_item(p, items, n + gridDim.x, v);
            if (t == 0 && nn < items) ok = move_k(ni + 1);
            if (!ok) break;
            const int j = w.s0 + (tid & 127), before = w.sq.kv_len - w.sq.q_len;
            // rows [ra, rb) of the sequence see slot j
            int ia = p.causal ? j - before : -before, ib = p.window ? j + p.window - before : w.sq.q_len;
            if (ia < 0) ia = 0;
            if (ib > w.sq.q_len) ib = w.sq.q_len;
            float total = 0.f;
            for (int rt = w.first; rt < w.last && ok; rt++, cnt++) {
                if (cnt % kGroups != t) continue;  // (counted over all items: a group waits for every use of its own buffers)
                const uint32_t bf = cnt % kBufs, lb = cnt % kLse;
                ok = warp_wait(&bar.lse[lb], (cnt / kLse) & 1) && warp_wait(&bar.s[bf], (cnt / kBufs) & 1);
                if (!ok) break;
                fence_after();
                // the tile's columns [a, e) see the slot; those past the last whole token are none
                const int ta = ia - rt * tok, te = ib - rt * tok;
                const int a = ta > 0 ? (ta < tok ? ta : tok) * p.group : 0, e = te > 0 ? (te < tok ? te : tok) * p.group : 0;
                const bool cut = __any_sync(~0u, a > 0 || e < 128);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    uint32_t x[64];
                    tm_ld64(tm + lanes + 128 * bf + 64 * q, x);
                    tm_ld_wait(x);
                    if (cut) {
#pragma unroll
                        for (int k = 0; k < 64; k++)
                            if (64 * q + k < a || 64 * q + k >= e) x[k] = 0xff800000u;
                    }
#pragma unroll
                    for (int k = 0; k < 64; k += 4) {
                        const float4 z = *reinterpret_cast<const float4 *>(&s_lse[lb][64 * q + k]);
                        const float2 f0 = unpack2(fma2(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), cc, pack2(z.x, z.y)));
                        const float2 f1 = unpack2(fma2(pack2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), cc, pack2(z.z, z.w)));
                        sum[0] = add2(sum[0], pack2(ex2(f0.x), ex2(f0.y)));
                        sum[1] = add2(sum[1], pack2(ex2(f1.x), ex2(f1.y)));
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bar.free[bf]), bar_arrive(&bar.lfree[lb]);
                const float2 f = unpack2(add2(sum[0], sum[1]));
                total += f.x + f.y;
            }
            // the other groups' sums join the first's, in order
            if (!ok) break;
            if (t > 0) {
                ok = warp_wait(&bar.read, (ni & 1) ^ 1);  // the last item's have been read
                s_part[t - 1][tid & 127] = total;
                __syncwarp();
                if (lane == 0) bar_arrive(&bar.joined);
            } else {
                ok = warp_wait(&bar.joined, ni & 1);
#pragma unroll
                for (int k = 0; k < kGroups - 1; k++) total += s_part[k][tid];
                if (ok && j >= w.vis.lo && j < w.vis.hi) {
                    if (p.mass_split > 1)
                        p.mass_parts[((int64_t)w.piece * p.bt.batch * p.c.kv_heads + w.b * p.c.kv_heads + w.hk) * p.logit_stride + j] = total;
                    else
                        p.mass[w.b * p.mass_seq + w.hk * p.mass_head + j] += total;
                }
                __syncwarp();
                if (lane == 0) bar_arrive(&bar.read);
            }
            ni++;
            n = nn, w = v;
        }
    } else if (warp == kCopyWarp) {  // ------------------------------------- K, queries
        const int box = 1 << (p.c.page_shift < 7 ? p.c.page_shift : 7), boxes = kTileSlots / box, halves = D / 64;
        const int mine = lane % boxes, half = lane / boxes;
        uint32_t nk = 0, nq = 0;
        auto copy_k = [&](const Slots &v) {
            const int slot = v.s0 + mine * box;
            int page = -1;
            if (half < halves && slot < v.vis.hi && slot + box > v.vis.lo) {
                page = p.bt.table[(int64_t)v.b * p.bt.table_stride + (slot >> p.c.page_shift)];
                if ((uint32_t)page >= (uint32_t)p.c.num_pages) page = -1;  // recorded by the pass before
            }
            const uint32_t bytes = __popc(__ballot_sync(~0u, page >= 0)) * box * 128;
            if (nk > 0 && !warp_wait(&bar.kread, (nk - 1) & 1)) return false;
            if (lane == 0) bar_expect(&bar.kfull, bytes);
            __syncwarp();
            if (page >= 0)
                tma4(ks + half * S::kHalf + mine * box * 128, &kmap, 64 * half, slot & ((1 << p.c.page_shift) - 1), v.hk, page, &bar.kfull);
            nk++;
            return true;
        };
        Slots v;
        int n = next_item(p, items, blockIdx.x, w);
        if (n < items) ok = copy_k(w);
        while (n < items && ok) {
            // the next item's K goes before this one's queries: it is moved before this item is summed
            const int nn = next_item(p, items, n + gridDim.x, v);
            if (nn < items) ok = copy_k(v);
            if (!ok) break;
            for (int rt = w.first; rt < w.last; rt++, nq++) {
                const uint32_t st = nq % S::kStages;
                if (!warp_wait(&bar.qempty[st], ((nq / S::kStages) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) bar_expect(&bar.qfull[st], halves * tok * p.group * 128);
                __syncwarp();
                if (lane < halves)
                    tma3(qs + st * S::kTile + lane * S::kHalf, &qmap, 64 * lane, w.hk * p.group, w.sq.q0 + rt * tok, &bar.qfull[st]);
            }
            n = nn, w = v;
        }
        if (!ok) {  // wait (bounded) until the copies already issued have landed
            if (nk > 0) wait_bar(&bar.kfull, (nk - 1) & 1);
            for (uint32_t c = nq < S::kStages ? 0 : nq - S::kStages; c < nq; c++) wait_bar(&bar.qfull[c % S::kStages], (c / S::kStages) & 1);
        }
    } else if (warp == kMmaWarp) {  // -------------------------------------- products
        constexpr uint32_t IS = kInstr<BF, 128, false>;
        const uint32_t one = elect_one();
        const uint32_t qd = desc_lo(qs, 16);
        uint32_t nk = 0, cnt = 0;
        for (int n = blockIdx.x; n < items && ok; n += gridDim.x) {
            if (!slots_of(p, n, w)) continue;
            const int tiles = __shfl_sync(~0u, w.last - w.first, 0);
            ok = warp_wait(&bar.ktm[nk & 1], (nk >> 1) & 1);
            for (int i = 0; i < tiles && ok; i++, cnt++) {
                const uint32_t st = cnt % S::kStages, bf = cnt % kBufs;
                ok = warp_wait(&bar.qfull[st], (cnt / S::kStages) & 1) && warp_wait(&bar.free[bf], ((cnt / kBufs) & 1) ^ 1);
                if (!ok) break;
                fence_after();
                uint32_t a = tm + kKCol + 64 * (nk & 1), b = qd + st * (S::kTile / 16), acc = 0;
#pragma unroll 1
                for (int e = 0; e < D / 64; e++) {
#pragma unroll
                    for (int k = 0; k < 4; k++, acc = 1) mma_ts<IS>(one, tm + 128 * bf, a + 8 * k, b + 2 * k, acc);
                    a += 32, b += S::kHalf / 16;
                }
                commit(one, &bar.s[bf]);
                commit(one, &bar.qempty[st]);
            }
            commit(one, &bar.kempty[nk & 1]);
            nk++;
        }
        commit(one, &bar.done);
        warp_wait(&bar.done, 0);
    } else {  // -------------------------------------------------------------- log-sum-exps
        // one the even, one the odd tiles of the whole line; a lane's four rows sit at the same
        // places of every tile, and the next tile's values are under way while this one's wait
        int at[4], i4[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const int r = lane + 32 * k;
            i4[k] = r / (uint32_t)p.group;
            at[k] = i4[k] * p.q_heads + r - i4[k] * p.group;
            if (i4[k] >= tok) i4[k] = 1 << 30;
        }
        uint32_t cnt = warp - kLseWarp, base = 0;
        float z[4];
        bool have = false;
        auto put = [&] {  // the values of tile cnt
            const uint32_t lb = cnt % kLse;
            if (!warp_wait(&bar.lfree[lb], ((cnt / kLse) & 1) ^ 1)) return false;
#pragma unroll
            for (int k = 0; k < 4; k++) s_lse[lb][lane + 32 * k] = z[k];
            __syncwarp();
            if (lane == 0) bar_arrive(&bar.lse[lb]);
            cnt += 2;
            return true;
        };
        for (int n = blockIdx.x; n < items && ok; n += gridDim.x) {
            if (!slots_of(p, n, w)) continue;
            const uint32_t tiles = w.last - w.first;
            const float *src = p.lse2 + (int64_t)w.sq.q0 * p.q_heads + w.hk * p.group;
            for (uint32_t c = cnt + (have ? 2 : 0); c < base + tiles && ok; c += 2) {
                const int t0 = (w.first + (int)(c - base)) * tok;
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    y[k] = -INFINITY;
                    if (i4[k] < w.sq.q_len - t0) y[k] = src[(int64_t)t0 * p.q_heads + at[k]];
                }
                if (have) ok = put();
#pragma unroll
                for (int k = 0; k < 4; k++) z[k] = y[k] == -INFINITY ? y[k] : -y[k];  // a row that sees nothing adds nothing
                have = true;
            }
            base += tiles;
        }
        if (have && ok) ok = put();
    }
    if (!ok && lane == 0) flag(p.c.status, FTMOE_ERR_STATE);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
}

// mass += the pieces' sums, in order: one thread a slot.
__global__ void __launch_bounds__(128) mass_join(const AttendParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int per = p.bt.batch * p.c.kv_heads, n = (blockIdx.x * per + blockIdx.z * p.c.kv_heads + blockIdx.y) * p.mass_split;
    const int j = blockIdx.x * kTileSlots + threadIdx.x;
    float sum = 0.f;
    Slots w;
    bool any = false;
    for (int k = 0; k < p.mass_split; k++)
        if (slots_of(p, n + k, w) && j >= w.vis.lo && j < w.vis.hi) {
            sum += p.mass_parts[((int64_t)k * per + w.b * p.c.kv_heads + w.hk) * p.logit_stride + j];
            any = true;
        }
    if (any) p.mass[blockIdx.z * p.mass_seq + blockIdx.y * p.mass_head + j] += sum;
}

template <bool BF, int D>
cudaError_t launch(const AttendParams &p, int num_sms, cudaStream_t st) {
    using S = Shape<D>;
    CUtensorMap qm, km;
    if (!query_map(qm, p, BF) || !page_map(km, p.c, true, BF, p.c.page_shift < 7 ? 1 << p.c.page_shift : 128)) return cudaErrorInvalidValue;
    const int64_t tiles = ((int64_t)p.bt.max_kv + kTileSlots - 1) / kTileSlots, items = tiles * p.bt.batch * p.c.kv_heads * p.mass_split;
    if (items >= (int64_t)1 << 31) return cudaErrorInvalidValue;
    if (items == 0) return cudaSuccess;
    cudaError_t e = allow_smem<mass_kernel<BF, D>>(S::kSmem);
    if (e != cudaSuccess) return e;
    mass_kernel<BF, D><<<(unsigned)(items < num_sms ? items : num_sms), kThreads, S::kSmem, st>>>(p, (int)items, qm, km);
    if ((e = cudaGetLastError()) != cudaSuccess || p.mass_split == 1) return e;
    return launch_after(mass_join, dim3((unsigned)tiles, p.c.kv_heads, p.bt.batch), 128, 0, st, p);
}

}  // namespace

// Pieces that each item's rows are cut into: about four items for every SM, but no piece below four row tiles.
// (A prompt of 4096 tokens, 128 items of unequal rows on 152 SMs: 167 us whole, 113 us in four pieces.)
int mass_split(const AttendParams &p, int num_sms) {
    const int64_t items = ((int64_t)p.bt.max_kv + kTileSlots - 1) / kTileSlots * p.bt.batch * p.c.kv_heads;
    const int64_t rows = ((int64_t)p.bt.max_q + p.item_tokens / 2 - 1) / (p.item_tokens / 2);
    int64_t n = items > 0 ? 4 * (int64_t)num_sms / items : 1;
    if (n > rows / 4) n = rows / 4;
    return n < 1 ? 1 : (n > 8 ? 8 : (int)n);
}

cudaError_t launch_mass(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    if (p.c.dim == 64) return bf16 ? launch<true, 64>(p, num_sms, st) : launch<false, 64>(p, num_sms, st);
    return bf16 ? launch<true, 128>(p, num_sms, st) : launch<false, 128>(p, num_sms, st);
}

}  // namespace kv
}  // namespace ftmoe

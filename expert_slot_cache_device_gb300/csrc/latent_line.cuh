// How the latent-attention kernels cut their work: as in kv_split.cuh, an item being a tile of tokens of one sequence and
// one block of heads. Items stand in one line, sequence by sequence, block by block, tile by tile, each as long as its
// visible slots have steps of 128 (and kItemCost for its start and end); CTA c of C takes an even piece of it. A warp of
// each CTA walks its piece and hands the parts out through a small ring.
#pragma once

#include "kv_tc05.cuh"
#include "latent.cuh"

namespace ftmoe {
namespace latent {

using kv::bar_arrive;
using kv::su32;
using kv::warp_wait;

constexpr int kStep = 128;    // slots of a step
constexpr int kItemCost = 2;  // what an item's start and end take, in steps (its queries, its first S, its outputs: 6000 to 9000 cycles)
constexpr int kParts = 4;     // entries of the ring of parts

// Whether `items` of at most `steps` steps are cut evenly for `have` places and joined, or each goes whole to a place, in as many waves. The
// join, and starts in the middle of items, cost about 8 steps where every place has a part (what an item's joining kernel reads), less with
// fewer. The host knows bounds of the lengths only: a mean of 3/4 is assumed. `waves`: the most that whole items may need.
inline bool cut_pays(int64_t items, int64_t steps, int64_t have, int64_t waves, int64_t extra) {
    const int64_t n = (items + have - 1) / have;
    if (n > waves) return true;
    const int64_t share = (items * (3 * steps / 4 + kItemCost) + have - 1) / have;
    return n * (steps + kItemCost) > share + kItemCost + 8 * (items < have ? items : have) / have + extra;
}

__device__ __forceinline__ int item_count(const Line &l, const kv::Seq &s) {
    return (int)((uint32_t)(s.q_len + l.item_tokens - 1) / (uint32_t)l.item_tokens);
}
// Slots [0, item_hi) are what at least one row of the item sees.
__device__ __forceinline__ int item_hi(const Line &l, const kv::Seq &s, int qt) {
    const int i0 = qt * l.item_tokens, i1 = l.item_tokens < s.q_len - i0 ? i0 + l.item_tokens : s.q_len;
    const kv::Range r = kv::visible(s, i0, i1, 0, l.causal);
    return r.hi;
}
__device__ __forceinline__ int item_steps(int hi) { return hi > 0 ? (hi + kStep - 1) / kStep : 1; }

// Units of one (sequence, block) in its first `end` items; the whole warp calls. Counted in 64 bits; the warp's 32-bit sums
// take the low 16 bits and the rest apart, which lanes below 2^43 fit.
__device__ __forceinline__ long long seq_units(const Line &l, const kv::Seq &s, int end) {
    long long n = 0;
    for (int qt = threadIdx.x & 31; qt < end; qt += 32) n += item_steps(item_hi(l, s, qt)) + kItemCost;
    return ((long long)__reduce_add_sync(~0u, (uint32_t)(n >> 16)) << 16) + __reduce_add_sync(~0u, (uint32_t)n & 0xffffu);
}

// A part of an item, as the roles take it from the ring.
struct Part {
    int b, block;
    int token, left;         // first token row of the item; new tokens from there to the sequence's end
    int slot, kv_len;        // the first token's slot
    int hi;                  // item_hi
    int first, last, steps;  // steps [first, last) of the item's; steps = 0: no more parts
};

// The walk along the line. P: `line`, and seq(b, status).
template <class P>
struct Walk {
    long long left;
    int b, block, qt, n_qt, at;  // at: units into the item (its kItemCost first)
    kv::Seq sq;
    __device__ __forceinline__ bool next(const P &p, Part &w) {
        while (left > 0) {
            const int hi = item_hi(p.line, sq, qt), steps = item_steps(hi);
            const int n = steps + kItemCost, end = left < n - at && p.line.join ? at + (int)left : n;
            w.b = b, w.block = block;
            w.token = sq.q0 + qt * p.line.item_tokens, w.left = sq.q_len - qt * p.line.item_tokens;
            w.slot = sq.kv_len - sq.q_len + qt * p.line.item_tokens, w.kv_len = sq.kv_len, w.hi = hi, w.steps = steps;
            w.first = at > kItemCost ? at - kItemCost : 0, w.last = end - kItemCost;
            left = p.line.join ? left - (end - at) : 0;
            at = 0;
            if (left > 0 && ++qt == n_qt) {
                qt = 0;
                if (++block == p.line.blocks) {
                    block = 0;
                    do {
                        sq = p.seq(++b, nullptr);
                        n_qt = item_count(p.line, sq);
                    } while (n_qt == 0);
                }
            }
            if (w.last > w.first) return true;
        }
        w.steps = 0;
        return false;
    }
};

// Where this CTA stands: its place in the line, the places there are, and its index in join, where those of one line follow one
// another (a pair's CTAs have the same place, and a line each).
struct Where {
    int at, of, id;
};
__device__ __forceinline__ Where where(const Line &l) {
    const int at = blockIdx.x >> l.pair, of = gridDim.x >> l.pair;
    return Where{at, of, l.pair ? (int)(blockIdx.x & 1) * of + at : at};
}

// Calls whose walk one warp finds by itself, while the others set up: a CTA an item (no line to walk), or few sequences of few
// items each, which a lane counts for its sequence. A start of 2 us less than plan's, whose loads, barriers and scans all warps wait for.
__device__ __forceinline__ bool plans_alone(const Line &l) { return !l.join || (l.max_q <= 16 * l.item_tokens && l.batch <= 256); }

template <class P>
__device__ __forceinline__ void plan_alone(const P &p, Walk<P> &w, int32_t *status) {
    const Line &l = p.line;
    const Where me = where(l);
    const int lane = threadIdx.x & 31;
    if (!l.join) {
        const int most = (l.max_q + l.item_tokens - 1) / l.item_tokens, block = me.at / most;
        w.qt = me.at - block * most, w.b = block / l.blocks, w.block = block - w.b * l.blocks;
        w.sq = p.seq(w.b, w.qt == 0 && w.block == 0 && lane == 0 ? status : nullptr);
        w.n_qt = item_count(l, w.sq), w.at = 0, w.left = w.qt < w.n_qt;
        return;
    }
    auto units = [&](const kv::Seq &x) {  // of a block
        int n = 0;
        for (int qt = 0; qt < item_count(l, x); qt++) n += item_steps(item_hi(l, x, qt)) + kItemCost;
        return n;
    };
    long long W = 0;
    for (int b = lane; b < l.batch; b += 32) W += units(p.seq(b, me.at == 0 ? status : nullptr));
#pragma unroll
    for (int o = 16; o; o >>= 1) W += __shfl_xor_sync(~0u, W, o);
    W *= l.blocks;
    const int C = kv::used_ctas(me.of, W);
    w.left = 0;
    if (me.at >= C) return;
    const long long u0 = kv::unit_start(me.at, C, W), u1 = kv::unit_start(me.at + 1, C, W);
    long long before = 0;  // units of the sequences before these
    for (int b0 = 0; b0 < l.batch; b0 += 32) {
        const kv::Seq s = b0 + lane < l.batch ? p.seq(b0 + lane, nullptr) : kv::Seq{0, 0, 0};
        const int per = units(s);
        long long x = (long long)per * l.blocks;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            if (lane >= o) x += y;
        }
        const unsigned past = __ballot_sync(~0u, u0 < before + x);
        if (past) {
            const int owner = __ffs(past) - 1;
            long long rest = u0 - (before + x - (long long)per * l.blocks);
            int block = 0, qt = 0, at = 0;
            if (lane == owner) {
                if (l.blocks > 1) block = (int)(rest / per);
                at = (int)(rest - (long long)block * per);
                for (int n; at >= (n = item_steps(item_hi(l, s, qt)) + kItemCost); qt++) at -= n;
            }
            w.b = b0 + owner, w.block = __shfl_sync(~0u, block, owner), w.at = __shfl_sync(~0u, at, owner);
            w.qt = __shfl_sync(~0u, qt, owner), w.n_qt = __shfl_sync(~0u, item_count(l, s), owner);
            w.sq.q0 = __shfl_sync(~0u, s.q0, owner), w.sq.q_len = __shfl_sync(~0u, s.q_len, owner), w.sq.kv_len = __shfl_sync(~0u, s.kv_len, owner);
            w.left = u1 - u0;
            return;
        }
        before += __shfl_sync(~0u, x, 31);
    }
}

// Total units and this CTA's start, for kWarps warps. s_sum: 32 kWarps entries, s_warp: kWarps.
template <int kWarps, class P>
__device__ __noinline__ bool plan(const P &p, Walk<P> &w, long long *s_warp, long long *s_sum, Walk<P> *s_walk, int32_t *status) {
    constexpr int T = kWarps * 32;
    const Line &l = p.line;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Where me = where(l);
    // one item a sequence at most: a thread a sequence, which then knows its start without reading it again
    const bool single = l.max_q <= l.item_tokens;
    kv::Seq mine{};
    auto sums = [&](int b0, int32_t *st) {
        if (single) {
            if (b0 + tid < l.batch) {
                mine = p.seq(b0 + tid, st);
                s_sum[tid] = mine.q_len > 0 ? item_steps(item_hi(l, mine, 0)) + kItemCost : 0;
            }
            __syncthreads();
            return;
        }
        for (int i = warp; i < T && b0 + i < l.batch; i += kWarps) {
            const kv::Seq s = p.seq(b0 + i, lane == 0 ? st : nullptr);
            const long long n = seq_units(l, s, item_count(l, s));
            if (lane == 0) s_sum[i] = n;
        }
        __syncthreads();
    };
    long long sum = 0, total;
    for (int b0 = 0; b0 < l.batch; b0 += T) {
        sums(b0, me.at == 0 ? status : nullptr);
        if (b0 + tid < l.batch) sum += s_sum[tid];
        if (b0 + T < l.batch) __syncthreads();
    }
    kv::block_scan<T>(sum, total, s_warp);
    const long long W = total * l.blocks;
    const int C = kv::used_ctas(me.of, W);
    if (me.at >= C) return false;
    const long long u0 = kv::unit_start(me.at, C, W), u1 = kv::unit_start(me.at + 1, C, W);
    long long base = 0;
    for (int b0 = 0; b0 < l.batch; b0 += T) {
        if (l.batch > T) {  // the sums of the last round are not these
            __syncthreads();
            sums(b0, nullptr);
        }
        const long long n = b0 + tid < l.batch ? s_sum[tid] * l.blocks : 0;
        const long long at = base + kv::block_scan<T>(n, total, s_warp);
        if (u0 >= at && u0 < at + n) {
            s_walk->b = b0 + tid;
            s_walk->left = u0 - at;  // for now: the start within the sequence
            if (single) {
                const uint32_t from = (uint32_t)(u0 - at), per = (uint32_t)s_sum[tid];  // below 2^16 blocks of 2^24 units
                const long long block = l.blocks == 1 ? 0 : (u0 - at) >> 32 ? (u0 - at) / per : from / per;
                s_walk->block = (int)block, s_walk->qt = 0, s_walk->n_qt = 1, s_walk->at = (int)(u0 - at - block * per), s_walk->sq = mine;
                s_walk->left = u1 - u0;
            }
        }
        base += total;
        if (base > u0) break;
    }
    __syncthreads();
    if (warp == 0 && !single) {
        const int b = s_walk->b;
        const kv::Seq s = p.seq(b, nullptr);
        const int n_qt = item_count(l, s);
        const long long per = seq_units(l, s, n_qt), from = s_walk->left;
        // (a 64-bit division takes longer than the rest)
        const int block = (from | per) >> 32 ? (int)(from / per) : (int)((uint32_t)from / (uint32_t)per);
        const long long rem = from - block * per;
        long long before = 0;
        int qt = -1, at = 0;
        for (int q0 = 0; q0 < n_qt && qt < 0; q0 += 32) {
            const int n = q0 + lane < n_qt ? item_steps(item_hi(l, s, q0 + lane)) + kItemCost : 0;  // 32 of them: below 2^30
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            const long long r = rem - before;
            const unsigned hit = __ballot_sync(~0u, n > 0 && r >= x - n && r < x);
            if (hit) {
                const int k = __ffs(hit) - 1;
                qt = q0 + k;
                at = (int)(r - __shfl_sync(~0u, x - n, k));
            }
            before += __shfl_sync(~0u, x, 31);
        }
        __syncwarp();
        if (lane == 0) {
            s_walk->block = block, s_walk->qt = qt, s_walk->n_qt = n_qt, s_walk->at = at, s_walk->sq = s;
            s_walk->left = u1 - u0;
        }
    }
    __syncthreads();
    w = *s_walk;
    return true;
}

// A place in a ring of N and the phase of its barriers.
template <int N>
struct Turn {
    int at = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) at = 0, ph ^= 1;
    }
};

struct PartRing {
    Part part[kParts];
    uint64_t full[kParts], empty[kParts];
};

// Takes the next part; the whole warp calls. False at the end (or when the wait ran out: ok).
__device__ __forceinline__ bool take(PartRing &ring, uint32_t &n, Part &w, bool &ok) {
    const uint32_t e = n % kParts;
    ok = warp_wait(&ring.full[e], (n / kParts) & 1);
    if (!ok) return false;
    w = ring.part[e];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) bar_arrive(&ring.empty[e]);
    n++;
    return __shfl_sync(~0u, w.steps, 0) > 0;
}

// Hands out all parts of the walk and leaves what the joining kernel needs; the whole warp calls. False when a wait ran out.
template <class P>
__device__ __forceinline__ bool hand_out(const P &p, PartRing &ring, Walk<P> &walk) {
    const int lane = threadIdx.x & 31;
    int4 join = make_int4(0, 0, 0, kv::kJoinNone);
    bool ok = true, more = true;
    for (uint32_t n = 0; more; n++) {
        if (n >= kParts && !warp_wait(&ring.empty[n % kParts], (n / kParts - 1) & 1)) {
            ok = false;
            break;
        }
        Part w;
        more = walk.next(p, w);
        if (more && (w.first > 0 || w.last < w.steps)) {
            if (w.first == 0)
                join.x = w.left, join.y = w.block, join.z = w.token;
            else
                join.w = w.last == w.steps ? kv::kJoinEnd : kv::kJoinOn;
        }
        __syncwarp();
        if (lane == 0) {
            ring.part[n % kParts] = w;
            bar_arrive(&ring.full[n % kParts]);
        }
        __syncwarp();
    }
    if (lane == 0 && p.line.join) p.line.join[where(p.line).id] = join;
    return ok;
}

}  // namespace latent
}  // namespace ftmoe

// Expanded latent attention on the 5th-generation tensor cores: keys of nope + rope elements (the rope part shared by the
// heads), values of D = nope elements, both as rows. An item is 256 consecutive tokens of one (sequence, head), as two tiles of
// M = 128 that read K and V from shared memory once. Bound by the tensor cores: 2 (nope + rope + D) flops a (token, row) against
// one exponential.
//
// Persistent, one CTA an SM, work cut by latent_line.cuh in steps of 128 rows. The softmax warps work as in kv_chunk.cu: P in
// tensor memory, formed with the maximum of the steps before. Roles:
//   warps 0-3, 4-7  softmax of tile 0 and 1, a thread a token; warps 0-3 also zero the V rows that no token sees in the last step.
//   warp 8          tensor copies (boxes of 128 rows x 64 elements, 128-byte swizzle): K into a ring of such chunks, each with
//                   barriers of its own, as a step's three fill the ring and are needed again soonest; V into a ring of steps; and the queries.
//   warp 9          issues tcgen05.mma, tile 0's and tile 1's in turn: O_t += P_t V, then S_t = Q_t K^T of the next step.
//   warp 11         walks the work and hands the parts out.
// Every wait is bounded; one that runs out is recorded and ends the role.
//
// Measured: a prompt of 4096, 32 heads: 133 us, 1.29 PFLOP/s of the 1.94 of a large library product (tensor pipe 66 % busy: 32 heads x 16
// items of unequal length, their starts and ends, and 6 us of join); 2048 tokens over 25000 rows, 16 heads: 338 us, 1.49 PFLOP/s; five
// chunks of at most 301: 26 us, cold starts of two kernels and a few steps' latency.
#include "latent_line.cuh"

namespace ftmoe {
namespace latent {
namespace {

using kv::add2;
using kv::bar_expect;
using kv::bar_init;
using kv::commit;
using kv::desc_lo;
using kv::ex2;
using kv::fence_after;
using kv::fence_async;
using kv::fence_before;
using kv::fma2;
using kv::from_f2;
using kv::max3;
using kv::mma_ss;
using kv::mma_ts;
using kv::pack2;
using kv::tm_ld32;
using kv::tm_ld64;
using kv::tm_ld_wait;
using kv::tm_st16;
using kv::tm_st32;
using kv::tm_st_wait;
using kv::tma3;
using kv::unpack2;
using kv::wait_bar;

constexpr int kWarps = 12, kThreads = kWarps * 32, kRows = 256, kTileSlots = kStep;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kWalkWarp = 11;
constexpr float kSlack = 8.f;
// The largest sum of 64 P that is let through: P below it is finite in its type, sums in fp32.
template <bool BF>
constexpr float kMost = BF ? 18446744073709551616.f : 16384.f;
constexpr int kChunk = kTileSlots * 128;

template <int D>
struct Shape {
    static constexpr int kK = D / 64 + 1, kV = D / 64;  // chunks of a step
    static constexpr int kKRing = D == 128 ? 3 : 6, kVRing = D == 128 ? 2 : 3;  // chunks of K, whole steps of V
    static constexpr int kQ = 2 * kK * kChunk;
    static constexpr int kOut = 8 * 32 * 64;  // a warp's 32 output rows, 32 elements at a time; the plan's sums before
    static constexpr int kSmem = 1024 + (kKRing + kVRing * kV) * kChunk + kQ + kOut;
    static constexpr uint32_t kO = 256, kP = D == 128 ? 0 : 384;  // columns of O_0 and P_0
    static constexpr uint32_t kPStep = D == 128 ? 128 : 64;       // from P_0 to P_1
};
constexpr int kMaxK = 6, kMaxV = 3;

struct Maps {
    CUtensorMap q, k, key, v;
};
struct Bars {
    uint64_t k_full[kMaxK], k_empty[kMaxK], v_full[kMaxV], v_empty[kMaxV];
    uint64_t qfull, qempty, s[2], p[2][2], half[2], o[2], done;
};

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
__global__ void __launch_bounds__(kThreads, 1) expand_kernel(const __grid_constant__ ExpandParams p, const __grid_constant__ Maps maps) {
    using S = Shape<D>;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ Bars bar;
    __shared__ PartRing parts;
    __shared__ uint32_t s_tmem;
    __shared__ long long s_warp[kWarps];
    __shared__ Walk<ExpandParams> s_walk;
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;  // (uniform, for the products' descriptors)
    const uint32_t ks = (su32(sm_raw) + 1023u) & ~1023u, vs = ks + S::kKRing * kChunk, qs = vs + S::kVRing * S::kV * kChunk, stage_out = qs + S::kQ;

    if (tid == 0) {
        for (int i = 0; i < S::kKRing; i++) bar_init(&bar.k_full[i], 1), bar_init(&bar.k_empty[i], 1);
        for (int i = 0; i < S::kVRing; i++) bar_init(&bar.v_full[i], 1), bar_init(&bar.v_empty[i], 1);
        for (int i = 0; i < kParts; i++) bar_init(&parts.full[i], 1), bar_init(&parts.empty[i], 10);  // softmax, copies, products
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
    Walk<ExpandParams> walk;
    bool any = true;
    if (!plans_alone(p.line))
        any = plan<kWarps>(p, walk, s_warp, reinterpret_cast<long long *>(sm_raw + (stage_out - su32(sm_raw))), &s_walk, p.status);
    else if (warp == kWalkWarp)
        plan_alone(p, walk, p.status);
    asm volatile("griddepcontrol.launch_dependents;" :::);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tm = *reinterpret_cast<volatile uint32_t *>(&s_tmem);
    if (!any) {  // the whole CTA
        if (tid == 0 && p.line.join) p.line.join[where(p.line).id] = make_int4(0, 0, 0, kv::kJoinNone);
        if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
        return;
    }
    bool ok = true;
    Part w;
    uint32_t n_part = 0;

    // registers: 384 threads x 168 at launch = 256 x 208 + 128 x 88
    if (warp < 8) {  // ---------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tm + lanes + 128 * t, tO = tm + lanes + S::kO + D * t, tP = tm + lanes + S::kP + S::kPStep * t;
        const float c2 = p.scale * kv::kLog2e;
        const int row_i = tid;  // this thread's token of the item
        uint32_t ns = 0, no = 0, step = 0;  // step: steps of this CTA, both tiles' or not
        while (take(parts, n_part, w, ok)) {
            if (w.left <= t * 128) continue;  // the second tile has no tokens
            const bool live = row_i < w.left;
            const int at = w.slot + row_i;
            const int end = !live || at < 0 ? 0 : (p.causal ? at + 1 : w.kv_len);
            float m = live ? -INFINITY : 0.f, l = 0.f, up = 1.f;  // rows that are none stay at P = 0
            bool raise = false;  // O is to be multiplied by up
            for (int j = w.first; j < w.last && ok; j++, ns++, step++) {
                const int s0 = j * kTileSlots;
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
                const bool cut = __any_sync(~0u, end < s0 + kTileSlots);
                // slots that the row does not see, in the groups of 32 that some row of the warp does not see whole
                auto hide = [&](int q) {
#pragma unroll
                    for (int g = 64 * q; g < 64 * q + 64; g += 32) {
                        const int e = end - s0 - g;
                        if (__any_sync(~0u, e < 32)) {
#pragma unroll
                            for (int k = 0; k < 32; k++)
                                if (k >= e) x[g + k] = 0xff800000u;
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
                if (t == 0 && s0 + kTileSlots > w.hi) {  // V of rows that no token sees: what they hold must not reach 0 * V
                    const int r0 = w.hi > s0 ? w.hi - s0 : 0, place = step % S::kVRing;
                    if (!warp_wait(&bar.v_full[place], (step / S::kVRing) & 1)) ok = false;
                    for (int i = tid; i < (kTileSlots - r0) * 8 * S::kV; i += 128) {
                        const int c = i / ((kTileSlots - r0) * 8), r = i - c * ((kTileSlots - r0) * 8);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vs + (place * S::kV + c) * kChunk + r0 * 128 + r * 16), "r"(0) : "memory");
                    }
                    fence_async();
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
            const bool whole = w.first == 0 && w.last == w.steps;
            const int64_t token = w.token + row_i;
            const int part = 2 * blockIdx.x + (w.first == 0 ? 1 : 0);
            float f = raise ? up : 1.f;
            if (whole) f = l == 0.f ? 0.f : f / l;
            // 32 elements of the warp's rows at a time, in a loop: run once an item, unrolled code took most of its
            // time to be fetched
            const uint32_t st = stage_out + warp * 2048;
            uint16_t *out = p.out.d + (int64_t)(w.token + 32 * warp) * p.out.token + w.block * p.out.head;
            const int rows = w.left - 32 * warp;  // of this warp's 32
            float *po = p.part_o + (int64_t)part * kRows * D + tid;
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
                        uint4 z;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(z.x), "=r"(z.y), "=r"(z.z), "=r"(z.w)
                                     : "r"(st + r * 64 + (((lane ^ (r >> 1)) & 3) << 4))
                                     : "memory");
                        if (r < rows) *reinterpret_cast<uint4 *>(out + r * p.out.token + k + 8 * (lane & 3)) = z;
                    }
                    __syncwarp();
                } else {  // parts are kept element by element, rows consecutive: a warp's store is one line
#pragma unroll
                    for (int e = 0; e < 32; e++) po[(k + e) * kRows] = __uint_as_float(y[e]) * f;
                }
            }
            if (!whole)
                p.part_ml[(int64_t)part * kRows + tid] = make_float2(m, l);
            else if (live && p.lse)
                p.lse[token * p.heads + w.block] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            fence_before();  // O is read before the next item's first P is announced
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    }
    if (warp == kCopyWarp) {  // ---------------------------------------------- K, V and the queries
        Turn<S::kKRing> k;
        Turn<S::kVRing> v;
        uint32_t nq = 0;
        const bool lead = lane == 0;
        while (ok && take(parts, n_part, w, ok)) {
            const int row0 = p.first_row(w.b);
            for (int j = w.first; j < w.last && ok; j++) {
                const int row = row0 + j * kTileSlots;
                for (int c = 0; c < S::kK; c++, k.next()) {
                    ok = ok && warp_wait(&bar.k_empty[k.at], k.ph ^ 1);
                    if (!ok) break;
                    if (lead) {
                        bar_expect(&bar.k_full[k.at], kChunk);
                        if (c == S::kK - 1)
                            tma3(ks + k.at * kChunk, &maps.key, 0, row, 0, &bar.k_full[k.at]);
                        else
                            tma3(ks + k.at * kChunk, &maps.k, 64 * c, w.block, row, &bar.k_full[k.at]);
                    }
                    __syncwarp();
                }
                if (ok && j == w.first) {  // the item's queries, after its first K
                    if (nq > 0 && !warp_wait(&bar.qempty, (nq - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    nq++;
                    const int n = (w.left > 128 ? 2 : 1) * S::kK;
                    if (lead) bar_expect(&bar.qfull, n * kChunk);
                    __syncwarp();
                    if (lane < n) tma3(qs + lane * kChunk, &maps.q, 64 * (lane % S::kK), w.block, w.token + 128 * (lane / S::kK), &bar.qfull);
                }
                ok = ok && warp_wait(&bar.v_empty[v.at], v.ph ^ 1);
                if (!ok) break;
                if (lead) bar_expect(&bar.v_full[v.at], S::kV * kChunk);
                __syncwarp();
                if (lane < S::kV) tma3(vs + (v.at * S::kV + lane) * kChunk, &maps.v, 64 * lane, w.block, row, &bar.v_full[v.at]);
                v.next();
            }
        }
        if (!ok) {  // wait (bounded) until the copies already issued have landed
            for (int i = 0; i < S::kKRing; i++, k.next()) wait_bar(&bar.k_full[k.at], k.ph ^ 1);
            for (int i = 0; i < S::kVRing; i++, v.next()) wait_bar(&bar.v_full[v.at], v.ph ^ 1);
            if (nq > 0) wait_bar(&bar.qfull, (nq - 1) & 1);
        }
    } else if (warp == kMmaWarp) {  // -------------------------------------- products
        constexpr uint32_t IS = kv::kInstr<BF, kTileSlots, false>, IO = kv::kInstr<BF, D, true>;
        const uint32_t one = kv::elect_one();
        const uint32_t qd = desc_lo(qs, 16), kd = desc_lo(ks, 16), vd = desc_lo(vs, kChunk);
        const int rope_steps = p.rope >> 4;
        uint32_t np = 0, ni = 0;  // bit t of np: the phase of tile t's P
        Turn<S::kKRing> k;
        Turn<S::kVRing> v;
        // Loops, not unrolled code: fetching instructions between the softmax's long code took longer than the products.
        auto scores = [&](int t, bool last) {  // over the K chunks from k on; `last`: their last use
            uint32_t a = qd + t * (S::kK * kChunk / 16), acc = 0;
            Turn<S::kKRing> at = k;
#pragma unroll 1
            for (int e = 0; e < S::kK; e++, at.next()) {
                ok = ok && warp_wait(&bar.k_full[at.at], at.ph);
                if (!ok) return;
                fence_after();
                const uint32_t b = kd + at.at * (kChunk / 16);
                if (e < S::kK - 1) {
#pragma unroll
                    for (int i = 0; i < 4; i++, acc = 1) mma_ss<IS>(one, tm + 128 * t, a + 2 * i, b + 2 * i, acc);
                } else {
#pragma unroll 1
                    for (int i = 0; i < rope_steps; i++) mma_ss<IS>(one, tm + 128 * t, a + 2 * i, b + 2 * i, 1);
                }
                a += kChunk / 16;
                if (last) commit(one, &bar.k_empty[at.at]);
            }
            commit(one, &bar.s[t]);
            if (last) k = at;
        };
        auto values = [&](int t, uint32_t acc) {
            uint32_t b = vd + v.at * (S::kV * kChunk / 16), a = tm + S::kP + S::kPStep * t;
#pragma unroll 1
            for (int q = 0; q < 2; q++) {
                ok = ok && warp_wait(&bar.p[t][q], (np >> t) & 1);
                if (!ok) return;
                fence_after();
#pragma unroll
                for (int i = 0; i < 4; i++, acc = 1) mma_ts<IO>(one, tm + S::kO + D * t, a + 8 * i, b + i * (2048 / 16), acc);
                if (q == 0) commit(one, &bar.half[t]);
                a += 32, b += 4 * 2048 / 16;
            }
            np ^= 1 << t;
        };
        while (ok && take(parts, n_part, w, ok)) {
            // uniform values keep the loop's addresses in uniform registers
            const int n = __shfl_sync(~0u, w.last - w.first, 0), two = __shfl_sync(~0u, w.left > 128 ? 1 : 0, 0);
            ok = warp_wait(&bar.qfull, ni++ & 1);
            if (!ok) break;
            fence_after();
#pragma unroll 1
            for (int t = 0; t <= two && ok; t++) scores(t, t == two);
            if (n == 1) commit(one, &bar.qempty);
#pragma unroll 1
            for (int j = 0; j < n && ok; j++) {  // O_t += P_t V_j, S_t = Q_t K_{j+1}
                ok = warp_wait(&bar.v_full[v.at], v.ph);
                const bool more = j + 1 < n;
#pragma unroll 1
                for (int t = 0; t <= two && ok; t++) {
                    values(t, j > 0);
                    if (!ok) break;
                    if (t == two) commit(one, &bar.v_empty[v.at]);
                    if (more)
                        scores(t, t == two);
                    else
                        commit(one, &bar.o[t]);
                }
                v.next();
                if (j + 2 == n) commit(one, &bar.qempty);
            }
        }
        commit(one, &bar.done);  // every product is done when this arrives
        warp_wait(&bar.done, 0);
    } else if (warp == kWalkWarp) {
        ok = hand_out(p, parts, walk);
    }
    if (!ok && lane == 0) kv::flag(p.status, FTMOE_ERR_STATE);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
}

// Joins the parts of the item that CTA c of the kernel before started. A CTA takes 32 tokens, a lane a token
// and a warp an eighth of the elements; rows go out through shared memory.
constexpr int kJoinThreads = 256, kJoinRows = 32;

template <bool BF, int D>
__global__ void __launch_bounds__(kJoinThreads) expand_combine(const ExpandParams p) {
    constexpr int E = D / 8;  // elements a thread
    __shared__ __align__(16) uint16_t s_out[kJoinRows][D + 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 join = p.line.join[c];
    const int row0 = blockIdx.y * kJoinRows, row = row0 + lane;
    if (row0 >= join.x) return;
    const bool live = row < join.x;
    const int n = kv::count_parts(p.line.join, c, gridDim.x);
    // the first four parts, which are mostly all, load at once
    constexpr int K = 4;
    auto slot = [&](int k) { return (int64_t)(2 * (c + k) + (k == 0)); };
    auto part = [&](int k) { return p.part_o + (slot(k) * D + warp * E) * kRows + row; };
    float2 ml[K];
    float v[K][E], M = -INFINITY, L = 0.f, x[E];
#pragma unroll
    for (int k = 0; k < K; k++) {
        ml[k] = k < n ? p.part_ml[slot(k) * kRows + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; e++) v[k][e] = k < n ? part(k)[e * kRows] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; k++) M = fmaxf(M, ml[k].x);
    for (int k = K; k < n; k++) M = fmaxf(M, p.part_ml[slot(k) * kRows + row].x);
#pragma unroll
    for (int e = 0; e < E; e++) x[e] = 0.f;
    auto add = [&](float2 y, const float *o, int step) {
        const float a = y.x == -INFINITY ? 0.f : ex2(y.x - M);
        L += y.y * a;
#pragma unroll
        for (int e = 0; e < E; e++) x[e] += o[e * step] * a;
    };
#pragma unroll
    for (int k = 0; k < K; k++) add(ml[k], v[k], 1);
    for (int k = K; k < n; k++) add(p.part_ml[slot(k) * kRows + row], part(k), kRows);
    const float f = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(&s_out[lane][warp * E + e]) = from_f2<BF>(x[e] * f, x[e + 1] * f);
    if (warp == 0 && live && p.lse)
        p.lse[(int64_t)(join.z + row) * p.heads + join.y] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    __syncthreads();
    for (int k = threadIdx.x; k < kJoinRows * D / 8; k += kJoinThreads) {
        const int r = k / (D / 8), ch = k % (D / 8);
        if (row0 + r < join.x)
            *reinterpret_cast<uint4 *>(p.out.d + (int64_t)(join.z + row0 + r) * p.out.token + join.y * p.out.head + 8 * ch) =
                *reinterpret_cast<const uint4 *>(&s_out[r][8 * ch]);
    }
}

template <bool BF, int D>
cudaError_t launch(const ExpandParams &p, int C, cudaStream_t st) {
    using S = Shape<D>;
    Maps m;
    const bool keys = p.rows > 0;  // (without one, no chunk's rows are ever seen)
    const void *some = p.q.d;
    if (!kv::box_map(m.q, BF, p.q.d, {p.nope + p.rope, p.heads, p.tokens}, 2 * p.q.head, 2 * p.q.token, {64, 1, 128}, true) ||
        !kv::box_map(m.k, BF, keys ? p.k.d : some, {p.nope, p.heads, keys ? p.rows : 1}, keys ? 2 * p.k.head : 16, keys ? 2 * p.k.token : 16, {64, 1, 128}, true) ||
        !kv::box_map(m.v, BF, keys ? p.v.d : some, {p.vdim, p.heads, keys ? p.rows : 1}, keys ? 2 * p.v.head : 16, keys ? 2 * p.v.token : 16, {64, 1, 128}, true) ||
        !kv::box_map(m.key, BF, keys ? p.key : some, {p.rope, keys ? p.rows : 1, 1}, keys ? 2 * p.key_stride : 16, keys ? 2 * p.key_stride : 16, {64, 128, 1}, true))
        return cudaErrorInvalidValue;
    cudaError_t rc = kv::allow_smem<expand_kernel<BF, D>>(S::kSmem);
    if (rc != cudaSuccess) return rc;
    expand_kernel<BF, D><<<C, kThreads, S::kSmem, st>>>(p, m);
    if ((rc = cudaGetLastError()) != cudaSuccess || !p.line.join) return rc;
    return kv::launch_after(expand_combine<BF, D>, dim3(C, kRows / kJoinRows), kJoinThreads, 0, st, p);
}

int64_t most_items(const ExpandParams &p) { return (int64_t)((p.max_q + kRows - 1) / kRows) * p.batch * p.heads; }
// 8 items of two steps 10.9 us cut, 9.2 whole, of four 11.4 and 12.8; 64 of eight steps 23.9 and 20.8, of 16 steps 32.0 and 34.0; 152 of 16
// steps 38.9 and 35.5; 304 of four, two waves, 34.7 and 36.5.
bool cut(const ExpandParams &p, int num_sms) { return cut_pays(most_items(p), ((int64_t)p.max_kv + kStep - 1) / kStep, num_sms, 1, 1); }
int ctas(const ExpandParams &p, int num_sms) {
    const int64_t items = most_items(p);
    if (!cut(p, num_sms)) return (int)items;
    const int64_t most = items < num_sms ? items * (p.max_kv / kStep + 1 + kItemCost) : num_sms;
    return (int)(most < num_sms ? (most > 0 ? most : 1) : num_sms);
}

}  // namespace

size_t expand_workspace(ExpandParams &p, int num_sms, unsigned char *base) {
    p.line.batch = p.batch, p.line.blocks = p.heads, p.line.item_tokens = kRows, p.line.max_q = p.max_q, p.line.causal = p.causal;
    p.line.pair = 0, p.line.join = nullptr, p.part_o = nullptr, p.part_ml = nullptr;
    if (!cut(p, num_sms)) return 0;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char *at = base ? base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t C = ctas(p, num_sms), n = 2 * C * kRows;  // a part that starts an item and one that goes on with one for each CTA
    p.part_o = reinterpret_cast<float *>(take(n * p.vdim * 4));
    p.part_ml = reinterpret_cast<float2 *>(take(n * 8));
    p.line.join = reinterpret_cast<int4 *>(take(C * 16));
    return off;
}

cudaError_t launch_expand(const ExpandParams &p, bool bf16, int num_sms, cudaStream_t st) {
    const int C = ctas(p, num_sms);
    if (p.vdim == 64) return bf16 ? launch<true, 64>(p, C, st) : launch<false, 64>(p, C, st);
    return bf16 ? launch<true, 128>(p, C, st) : launch<false, 128>(p, C, st);
}

}  // namespace latent
}  // namespace ftmoe

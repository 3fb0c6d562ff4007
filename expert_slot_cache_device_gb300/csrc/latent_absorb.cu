// Absorbed latent attention on the 5th-generation tensor cores. All heads read the same cached vectors, so the rows of an
// item are (token, head) pairs, NR = 16, 32 or 64 of them, and a tile is 128 slots (64 of an 8-bit cache). Both products have the
// cache as their A operand, straight from shared memory in the one layout that the copies leave it in:
//   S^T [slots, NR rows]   = [C | K] [Q | Q_rope]^T    A: slots are M, latents K (K-major)
//   O^T [latent, NR rows] += C^T P^T                   A: latents are M = 128, slots K (M-major)
// so that O takes latent / 128 * NR columns of tensor memory (256 of 512 at most), and few rows cost few columns instead of an
// unused part of M = 128. (128 rows would take all 512 columns for O and leave none for S.) P^T goes to shared memory as B.
//
// Persistent, one CTA an SM, work cut by latent_line.cuh. Roles:
//   warps 0-3   (64 rows: 8-11 too, which take the last 32) softmax of a tile: a warp has a quarter of the slots, a thread four (two)
//               slots of every eighth pair of rows. P = 2^(s scale log2 e - m) in fp32 with the maximum m of the tiles before; one vote tells
//               whether a P is above 2^8, and only then maxima are taken across the slots, m is raised and O multiplied. P is rounded to
//               the cache's type, as the tensor cores take it; the sums are of P in fp32, kept by each thread for its slots and added at
//               the item's end.
//   warp 4      (16 bits) tensor copies of units of 64 latents of a tile (128-byte swizzle), a lane each: one lane after another, with a wait
//               each, they took 450 cycles a unit and held everything up. Then the next tile's prefetch to L2.
//   warp 5      issues tcgen05.mma. The warp's number comes from a shuffle, by which the compiler knows its branches to be uniform and
//               keeps descriptors in uniform registers (without: 70 cycles a product).
//   warp 6      walks the work and hands the parts out.
//   warp 7      tensor copies of queries and rotary parts.
//   warps 8-15  (8 bits, instead of warp 4) load codes and powers, a warp a unit, and turn them into elements. Codes stay in registers on
//               their way: shared memory has no place for more than a quarter of a tile's, which let too few be under way.
// Every wait is bounded; one that runs out is recorded and ends the role.
//
// Measured: 48 sequences of 9000 tokens, 128 heads: 94 us with the join, 3.2 TB/s of the 6.8 of a plain copy (this kernel alone: 3.4, DRAM
// read once, 307 MB, the tensor pipe 34 % busy). Shared memory holds one tile (128 KB) beside 72 KB of queries, so an SM's time is the chain of a
// tile: its scores (36 products of 50 cycles: M128 N64 runs no faster), softmax, outputs (32), and the refill behind them. 8 bits, 96
// of 7000, 32 heads: 98 us, 2.3 TB/s; there the chain is conversion (about 1500 cycles of 64 slots), scores, softmax, outputs over two places,
// and shared memory passes 4 KB a slot, half its bandwidth over the call. More than 32 rows are blocks of 32 in 8 bits, each of which converts the
// cache for itself: 48 of 9000, 64 heads 126 us, 128 heads 229. One sequence of 777: 12 us, latency (launch, plan, one tile, join).
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
using kv::mma_ss;
using kv::pack2;
using kv::tma3;
using kv::unpack2;
using kv::wait_bar;

constexpr int kCopyWarp = 4, kMmaWarp = 5, kWalkWarp = 6, kRopeWarp = 7, kConvWarps = 8;
constexpr float kMost = 256.f;   // P that is let through without raising m
constexpr float kLeast = 5.9604645e-8f;  // 2^-24

template <bool Q8, int NR>
struct Shape {
    // Softmax warps, and the columns (rows of the item) of each: of 64 columns a warp takes half, two warps a quarter of the lanes
    // (48 x 9000 tokens, 128 heads: 93.4 us, 99.3 with all 64 in one).
    static constexpr int kCols = NR == 64 ? 32 : NR, kSoft = 4 * NR / kCols;
    static constexpr int kWarps = Q8 ? 16 : 4 + kSoft, kThreads = kWarps * 32;
    // Slots of a tile. 128 issue the fewest products (16 heads, 64 x 2000: 39 us, 46 with 64; 64 rows, 48 x 9000: 94, 113 with 64 slots
    // and four softmax warps). Of codes 64, with places for two tiles: one is turned into elements while the other is worked on (98 us,
    // 108 with 128), and its scores are formed during the other's softmax (104 without).
    static constexpr int kTile = Q8 ? 64 : 128, kHalves = kTile / 64;
    static constexpr bool kTwo = Q8;
    static constexpr int kUnit = kTile * 128;   // 64 latents of a tile's slots
    static constexpr int kUnits = Q8 ? 16 : 8;  // places for them; two are an operand of the second product
    static constexpr int kRopes = NR == 64 ? 1 : 2;
    static constexpr int kQ = 9 * NR * 128;
    // P lies over the rotary part, which S has read by then, where shared memory would not hold both
    static constexpr bool kOver = NR == 64;
    static constexpr int kPOne = NR * 2 * kTile, kP = kOver ? 0 : kTwo ? 2 * kPOne : kPOne, kScratch = kOver ? 2048 : 0;
    static constexpr int kSmem = 1024 + kUnits * kUnit + kRopes * kUnit + kQ + kP + kScratch;
    static constexpr uint32_t kS = 256, kSTwo = kTwo ? NR : 0;  // column of S, from one tile's to the next one's; O is at 0
};
constexpr int kMaxRopes = 2;

struct Maps {
    CUtensorMap q, q_rope, lat, rope, all;  // all: whole slots, for prefetches
};

struct Bars {
    uint64_t unit_full[16], pair_empty[8], rope_full[kMaxRopes], rope_empty[kMaxRopes];
    uint64_t qfull, qempty, s[2], p[2], pv, o, done;
};

// Sixteen lanes of tensor memory as fragments: a thread's registers 4 j .. 4 j + 3 are columns 8 j + 2 (lane % 4), + 1 of lane
// lane / 4, then of lane / 4 + 8.
template <int NR>
__device__ __forceinline__ void load_s(uint32_t a, uint32_t *x) {
    if constexpr (NR == 32) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : FTMOE_R4(x, 0), FTMOE_R4(x, 4), FTMOE_R4(x, 8), FTMOE_R4(x, 12)
            : "r"(a)
            : "memory");
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : FTMOE_R4(x, 0), FTMOE_R4(x, 4)
            : "r"(a)
            : "memory");
    }
}
// 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : FTMOE_R4(x, 0), FTMOE_R4(x, 4), FTMOE_R4(x, 8), FTMOE_R4(x, 12)
        : "r"(a)
        : "memory");
}

// Barrier of the softmax warps' N threads; true if any thread brings it.
template <int N>
__device__ __forceinline__ bool vote_of(bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)mine), "n"(N)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float ld_f(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void st_f(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory"); }

// Out of line: rare, and copies of it between the plain ones' cost instruction fetches.
template <bool BF>
__device__ __noinline__ void decode16_far(const uint4 u, uint32_t byte, uint4 &lo, uint4 &hi) {
    decode16_floats<BF>(u, byte, lo, hi);
}
__device__ __forceinline__ void prefetch(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
constexpr int kWide = 192;  // 16-bit elements of a slot that one prefetch has

// Tiles of a part.
template <int kTile>
struct Tiles {
    int first, last;
    __device__ __forceinline__ explicit Tiles(const Part &w) {
        first = w.first * (kStep / kTile), last = w.last * (kStep / kTile);
        const int end = (w.hi + kTile - 1) / kTile;
        if (last > end) last = end > first ? end : first + 1;
    }
};

template <bool BF, bool Q8, int NR>
__global__ void __launch_bounds__((Shape<Q8, NR>::kThreads), 1) absorb_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ Maps maps) {
    using S = Shape<Q8, NR>;
    constexpr int kTile = S::kTile, kUnit = S::kUnit, kUnits = S::kUnits;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ Bars bar;
    __shared__ PartRing parts;
    __shared__ uint32_t s_tmem;
    __shared__ long long s_warp[S::kWarps];
    __shared__ Walk<AttendParams> s_walk;
    __shared__ uint16_t s_tok[NR];  // token of a row in its item
    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid >> 5, 0), lane = tid & 31;  // (uniform, for the products' descriptors)
    const uint32_t units = (su32(sm_raw) + 1023u) & ~1023u, ropes = units + kUnits * kUnit;
    const uint32_t qs = ropes + S::kRopes * kUnit, ps = S::kOver ? ropes : qs + S::kQ, scratch = S::kOver ? qs + S::kQ : ps;
    const int L = p.c.latent >> 6;  // units of a tile
    const int pair = p.line.pair, rank = pair & blockIdx.x;

    if (tid == 0) {
        for (int i = 0; i < kUnits; i++) bar_init(&bar.unit_full[i], 1);
        for (int i = 0; i < kUnits / 2; i++) bar_init(&bar.pair_empty[i], 1);
        for (int i = 0; i < S::kRopes; i++) bar_init(&bar.rope_full[i], 1), bar_init(&bar.rope_empty[i], 1);
        for (int i = 0; i < kParts; i++) bar_init(&parts.full[i], 1), bar_init(&parts.empty[i], S::kSoft + (Q8 ? 2 + kConvWarps : 3));
        bar_init(&bar.qfull, 1), bar_init(&bar.qempty, 1), bar_init(&bar.pv, 1), bar_init(&bar.o, 1), bar_init(&bar.done, 1);
        for (int i = 0; i < 2; i++) bar_init(&bar.s[i], 1), bar_init(&bar.p[i], S::kSoft);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kCopyWarp && lane < 5 && (lane != 2 || !Q8))  // (their first use would wait for them)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps) + lane * sizeof(CUtensorMap)) : "memory");
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&s_tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    const int used = p.heads * p.line.item_tokens;  // rows of an item
    if (tid < NR) s_tok[tid] = tid < used ? tid / p.heads : 0;
    // rows past those are zeros: no copy writes them
    for (int i = tid; i < 9 * (NR - used) * 8; i += S::kThreads) {
        const int c = i / ((NR - used) * 8), r = i - c * ((NR - used) * 8);
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(qs + c * NR * 128 + used * 128 + r * 16), "r"(0) : "memory");
    }
    Walk<AttendParams> walk;
    bool any = true;
    if (!plans_alone(p.line))
        any = plan<S::kWarps>(p, walk, s_warp, reinterpret_cast<long long *>(sm_raw + (ps - su32(sm_raw))), &s_walk, p.c.status);
    else if (warp == kWalkWarp)
        plan_alone(p, walk, p.c.status);
    fence_async();  // of the zeros above, and of the plan's sums, over which tensor copies may go
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

    const int wide = ((rope_at(p.c.latent, p.c.bits) >> 1) + p.c.rope + kWide - 1) / kWide;  // copies of kWide elements of a slot: 4 at most

    if (warp < 4 || (S::kSoft == 8 && warp >= 8)) {  // ---------------------------------------------------- softmax
        constexpr int W = S::kCols, kThreads = 32 * S::kSoft;
        auto vote = [](bool mine) { return vote_of<kThreads>(mine); };
        // quarter of the lanes, first column, thread of the group
        const int quarter = warp & 3, half = S::kSoft == 8 ? warp >> 3 : 0, cb = half * W, st = half * 128 + (tid & 127);
        const uint32_t lanes = tm + ((uint32_t)(32 * quarter) << 16);
        const float c2 = p.scale * kv::kLog2e;
        const int row0 = kTile / 4 * quarter + (lane >> 2), col0 = cb + 2 * (lane & 3);
        constexpr int NB = W / 8;
        uint32_t ns = 0, no = 0;
        while (!vote(!take(parts, n_part, w, ok))) {
            const Tiles<kTile> tl(w);
            const int block = (w.block << pair) + rank;
            const bool dead = w.left < p.line.item_tokens;  // some of the item's tokens are none
            auto limit = [&](int c) {                       // slots that row c sees
                const int t = s_tok[c], at = w.slot + t;
                return t >= w.left || at < 0 ? 0 : (p.line.causal ? at + 1 : w.kv_len);
            };
            const int least = dead || w.slot < 0 ? 0 : (p.line.causal ? w.slot + 1 : w.kv_len);
            // Rows c and c + 1 of eight i: z = -m, sums of P. m starts at 0: a first tile whose P are neither above 2^8 nor, for any thread
            // and row, all below 2^-24 needs no maximum (bf16: P keeps its precision there; f16 would lose it below 2^-14).
            float z[2 * NB];
            uint64_t l[NB];
#pragma unroll
            for (int i = 0; i < NB; i++) z[2 * i] = z[2 * i + 1] = 0.f, l[i] = 0;
            for (int j = tl.first; j < tl.last; j++, ns++) {
                const int s0 = j * kTile;
                const int turn = S::kTwo ? ns & 1 : 0;
                const uint32_t phase = S::kTwo ? ns >> 1 & 1 : ns & 1;
                const uint32_t tS = lanes + S::kS + turn * S::kSTwo + cb, pt = ps + turn * S::kPOne, sp = S::kOver ? scratch : pt;
                ok = ok && warp_wait(&bar.s[turn], phase);
                fence_after();
                constexpr int X = S::kHalves * W / 2;
                uint32_t x[X];  // slots of the warp's first 16 lanes, then of the others
                auto scores = [&] {
                    load_s<W>(tS, x);
                    if (S::kHalves == 2) load_s<W>(tS + (16u << 16), x + X - W / 2);
                    if (s0 + kTile <= least) return;
#pragma unroll
                    for (int k = 0; k < 2 * S::kHalves; k++)
#pragma unroll
                        for (int i = 0; i < NB; i++)
#pragma unroll
                            for (int e = 0; e < 2; e++)
                                if (s0 + row0 + 8 * k >= limit(8 * i + col0 + e)) x[(k >> 1) * (W / 2) + 4 * i + 2 * (k & 1) + e] = 0xff800000u;
                };
                // P in place of the scores; whether one is above 2^8
                auto form = [&] {
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < X; k += 2) {
                        const int i = (k % (W / 2)) >> 2;
                        const float2 f = unpack2(fma2(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), pack2(c2, c2), pack2(z[2 * i], z[2 * i + 1])));
                        const float a = ex2(f.x), b = ex2(f.y);
                        top = kv::max3(top, a, b);
                        x[k] = __float_as_uint(a), x[k + 1] = __float_as_uint(b);
                    }
                    return top > kMost;
                };
                scores();
                const bool fresh = j == tl.first;
                bool raise = form() || !ok || (fresh && !BF);
                if (fresh) {
#pragma unroll
                    for (int i = 0; i < 2 * NB; i++) {
                        const int r = 4 * (i >> 1) + (i & 1);
                        float t = fmaxf(__uint_as_float(x[r]), __uint_as_float(x[r + 2]));
                        if (S::kHalves == 2) t = kv::max3(t, __uint_as_float(x[X - W / 2 + r]), __uint_as_float(x[X - W / 2 + r + 2]));
                        raise = raise || t < kLeast;
                    }
                }
                if (vote(raise)) {
                    if (vote(!ok)) break;
                    scores();
                    // m to at least each row's maximum over the tile
#pragma unroll
                    for (int i = 0; i < 2 * NB; i++) {
                        const int r = 4 * (i >> 1) + (i & 1);
                        float t = fmaxf(__uint_as_float(x[r]), __uint_as_float(x[r + 2]));
                        if (S::kHalves == 2) t = kv::max3(t, __uint_as_float(x[X - W / 2 + r]), __uint_as_float(x[X - W / 2 + r + 2]));
                        t *= c2;
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, o));
                        if (lane < 4) st_f(sp + (quarter * NR + 8 * (i >> 1) + col0 + (i & 1)) * 4, t);
                    }
                    vote(false);
#pragma unroll
                    for (int i = 0; i < NB; i++) {
                        float f[2];
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const uint32_t a = sp + (8 * i + col0 + e) * 4;
                            const float t = fmaxf(fmaxf(ld_f(a), ld_f(a + NR * 4)), fmaxf(ld_f(a + 2 * NR * 4), ld_f(a + 3 * NR * 4)));
                            const float m = -z[2 * i + e], n = fresh ? (t == -INFINITY ? 0.f : t) : fmaxf(m, t);
                            f[e] = fresh ? 0.f : ex2(m - n);
                            z[2 * i + e] = -n;
                            if (quarter == 0 && lane < 4) st_f(a + 4 * NR * 4, f[e]);
                        }
                        const float2 y = unpack2(l[i]);
                        l[i] = pack2(y.x * f[0], y.y * f[1]);
                    }
                    if (S::kTwo && !fresh) ok = warp_wait(&bar.pv, (ns - 1) & 1);  // O holds all P so far (one tile: before this one's S)
                    if (vote(!ok)) break;
                    if (S::kTwo) fence_after();
                    if (!fresh) {
#pragma unroll 1
                        for (int k = 16 * half; k < (L >> 1) * NR; k += 4 * S::kSoft) {
                            uint32_t y[16];
                            tm_ld16(lanes + k, y);
#pragma unroll
                            for (int e = 0; e < 16; e++) y[e] = __float_as_uint(__uint_as_float(y[e]) * ld_f(sp + (4 * NR + (k + e) % NR) * 4));
                            kv::tm_st16(lanes + k, y);
                        }
                        kv::tm_st_wait();
                    }
                    vote(false);  // the scratch has been read
                    form();
                }
#pragma unroll
                for (int h = 0; h < S::kHalves; h++)
#pragma unroll
                    for (int i = 0; i < NB; i += 2) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 2; k++) {  // rows 8 i, then 8 (i + 1); slots, then slots + 8
                            const uint32_t *v = x + h * (W / 2) + 4 * (i + k);
                            const float a = __uint_as_float(v[0]), b = __uint_as_float(v[1]), c = __uint_as_float(v[2]), d = __uint_as_float(v[3]);
                            l[i + k] = add2(l[i + k], add2(pack2(a, b), pack2(c, d)));
                            y[2 * k] = from_f2<BF>(a, b), y[2 * k + 1] = from_f2<BF>(c, d);
                        }
                        // transposed: a row's slots consecutive, 64 in 128 bytes, 16-byte piece c of row r at c ^ (r % 8)
                        const int r = lane & 7, k = lane >> 3;
                        const int piece = 2 * S::kHalves * quarter + 2 * h + (k & 1);
                        const uint32_t at = pt + (piece >> 3) * (NR * 128) + (cb + 8 * (i + (k >> 1)) + r) * 128 + (((piece & 7) ^ r) << 4);
                        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                                     "r"(y[3])
                                     : "memory");
                    }
                if (s0 + kTile > w.hi) {  // latents of slots that no row sees: what they hold must not reach 0 * C
                    const int r0 = w.hi > s0 ? w.hi - s0 : 0;
                    for (int u = 0; u < L; u++) {
                        const uint32_t n = ns * L + u, at = n % kUnits;
                        ok = ok && warp_wait(&bar.unit_full[at], n / kUnits & 1);
                        for (int i = st; i < (kTile - r0) * 8; i += kThreads)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(units + at * kUnit + r0 * 128 + i * 16), "r"(0) : "memory");
                    }
                }
                fence_async();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&bar.p[turn]);
            }
            ok = ok && warp_wait(&bar.o, no++ & 1);
            if (vote(!ok)) break;
            fence_after();
            const bool whole = w.first == 0 && w.last == w.steps;
            const int part = 2 * where(p.line).id + (w.first == 0 ? 1 : 0);
#pragma unroll
            for (int i = 0; i < NB; i++) {
                const float2 y = unpack2(l[i]);
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float t = e ? y.y : y.x;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(~0u, t, o);
                    const int c = 8 * i + col0 + e;
                    if (lane < 4) st_f(scratch + (quarter * NR + c) * 4, t);
                    if (quarter == 0 && lane < 4) st_f(scratch + (5 * NR + c) * 4, -z[2 * i + e]);
                }
            }
            vote(false);
            if (tid < NR) {
                const int c = tid, t = s_tok[c], h = block * p.heads + c - t * p.heads;
                const float sum = (ld_f(scratch + c * 4) + ld_f(scratch + (NR + c) * 4)) + (ld_f(scratch + (2 * NR + c) * 4) + ld_f(scratch + (3 * NR + c) * 4));
                const float top = ld_f(scratch + (5 * NR + c) * 4);
                if (!whole)
                    p.part_ml[(int64_t)part * NR + c] = make_float2(sum == 0.f ? -INFINITY : top, sum);
                else if (p.lse && c < used && t < w.left && h < p.q_heads)
                    p.lse[(int64_t)(w.token + t) * p.q_heads + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
                st_f(scratch + (4 * NR + c) * 4, !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum);
            }
            vote(false);
            // a warp has 32 latents of each 128, a lane one, columns are rows of the item
            if (whole) {  // two lanes swap, so that each writes two latents of one row
                uint16_t *out = p.out.d + (int64_t)w.token * p.out.token + (int64_t)block * p.heads * p.out.head + 32 * quarter + (lane & ~1);
                const int rows = p.line.item_tokens < w.left ? used : w.left * p.heads, heads = p.q_heads - block * p.heads;
#pragma unroll 1
                for (int k = 16 * half; k < NR; k += 4 * S::kSoft) {
                    float f[16];
                    uint16_t *row[8];
#pragma unroll
                    for (int e = 0; e < 16; e++) f[e] = ld_f(scratch + (4 * NR + k + e) * 4);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int r = k + 2 * e + (lane & 1), t = s_tok[r], h = r - t * p.heads;
                        row[e] = r < rows && h < heads ? out + t * p.out.token + h * p.out.head : nullptr;
                    }
#pragma unroll 1
                    for (int u = 0; u < L >> 1; u++) {
                        uint32_t y[16];
                        tm_ld16(lanes + u * NR + k, y);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float a = __uint_as_float(y[e]) * f[e], b = __uint_as_float(y[e + 1]) * f[e + 1];
                            const float got = __shfl_xor_sync(~0u, lane & 1 ? a : b, 1);
                            if (row[e >> 1]) *reinterpret_cast<uint32_t *>(row[e >> 1] + 128 * u) = lane & 1 ? from_f2<BF>(got, b) : from_f2<BF>(a, got);
                        }
                    }
                }
            } else {
                float *po = p.part_o + ((int64_t)part * NR + cb) * p.c.latent + 32 * quarter + lane;
#pragma unroll 1
                for (int u = 0; u < L >> 1; u++) {
                    float *to = po + 128 * u;
                    uint32_t y[W];
                    if constexpr (W == 32)
                        kv::tm_ld32(lanes + u * NR + cb, y);
                    else
                        tm_ld16(lanes + u * NR, y);
#pragma unroll
                    for (int e = 0; e < W; e++, to += p.c.latent) *to = __uint_as_float(y[e]);
                }
            }
            fence_before();  // O is read before the next part's first P is announced
        }
    } else if (!Q8 && warp == kCopyWarp) {  // ------------------------------------- latents
        // four units at a time, eight lanes a unit, a page of the tile each
        const int box = 1 << p.c.page_shift < kTile ? 1 << p.c.page_shift : kTile, boxes = kTile / box;
        const int blk = lane & 7;
        const bool lead = blk == 0, mine = blk < boxes;
        const uint32_t to = units + blk * box * 128;
        uint32_t n = 0, sent = 0;  // units before this tile, those of this tile that went out
        while (ok && take(parts, n_part, w, ok)) {
            const int32_t *tab = p.bt.table + (int64_t)w.b * p.bt.table_stride;
            auto page_at = [&](int j) {
                const int slot = j * kTile + blk * box;
                return mine && slot < w.hi ? tab[slot >> p.c.page_shift] : -1;
            };
            const Tiles<kTile> tl(w);
            int next = page_at(tl.first);
            for (int j = tl.first; j < tl.last && ok; j++, n += L, sent = 0) {
                const int page = (uint32_t)next < (uint32_t)p.c.num_pages ? next : -1;  // (warp 7 records bad ones)
                next = page_at(j + 1);  // on its way while this tile waits for its places
                const int row = (j * kTile + blk * box) & ((1 << p.c.page_shift) - 1);
                const int bytes = __popc(__ballot_sync(~0u, lane < 8 && page >= 0)) * box * 128;  // of a unit
                for (int u0 = 0; u0 < L && ok; u0 += 4) {
                    const int u = u0 + (lane >> 3), at = (n + u) % kUnits, ph = (n + u) / kUnits & 1;
                    uint64_t *free = &bar.pair_empty[at >> 1];
                    // units go out as their places come free, those that are free already together
                    bool todo = u < L;
                    for (int k = 0; k < 5; k++) {
                        const unsigned ready = __ballot_sync(~0u, todo && lead && kv::test_bar(su32(free), ph ^ 1));
                        const bool go = todo && (ready >> (lane & ~7) & 1);
                        if (go && lead) bar_expect(&bar.unit_full[at], bytes);
                        __syncwarp();
                        if (go && page >= 0) tma3(to + at * kUnit, &maps.lat, 64 * u, row, page, &bar.unit_full[at]);
                        sent |= (ready & 1) << u0 | (ready >> 8 & 1) << (u0 + 1) | (ready >> 16 & 1) << (u0 + 2) | (ready >> 24 & 1) << (u0 + 3);
                        todo = todo && !go;
                        const unsigned left = __ballot_sync(~0u, todo);
                        if (!left) break;
                        const int from = __ffs(left) - 1, first = __shfl_sync(~0u, at >> 1, from), phase = __shfl_sync(~0u, ph, from);
                        ok = warp_wait(&bar.pair_empty[first], phase ^ 1);
                        if (!ok) break;
                    }
                }
                // The next tile on its way to L2: shared memory holds one, and what comes from memory only when its places are
                // free comes too late. (After this tile's copies, which would queue behind it.)
                if (lane >> 3 < wide && (uint32_t)next < (uint32_t)p.c.num_pages)
                    prefetch(&maps.all, kWide * (lane >> 3), ((j + 1) * kTile + blk * box) & ((1 << p.c.page_shift) - 1), next);
            }
        }
        if (!ok) {  // wait (bounded) until the copies already issued have landed: each place's last
            for (int i = 0; i < kUnits; i++) {
                int last = -1;
                for (int x = (int)n + i - kUnits; x < (int)n + kUnits; x += kUnits)
                    if (x >= 0 && (x < (int)n || (sent >> (x - n) & 1))) last = x;
                if (last >= 0) wait_bar(&bar.unit_full[last % kUnits], last / kUnits & 1);
            }
        }
    } else if (warp == kRopeWarp) {  // ------------------------------------- queries, rotary parts, powers of two
        const int box = 1 << p.c.page_shift < kTile ? 1 << p.c.page_shift : kTile, boxes = kTile / box;
        const int blk = lane & 7;
        Turn<S::kRopes> ro;
        uint32_t nq = 0;
        while (ok && take(parts, n_part, w, ok)) {
            const int32_t *tab = p.bt.table + (int64_t)w.b * p.bt.table_stride;
            auto page_at = [&](int j) {
                const int slot = j * kTile + blk * box;
                return blk < boxes && slot < w.hi ? tab[slot >> p.c.page_shift] : -1;
            };
            const Tiles<kTile> tl(w);
            int next = page_at(tl.first);
            if (nq > 0 && !warp_wait(&bar.qempty, (nq - 1) & 1)) {
                ok = false;
                break;
            }
            nq++;
            if (lane == 0) bar_expect(&bar.qfull, (L + 1) * used * 128);
            __syncwarp();
            if (lane <= L)
                tma3(qs + lane * NR * 128, lane < L ? &maps.q : &maps.q_rope, lane < L ? 64 * lane : 0, ((w.block << pair) + rank) * p.heads, w.token, &bar.qfull);
            for (int j = tl.first; j < tl.last && ok; j++) {
                const int slot = j * kTile + blk * box, row = slot & ((1 << p.c.page_shift) - 1);
                int page = next;
                next = page_at(j + 1);
                if ((uint32_t)page >= (uint32_t)p.c.num_pages) {
                    if (blk < boxes && slot < w.hi) kv::flag(p.c.status, FTMOE_ERR_ID_RANGE);
                    page = -1;
                }
                const bool mine = lane < 8 && page >= 0;
                const int valid = __popc(__ballot_sync(~0u, mine)) * box;
                ok = warp_wait(&bar.rope_empty[ro.at], ro.ph ^ 1);
                if (!ok) break;
                if (lane == 0) bar_expect(&bar.rope_full[ro.at], valid * 128);
                __syncwarp();
                if (mine) tma3(ropes + ro.at * kUnit + lane * box * 128, &maps.rope, 0, row, page, &bar.rope_full[ro.at]);
                ro.next();
                if (Q8 && lane >> 3 < wide && (uint32_t)next < (uint32_t)p.c.num_pages)  // (as warp 4 does)
                    prefetch(&maps.all, kWide * (lane >> 3), (slot + kTile) & ((1 << p.c.page_shift) - 1), next);
            }
        }
        if (!ok) {  // wait (bounded) until the copies already issued have landed
            if (nq > 0) wait_bar(&bar.qfull, (nq - 1) & 1);
            for (int i = 0; i < S::kRopes; i++, ro.next()) wait_bar(&bar.rope_full[ro.at], ro.ph ^ 1);
        }
    } else if (warp == kMmaWarp) {  // --------------------------------------- products
        constexpr uint32_t IS = kv::kInstrM<BF, kTile, NR, false, false>, IO = kv::kInstrM<BF, 128, NR, true, false>;
        const uint32_t one = kv::elect_one();
        const uint32_t qd = desc_lo(qs, 16), pd = desc_lo(ps, 16), ud = desc_lo(units, 16), rd = desc_lo(ropes, 16), vd = desc_lo(units, kUnit);
        const int rope_steps = p.c.rope >> 4;
        uint32_t nq = 0, n = 0, np = 0;  // items, tiles whose S and whose O product is issued
        Turn<kUnits> us, uv;  // of the scores and of the outputs
        Turn<S::kRopes> ro;
        // each unit's barrier is tested while the products of the one before are issued (a test takes 100 cycles)
        auto scores = [&](bool last) {
            const int turn = S::kTwo ? n & 1 : 0;
            const uint32_t d = tm + S::kS + turn * S::kSTwo;
            uint32_t b = qd, acc = 0;
            // Two tiles' places: one test of all that this tile needs, a lane each (a test takes 100 cycles); it is mostly there. Else each
            // unit's barrier is tested while the products of the one before are issued.
            bool there;
            if (S::kTwo) {
                const int at = us.at + lane, over = at >= kUnits;
                const uint32_t mine = lane < L ? su32(&bar.unit_full[over ? at - kUnits : at]) : su32(&bar.rope_full[ro.at]);
                there = __all_sync(~0u, kv::test_bar(mine, lane < L ? us.ph ^ over : ro.ph)) != 0;
            } else {
                there = kv::test_bar(su32(&bar.unit_full[us.at]), us.ph);
            }
            if (L == 8 && (there || !S::kTwo)) {  // places known here but for the first: 50 cycles a product, what it runs, against 77
                if (S::kTwo) fence_after();
                const uint32_t a = ud + us.at * (kUnit / 16);
#pragma unroll
                for (int u = 0; u < 8; u++) {
                    if (!S::kTwo) {
                        if (!__all_sync(~0u, there)) ok = ok && warp_wait(&bar.unit_full[u], us.ph);
                        fence_after();
                        there = kv::test_bar(su32(u < 7 ? &bar.unit_full[u + 1] : &bar.rope_full[ro.at]), u < 7 ? us.ph : ro.ph);
                    }
#pragma unroll
                    for (int k = 0; k < 4; k++, acc = 1) mma_ss<IS>(one, d, a + u * (kUnit / 16) + 2 * k, qd + u * (NR * 128 / 16) + 2 * k, acc);
                }
                us.at += 8, b = qd + 8 * (NR * 128 / 16);
                if (us.at == kUnits) us.at = 0, us.ph ^= 1;
            } else {
#pragma unroll 1
                for (int u = 0; u < L && ok; u++, b += NR * 128 / 16) {
                    if (S::kTwo && u == 0) there = kv::test_bar(su32(&bar.unit_full[us.at]), us.ph);
                    if (!__all_sync(~0u, there)) ok = warp_wait(&bar.unit_full[us.at], us.ph);
                    fence_after();
                    const uint32_t a = ud + us.at * (kUnit / 16);
                    us.next();
                    there = kv::test_bar(su32(u + 1 < L ? &bar.unit_full[us.at] : &bar.rope_full[ro.at]), u + 1 < L ? us.ph : ro.ph);
#pragma unroll
                    for (int k = 0; k < 4; k++, acc = 1) mma_ss<IS>(one, d, a + 2 * k, b + 2 * k, acc);
                }
            }
            if (!__all_sync(~0u, there)) ok = ok && warp_wait(&bar.rope_full[ro.at], ro.ph);
            if (!ok) return;
            fence_after();
            const uint32_t r = rd + ro.at * (kUnit / 16);
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (k < rope_steps) mma_ss<IS>(one, d, r + 2 * k, b + 2 * k, 1);
            commit(one, &bar.s[turn]);
            if (!S::kOver) commit(one, &bar.rope_empty[ro.at]), ro.next();
            if (last) commit(one, &bar.qempty);
            n++;
        };
        auto values = [&](uint32_t acc0) {
            const int turn = S::kTwo ? np & 1 : 0;
            ok = ok && warp_wait(&bar.p[turn], S::kTwo ? np >> 1 & 1 : np & 1);
            if (!ok) return;
            fence_after();
            const uint32_t b = pd + turn * (S::kPOne / 16);
#pragma unroll 1
            for (int u = 0; u < L; u += 2) {
                const uint32_t a = vd + uv.at * (kUnit / 16), d = tm + (u >> 1) * NR;
                uint32_t acc = acc0;
#pragma unroll
                for (int k = 0; k < kTile / 16; k++, acc = 1)
                    mma_ss<IO>(one, d, a + k * (2048 / 16), b + (k >> 2) * (NR * 128 / 16) + 2 * (k & 3), acc);
                commit(one, &bar.pair_empty[uv.at >> 1]);
                uv.next(), uv.next();
            }
            if (S::kOver) commit(one, &bar.rope_empty[ro.at]), ro.next();
            if (S::kTwo) commit(one, &bar.pv);
            np++;
        };
        while (ok && take(parts, n_part, w, ok)) {
            const Tiles<kTile> tl(w);
            const int nt = __shfl_sync(~0u, tl.last - tl.first, 0);
            ok = warp_wait(&bar.qfull, nq++ & 1);
            fence_after();
#pragma unroll 1
            for (int j = 0; j < nt && ok;) {
                scores(j + 1 == nt);
                // the next tile's scores too, if it is there before this one's P: they are formed during its softmax
                bool two = false;
                if (S::kTwo && j + 1 < nt && ok) {
                    const int at = us.at + lane, over = at >= kUnits;
                    const uint32_t watch = lane < L ? su32(&bar.unit_full[over ? at - kUnits : at]) : su32(&bar.p[np & 1]);
                    const uint32_t phase = lane < L ? us.ph ^ over : np >> 1 & 1;
                    for (int i = 0; i < 1 << 21; i++) {
                        const unsigned there = __ballot_sync(~0u, kv::test_bar(watch, phase));
                        two = (there & ((1u << L) - 1)) == (1u << L) - 1;
                        if (two || there >> 31) break;
                    }
                    if (two) scores(j + 2 == nt);
                }
                values(j > 0);
                if (two) values(1);
                j += 1 + two;
            }
            if (ok) commit(one, &bar.o);
        }
        commit(one, &bar.done);  // every product is done when this arrives
        warp_wait(&bar.done, 0);
    } else if (warp == kWalkWarp) {
        ok = hand_out(p, parts, walk);
    } else if (Q8 && warp >= 8) {  // --------------------------------------- codes to elements
        // every eighth unit a warp; four lanes have a slot's 64 codes, a warp eight slots at a time. The next unit's codes are loaded while
        // this one's are turned, and the pages of the one after that looked up.
        const int sub = lane >> 2, q = lane & 3;
        const int steps = 8 / L, rest = 8 - steps * L;  // tiles from a unit to this warp's next, and units
        const int64_t off = sub * p.c.slot + 16 * q, off8 = off + 8 * p.c.slot, offp = (lane & 15) * p.c.slot + p.c.latent;
        const uint32_t at0 = units + sub * 128 + (((2 * q) ^ sub) << 4), at1 = units + sub * 128 + (((2 * q + 1) ^ sub) << 4);
        uint32_t n = 0;  // units before this part
        while (ok && take(parts, n_part, w, ok)) {
            const Tiles<kTile> tl(w);
            const int32_t *tab = p.bt.table + (int64_t)w.b * p.bt.table_stride;
            struct Unit {  // tile and unit in it, pages of its 4 x 16 slots (-1: none)
                int j, m, page[4];
            };
            auto find = [&](Unit &x) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int slot = x.j * kTile + 16 * k;
                    x.page[k] = x.j < tl.last && slot < w.hi ? tab[slot >> p.c.page_shift] : -1;
                }
            };
            auto after = [&](const Unit &x) {
                Unit y;
                y.j = x.j + steps, y.m = x.m + rest;
                if (y.m >= L) y.m -= L, y.j++;
                find(y);
                return y;
            };
            auto load = [&](const Unit &x, uint4 (&in)[8], uint32_t (&power)[2]) {  // (of page 0 where there is none: not used)
                const unsigned char *at[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    at[k] = cell(p.c, (uint32_t)x.page[k] < (uint32_t)p.c.num_pages ? x.page[k] : 0, x.j * kTile + 16 * k) + 64 * x.m;
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        uint4 &v = in[2 * k + i];
                        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "l"(at[k] + (i ? off8 : off)));
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; k++)  // both powers of a slot's two groups, slots lane and lane + 32
                    asm volatile("ld.global.u16 %0, [%1];" : "=r"(power[k]) : "l"((lane & 16 ? at[2 * k + 1] : at[2 * k]) + (offp - 62 * x.m)));
            };
            uint32_t x = n + ((warp - 8 - n) & 7);  // of all units
            auto turn = [&](const uint4 (&in)[8], const uint32_t (&power)[2]) {
                const uint32_t un = x % kUnits;
                const bool free = kv::test_bar(su32(&bar.pair_empty[un >> 1]), x / kUnits & 1 ^ 1);
                bool plain = true;
#pragma unroll
                for (int k = 0; k < 2; k++) plain = plain && plain_power<BF>(power[k] & 255) && plain_power<BF>(power[k] >> 8);
                plain = __all_sync(~0u, plain);
                if (!__all_sync(~0u, free)) ok = ok && warp_wait(&bar.pair_empty[un >> 1], x / kUnits & 1 ^ 1);
                if (!ok) return;
                auto byte = [&](int i) { return __shfl_sync(~0u, power[i >> 2], 8 * (i & 3) + sub) >> (q & 2) * 4 & 255; };
                auto put = [&](int i, const uint4 &lo, const uint4 &hi) {
                    const uint32_t o = un * kUnit + 1024 * i;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at0 + o), "r"(lo.x), "r"(lo.y), "r"(lo.z), "r"(lo.w) : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at1 + o), "r"(hi.x), "r"(hi.y), "r"(hi.z), "r"(hi.w) : "memory");
                };
                uint4 lo, hi;
                if (plain) {
#pragma unroll
                    for (int i = 0; i < 8; i++) decode16_plain<BF>(in[i], byte(i), lo, hi), put(i, lo, hi);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) decode16_far<BF>(in[i], byte(i), lo, hi), put(i, lo, hi);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) bar_arrive(&bar.unit_full[un]);
                x += 8;
            };
            Unit y{tl.first + (int)(x - n) / L, (int)(x - n) % L, {-1, -1, -1, -1}};
            find(y);
            uint4 a[8], b[8];
            uint32_t pa[2], pb[2];
            load(y, a, pa);
            Unit z = after(y);
            while (y.j < tl.last && ok) {
                load(z, b, pb);
                y = after(z);
                turn(a, pa);
                if (z.j >= tl.last || !ok) break;
                load(y, a, pa);
                z = after(y);
                turn(b, pb);
            }
            n += (tl.last - tl.first) * L;
        }
    }
    if (!ok && lane == 0) kv::flag(p.c.status, FTMOE_ERR_STATE);
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
}

// Joins the parts of the item that CTA c of the kernel before started: a warp a row, a lane four latents at a time. What the
// first FIRST parts may have is loaded before it is known how many there are, one trip instead of four: eight where the grid is
// small (16 rows an SM at most) and has nothing else to wait for, else the two that an item that is joined has, in few registers
// (seven parts of one sequence, 16 heads: 13.5 us with the kernel before, two first 15.5; 48 sequences of 128 heads: 97 us, 100 with four
// first).
// Rows of a CTA: two of a small grid, over more SMs (one sequence of 777, 16 heads: 11.9 us, with eight 12.4, with sixteen 15.1).
template <int FIRST>
constexpr int kJoinRows = FIRST == 2 ? 8 : 2;

template <bool BF, int FIRST>
__global__ void __launch_bounds__(32 * kJoinRows<FIRST>, FIRST == 2 ? 4 : 1) absorb_combine(const AttendParams p, int rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x, row = blockIdx.y * kJoinRows<FIRST> + warp;
    const int of = gridDim.x >> p.line.pair, rank = p.line.pair && c >= of ? 1 : 0, end = (rank + 1) * of;  // (Where)
    const int t = row / p.heads;
    if (t >= p.line.item_tokens) return;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 mine = c + lane < end ? p.line.join[c + lane] : make_int4(0, 0, 0, kv::kJoinEnd);
    auto slot = [&](int k) { return (int64_t)(2 * (c + k) + (k == 0)) * rows + row; };
    auto part = [&](int k) { return reinterpret_cast<const float4 *>(p.part_o + slot(k) * p.c.latent) + lane; };
    const float2 none = make_float2(-INFINITY, 0.f);
    float2 ml = c + lane < end ? p.part_ml[slot(lane)] : none;
    float4 v[FIRST][4];
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (128 * i < p.c.latent) v[k][i] = part(k)[32 * i];
    };
#pragma unroll
    for (int k = 0; k < FIRST; k++)
        if (c + k < end) fetch(k);
    const int left = __shfl_sync(~0u, mine.x, 0), block = __shfl_sync(~0u, mine.y, 0), token = __shfl_sync(~0u, mine.z, 0);
    const int h = ((block << p.line.pair) + rank) * p.heads + row - t * p.heads;
    if (t >= left || h >= p.q_heads) return;
    const unsigned ends = __ballot_sync(~0u, lane > 0 && mine.w == kv::kJoinEnd);
    const int n = ends ? __ffs(ends) : kv::count_parts(p.line.join, c, end);
    if (lane >= n) ml = none;
    float M = ml.x;
    for (int k = lane + 32; k < n; k += 32) M = fmaxf(M, p.part_ml[slot(k)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    float sum = 0.f;
    float4 x[4] = {};
    auto add = [&](float2 y, const float4 *o, int step) {
        const float a = y.x == -INFINITY ? 0.f : ex2(y.x - M);
        sum += y.y * a;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (128 * i >= p.c.latent) break;
            const float4 f = o[step * i];
            x[i].x += f.x * a, x[i].y += f.y * a, x[i].z += f.z * a, x[i].w += f.w * a;
        }
    };
#pragma unroll
    for (int k = 0; k < FIRST; k++) {
        const float2 y = make_float2(__shfl_sync(~0u, ml.x, k), __shfl_sync(~0u, ml.y, k));
        if (k < n) add(y, v[k], 1);
    }
    for (int k = FIRST; k < n; k++) add(p.part_ml[slot(k)], part(k), 32);
    const float f = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *out = p.out.d + (int64_t)(token + t) * p.out.token + (int64_t)h * p.out.head + 4 * lane;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (128 * i >= p.c.latent) break;
        *reinterpret_cast<uint2 *>(out + 128 * i) = make_uint2(from_f2<BF>(x[i].x * f, x[i].y * f), from_f2<BF>(x[i].z * f, x[i].w * f));
    }
    if (lane == 0 && p.lse) p.lse[(int64_t)(token + t) * p.q_heads + h] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

// Rows of an item: as few as hold the tokens of the longest sequence, since they cost products and queries' place (64 x 2000 tokens: 16
// heads 39 us, 43 as 32 rows, 53 as 64; 32 heads 42, 54 as 64). With 8 bits 32 at most: two tiles of elements and more queries do not fit
// shared memory (64 rows are two blocks there, 48 x 9000 tokens of 64 heads 126 us, 16 bits 73).
int rows_of(const AttendParams &p) {
    const int64_t n = (int64_t)p.q_heads * p.bt.max_q;
    return n <= 16 ? 16 : n <= 32 || p.c.bits == 8 ? 32 : 64;
}

// Items (or pairs of them), if no sequence has more tokens than max_q.
int64_t most_items(const AttendParams &p) {
    return (int64_t)((p.bt.max_q + p.line.item_tokens - 1) / p.line.item_tokens) * p.bt.batch * p.line.blocks;
}
// One sequence of 16 heads and two steps 9.6 us cut, 10.1 whole; 64 sequences of four steps 20.4 and 16.0, of 16 steps 39.7 and 45.9; 152
// of eight steps 47.0 and 39.2; two waves: 256 of eight steps 69.8 and 63.6, 160 of 16 steps 76.6 and 100.
bool cut(const AttendParams &p, int num_sms) {
    return cut_pays(most_items(p), ((int64_t)p.bt.max_kv + kStep - 1) / kStep, num_sms >> p.line.pair, 2, 0);
}
int ctas(const AttendParams &p, int num_sms) {
    const int64_t items = most_items(p);
    if (!cut(p, num_sms)) return (int)items << p.line.pair;
    const int64_t have = num_sms >> p.line.pair, most = items < have ? items * (p.bt.max_kv / kStep + 1 + kItemCost) : have;
    return (int)(most < have ? (most > 0 ? most : 1) : have) << p.line.pair;
}

template <bool BF, bool Q8, int NR>
cudaError_t launch(const AttendParams &p, int C, int num_sms, cudaStream_t st) {
    using S = Shape<Q8, NR>;
    const int box = 1 << p.c.page_shift < S::kTile ? 1 << p.c.page_shift : S::kTile, slots = 1 << p.c.page_shift, per = p.line.item_tokens;
    Maps m;
    bool ok = kv::box_map(m.q, BF, p.q.d, {p.c.latent, p.q_heads, p.bt.tokens}, 2 * p.q.head, 2 * p.q.token, {64, p.heads, per}, true) &&
              kv::box_map(m.q_rope, BF, p.q_rope.d, {p.c.rope, p.q_heads, p.bt.tokens}, 2 * p.q_rope.head, 2 * p.q_rope.token, {64, p.heads, per}, true) &&
              kv::box_map(m.rope, BF, p.c.pages + rope_at(p.c.latent, p.c.bits), {p.c.rope, slots, p.c.num_pages}, p.c.slot, p.c.page, {64, box, 1}, true);
    const int row = rope_at(p.c.latent, p.c.bits) / 2 + p.c.rope;
    ok = ok && kv::box_map(m.all, BF, p.c.pages, {row, slots, p.c.num_pages}, p.c.slot, p.c.page, {kWide, box, 1}, false);
    if (!Q8)
        ok = ok && kv::box_map(m.lat, BF, p.c.pages, {p.c.latent, slots, p.c.num_pages}, p.c.slot, p.c.page, {64, box, 1}, true);
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t rc = kv::allow_smem<absorb_kernel<BF, Q8, NR>>(S::kSmem);
    if (rc != cudaSuccess) return rc;
    absorb_kernel<BF, Q8, NR><<<C, S::kThreads, S::kSmem, st>>>(p, m);
    if ((rc = cudaGetLastError()) != cudaSuccess || !p.line.join) return rc;
    auto join = [&](auto kern, int per) { return kv::launch_after(kern, dim3(C, NR / per), 32 * per, 0, st, p, NR); };
    return C * NR <= 16 * num_sms ? join(absorb_combine<BF, 8>, kJoinRows<8>) : join(absorb_combine<BF, 2>, kJoinRows<2>);
}

template <bool BF>
cudaError_t launch_rows(const AttendParams &p, int C, int num_sms, cudaStream_t st) {
    const int n = rows_of(p);
    if (p.c.bits == 8) return n == 16 ? launch<BF, true, 16>(p, C, num_sms, st) : launch<BF, true, 32>(p, C, num_sms, st);
    if (n == 16) return launch<BF, false, 16>(p, C, num_sms, st);
    return n == 32 ? launch<BF, false, 32>(p, C, num_sms, st) : launch<BF, false, 64>(p, C, num_sms, st);
}

}  // namespace

size_t attend_workspace(AttendParams &p, int num_sms, unsigned char *base) {
    const int rows = rows_of(p);
    p.line.blocks = (p.q_heads + rows - 1) / rows, p.heads = (p.q_heads + p.line.blocks - 1) / p.line.blocks;
    p.line.blocks = (p.q_heads + p.heads - 1) / p.heads;
    p.line.item_tokens = rows / p.heads, p.line.batch = p.bt.batch, p.line.max_q = p.bt.max_q, p.line.causal = p.causal;
    // Two blocks of heads read the same cached tokens at the same time, on two SMs: one of them mostly finds them in L2 (one after the
    // other, 128 heads read them from memory twice: 32 x 4000 tokens 74 us, in pairs 61; 64 x 2000 of 32 heads are one block).
    p.line.pair = p.line.blocks % 2 == 0 ? 1 : 0;
    p.line.blocks >>= p.line.pair;
    p.line.join = nullptr, p.part_o = nullptr, p.part_ml = nullptr;
    if (!cut(p, num_sms)) return 0;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char *at = base ? base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t C = ctas(p, num_sms), n = 2 * C * rows;  // a part that starts an item and one that goes on with one for each CTA
    p.part_o = reinterpret_cast<float *>(take(n * p.c.latent * 4));
    p.part_ml = reinterpret_cast<float2 *>(take(n * 8));
    p.line.join = reinterpret_cast<int4 *>(take(C * 16));
    return off;
}

cudaError_t launch_attend(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    const int C = ctas(p, num_sms);
    return bf16 ? launch_rows<true>(p, C, num_sms, st) : launch_rows<false>(p, C, num_sms, st);
}

}  // namespace latent
}  // namespace ftmoe

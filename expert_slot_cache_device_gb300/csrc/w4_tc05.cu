// Products with 4-bit weights for more than 16 tokens, on the 5th-generation tensor cores: y^T = W x^T with the
// decoded weights as the A operand (M = 128 rows) in tensor memory and 32, 64 or 128 tokens as N.
//
// The packed order of w4.cu holds what a lane of mma.sync m16n8k16 takes of a row tile, which is what
// tcgen05.st.16x128b takes of it too: a lane decodes its 16 bytes to sixteen registers and stores
// them, with no exchange. Each group of k has products of its own, summed by the tensor cores from zero in
// fp32; a thread reads its row of them back, and adds them times the group's scale to its sums in fp32, so no
// weight is rounded.
//
// A CTA is 128 rows and ten warps, two CTAs an SM for 32 tokens; work goes by blocks of 64 k:
//   warps 0-3, 4-7  decode: two teams take the blocks (of groups of 128: pairs of them) in turn. Codes, scales and
//                   zeros come through a ring of the warp's own, so no warp waits for another there. A block's
//                   products are read LAG blocks later and run meanwhile;
//   warp 8          issues the products;
//   warp 9          copies x by tensor map. (Copied by lanes in the order of the former pack, 4 bytes at a time with a
//                   proxy fence a block, x took longer than all the rest: 37 us at 24 tokens.)
// Up to eight CTAs of a cluster cut k and join their sums in rank order. Every wait is bounded; a CTA in which one runs
// out gives NaN.
//
// 16384 x 7168 with 24 tokens takes 26.7 us (2.4 TB/s). Decoding, about 230 instructions a warp for 32 x 64 codes, fills 63 % of the
// issue slots at two CTAs an SM, but takes only 6 of the 26.7: with no codes decoded it is 21. The rest is each block's chain of
// copy, store, product and read-back of every group's sums, and the cut: whole clusters take row groups, here 256 CTAs on 304
// places, so SMs with two set the time. With 128 tokens 45 us (0.67 PFLOP/s), where a decoded block serves four
// times the tokens and is decoded again for the next 128 (64 in groups of 32).
#include <cmath>
#include "kv_tc05.cuh"
#include "w4.cuh"

namespace ftmoe {
namespace w4 {
namespace {

using kv::cp16;
using kv::from_f;
using kv::to_f;

constexpr int kDecode = 8, kMmaWarp = 8, kThreads = 320, kRowsCta = 128;
constexpr int kBound = 384;  // registers are given out by quarters of an SM: ten warps take those of twelve
constexpr int kXStages = 8;

// NT tokens (the products' N).
template <int GROUP, int NT>
struct Tile {
    static constexpr int CTAS = NT > 32 ? 1 : 2;    // an SM
    static constexpr int UB = GROUP > 64 ? 2 : 1;   // blocks of 64 k that share their products
    static constexpr int NG = GROUP < 64 ? 2 : 1;   // groups of a block
    static constexpr int ACOL = 0, DCOL = 128;      // tensor memory: two A buffers of 32 columns a team, then the products
    static constexpr int COLS = 512 / CTAS;
    static constexpr int LAG = DCOL + 4 * NG * NT > COLS ? 1 : 2;  // blocks between the decoding of one and the reading of its products: their buffers
    static constexpr int STAGES = 6;
    static constexpr int PC = 2 * NG;               // (row tile, group) pairs of a warp and block
    static constexpr int META = 2 * 512;            // after a stage's codes: scales [pair][8 pairs of rows], zeros likewise
    static constexpr int STAGE = META + PC * 48;
    static constexpr int X = NT * 128;              // bytes of an x stage
    static constexpr int SMEM = 1024 + kXStages * X + kDecode * STAGES * STAGE;
    static_assert(DCOL + 2 * LAG * NG * NT <= COLS, "the products fit tensor memory");
    static_assert(2 * NT * kRowsCta * 4 <= kXStages * X + kDecode * STAGES * STAGE, "the teams' sums fit the rings");
    // first column of the products of a team's block j
    static __device__ __forceinline__ uint32_t dcol(int team, int j) {
        return DCOL + (team * LAG + (LAG > 1 ? j / UB & 1 : 0)) * NG * NT;
    }
};

struct Bars {
    uint64_t a[2][2], d[2][2], xfull[kXStages], xempty[kXStages], done;
};

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sixteen rows (lanes of tensor memory) x 32 columns: registers 4 s .. 4 s + 3 are an A fragment of m16n8k16.
__device__ __forceinline__ void tm_st_rows16(uint32_t a, const uint32_t *x) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
        FTMOE_I4(x, 0), FTMOE_I4(x, 4), FTMOE_I4(x, 8), FTMOE_I4(x, 12)
        : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t *x) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : FTMOE_R4(x, 0), FTMOE_R4(x, 4), FTMOE_R4(x, 8), FTMOE_R4(x, 12)
        : "r"(a)
        : "memory");
}

template <bool BF, int GROUP, bool ZEROS, int NT>
__global__ void __launch_bounds__(kBound, (Tile<GROUP, NT>::CTAS)) w4_tc05_kernel(const MatvecParams p, const int split, const __grid_constant__ CUtensorMap xmap) {
    using T = Tile<GROUP, NT>;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ Bars bar;
    __shared__ uint32_t s_tmem;
    __shared__ int s_bad;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned char *const sm = sm_raw + ((1024u - (pipe::su32(sm_raw) & 1023u)) & 1023u);
    const uint32_t xs = pipe::su32(sm), ring = xs + kXStages * T::X;
    const int rank = split > 1 ? (int)kv::cluster_rank() : 0;
    const int group8 = blockIdx.x / split, tok0 = blockIdx.y * NT;
    const int live = p.tokens - tok0 < NT ? p.tokens - tok0 : NT;
    const int units = (p.g.k_blocks + T::UB - 1) / T::UB;
    const int u0 = (int)((uint32_t)(rank * units) / (uint32_t)split), u1 = (int)((uint32_t)((rank + 1) * units) / (uint32_t)split);

    if (tid == 0) {
        for (int i = 0; i < 4; i++) kv::bar_init(&bar.a[i >> 1][i & 1], 4), kv::bar_init(&bar.d[i >> 1][i & 1], 1);
        for (int i = 0; i < kXStages; i++) kv::bar_init(&bar.xfull[i], 1), kv::bar_init(&bar.xempty[i], 1);
        kv::bar_init(&bar.done, 1);
        s_bad = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(pipe::su32(&s_tmem)), "n"(T::COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    kv::fence_before();
    __syncthreads();
    kv::fence_after();
    const uint32_t tm = *reinterpret_cast<volatile uint32_t *>(&s_tmem);
    const int mine0 = T::UB * ((u1 - u0 + 1) / 2), mine1 = T::UB * ((u1 - u0) / 2);  // blocks of the teams
    bool ok = true;
    uint64_t acc[NT / 2];
#pragma unroll
    for (int i = 0; i < NT / 2; i++) acc[i] = 0;

    if (warp < kDecode) {  // ------------------------------------------------- decode, sums
        const int team = warp >> 2, q = warp & 3, rt0 = group8 * 8 + 2 * q, mine = team ? mine1 : mine0;
        const uint32_t st0 = ring + warp * T::STAGES * T::STAGE, st1 = st0 + T::STAGES * T::STAGE;
        const uint32_t lanes = tm + ((uint32_t)(32 * q) << 16);
        // what this lane copies of a block: its codes of both row tiles, and one piece of scales or zeros
        // (row tiles past the last read the last again: their rows are not written)
        const int most = p.g.row_tiles - 1, rt_a = rt0 < most ? rt0 : most, rt_b = rt0 + 1 < most ? rt0 + 1 : most, u_first = u0 + team;
        const unsigned char *cp = p.packed + (((int64_t)rt_a * p.g.k_blocks + u_first * T::UB) * 32 + lane) * 16;
        const int64_t next_tile = (int64_t)(rt_b - rt_a) * p.g.k_blocks * 512;
        const bool z = ZEROS && lane >= 2 * T::PC;
        const int pj = z ? lane - 2 * T::PC : lane >> 1;
        const bool piece = lane < T::PC * (ZEROS ? 3 : 2);
        const int64_t at = (int64_t)(pj / T::NG ? rt_b : rt_a) * p.g.groups + u_first * T::NG + pj % T::NG;
        const unsigned char *mp = p.packed + p.g.code_bytes + (z ? (int64_t)p.g.row_tiles * p.g.groups * 32 + at * 16 : at * 32 + (lane & 1) * 16);
        const uint32_t m_step = 2 * T::NG * (z ? 16 : 32);
        uint32_t in = st0 + lane * 16;  // the stage that is filled next
        auto copy = [&](int i) {
            if (i < mine) {
                cp16(in, cp);
                cp16(in + 512, cp + next_tile);
                if (piece) cp16(in + T::META, mp);
                if (T::UB == 1 || (i & 1)) {
                    cp += T::UB > 1 ? 3 * 512 : 2 * 512, mp += m_step;
                } else {
                    cp += 512;
                }
                in = in + T::STAGE < st1 ? in + T::STAGE : in + T::STAGE - T::STAGES * T::STAGE;
            }
            cp_commit();
        };
        float s_old[T::LAG][T::NG];  // this thread's row's scales of the blocks whose products are not read yet
        // the products of block j times their scales onto the sums
        auto finish = [&](int j) {
            if (!kv::warp_wait(&bar.d[team][j & 1], (j >> 1) & 1)) return false;
            kv::fence_after();  // the block's A buffer is stored to next, whether its products are read here or with the next block's
            if (T::UB == 1 || (j & 1)) {
#pragma unroll
                for (int g = 0; g < T::NG; g++) {
                    const uint64_t s2 = kv::pack2(s_old[0][g], s_old[0][g]);
#pragma unroll
                    for (int h = 0; h < NT / 16; h++) {
                        uint32_t x[16];
                        tm_ld16(lanes + T::dcol(team, j) + g * NT + 16 * h, x);
#pragma unroll
                        for (int k = 0; k < 8; k++)
                            acc[8 * h + k] = kv::fma2(s2, kv::pack2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), acc[8 * h + k]);
                    }
                }
            }
            return true;
        };
#pragma unroll
        for (int i = 0; i < T::STAGES - 1; i++) copy(i);
        const unsigned char *wm = sm + (st0 - xs);
#pragma unroll 1
        for (int i = 0; i < mine; i++) {
            cp_wait<T::STAGES - 2>();
            __syncwarp();  // scales and zeros come from other lanes; and all have read the stage before
            copy(i + T::STAGES - 1);
            if (T::LAG > 1 && i > 1 && !(ok = finish(i - 2))) break;
            const unsigned char *meta = wm + T::META;
            const uint32_t a_col = lanes + T::ACOL + team * 64 + (i & 1) * 32;
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const uint4 w = *reinterpret_cast<const uint4 *>(wm + r * 512 + lane * 16);
                const uint32_t v[4] = {w.x, w.y, w.z, w.w};
                uint32_t a[16];
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    const uint32_t zz = ZEROS ? *reinterpret_cast<const uint16_t *>(meta + T::PC * 32 + (r * T::NG + (T::NG > 1 ? s >> 1 : 0)) * 16 + (lane >> 2) * 2) : 0x0808u;
                    const uint32_t o0 = offset2<BF>(zz & 255u), o1 = offset2<BF>(zz >> 8);
                    a[4 * s] = decode2<BF>(v[s], o0), a[4 * s + 1] = decode2<BF>(v[s] >> 4, o1);
                    a[4 * s + 2] = decode2<BF>(v[s] >> 8, o0), a[4 * s + 3] = decode2<BF>(v[s] >> 12, o1);
                }
                tm_st_rows16(a_col + ((uint32_t)(16 * r) << 16), a);
            }
            float s_now[T::NG];
#pragma unroll
            for (int g = 0; g < T::NG; g++)
                s_now[g] = to_f<BF>(*reinterpret_cast<const uint16_t *>(meta + ((lane >> 4) * T::NG + g) * 32 + (lane & 7) * 4 + (lane >> 3 & 1) * 2));
            if (T::LAG == 1 && i > 0 && !(ok = finish(i - 1))) break;
#pragma unroll
            for (int g = 0; g < T::NG; g++) {
                if (T::LAG > 1) s_old[0][g] = s_old[T::LAG - 1][g];
                s_old[T::LAG - 1][g] = s_now[g];
            }
            kv::tm_st_wait();
            kv::fence_before();
            __syncwarp();
            if (lane == 0) kv::bar_arrive(&bar.a[team][i & 1]);
            wm += (i + 1) % T::STAGES ? T::STAGE : -(T::STAGES - 1) * T::STAGE;
        }
        if (T::LAG > 1 && ok && mine > 1) ok = finish(mine - 2);
        if (T::LAG > 1) {
#pragma unroll
            for (int g = 0; g < T::NG; g++) s_old[0][g] = s_old[T::LAG - 1][g];
        }
        if (ok && mine > 0) ok = finish(mine - 1);
        cp_wait<0>();
    } else if (warp == kMmaWarp) {  // ------------------------------------------- products
        constexpr uint32_t I = kv::kInstr<BF, NT, false>;
        const uint32_t one = kv::elect_one(), xd = kv::desc_lo(xs, 16);
        uint32_t c = 0;
        for (int n = 0; n < 2 * mine0 && ok; n++) {
            const int team = n & 1, i = n >> 1;
            if (team && i >= mine1) continue;
            const uint32_t st = c % kXStages;
            ok = kv::warp_wait(&bar.xfull[st], (c / kXStages) & 1) && kv::warp_wait(&bar.a[team][i & 1], (i >> 1) & 1);
            if (!ok) break;
            c++;
            kv::fence_after();
            const uint32_t d = tm + T::dcol(team, i), a = tm + T::ACOL + team * 64 + (i & 1) * 32;
#pragma unroll
            for (int s = 0; s < 4; s++)
                kv::mma_ts<I>(one, d + (T::NG > 1 ? (s >> 1) * NT : 0), a + 8 * s, xd + st * (T::X / 16) + 2 * s,
                              T::NG > 1 ? s & 1 : (s > 0 || (T::UB > 1 && (i & 1))));
            kv::commit(one, &bar.d[team][i & 1]);
            kv::commit(one, &bar.xempty[st]);
        }
        kv::commit(one, &bar.done);
        kv::warp_wait(&bar.done, 0);
    } else {  // ---------------------------------------------------------------- x
        int c = 0;
        for (int n = 0; n < 2 * mine0; n++) {
            const int team = n & 1, i = n >> 1;
            if (team && i >= mine1) continue;
            const uint32_t st = c % kXStages;
            ok = kv::warp_wait(&bar.xempty[st], ((c / kXStages) & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) {
                kv::bar_expect(&bar.xfull[st], T::X);
                kv::tma3(xs + st * T::X, &xmap, ((u0 + team + i / T::UB * 2) * T::UB + i % T::UB) * 64, tok0, 0, &bar.xfull[st]);
            }
            c++;
        }
        for (int i = c > kXStages ? c - kXStages : 0; i < c; i++) kv::warp_wait(&bar.xfull[i % kXStages], (i / kXStages) & 1);  // all have landed
    }
    if (!ok) s_bad = 1;
    kv::fence_before();
    __syncthreads();
    kv::fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tm), "n"(T::COLS) : "memory");

    // ---- join the teams' sums, [team][token][row], then the ranks'
    float *so = reinterpret_cast<float *>(sm);
    constexpr int SUMS = NT * kRowsCta;
    const bool bad = s_bad != 0;
    if (warp < kDecode) {
#pragma unroll
        for (int i = 0; i < NT / 2; i++) {
            const float2 v = kv::unpack2(acc[i]);
            float *to = so + (warp >> 2) * SUMS + 2 * i * kRowsCta + 32 * (warp & 3) + lane;
            to[0] = bad ? NAN : v.x, to[kRowsCta] = bad ? NAN : v.y;
        }
    }
    __syncthreads();
    auto sum = [&](int i) {
        float4 v = *reinterpret_cast<const float4 *>(so + i);
        const float4 u = *reinterpret_cast<const float4 *>(so + SUMS + i);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        return v;
    };
    const int used = live * kRowsCta;
    if (split > 1) {
        for (int i = tid * 4; i < used; i += kThreads * 4) *reinterpret_cast<float4 *>(so + i) = sum(i);
        kv::cluster_sync();
    }
    for (int i = (tid + rank * kThreads) * 4; i < used; i += kThreads * split * 4) {
        float4 v;
        if (split > 1) {
            v = kv::ld_rank(pipe::su32(so + i), 0);
            for (int k = 1; k < split; k++) {
                const float4 u = kv::ld_rank(pipe::su32(so + i), k);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
        } else {
            v = sum(i);
        }
        const int n = group8 * kRowsCta + i % kRowsCta;
        uint16_t *y = p.y + (int64_t)(tok0 + i / kRowsCta) * p.y_stride + n;
        const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (n + k < p.g.N) y[k] = from_f<BF>(e[k]);
    }
    if (split > 1) kv::cluster_sync();  // no rank leaves while its sums are read
}

template <bool BF, int GROUP, bool ZEROS, int NT>
cudaError_t launch_nt(const MatvecParams &p, cudaStream_t st) {
    using T = Tile<GROUP, NT>;
    const int groups = (p.g.row_tiles + 7) / 8, tiles = (p.tokens + NT - 1) / NT;
    const int units = (p.g.k_blocks + T::UB - 1) / T::UB;
    const cudaError_t e = kv::allow_smem<w4_tc05_kernel<BF, GROUP, ZEROS, NT>>(T::SMEM);
    if (e != cudaSuccess) return e;
    // The largest clusters that all run at once, four blocks a CTA at least (6000 rows of 7168, 24 tokens: 15 us with 5 CTAs a
    // cluster, 20.7 with 6, which take a second round; 2048 rows, 64 tokens: 12.4 with 6, 20.6 with 7). The device's own
    // count is of one CTA an SM; where two fit, both run (1.8 counted as active at a time).
    auto fit = [&](int s) { return T::CTAS * kv::most_clusters<w4_tc05_kernel<BF, GROUP, ZEROS, NT>>(s, kThreads, T::SMEM); };
    int split = 8;
    while (split > 1 && (units < 4 * split || (int64_t)groups * tiles > fit(split))) split--;
    CUtensorMap m;
    if (!kv::row_map(m, p.x, p.g.K, p.tokens, p.x_stride, NT, BF)) return cudaErrorInvalidValue;
    return kv::launch_clusters(w4_tc05_kernel<BF, GROUP, ZEROS, NT>, dim3(groups * split, tiles), split, kThreads, T::SMEM, st, p, split, m);
}

template <bool BF, int GROUP, bool ZEROS>
cudaError_t launch_group(const MatvecParams &p, cudaStream_t st) {
    // Codes are decoded once for the tokens of a tile; more than 32 take an SM's registers and tensor memory for one CTA.
    if (p.tokens <= 32) return launch_nt<BF, GROUP, ZEROS, 32>(p, st);
    if (GROUP < 64 || p.tokens <= 64) return launch_nt<BF, GROUP, ZEROS, 64>(p, st);
    return launch_nt<BF, GROUP, ZEROS, GROUP < 64 ? 64 : 128>(p, st);
}
template <bool BF, int GROUP>
cudaError_t launch_zeros(const MatvecParams &p, cudaStream_t st) {
    return p.g.zeros ? launch_group<BF, GROUP, true>(p, st) : launch_group<BF, GROUP, false>(p, st);
}

template <bool BF>
cudaError_t launch(const MatvecParams &p, cudaStream_t st) {
    if (p.g.group == 32) return launch_zeros<BF, 32>(p, st);
    return p.g.group == 64 ? launch_zeros<BF, 64>(p, st) : launch_zeros<BF, 128>(p, st);
}

}  // namespace

cudaError_t launch_tc05(const MatvecParams &p, bool bf16, cudaStream_t st) {
    return bf16 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace w4
}  // namespace ftmoe

// Products with 4-bit weights: y[t, n] = sum over groups G of s[n, G] sum_{k in G} (q[n, k] - z[n, G]) x[t, k].
//
// The codes are laid out once, in the order in which mma.sync m16n8k16 takes its A operand, so
// a warp's load of a tile of 16 rows x 64 k is 512 consecutive bytes: lane (g, t) = (lane / 4,
// lane % 4) holds four words, word s the eight codes of the 16 k of step s: nibble i of the low half is the
// first and nibble i of the high half the second element of fragment register a_i (a0: row g, a1:
// row g + 8 at k = 2 t; a2, a3 the same at 2 t + 8). (w >> 4i) & 0x000f000f OR'ed into the bits of
// (128, 128) in bf16, or (1024, 1024) in f16, makes 128 + q (1024 + q) exactly, and subtracting
// 128 + z leaves the exact integer q - z. A group's products are summed by the tensor cores in
// fp32 from zero; its scale multiplies that sum in fp32, so no weight is rounded.
//   packed: codes [row tile][64-k block][lane][16 B], then scales [row tile][group][8] pairs (rows g,
//   g + 8), then zeros [row tile][group][8] pairs of bytes. Rows past N and k past K hold zeros.
//
// This kernel is for up to 16 tokens, w4_tc05.cu for more. Bound by the instructions that decode (about 100 a warp for 16 x 64 codes)
// and by a call's start and end; the codes alone are 1.2 us of the 6.2 us of one token times 2048 x 7168, and 8.8 of the 18.5
// (3.6 TB/s) of 16384 x 7168. A CTA is eight warps: WR row tiles times WK slices of k, so that several
// warps share the x that a chunk of k stages in shared memory. Codes and scales go to shared memory too (each lane
// copies the 16 bytes of codes that it reads itself), kStages chunks deep: held in registers instead, two
// chunks of them spilled. Where row tiles alone do not fill the SMs, up to eight CTAs of a cluster split k and join their sums
// through distributed shared memory in rank order, so results repeat bit for bit.
#include "kv_attend.cuh"
#include "pipeline.cuh"
#include "w4.cuh"

namespace ftmoe {
namespace w4 {
namespace {

using kv::cp16;
using kv::from_f;
using kv::to_f;

__global__ void pack_kernel(const Geometry g, const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                            unsigned char *packed) {
    const int64_t words = (int64_t)g.row_tiles * g.k_blocks * 128;
    const int64_t metas = (int64_t)g.row_tiles * g.groups * 8;
    const int ng = g.K / g.group;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < words + metas; i += (int64_t)gridDim.x * blockDim.x) {
        if (i < words) {
            const int s = (int)(i & 3), lane = (int)(i >> 2 & 31);
            const int64_t tile = i >> 7;
            const int kb = (int)(tile % g.k_blocks), rt = (int)(tile / g.k_blocks);
            uint32_t w = 0;
#pragma unroll
            for (int r = 0; r < 4; r++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int n = rt * 16 + (lane >> 2) + 8 * (r & 1);
                    const int k = kb * 64 + 16 * s + 8 * (r >> 1) + 2 * (lane & 3) + e;
                    uint32_t q = 0;
                    if (n < g.N && k < g.K) q = codes[(int64_t)n * (g.K / 2) + (k >> 1)] >> (4 * (k & 1)) & 15;
                    w |= q << (4 * r + 16 * e);
                }
            reinterpret_cast<uint32_t *>(packed)[i] = w;
        } else {
            const int64_t m = i - words;
            const int r = (int)(m & 7), gi = (int)(m >> 3) % g.groups, rt = (int)((m >> 3) / g.groups);
            uint32_t s = 0, z = 0;
            for (int e = 0; e < 2; e++) {
                const int n = rt * 16 + r + 8 * e;
                if (n < g.N && gi < ng) {
                    s |= (uint32_t)scales[(int64_t)n * ng + gi] << (16 * e);
                    if (zeros) z |= (uint32_t)(zeros[(int64_t)n * ng + gi] & 15) << (8 * e);
                }
            }
            reinterpret_cast<uint32_t *>(packed + g.code_bytes)[m] = s;
            if (zeros) reinterpret_cast<uint16_t *>(packed + g.code_bytes + metas * 4)[m] = (uint16_t)z;
        }
    }
}

constexpr int kWarps = 8, kThreads = kWarps * 32, kStages = 3;

// TN tiles of eight tokens; WK_ slices of k a CTA.
template <int GROUP, int TN, int WK_>
struct Shape {
    static constexpr int WK = WK_, WR = kWarps / WK;
    static constexpr int CTAS = TN == 1 ? 3 : 2;             // CTAs an SM
    static constexpr int KPW = 4;                            // 64-k blocks of a warp and chunk
    static constexpr int CB = KPW * WK;                      // blocks of a chunk
    static constexpr int RS = CB * 128 + 16;                 // bytes of an x row: eight rows' 16 bytes cover the banks
    static constexpr int NG = GROUP < 64 ? KPW * 2 : KPW * 64 / GROUP;  // groups of a warp's blocks
    static constexpr int META = NG * 48;                     // scales [group][8 pairs], zeros likewise
    static constexpr int WARP = KPW * 512 + META;
    static constexpr int MOST = (8 * TN + 1) * RS + kWarps * WARP; // bytes of a stage with every row of x
    static constexpr int ROWS = WR * 16;
    static constexpr int TILE = 8 * TN * ROWS;               // sums of a CTA; one copy a k slice, over the stages
    static_assert(WK * TILE * 4 <= kStages * kWarps * WARP, "the sums fit the stages");
};

template <bool BF>
__device__ __forceinline__ void mma_next(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        pipe::mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else
        pipe::mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}
// The same from zero.
template <bool BF>
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        pipe::mma_f16_16816_z(d, a[0], a[1], a[2], a[3], b0, b1);
}

// `split` CTAs of a cluster share k; grid (row groups * split, token tiles of 8 TN); a stage holds `rows`
// rows of x: those that the call has, and one of zeros where they do not fill the token tiles.
template <bool BF, int GROUP, bool ZEROS, int TN, int WK>
__global__ void __launch_bounds__(kThreads, Shape<GROUP, TN, WK>::CTAS) matvec_kernel(const MatvecParams p, const int split, const int rows) {
    using S = Shape<GROUP, TN, WK>;
    constexpr int GK = GROUP > 64 ? 2 : 1;  // blocks that share a scale
    extern __shared__ __align__(128) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rank = split > 1 ? (int)kv::cluster_rank() : 0, wr = warp / S::WK, wk = warp % S::WK;
    const int rt0 = blockIdx.x / split * S::WR + wr, tok0 = blockIdx.y * 8 * TN;
    const int live_x = p.tokens - tok0 < 8 * TN ? p.tokens - tok0 : 8 * TN;
    // this CTA's blocks of k, whole groups
    const int pairs = (p.g.k_blocks + GK - 1) / GK;
    const int kb0 = (int)((int64_t)rank * pairs / split) * GK, kb1_ = (int)((int64_t)(rank + 1) * pairs / split) * GK;
    const int kb1 = kb1_ < p.g.k_blocks ? kb1_ : p.g.k_blocks;
    const int chunks = (kb1 - kb0 + S::CB - 1) / S::CB;

    const uint32_t base = pipe::su32(sm), stage = rows * S::RS + kWarps * S::WARP, mine = rows * S::RS + warp * S::WARP;  // x, the warps' parts

    // What this thread copies of each chunk stays at one place of it: pointers advance by the chunk.
    // Codes: KPW blocks of each row tile.
    const int kb_w = kb0 + wk * S::KPW;
    const unsigned char *cp = p.packed + (((int64_t)rt0 * p.g.k_blocks + kb_w) * 32 + lane) * 16;
    const bool live_r = rt0 < p.g.row_tiles;
    // Scales and zeros: 16-byte pieces, two of scales and one of zeros a group, PC groups.
    constexpr int PC = S::NG, PIECES = PC * (ZEROS ? 3 : 2), STEP = GROUP > 64 ? S::CB / 2 : (GROUP < 64 ? S::CB * 2 : S::CB);
    static_assert(PIECES <= 64, "two pieces a lane at most");
    const unsigned char *mp[PIECES > 32 ? 2 : 1];
    int m_left[PIECES > 32 ? 2 : 1], m_step[PIECES > 32 ? 2 : 1];  // groups before the row's end; bytes a chunk
#pragma unroll
    for (int q = 0; q < (PIECES > 32 ? 2 : 1); q++) {
        const int i = lane + 32 * q;
        const bool z = ZEROS && i >= 2 * PC;
        const int j = z ? i - 2 * PC : i >> 1, rt = rt0;
        const int gi = (GROUP > 64 ? kb_w / 2 : (GROUP < 64 ? kb_w * 2 : kb_w)) + j % S::NG;
        const unsigned char *sp = p.packed + p.g.code_bytes;
        const int64_t at = (int64_t)rt * p.g.groups + gi;
        mp[q] = z ? sp + (int64_t)p.g.row_tiles * p.g.groups * 32 + at * 16 : sp + at * 32 + (i & 1) * 16;
        m_left[q] = i < PIECES && rt < p.g.row_tiles ? p.g.groups - gi : 0;
        m_step[q] = STEP * (z ? 16 : 32);
    }
    // x: chunk tid % (8 CB) of rows tid / (8 CB), ...
    constexpr int XC = S::CB * 8, XR = kThreads / XC;  // 16-byte chunks a row, rows a round
    const int xr = tid / XC, k1 = kb1 * 64 < p.g.K ? kb1 * 64 : p.g.K;
    int xk = kb0 * 64 + 8 * (tid % XC);
    const uint16_t *xp = p.x + (int64_t)(tok0 + xr) * p.x_stride + xk;
    const uint32_t xd = xr * S::RS + 16 * (tid % XC);
    int kb_next = kb_w;

    // the row of x in a stage, one for each token tile, whose address this lane gives to ldmatrix; tokens that are none read a
    // row of zeros
    uint32_t xo[TN];
#pragma unroll
    for (int n = 0; n < TN; n++) xo[n] = (8 * n + (lane & 7) < live_x ? 8 * n + (lane & 7) : rows - 1) * S::RS + wk * S::KPW * 128 + 16 * (lane >> 3);
    if (live_x < 8 * TN)
        for (int i = tid; i < kStages * (S::RS / 16); i += kThreads)
            *reinterpret_cast<uint4 *>(sm + i / (S::RS / 16) * stage + (rows - 1) * S::RS + i % (S::RS / 16) * 16) = make_uint4(0, 0, 0, 0);

    auto copy = [&](int c) {
        if (c < chunks) {
            const uint32_t st = base + (c % kStages) * stage;
            const int n = kb1 - kb_next;
#pragma unroll
            for (int i = 0; i < S::KPW; i++) {
                const bool ok = live_r && i < n;
                cp16(st + mine + i * 512 + lane * 16, ok ? cp + i * 512 : p.packed, ok ? 16 : 0);
            }
#pragma unroll
            for (int q = 0; q < (PIECES > 32 ? 2 : 1); q++) {
                if (lane + 32 * q < PIECES) cp16(st + mine + S::KPW * 512 + (lane + 32 * q) * 16, m_left[q] > 0 ? mp[q] : p.packed, m_left[q] > 0 ? 16 : 0);
                mp[q] += m_step[q], m_left[q] -= STEP;
            }
            const bool in = xk < k1;
#pragma unroll
            for (int r = 0; r < 8 * TN; r += XR)
                if (xr + r < live_x) cp16(st + xd + r * S::RS, in ? xp + (int64_t)r * p.x_stride : p.x, in ? 16 : 0);
            cp += S::CB * 512, kb_next += S::CB, xk += S::CB * 64, xp += S::CB * 64;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    float acc[TN][4];
#pragma unroll
    for (int n = 0; n < TN; n++) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int c = 0; c < kStages - 1; c++) copy(c);
    for (int c = 0; c < chunks; c++) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();  // this chunk is there, and the stage of the one before is read
        copy(c + kStages - 1);
        const unsigned char *st = sm + (c % kStages) * stage;
        const unsigned char *wm = st + mine;
        const uint32_t *sc = reinterpret_cast<const uint32_t *>(wm + S::KPW * 512) + g;
        const uint16_t *zc = reinterpret_cast<const uint16_t *>(wm + S::KPW * 512 + S::NG * 32) + g;
        float part[TN][4];
#pragma unroll
        for (int i = 0; i < S::KPW; i++) {
            const uint4 w = *reinterpret_cast<const uint4 *>(wm + i * 512 + lane * 16);
#pragma unroll
            for (int h = 0; h < 2; h++) {  // 32 k: two steps
                const int gi = GROUP > 64 ? i / 2 : (GROUP < 64 ? 2 * i + h : i);
                const bool begin = GROUP < 64 || (h == 0 && i % GK == 0), end = GROUP < 64 || (h == 1 && i % GK == GK - 1);
                const uint32_t z = ZEROS ? zc[gi * 8] : 0x0808u;
                const uint32_t o0 = offset2<BF>(z & 255u), o1 = offset2<BF>(z >> 8);
                const uint32_t v[2] = {h ? w.z : w.x, h ? w.w : w.y};
                uint32_t a[2][4];
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    a[s][0] = decode2<BF>(v[s], o0), a[s][1] = decode2<BF>(v[s] >> 4, o1);
                    a[s][2] = decode2<BF>(v[s] >> 8, o0), a[s][3] = decode2<BF>(v[s] >> 12, o1);
                }
#pragma unroll
                for (int n = 0; n < TN; n++) {
                    uint32_t b[4];
                    pipe::ldsm_x4(b, st + xo[n] + i * 128 + h * 64);
                    if (begin)
                        mma_first<BF>(part[n], a[0], b[0], b[1]);
                    else
                        mma_next<BF>(part[n], a[0], b[0], b[1]);
                    mma_next<BF>(part[n], a[1], b[2], b[3]);
                }
                if (end) {
                    const uint32_t s2 = sc[gi * 8];
                    const float s0 = to_f<BF>((uint16_t)s2), s1 = to_f<BF>((uint16_t)(s2 >> 16));
#pragma unroll
                    for (int n = 0; n < TN; n++) {
                        acc[n][0] += s0 * part[n][0], acc[n][1] += s0 * part[n][1];
                        acc[n][2] += s1 * part[n][2], acc[n][3] += s1 * part[n][3];
                    }
                }
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // ---- join the k slices: [wk][token][row] over the stages, then the ranks
    __syncthreads();
    float *so = reinterpret_cast<float *>(sm);
    constexpr int TILE = S::TILE;
#pragma unroll
    for (int n = 0; n < TN; n++)
#pragma unroll
        for (int i = 0; i < 4; i++) so[wk * TILE + (8 * n + 2 * t + (i & 1)) * S::ROWS + wr * 16 + g + 8 * (i >> 1)] = acc[n][i];
    __syncthreads();
    if (split > 1) {
        for (int i = tid * 4; i < TILE; i += kThreads * 4) {
            float4 v = *reinterpret_cast<const float4 *>(so + i);
#pragma unroll
            for (int k = 1; k < S::WK; k++) {
                const float4 u = *reinterpret_cast<const float4 *>(so + k * TILE + i);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            *reinterpret_cast<float4 *>(so + i) = v;
        }
        kv::cluster_sync();
    }
    const int row0 = blockIdx.x / split * S::ROWS;
    for (int i = (tid + rank * kThreads) * 4; i < TILE; i += kThreads * split * 4) {
        float4 v;
        if (split > 1) {
            v = kv::ld_rank(pipe::su32(so + i), 0);
            for (int k = 1; k < split; k++) {
                const float4 u = kv::ld_rank(pipe::su32(so + i), k);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
        } else {
            v = *reinterpret_cast<const float4 *>(so + i);
#pragma unroll
            for (int k = 1; k < S::WK; k++) {
                const float4 u = *reinterpret_cast<const float4 *>(so + k * TILE + i);
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
        }
        const int tok = tok0 + i / S::ROWS, n = row0 + i % S::ROWS;
        if (tok < p.tokens) {
            uint16_t *y = p.y + (int64_t)tok * p.y_stride + n;
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; k++)
                if (n + k < p.g.N) y[k] = from_f<BF>(e[k]);
        }
    }
    if (split > 1) kv::cluster_sync();  // no rank leaves while its sums are read
}

template <bool BF, int GROUP, bool ZEROS, int TN, int WK>
cudaError_t launch_tn(const MatvecParams &p, int num_sms, cudaStream_t st) {
    using S = Shape<GROUP, TN, WK>;
    const int groups = (p.g.row_tiles + S::WR - 1) / S::WR, tiles = (p.tokens + 8 * TN - 1) / (8 * TN);
    // k is split where that shortens the busiest SM's work: its CTAs (S::CTAS at once), each as long as its
    // chunks and about two more for its start and end
    const int64_t ctas = (int64_t)groups * tiles;
    int split = 1;
    int64_t best = INT64_MAX;
    for (int s = 1; s <= 8; s++) {
        const int per = (p.g.k_blocks + s - 1) / s, chunks = (per + S::CB - 1) / S::CB;
        const int64_t an_sm = (ctas * s + num_sms - 1) / num_sms, cost = an_sm * chunks + (an_sm + S::CTAS - 1) / S::CTAS * 4;
        if (cost < best) best = cost, split = s;
        if (per <= S::CB) break;
    }
    cudaError_t e = kv::allow_smem<matvec_kernel<BF, GROUP, ZEROS, TN, WK>>(kStages * S::MOST);
    const int rows = p.tokens % (8 * TN) == 0 ? 8 * TN : (p.tokens < 8 * TN ? p.tokens : 8 * TN) + 1;
    if (e != cudaSuccess) return e;
    return kv::launch_clusters(matvec_kernel<BF, GROUP, ZEROS, TN, WK>, dim3(groups * split, tiles), split, kThreads,
                               kStages * (rows * S::RS + kWarps * S::WARP), st, p, split, rows);
}

template <bool BF, int GROUP, bool ZEROS>
cudaError_t launch_group(const MatvecParams &p, int num_sms, cudaStream_t st) {
    // One token tile and at most a row tile an SM: all warps of a CTA on one row tile, k cut inside the CTA rather than
    // over clusters (2048 rows of 7168, one token: 6.3 us against 8.3; 6000 rows, eight tokens: 14.5 against 10.4).
    if (p.tokens <= 8)
        return p.g.row_tiles <= num_sms ? launch_tn<BF, GROUP, ZEROS, 1, 8>(p, num_sms, st) : launch_tn<BF, GROUP, ZEROS, 1, 2>(p, num_sms, st);
    return launch_tn<BF, GROUP, ZEROS, 2, 2>(p, num_sms, st);
}

template <bool BF>
cudaError_t launch(const MatvecParams &p, int num_sms, cudaStream_t st) {
    if (p.g.zeros) {
        if (p.g.group == 32) return launch_group<BF, 32, true>(p, num_sms, st);
        return p.g.group == 64 ? launch_group<BF, 64, true>(p, num_sms, st) : launch_group<BF, 128, true>(p, num_sms, st);
    }
    if (p.g.group == 32) return launch_group<BF, 32, false>(p, num_sms, st);
    return p.g.group == 64 ? launch_group<BF, 64, false>(p, num_sms, st) : launch_group<BF, 128, false>(p, num_sms, st);
}

}  // namespace

Geometry geometry(int32_t N, int32_t K, int32_t group, int32_t zeros) {
    Geometry g;
    g.N = N, g.K = K, g.group = group, g.zeros = zeros;
    g.row_tiles = (N + 15) / 16;
    g.k_blocks = (K + 63) / 64;
    g.groups = group > 64 ? K / group : g.k_blocks * (64 / group);
    g.code_bytes = (int64_t)g.row_tiles * g.k_blocks * 512;
    g.meta_bytes = (int64_t)g.row_tiles * g.groups * (zeros ? 48 : 32);
    return g;
}

cudaError_t launch_pack(const Geometry &g, const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                        unsigned char *packed, cudaStream_t st) {
    const int64_t items = (int64_t)g.row_tiles * (g.k_blocks * 128 + (int64_t)g.groups * 8);
    const int64_t blocks = (items + 255) / 256;
    pack_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(g, codes, scales, zeros, packed);
    return cudaGetLastError();
}

constexpr int32_t kMostTokens = 1 << 21;  // of one launch

cudaError_t launch_matvec(const MatvecParams &p, bool bf16, int num_sms, cudaStream_t st) {
    // More than 16 tokens go to the tensor-memory kernel (16384 rows of 7168: with 24 tokens 26.7 us against 28.7 here, with 32
    // 26.7 against 36.9; 2048 rows, 32 tokens: 12.4 against 15.5). At 16 tokens this one takes 24.7 as that one does, and 12.4
    // against 14.6 for 6000 rows, 8.5 against 12.3 for 2048.
    if (p.tokens > 16) {
        MatvecParams q = p;  // a grid has 65535 tiles of 64 tokens at most
        for (int64_t t = 0; t < p.tokens; t += kMostTokens) {
            q.x = p.x + t * p.x_stride, q.y = p.y + t * p.y_stride;
            q.tokens = p.tokens - t < kMostTokens ? (int32_t)(p.tokens - t) : kMostTokens;
            if (const cudaError_t e = launch_tc05(q, bf16, st)) return e;
        }
        return cudaSuccess;
    }
    return bf16 ? launch<true>(p, num_sms, st) : launch<false>(p, num_sms, st);
}

}  // namespace w4
}  // namespace ftmoe

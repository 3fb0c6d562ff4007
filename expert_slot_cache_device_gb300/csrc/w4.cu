// Products with 4-bit weights: y[t, n] = sum over groups G of s[n, G] sum_{k in G} (q[n, k] - z[n, G]) x[t, k].
//
// The codes are laid out once, in the order in which mma.sync m16n8k16 takes its A operand, so
// a warp's load of a tile of 16 rows x 64 k is 512 consecutive bytes: lane (g, t) = (lane / 4,
// lane % 4) holds four words, word s the eight codes of k step s (16 k): nibble i of the low half is
// the first and nibble i of the high half the second element of fragment register a_i (a0: row
// g, k 2t; a1: row g + 8; a2, a3: the same at k 2t + 8). (w >> 4i) & 0x000f000f OR'ed into the
// bits of (128, 128) in bf16, or (1024, 1024) in f16, makes 128 + q (1024 + q) exactly, and
// subtracting 128 + z leaves the exact integer q - z. A group's products are summed by the
// tensor cores in fp32 from zero; its scale multiplies that sum in fp32, so no weight is rounded.
//   packed: codes [row tile][64-k block][lane][16 B], then scales [row tile][group][8] pairs (rows g,
//   g + 8), then zeros [row tile][group][8] pairs of bytes. Rows past N and k past K hold zeros.
#include "kv.cuh"
#include "pipeline.cuh"

namespace ftmoe {
namespace w4 {
namespace {

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
                    const int k = kb * 64 + s * 16 + 2 * (lane & 3) + 8 * (r >> 1) + e;
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

// (128 + z, 128 + z) in bf16 or (1024 + z, 1024 + z) in f16.
template <bool BF>
__device__ __forceinline__ uint32_t offset2(uint32_t z) {
    return (BF ? 0x43004300u : 0x64006400u) | z | z << 16;
}
template <bool BF>
__device__ __forceinline__ uint32_t decode2(uint32_t w, uint32_t off) {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w), "r"(0x000f000fu), "r"(BF ? 0x43004300u : 0x64006400u));
    if (BF) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&off));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&d);
}

constexpr int kWarps = 8;

template <bool BF, int GROUP>
__global__ void __launch_bounds__(kWarps * 32) matvec_kernel(const MatvecParams p) {
    constexpr int KB = GROUP > 64 ? GROUP / 64 : 1;      // 64-k blocks of one step
    constexpr int GPB = GROUP < 64 ? 64 / GROUP : 1;     // groups of one 64-k block
    __shared__ float s_acc[kWarps][32][4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int rt = blockIdx.x, tok = blockIdx.y * 8 + g;
    const uint4 *codes = reinterpret_cast<const uint4 *>(p.packed) + (int64_t)rt * p.g.k_blocks * 32 + lane;
    const uint32_t *scales = reinterpret_cast<const uint32_t *>(p.packed + p.g.code_bytes) + (int64_t)rt * p.g.groups * 8 + g;
    const uint16_t *zeros = reinterpret_cast<const uint16_t *>(p.packed + p.g.code_bytes + (int64_t)p.g.row_tiles * p.g.groups * 32) +
                            (int64_t)rt * p.g.groups * 8 + g;
    const uint16_t *x = p.x + (int64_t)tok * p.x_stride + 2 * t;
    const bool live = tok < p.tokens;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int kb = warp * KB; kb < p.g.k_blocks; kb += kWarps * KB) {
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < KB; u++) {
            const uint4 c = codes[(int64_t)(kb + u) * 32];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int s = 0; s < 4; s++) {
                const int gi = GROUP > 64 ? kb / KB : kb * GPB + s * GPB / 4;
                const uint32_t z = p.g.zeros ? zeros[(int64_t)gi * 8] : 0x0808u;
                const uint32_t o0 = offset2<BF>(z & 255u), o1 = offset2<BF>(z >> 8);
                const int k = (kb + u) * 64 + s * 16;
                uint32_t b0 = 0, b1 = 0;
                if (live && k < p.g.K) {
                    b0 = *reinterpret_cast<const uint32_t *>(x + k);
                    b1 = *reinterpret_cast<const uint32_t *>(x + k + 8);
                }
                const uint32_t a0 = decode2<BF>(w[s], o0), a1 = decode2<BF>(w[s] >> 4, o1);
                const uint32_t a2 = decode2<BF>(w[s] >> 8, o0), a3 = decode2<BF>(w[s] >> 12, o1);
                if (BF)
                    pipe::mma_bf16_16816(part, a0, a1, a2, a3, b0, b1);
                else
                    pipe::mma_f16_16816(part, a0, a1, a2, a3, b0, b1);
                const bool last = GROUP > 64 ? (u == KB - 1 && s == 3) : (s + 1) % (4 / GPB) == 0;
                if (last) {
                    const uint32_t sc = scales[(int64_t)gi * 8];
                    const float s0 = to_f<BF>((uint16_t)sc), s1 = to_f<BF>((uint16_t)(sc >> 16));
                    acc[0] += s0 * part[0], acc[1] += s0 * part[1], acc[2] += s1 * part[2], acc[3] += s1 * part[3];
                    part[0] = part[1] = part[2] = part[3] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) s_acc[warp][lane][i] = acc[i];
    __syncthreads();
    if (warp == 0) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) v += s_acc[w][lane][i];
            const int n = rt * 16 + g + 8 * (i >> 1), to = blockIdx.y * 8 + 2 * t + (i & 1);
            if (n < p.g.N && to < p.tokens) p.y[to * p.y_stride + n] = from_f<BF>(v);
        }
    }
}

template <bool BF>
cudaError_t launch(const MatvecParams &p, cudaStream_t st) {
    const dim3 grid(p.g.row_tiles, (p.tokens + 7) / 8);
    if (p.g.group == 32)
        matvec_kernel<BF, 32><<<grid, kWarps * 32, 0, st>>>(p);
    else if (p.g.group == 64)
        matvec_kernel<BF, 64><<<grid, kWarps * 32, 0, st>>>(p);
    else
        matvec_kernel<BF, 128><<<grid, kWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
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

cudaError_t launch_matvec(const MatvecParams &p, bool bf16, int, cudaStream_t st) {
    return bf16 ? launch<true>(p, st) : launch<false>(p, st);
}

}  // namespace w4
}  // namespace ftmoe

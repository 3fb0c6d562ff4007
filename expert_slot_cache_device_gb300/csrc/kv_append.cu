// Rotary positions on the new tokens' queries and keys, and the write of keys and values to
// their slots of the paged cache.
//
// Pair i of a head turns by the angle 2 pi f_i pos, f_i in turns a position. In fp32,
// pos * f_i alone is off by up to half an ulp of the whole number of turns (0.008 turns at
// position 2^17), so f_i comes as hi + lo: r = pos * hi is rounded, e = fma(pos, hi, -r) is what
// the rounding lost (exact), and the fraction (r - rint(r)) + e + pos * lo, whose first
// difference is exact too, holds the angle to about 2^-24 turns at any |pos| < 2^24.
//
// One CTA a token. Thread t takes the same pair of 16-byte chunks c = t % (dim / 16) of one head
// after another, so its eight angles' sines and cosines stay in registers; every chunk pair is
// two 16-byte loads and two 16-byte stores. Bound by reading and writing the rows once: a prompt of 3 x
// up to 4001 tokens of 64 + 2 x 8 heads of 128 (318 MB) takes 51 us, 6.2 TB/s, 0.93 of a plain copy; 16
// single tokens take 3.2 us, a kernel's start and end.
#include "kv.cuh"

namespace ftmoe {
namespace kv {
namespace {

constexpr int kThreads = 128;

template <bool BF>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    __shared__ float2 s_cs[128];  // (cos, sin) * factor of each pair
    __shared__ long long s_seq;   // of this token: (sequence, slot), -1 without one; one store, so that of two sequences that claim it one does
    const int t = blockIdx.x, tid = threadIdx.x;
    if (tid == 0) s_seq = -1;
    __syncthreads();
    const float pos = (float)p.pos[t];
    for (int b = tid; b < p.bt.batch; b += kThreads) {
        const Seq s = seq_info(p.bt, b, p.c.status);
        if (t >= s.q0 && t < s.q0 + s.q_len) s_seq = seq_slot(b, s.kv_len - s.q_len + (t - s.q0));
    }
    for (int i = tid; i < p.rot / 2; i += kThreads) {
        const float2 f = p.freq[i];
        const float r = pos * f.x;
        const float turn = (r - rintf(r)) + fmaf(pos, f.x, -r) + pos * f.y;
        float sn, cs;
        sincospif(2.0f * turn, &sn, &cs);
        s_cs[i] = make_float2(cs * p.factor, sn * p.factor);
    }
    __syncthreads();
    const int b = (int)(s_seq >> 32), slot = (int)s_seq;
    if (b < 0) return;  // a row that no sequence covers
    const int page = slot < 0 ? -1 : page_of(p.c, p.bt, b, slot);
    const int row = slot & ((1 << p.c.page_shift) - 1);

    const int pairs = p.c.dim >> 4, c = tid % pairs, per = kThreads / pairs;
    if (tid >= per * pairs) return;
    const bool turned = c < (p.rot >> 4);
    float2 cs[8];
    if (turned) {
#pragma unroll
        for (int i = 0; i < 8; i++) cs[i] = s_cs[8 * c + i];
    }
    // element offsets of the two chunks
    const int e0 = turned && !p.interleaved ? 8 * c : 16 * c;
    const int e1 = turned && !p.interleaved ? p.rot / 2 + 8 * c : 16 * c + 8;
    const int heads = p.q_heads + 2 * p.c.kv_heads;
    for (int h = tid / pairs; h < heads; h += per) {
        const uint16_t *src;
        uint16_t *dst;
        bool rot = turned;
        if (h < p.q_heads) {
            src = p.q.d + t * p.q.token + h * p.q.head;
            dst = p.q_out.d + t * p.q_out.token + h * p.q_out.head;
        } else {
            if (page < 0) continue;  // no slot, or a bad page (recorded)
            const int hk = h - p.q_heads;
            if (hk < p.c.kv_heads) {
                src = p.k.d + t * p.k.token + hk * p.k.head;
                dst = p.c.k + k_at(p.c, page, row, hk);
            } else {
                src = p.v.d + t * p.v.token + (hk - p.c.kv_heads) * p.v.head;
                dst = p.c.v + v_at(p.c, page, row, hk - p.c.kv_heads);
                rot = false;
            }
        }
        // values have no pairs: their chunks are copied in place
        uint4 a = *reinterpret_cast<const uint4 *>(src + e0), d = *reinterpret_cast<const uint4 *>(src + e1);
        if (rot) {
            uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ud[4] = {d.x, d.y, d.z, d.w};
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 x = to_f2<BF>(ua[i]), y = to_f2<BF>(ud[i]);
                    ua[i] = from_f2<BF>(x.x * cs[i].x - x.y * cs[i].y, x.y * cs[i].x + x.x * cs[i].y);
                    ud[i] = from_f2<BF>(y.x * cs[4 + i].x - y.y * cs[4 + i].y, y.y * cs[4 + i].x + y.x * cs[4 + i].y);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 x = to_f2<BF>(ua[i]), y = to_f2<BF>(ud[i]);
                    const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
                    ua[i] = from_f2<BF>(x.x * c0.x - y.x * c0.y, x.y * c1.x - y.y * c1.y);
                    ud[i] = from_f2<BF>(y.x * c0.x + x.x * c0.y, y.y * c1.x + x.y * c1.y);
                }
            }
            a = make_uint4(ua[0], ua[1], ua[2], ua[3]);
            d = make_uint4(ud[0], ud[1], ud[2], ud[3]);
        }
        *reinterpret_cast<uint4 *>(dst + e0) = a;
        *reinterpret_cast<uint4 *>(dst + e1) = d;
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, bool bf16, cudaStream_t st) {
    if (bf16)
        append_kernel<true><<<p.bt.tokens, kThreads, 0, st>>>(p);
    else
        append_kernel<false><<<p.bt.tokens, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kv
}  // namespace ftmoe

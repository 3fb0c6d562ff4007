// Write of new tokens to a latent cache (norm, rotary positions, 16 or 8 bits) and its reading
// back as rows.
#include "latent.cuh"

namespace ftmoe {
namespace latent {
namespace {

using kv::from_f2;
using kv::to_f2;

constexpr int kThreads = 128;

// 2^-e and the stored byte of the least e in [-127, 127] with top <= 448 * 2^e. top = 1.f * 2^k: e = k - 8, or one
// more above 1.75 * 2^k.
__device__ __forceinline__ uint32_t power_byte(float top) {
    const uint32_t u = __float_as_uint(top);
    if (u >= 0x7f800000u) return 255;
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);  // biased; subnormals cut to 0
    return e > 0 ? e : 0;
}

// One CTA a token. Thread t < latent / 8 holds 8 latents; a group of 32 is four neighbouring lanes. For the rotary
// parts, thread t takes the same pair of 16-byte chunks of one head after another (the key is one more head), with
// its eight angles in registers; angles as in kv_append.cu. Bound by memory for a prompt (7690 tokens with 128 heads' queries: 47 us,
// 5.8 TB/s, 0.85 of a plain copy's rate), by the launch and two dependent loads for a step (64 tokens: 2.8 us).
template <bool BF, bool Q8>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    __shared__ float2 s_cs[32];
    __shared__ float s_sum[kThreads / 32];
    __shared__ long long s_seq;  // of this token: (sequence, slot), -1 without one; one store, so that of two sequences that claim it one does
    const int t = blockIdx.x, tid = threadIdx.x, rope = p.c.rope, latent = p.c.latent;
    if (tid == 0) s_seq = -1;
    uint4 x = make_uint4(0, 0, 0, 0), w = x;
    if (tid < latent >> 3) {
        x = *reinterpret_cast<const uint4 *>(p.lat + t * p.lat_stride + 8 * tid);
        if (p.weight) w = *reinterpret_cast<const uint4 *>(p.weight + 8 * tid);
    }
    __syncthreads();
    for (int b = tid; b < p.bt.batch; b += kThreads) {
        const kv::Seq s = kv::seq_info(p.bt, b, p.c.status);
        if (t >= s.q0 && t < s.q0 + s.q_len) s_seq = kv::seq_slot(b, s.kv_len - s.q_len + (t - s.q0));
    }
    if (tid < rope >> 1) {
        const float2 f = p.freq[tid];
        const float pos = (float)p.pos[t], r = pos * f.x;
        const float turn = (r - rintf(r)) + fmaf(pos, f.x, -r) + pos * f.y;
        float sn, cs;
        sincospif(2.0f * turn, &sn, &cs);
        s_cs[tid] = make_float2(cs * p.factor, sn * p.factor);
    }
    uint32_t ux[4] = {x.x, x.y, x.z, x.w}, uw[4] = {w.x, w.y, w.z, w.w};
    float y[8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = to_f2<BF>(ux[i]);
        y[2 * i] = f.x, y[2 * i + 1] = f.y;
        sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
    __syncthreads();
    const int b = (int)(s_seq >> 32), slot = (int)s_seq;
    if (b < 0) return;  // a row that no sequence covers
    const int page = slot < 0 ? -1 : page_of(p.c, p.bt, b, slot);
    unsigned char *dst = page < 0 ? nullptr : cell(p.c, page, slot);

    // latents (every lane takes part in the shuffles)
    {
        if (p.weight) {
            const float mean = (s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]) / (float)latent, rstd = rsqrtf(mean + p.eps);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = to_f2<BF>(uw[i]);
                ux[i] = from_f2<BF>(y[2 * i] * rstd * f.x, y[2 * i + 1] * rstd * f.y);
            }
        }
        if (!Q8) {
            if (dst && tid < latent >> 3) *reinterpret_cast<uint4 *>(dst + 16 * tid) = make_uint4(ux[0], ux[1], ux[2], ux[3]);
        } else {
            float top = 0.f;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = to_f2<BF>(ux[i]);
                y[2 * i] = f.x, y[2 * i + 1] = f.y;
                bad = bad || !(fabsf(f.x) < INFINITY) || !(fabsf(f.y) < INFINITY);
            }
            // 240 * 2^e of the type's last e: the next code up would read back as infinity
            const float most = BF ? __uint_as_float(0x7f700000u) : 61440.f;
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = fminf(fmaxf(y[i], -most), most);
#pragma unroll
            for (int i = 0; i < 8; i++) top = fmaxf(top, fabsf(y[i]));
            if (bad) top = INFINITY;
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const uint32_t byte = power_byte(top);
            const float up = byte >= 254 ? 0.f : __uint_as_float((254 - byte) << 23);
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                unsigned short h;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y[2 * i + 1] * up), "f"(y[2 * i] * up));
                c[i] = h;
            }
            if (dst && tid < latent >> 3) {
                *reinterpret_cast<uint2 *>(dst + 8 * tid) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
                if ((tid & 3) == 0) dst[latent + (tid >> 2)] = (unsigned char)byte;
            }
        }
    }

    const int pairs = rope >> 4, c = tid % pairs, per = kThreads / pairs;
    if (tid >= per * pairs) return;
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; i++) cs[i] = s_cs[8 * c + i];
    const int e0 = p.interleaved ? 16 * c : 8 * c, e1 = p.interleaved ? 16 * c + 8 : rope / 2 + 8 * c;
    for (int h = tid / pairs; h <= p.q_heads; h += per) {
        const uint16_t *src;
        uint16_t *to;
        if (h < p.q_heads) {
            src = p.q.d + t * p.q.token + h * p.q.head;
            to = p.q_out.d + t * p.q_out.token + h * p.q_out.head;
        } else {
            if (!dst) continue;  // no slot, or a bad page (recorded)
            src = p.key + t * p.key_stride;
            to = reinterpret_cast<uint16_t *>(dst + rope_at(latent, p.c.bits));
        }
        const uint4 a = *reinterpret_cast<const uint4 *>(src + e0), d = *reinterpret_cast<const uint4 *>(src + e1);
        uint32_t ua[4] = {a.x, a.y, a.z, a.w}, ud[4] = {d.x, d.y, d.z, d.w};
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = to_f2<BF>(ua[i]), g = to_f2<BF>(ud[i]);
                ua[i] = from_f2<BF>(f.x * cs[i].x - f.y * cs[i].y, f.y * cs[i].x + f.x * cs[i].y);
                ud[i] = from_f2<BF>(g.x * cs[4 + i].x - g.y * cs[4 + i].y, g.y * cs[4 + i].x + g.x * cs[4 + i].y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 f = to_f2<BF>(ua[i]), g = to_f2<BF>(ud[i]);
                const float2 c0 = cs[2 * i], c1 = cs[2 * i + 1];
                ua[i] = from_f2<BF>(f.x * c0.x - g.x * c0.y, f.y * c1.x - g.y * c1.y);
                ud[i] = from_f2<BF>(g.x * c0.x + f.x * c0.y, g.y * c1.x + f.y * c1.y);
            }
        }
        *reinterpret_cast<uint4 *>(to + e0) = make_uint4(ua[0], ua[1], ua[2], ua[3]);
        *reinterpret_cast<uint4 *>(to + e1) = make_uint4(ud[0], ud[1], ud[2], ud[3]);
    }
}

// A CTA copies kReadRows slots of one sequence; a thread takes 16 bytes of a slot at a time, kReadAhead of them in flight (what an 8-bit
// slot's 40 pieces leave a thread: 8 x <= 30000 tokens 39.6 us, 6.0 TB/s, 46.4 with one in flight; 7 x <= 1500 in 16 bits 2.8 us, 4.3).
constexpr int kReadRows = 32, kReadThreads = 256, kReadAhead = 5;

template <bool BF, bool Q8>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const ReadParams p) {
    __shared__ int64_t s_src[kReadRows];  // offset of the slot, -1: none
    const int b = blockIdx.y, tid = threadIdx.x, j0 = blockIdx.x * kReadRows;
    int32_t *status = blockIdx.x == 0 && tid == 0 ? p.c.status : nullptr;
    const int n = kv::seq_kv_len(p.bt, b, status);
    const int a = p.cu_rows[b], e = p.cu_rows[b + 1];
    const int r0 = a < 0 ? 0 : (a > p.rows ? p.rows : a), r1 = e < r0 ? r0 : (e > p.rows ? p.rows : e);
    if (r0 != a || r1 != e || r1 - r0 != n) kv::flag(status, FTMOE_ERR_STATE);
    const int m = min(n, r1 - r0) - j0, here = m < kReadRows ? m : kReadRows;
    if (here <= 0) return;
    if (tid < here) {
        const int page = page_of(p.c, p.bt, b, j0 + tid);
        s_src[tid] = page < 0 ? -1 : cell(p.c, page, j0 + tid) - p.c.pages;
    }
    __syncthreads();
    const int latent = p.c.latent, at = rope_at(latent, p.c.bits);
    const int lat = Q8 ? latent >> 4 : latent >> 3, per = lat + (p.c.rope >> 3);  // 16-byte pieces of a slot, 72 at most
    const uint32_t inv = ((1u << 20) + per - 1) / per;                            // i / per = i * inv >> 20 for i * per < 2^20
    for (int i0 = tid; i0 < here * per; i0 += kReadAhead * kReadThreads) {
        uint4 x[kReadAhead];
        uint32_t byte[kReadAhead];
        int row[kReadAhead], col[kReadAhead];  // row -1: none
#pragma unroll
        for (int k = 0; k < kReadAhead; k++) {
            const int i = i0 + k * kReadThreads, r = i * inv >> 20, c = i - r * per;
            const int64_t from = i < here * per ? s_src[r] : -1;
            row[k] = from < 0 ? -1 : r, col[k] = c, x[k] = make_uint4(0, 0, 0, 0), byte[k] = 0;
            if (from < 0) continue;
            const unsigned char *src = p.c.pages + from;
            x[k] = *reinterpret_cast<const uint4 *>(src + (c < lat ? 16 * c : at + 16 * (c - lat)));
            if (Q8 && c < lat) byte[k] = src[latent + (c >> 1)];
        }
#pragma unroll
        for (int k = 0; k < kReadAhead; k++) {
            if (row[k] < 0) continue;
            uint16_t *dst = p.out + (int64_t)(r0 + j0 + row[k]) * p.out_stride;
            const int c = col[k];
            if (!Q8 || c >= lat)
                *reinterpret_cast<uint4 *>(dst + (Q8 ? latent + 8 * (c - lat) : 8 * c)) = x[k];
            else {
                uint4 lo, hi;
                decode16<BF>(x[k], byte[k], lo, hi);
                *reinterpret_cast<uint4 *>(dst + 16 * c) = lo;
                *reinterpret_cast<uint4 *>(dst + 16 * c + 8) = hi;
            }
        }
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, bool bf16, cudaStream_t st) {
    const bool q8 = p.c.bits == 8;
    auto kern = bf16 ? (q8 ? append_kernel<true, true> : append_kernel<true, false>) : (q8 ? append_kernel<false, true> : append_kernel<false, false>);
    kern<<<p.bt.tokens, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_read(const ReadParams &p, bool bf16, cudaStream_t st) {
    const bool q8 = p.c.bits == 8;
    auto kern = bf16 ? (q8 ? read_kernel<true, true> : read_kernel<true, false>) : (q8 ? read_kernel<false, true> : read_kernel<false, false>);
    // no sequence has more rows than there are, however loose the bound (64 x <= 500 tokens, a bound of 131072: 21 us, without the cut
    // 134; a bound of 500: 7.2)
    const int most = p.bt.max_kv < p.rows ? p.bt.max_kv : p.rows;
    kern<<<dim3((most + kReadRows - 1) / kReadRows, p.bt.batch), kReadThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace latent
}  // namespace ftmoe

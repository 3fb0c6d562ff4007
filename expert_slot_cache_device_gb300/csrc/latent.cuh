// Device views of a paged latent cache and of expanded rows, parameters and launches of the
// latent-attention kernels.
#pragma once

#include <cuda_fp8.h>

#include "kv.cuh"

namespace ftmoe {
namespace latent {

using kv::Batch;
using kv::Rows;

constexpr int kGroup = 32;  // latents that share a power of two in 8 bits

struct View {
    unsigned char *pages;
    int64_t page, slot;  // bytes
    int32_t num_pages, page_shift, latent, rope, bits;
    int32_t *status;
};

// Bytes of a slot before its rotary part, and the byte where its powers of two start.
__host__ __device__ __forceinline__ int rope_at(int latent, int bits) {
    return bits == 16 ? 2 * latent : latent + ((latent / kGroup + 15) & ~15);
}

// Page of a slot of sequence b, or -1 (recorded) where the table names none.
__device__ __forceinline__ int page_of(const View &c, const Batch &bt, int b, int slot) {
    const int page = bt.table[(int64_t)b * bt.table_stride + (slot >> c.page_shift)];
    if ((uint32_t)page < (uint32_t)c.num_pages) return page;
    kv::flag(c.status, FTMOE_ERR_ID_RANGE);
    return -1;
}
__device__ __forceinline__ unsigned char *cell(const View &c, int page, int slot) {
    return c.pages + page * c.page + (slot & ((1 << c.page_shift) - 1)) * c.slot;
}

// 2^e of a stored byte e + 127 (255: NaN).
__device__ __forceinline__ float power(uint32_t byte) {
    return byte == 255 ? __uint_as_float(0x7fc00000u) : (byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u));
}
// Two e4m3 codes (low byte first) as floats: exact, as binary16 holds every code.
__device__ __forceinline__ float2 codes2(uint32_t u) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 16 codes of one group as elements. A code's exponent and fraction, put under the element type's, are its value times
// 2^-120 (bf16) or 2^-8 (f16), subnormals too, and one product with a power of two gives the element. Powers whose factor the type
// does not hold (not plain_power) go by floats. (A group with a NaN has the power NaN; the codes 0x7f and 0xff are not written.)
template <bool BF>
__device__ __forceinline__ bool plain_power(uint32_t byte) {
    return (BF || byte >= 127 - 22) && byte <= 127 + 7;
}
template <bool BF>
__device__ __forceinline__ void decode16_plain(const uint4 u, uint32_t byte, uint4 &lo, uint4 &hi) {
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    uint32_t out[8];
    // the factor twice: bf16 2^(e + 120), f16 2^(e + 8)
    const uint32_t f = BF ? (byte + 120) * 0x00800080u : (byte - 127 + 8 + 15) * 0x04000400u;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const uint32_t x = __byte_perm(in[i >> 1], 0, i & 1 ? 0x3424 : 0x1404);  // codes in the high bytes
        const uint32_t y = (x & 0x80008000u) | (BF ? x >> 4 & 0x07f007f0u : x >> 1 & 0x3f803f80u);
        if (BF)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(out[i]) : "r"(y), "r"(f));
        else
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(out[i]) : "r"(y), "r"(f));
    }
    lo = make_uint4(out[0], out[1], out[2], out[3]), hi = make_uint4(out[4], out[5], out[6], out[7]);
}
template <bool BF>
__device__ __forceinline__ void decode16_floats(const uint4 u, uint32_t byte, uint4 &lo, uint4 &hi) {
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
    uint32_t out[8];
    const float s = power(byte);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 a = codes2(in[i] & 0xffffu), b = codes2(in[i] >> 16);
        out[2 * i] = kv::from_f2<BF>(a.x * s, a.y * s), out[2 * i + 1] = kv::from_f2<BF>(b.x * s, b.y * s);
    }
    lo = make_uint4(out[0], out[1], out[2], out[3]), hi = make_uint4(out[4], out[5], out[6], out[7]);
}
template <bool BF>
__device__ __forceinline__ void decode16(const uint4 u, uint32_t byte, uint4 &lo, uint4 &hi) {
    if (plain_power<BF>(byte))
        decode16_plain<BF>(u, byte, lo, hi);
    else
        decode16_floats<BF>(u, byte, lo, hi);
}

// ---------------------------------------------------------------- launches
struct AppendParams {
    View c;
    Batch bt;
    const uint16_t *lat, *key, *weight;  // weight nullable: no norm
    int64_t lat_stride, key_stride;
    float eps, factor;
    Rows q, q_out;
    int32_t q_heads, interleaved;
    const float2 *freq;
    const int32_t *pos;
};
cudaError_t launch_append(const AppendParams &p, bool bf16, cudaStream_t st);

struct ReadParams {
    View c;
    Batch bt;
    const int32_t *cu_rows;
    int32_t rows;
    uint16_t *out;
    int64_t out_stride;
};
cudaError_t launch_read(const ReadParams &p, bool bf16, cudaStream_t st);

// How a call's work is cut (latent_line.cuh): an item is item_tokens tokens of one sequence and one of `blocks` blocks of heads.
struct Line {
    int32_t batch, blocks, item_tokens, max_q, causal;
    int32_t pair;  // 1: CTAs 2 i and 2 i + 1 have the same place in the line and a block each of a pair of blocks (`blocks` counts pairs)
    int4 *join;  // [CTAs] (kv_split.cuh), or NULL: a CTA an item, whole
};

struct AttendParams {
    View c;
    Batch bt;
    Rows q, q_rope, out;
    int32_t q_heads, causal;
    float scale;
    float *lse;  // [tokens, q_heads] (nullable)
    Line line;
    int32_t heads;  // of a block
    // workspace (attend_workspace): parts of split items
    float *part_o;
    float2 *part_ml;
    __device__ __forceinline__ kv::Seq seq(int b, int32_t *status) const { return kv::seq_info(bt, b, status); }
};
// Bytes of workspace; with `base` the pointers of p are set into it.
size_t attend_workspace(AttendParams &p, int num_sms, unsigned char *base);
cudaError_t launch_attend(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);

struct ExpandParams {
    const int32_t *cu_q, *cu_kv;
    int32_t batch, tokens, rows, max_q, max_kv;
    int32_t *status;
    Rows q, k, v, out;
    const uint16_t *key;  // shared rotary parts
    int64_t key_stride;
    int32_t heads, nope, rope, vdim, causal;
    float scale;
    float *lse;
    Line line;
    // workspace (expand_workspace): parts of split items
    float *part_o;
    float2 *part_ml;
    // First key row of sequence b, and the sequence, each value cut to its range (a cut is recorded).
    __device__ __forceinline__ int first_row(int b) const {
        const int a = cu_kv[b];
        return a < 0 ? 0 : (a > rows ? rows : a);
    }
    __device__ __forceinline__ kv::Seq seq(int b, int32_t *st) const {
        Batch bt{};
        bt.tokens = tokens, bt.max_q = max_q, bt.max_kv = max_kv;
        const int row0 = first_row(b), e = cu_kv[b + 1], end = e < row0 ? row0 : (e > rows ? rows : e);
        if (cu_kv[b] != row0 || end != e) kv::flag(st, FTMOE_ERR_STATE);
        return kv::seq_cut(bt, cu_q[b], cu_q[b + 1], end - row0, st);
    }
};
size_t expand_workspace(ExpandParams &p, int num_sms, unsigned char *base);
cudaError_t launch_expand(const ExpandParams &p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace latent
}  // namespace ftmoe

// Device views of a paged key/value cache and of the sequences of one call, shared by the
// append, attention and eviction kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ftmoe.h"

namespace ftmoe {
namespace kv {

struct View {
    uint16_t *k, *v;
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // elements
    int32_t num_pages, page_shift, kv_heads, dim;
    int32_t *status;
};

struct Batch {
    const int32_t *table;
    int64_t table_stride;
    const int32_t *kv_lens, *cu_q;
    int32_t batch, tokens, max_q, max_kv;
};

struct Rows {
    uint16_t *d;
    int64_t token, head;
};

__device__ __forceinline__ void flag(int32_t *status, int32_t code) {
    if (status) atomicCAS(status, 0, code);
}

// Sequence b: its first token row, new tokens and cached tokens, each cut to its range (a cut
// is recorded), so that no index formed from them leaves the caller's arrays.
struct Seq {
    int q0, q_len, kv_len;
};

__device__ __forceinline__ int seq_kv_len(const Batch &bt, int b, int32_t *status) {
    const int n = bt.kv_lens[b], c = n < 0 ? 0 : (n > bt.max_kv ? bt.max_kv : n);
    if (c != n) flag(status, FTMOE_ERR_STATE);
    return c;
}

__device__ __forceinline__ Seq seq_cut(const Batch &bt, int a, int e, int n, int32_t *status) {
    Seq s;
    s.q0 = a < 0 ? 0 : (a > bt.tokens ? bt.tokens : a);
    int end = e < s.q0 ? s.q0 : (e > bt.tokens ? bt.tokens : e);
    if (end - s.q0 > bt.max_q) end = s.q0 + bt.max_q;
    s.q_len = end - s.q0;
    s.kv_len = n < 0 ? 0 : (n > bt.max_kv ? bt.max_kv : n);
    if (s.q0 != a || end != e || s.kv_len != n) flag(status, FTMOE_ERR_STATE);
    return s;
}

__device__ __forceinline__ Seq seq_info(const Batch &bt, int b, int32_t *status) {
    return seq_cut(bt, bt.cu_q[b], bt.cu_q[b + 1], bt.kv_lens[b], status);
}

// A sequence and a slot of it (below 0: none) in one word.
__device__ __forceinline__ long long seq_slot(int b, int slot) { return (long long)b << 32 | (uint32_t)slot; }

// Page of a slot of sequence b, or -1 (recorded) where the table names none.
__device__ __forceinline__ int page_of(const View &c, const Batch &bt, int b, int slot) {
    const int page = bt.table[(int64_t)b * bt.table_stride + (slot >> c.page_shift)];
    if ((uint32_t)page < (uint32_t)c.num_pages) return page;
    flag(c.status, FTMOE_ERR_ID_RANGE);
    return -1;
}

__device__ __forceinline__ int64_t k_at(const View &c, int page, int row, int head) {
    return page * c.k_page + row * c.k_slot + head * c.k_head;
}
__device__ __forceinline__ int64_t v_at(const View &c, int page, int row, int head) {
    return page * c.v_page + row * c.v_slot + head * c.v_head;
}

template <bool BF>
__device__ __forceinline__ float to_f(uint16_t u) {
    if (BF) return __uint_as_float((uint32_t)u << 16);
    return __half2float(__ushort_as_half(u));
}
template <bool BF>
__device__ __forceinline__ uint16_t from_f(float f) {
    if (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    return __half_as_ushort(__float2half_rn(f));
}
// Two elements of a 32-bit word, low half first.
template <bool BF>
__device__ __forceinline__ float2 to_f2(uint32_t u) {
    if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
template <bool BF>
__device__ __forceinline__ uint32_t from_f2(float a, float b) {
    uint32_t u;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
    return u;
}

// ---------------------------------------------------------------- launches
struct AppendParams {
    View c;
    Batch bt;
    Rows q, q_out, k, v;
    int32_t q_heads, rot, interleaved;
    float factor;
    const float2 *freq;  // [rot / 2] turns a position, hi and lo
    const int32_t *pos;
};
cudaError_t launch_append(const AppendParams &p, bool bf16, cudaStream_t st);

struct AttendParams {
    View c;
    Batch bt;
    Rows q, out;
    int32_t q_heads, group, window, causal;
    int32_t item_tokens;  // tokens of an item of the tiled kernels: two tiles of 128 / group
    float scale;
    const float *sinks;
    float *lse;   // [tokens, q_heads] (nullable)
    float *mass;  // (nullable)
    int64_t mass_seq, mass_head;
    // workspace (attend_workspace): parts of split items, log-sum-exps in powers of two for the
    // mass pass, the scores that it reads
    float *part_o;
    float2 *part_ml;
    int4 *join;  // per CTA of the split kernels (Join)
    float *lse2;
    float *logits;  // [batch, kv_heads, logit_rows][logit_stride]
    float *mass_parts;  // [mass_split][batch, kv_heads][logit_stride], the mass pass of chunks cut by rows
    int32_t mass_split;
    int32_t logit_rows;
    int64_t logit_stride;
    uint16_t *q_copy;  // [tokens, q_heads, dim]: the queries of a call whose output replaces them before the mass pass of chunks
};
// Bytes of workspace; with `base` the pointers of p are set into it.
size_t attend_workspace(AttendParams &p, int num_sms, unsigned char *base);
cudaError_t launch_attend(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st);

struct EvictParams {
    View c;
    Batch bt;
    const float *mass;
    int64_t mass_seq, mass_head;
    int32_t budget, recent;
    const int32_t *new_table;
    int64_t new_stride;
    int32_t *kept;
    float *new_mass;
    int32_t *new_lens;
};
cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t st);

}  // namespace kv

namespace w4 {

// Packed layout (see w4.cu): sizes of its two parts.
struct Geometry {
    int32_t N, K, group, zeros;
    int32_t row_tiles, k_blocks, groups;  // 16-row tiles, 64-k blocks, groups with padding
    int64_t code_bytes, meta_bytes;
};
Geometry geometry(int32_t N, int32_t K, int32_t group, int32_t zeros);
cudaError_t launch_pack(const Geometry &g, const uint8_t *codes, const uint16_t *scales, const uint8_t *zeros,
                        unsigned char *packed, cudaStream_t st);
struct MatvecParams {
    Geometry g;
    const unsigned char *packed;
    const uint16_t *x;
    uint16_t *y;
    int64_t x_stride, y_stride;
    int32_t tokens;
};
cudaError_t launch_matvec(const MatvecParams &p, bool bf16, int num_sms, cudaStream_t st);

}  // namespace w4
}  // namespace ftmoe

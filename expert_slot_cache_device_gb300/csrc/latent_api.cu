// Host side of the latent-attention entry points: argument checks and launches. See include/ftmoe.h
// for the contract of every entry point.
#include <cmath>

#include "attn_checks.cuh"
#include "latent.cuh"

using namespace ftmoe;
using namespace ftmoe::checks;

namespace {

bool is16(int dtype) { return dtype == FTMOE_DT_BF16 || dtype == FTMOE_DT_F16; }

int check_latent(const ftmoe_latent_cache *c, latent::View &v) {
    if (!c) return fail(FTMOE_ERR_INVALID_ARG, "null cache view");
    if (!is16(c->dtype)) return fail(FTMOE_ERR_FORMAT, "cache dtype %d: bf16 or f16", c->dtype);
    if (c->bits != 16 && c->bits != 8) return fail(FTMOE_ERR_FORMAT, "bits=%d: 16 or 8", c->bits);
    if (c->latent < 128 || c->latent > 512 || c->latent % 128)
        return fail(FTMOE_ERR_FORMAT, "latent=%d: a multiple of 128, at most 512", c->latent);
    if (c->rope < 16 || c->rope > 64 || c->rope % 16) return fail(FTMOE_ERR_FORMAT, "rope=%d: a multiple of 16 from 16 to 64", c->rope);
    if (!c->d_pages || !aligned16(c->d_pages)) return fail(FTMOE_ERR_INVALID_ARG, "pages must be non-null and 16-byte aligned");
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(FTMOE_ERR_INVALID_ARG, "page_size=%d: a power of two in [16, 256]", c->page_size);
    if (c->num_pages <= 0) return fail(FTMOE_ERR_INVALID_ARG, "num_pages=%d", c->num_pages);
    const int row = latent::rope_at(c->latent, c->bits) + 2 * c->rope;
    if (c->page_stride <= 0 || c->page_stride % 16 || c->slot_stride < row || c->slot_stride % 16)
        return fail(FTMOE_ERR_INVALID_ARG, "strides must be multiples of 16 bytes, slots of %d bytes apart", row);
    v.pages = static_cast<unsigned char *>(c->d_pages), v.page = c->page_stride, v.slot = c->slot_stride;
    v.num_pages = c->num_pages, v.latent = c->latent, v.rope = c->rope, v.bits = c->bits, v.status = c->d_status;
    for (v.page_shift = 4; (1 << v.page_shift) < c->page_size;) v.page_shift++;
    return FTMOE_OK;
}

int attend_params(const ftmoe_latent_cache *kvc, const ftmoe_kv_batch *batch, int q_heads, int causal, latent::AttendParams &p) {
    int rc = check_latent(kvc, p.c);
    if (rc) return rc;
    if ((rc = check_batch(batch, p.c.page_shift, p.bt))) return rc;
    if (q_heads <= 0 || q_heads > 65535) return fail(FTMOE_ERR_INVALID_ARG, "q_heads=%d", q_heads);
    if ((int64_t)p.bt.tokens * q_heads > INT32_MAX)
        return fail(FTMOE_ERR_INVALID_ARG, "%d tokens of %d heads: more than 2^31 - 1 rows", p.bt.tokens, q_heads);
    p.q_heads = q_heads, p.causal = causal != 0;
    return FTMOE_OK;
}

int expand_params(const ftmoe_row_batch *b, int dtype, int heads, int nope, int rope, int v_dim, int causal, latent::ExpandParams &p) {
    if (!b) return fail(FTMOE_ERR_INVALID_ARG, "null batch");
    if (!is16(dtype)) return fail(FTMOE_ERR_FORMAT, "dtype %d: bf16 or f16", dtype);
    if (!((nope == 128 && v_dim == 128) || (nope == 64 && v_dim == 64)))
        return fail(FTMOE_ERR_FORMAT, "nope=%d, v_dim=%d: both 128 or both 64", nope, v_dim);
    if (rope < 16 || rope > 64 || rope % 16) return fail(FTMOE_ERR_FORMAT, "rope=%d: a multiple of 16 from 16 to 64", rope);
    if (heads <= 0 || heads > 65535) return fail(FTMOE_ERR_INVALID_ARG, "heads=%d", heads);
    if (b->batch < 0 || b->batch > 65535) return fail(FTMOE_ERR_INVALID_ARG, "batch=%d outside [0, 65535]", b->batch);
    if (b->tokens < 0 || b->rows < 0 || b->max_q < 0 || b->max_kv < 0)
        return fail(FTMOE_ERR_INVALID_ARG, "negative tokens, rows, max_q or max_kv");
    if (b->max_kv > 1 << 30) return fail(FTMOE_ERR_INVALID_ARG, "max_kv=%d above 2^30", b->max_kv);
    if (b->batch > 0 && (!b->d_cu_q || !b->d_cu_kv)) return fail(FTMOE_ERR_INVALID_ARG, "null cu_q or cu_kv");
    if ((int64_t)b->tokens * heads > INT32_MAX)
        return fail(FTMOE_ERR_INVALID_ARG, "%d tokens of %d heads: more than 2^31 - 1 rows", b->tokens, heads);
    p.cu_q = b->d_cu_q, p.cu_kv = b->d_cu_kv, p.batch = b->batch, p.tokens = b->tokens, p.rows = b->rows, p.status = b->d_status;
    p.max_q = b->max_q < b->tokens ? b->max_q : b->tokens, p.max_kv = b->max_kv < b->rows ? b->max_kv : b->rows;
    p.heads = heads, p.nope = nope, p.rope = rope, p.vdim = v_dim, p.causal = causal != 0;
    return FTMOE_OK;
}

int check_workspace(size_t need, void *d, size_t bytes) {
    if (need && (!d || ((uintptr_t)d & 255) || bytes < need))
        return fail(FTMOE_ERR_INVALID_ARG, "workspace: %zu bytes at a 256-byte boundary needed, %zu given", need, bytes);
    return FTMOE_OK;
}

}  // namespace

int ftmoe_latent_append(const ftmoe_latent_cache *kvc, const ftmoe_kv_batch *batch, const ftmoe_rotary *rotary, const void *d_c,
                        int64_t c_stride, const void *d_k_rope, int64_t k_stride, const void *d_weight, float eps,
                        const ftmoe_rows *q, const ftmoe_rows *q_out, int32_t q_heads, const int32_t *d_positions, void *stream) {
    NvtxRange range("ftmoe_latent_append");
    latent::AppendParams p{};
    int rc = check_latent(kvc, p.c);
    if (rc) return rc;
    if ((rc = check_batch(batch, p.c.page_shift, p.bt))) return rc;
    if (!rotary) return fail(FTMOE_ERR_INVALID_ARG, "null rotary plan");
    if (rotary->rot_dim != p.c.rope) return fail(FTMOE_ERR_INVALID_ARG, "rot_dim=%d: the cache's rope=%d", rotary->rot_dim, p.c.rope);
    if (!rotary->d_freq || ((uintptr_t)rotary->d_freq & 7)) return fail(FTMOE_ERR_INVALID_ARG, "d_freq must be non-null and 8-byte aligned");
    if (!std::isfinite(rotary->factor)) return fail(FTMOE_ERR_INVALID_ARG, "rotary factor is not finite");
    if (!d_c || !aligned16(d_c) || c_stride % 8 || c_stride < p.c.latent || !d_k_rope || !aligned16(d_k_rope) || k_stride % 8 || k_stride < p.c.rope)
        return fail(FTMOE_ERR_INVALID_ARG, "c and k_rope must be non-null and 16-byte aligned, rows a multiple of 8 elements apart");
    if (!aligned16(d_weight)) return fail(FTMOE_ERR_INVALID_ARG, "weight must be 16-byte aligned");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(FTMOE_ERR_INVALID_ARG, "eps must be finite and not negative");
    if (q_heads < 0 || q_heads > 65535) return fail(FTMOE_ERR_INVALID_ARG, "q_heads=%d", q_heads);
    if (q_heads > 0) {
        if ((rc = check_rows(q, "q", q_heads, p.c.rope, p.q))) return rc;
        if ((rc = check_rows(q_out, "q_out", q_heads, p.c.rope, p.q_out))) return rc;
        if (p.q_out.d == p.q.d && ((p.bt.tokens > 1 && p.q_out.token != p.q.token) || (q_heads > 1 && p.q_out.head != p.q.head)))
            return fail(FTMOE_ERR_INVALID_ARG, "q_out over q needs q's strides");
    }
    if (!d_positions) return fail(FTMOE_ERR_INVALID_ARG, "null positions");
    if (p.bt.tokens == 0 || p.bt.batch == 0) return FTMOE_OK;
    p.lat = static_cast<const uint16_t *>(d_c), p.key = static_cast<const uint16_t *>(d_k_rope);
    p.weight = static_cast<const uint16_t *>(d_weight), p.lat_stride = c_stride, p.key_stride = k_stride, p.eps = eps;
    p.q_heads = q_heads, p.interleaved = rotary->interleaved != 0, p.factor = rotary->factor;
    p.freq = reinterpret_cast<const float2 *>(rotary->d_freq), p.pos = d_positions;
    return cuda_rc(latent::launch_append(p, kvc->dtype == FTMOE_DT_BF16, static_cast<cudaStream_t>(stream)), "latent append kernel");
}

int ftmoe_latent_read(const ftmoe_latent_cache *kvc, const ftmoe_kv_batch *batch, const int32_t *d_cu_rows, int32_t rows, void *d_out,
                      int64_t out_stride, void *stream) {
    NvtxRange range("ftmoe_latent_read");
    latent::ReadParams p{};
    int rc = check_latent(kvc, p.c);
    if (rc) return rc;
    if ((rc = check_batch(batch, p.c.page_shift, p.bt))) return rc;
    if (rows < 0) return fail(FTMOE_ERR_INVALID_ARG, "rows=%d", rows);
    if (rows == 0 || p.bt.batch == 0 || p.bt.max_kv == 0) return FTMOE_OK;
    if (!d_cu_rows) return fail(FTMOE_ERR_INVALID_ARG, "null cu_rows");
    if (!d_out || !aligned16(d_out) || out_stride % 8 || out_stride < p.c.latent + p.c.rope)
        return fail(FTMOE_ERR_INVALID_ARG, "out must be non-null and 16-byte aligned, rows a multiple of 8 elements apart, at least latent + rope");
    p.cu_rows = d_cu_rows, p.rows = rows, p.out = static_cast<uint16_t *>(d_out), p.out_stride = out_stride;
    return cuda_rc(latent::launch_read(p, kvc->dtype == FTMOE_DT_BF16, static_cast<cudaStream_t>(stream)), "latent read kernel");
}

int ftmoe_latent_attention_workspace_bytes(const ftmoe_latent_cache *kvc, const ftmoe_kv_batch *batch, int32_t q_heads, int32_t causal,
                                           size_t *bytes) {
    if (!bytes) return fail(FTMOE_ERR_INVALID_ARG, "null bytes");
    latent::AttendParams p{};
    int rc = attend_params(kvc, batch, q_heads, causal, p), sms = 0;
    if (rc) return rc;
    if ((rc = num_sms(sms))) return rc;
    *bytes = latent::attend_workspace(p, sms, nullptr);
    return FTMOE_OK;
}

int ftmoe_latent_attention(const ftmoe_latent_cache *kvc, const ftmoe_kv_batch *batch, const ftmoe_rows *q, const ftmoe_rows *q_rope,
                           int32_t q_heads, float scale, int32_t causal, const ftmoe_rows *out, float *d_lse, void *d_workspace,
                           size_t workspace_bytes, void *stream) {
    NvtxRange range("ftmoe_latent_attention");
    latent::AttendParams p{};
    int rc = attend_params(kvc, batch, q_heads, causal, p), sms = 0;
    if (rc) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FTMOE_ERR_INVALID_ARG, "scale must be positive and finite");
    if ((rc = check_rows(q, "q", q_heads, p.c.latent, p.q))) return rc;
    if ((rc = check_rows(q_rope, "q_rope", q_heads, p.c.rope, p.q_rope))) return rc;
    if ((rc = check_rows(out, "out", q_heads, p.c.latent, p.out))) return rc;
    if (p.out.d == p.q.d && ((p.bt.tokens > 1 && p.out.token != p.q.token) || (q_heads > 1 && p.out.head != p.q.head)))
        return fail(FTMOE_ERR_INVALID_ARG, "out over q needs q's strides");
    if (p.bt.tokens == 0 || p.bt.batch == 0 || p.bt.max_q == 0) return FTMOE_OK;
    if ((rc = num_sms(sms))) return rc;
    p.scale = scale, p.lse = d_lse;
    if ((rc = check_workspace(latent::attend_workspace(p, sms, static_cast<unsigned char *>(d_workspace)), d_workspace, workspace_bytes))) return rc;
    return cuda_rc(latent::launch_attend(p, kvc->dtype == FTMOE_DT_BF16, sms, static_cast<cudaStream_t>(stream)), "latent attention kernels");
}

int ftmoe_expanded_attention_workspace_bytes(const ftmoe_row_batch *batch, int32_t dtype, int32_t heads, int32_t nope, int32_t rope,
                                             int32_t v_dim, int32_t causal, size_t *bytes) {
    if (!bytes) return fail(FTMOE_ERR_INVALID_ARG, "null bytes");
    latent::ExpandParams p{};
    int rc = expand_params(batch, dtype, heads, nope, rope, v_dim, causal, p), sms = 0;
    if (rc) return rc;
    if ((rc = num_sms(sms))) return rc;
    *bytes = latent::expand_workspace(p, sms, nullptr);
    return FTMOE_OK;
}

int ftmoe_expanded_attention(const ftmoe_row_batch *batch, int32_t dtype, int32_t heads, int32_t nope, int32_t rope, int32_t v_dim,
                             const ftmoe_rows *q, const ftmoe_rows *k, const void *d_k_rope, int64_t k_rope_stride, const ftmoe_rows *v,
                             float scale, int32_t causal, const ftmoe_rows *out, float *d_lse, void *d_workspace, size_t workspace_bytes,
                             void *stream) {
    NvtxRange range("ftmoe_expanded_attention");
    latent::ExpandParams p{};
    int rc = expand_params(batch, dtype, heads, nope, rope, v_dim, causal, p), sms = 0;
    if (rc) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FTMOE_ERR_INVALID_ARG, "scale must be positive and finite");
    if ((rc = check_rows(q, "q", heads, nope + rope, p.q))) return rc;
    if ((rc = check_rows(out, "out", heads, v_dim, p.out))) return rc;
    if (p.rows > 0) {
        if ((rc = check_rows(k, "k", heads, nope, p.k))) return rc;
        if ((rc = check_rows(v, "v", heads, v_dim, p.v))) return rc;
        if (!d_k_rope || !aligned16(d_k_rope) || k_rope_stride % 8 || k_rope_stride < rope)
            return fail(FTMOE_ERR_INVALID_ARG, "k_rope must be non-null and 16-byte aligned, rows a multiple of 8 elements apart");
    }
    if (p.tokens == 0 || p.batch == 0 || p.max_q == 0) return FTMOE_OK;
    if ((rc = num_sms(sms))) return rc;
    p.key = static_cast<const uint16_t *>(d_k_rope), p.key_stride = k_rope_stride, p.scale = scale, p.lse = d_lse;
    if ((rc = check_workspace(latent::expand_workspace(p, sms, static_cast<unsigned char *>(d_workspace)), d_workspace, workspace_bytes))) return rc;
    return cuda_rc(latent::launch_expand(p, dtype == FTMOE_DT_BF16, sms, static_cast<cudaStream_t>(stream)), "expanded attention kernels");
}

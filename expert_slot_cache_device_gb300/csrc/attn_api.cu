// Host side of the attention entry points: argument checks and launches. See include/ftmoe.h
// for the contract of every entry point.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include <nvtx3/nvToolsExt.h>

#include "internal.cuh"
#include "kv.cuh"

using namespace ftmoe;

namespace {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

int fail(int code, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return report_error(code, msg);
}

int cuda_rc(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return FTMOE_OK;
    cudaGetLastError();  // reported here: not again by the caller's next call
    return fail(FTMOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// SMs of the current device, asked for once a device.
int num_sms(int &n) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return FTMOE_OK;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return cuda_rc(e, "device query");
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0; }

int check_cache(const ftmoe_kv_cache *c, kv::View &v) {
    if (!c) return fail(FTMOE_ERR_INVALID_ARG, "null cache view");
    if (c->dtype != FTMOE_DT_BF16 && c->dtype != FTMOE_DT_F16)
        return fail(FTMOE_ERR_FORMAT, "cache dtype %d: bf16 or f16", c->dtype);
    if (!c->d_k || !c->d_v || !aligned16(c->d_k) || !aligned16(c->d_v))
        return fail(FTMOE_ERR_INVALID_ARG, "k and v pages must be non-null and 16-byte aligned");
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(FTMOE_ERR_INVALID_ARG, "page_size=%d: a power of two in [16, 256]", c->page_size);
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
        return fail(FTMOE_ERR_INVALID_ARG, "head_dim=%d: a multiple of 16, at most 256", c->head_dim);
    if (c->num_pages <= 0 || c->kv_heads <= 0 || c->kv_heads > 65535)
        return fail(FTMOE_ERR_INVALID_ARG, "num_pages=%d, kv_heads=%d", c->num_pages, c->kv_heads);
    if (!stride_ok(c->k_page) || !stride_ok(c->k_slot) || !stride_ok(c->k_head) || !stride_ok(c->v_page) ||
        !stride_ok(c->v_slot) || !stride_ok(c->v_head))
        return fail(FTMOE_ERR_INVALID_ARG, "cache strides must be positive multiples of 8 elements");
    v.k = static_cast<uint16_t *>(c->d_k), v.v = static_cast<uint16_t *>(c->d_v);
    v.k_page = c->k_page, v.k_slot = c->k_slot, v.k_head = c->k_head;
    v.v_page = c->v_page, v.v_slot = c->v_slot, v.v_head = c->v_head;
    v.num_pages = c->num_pages, v.kv_heads = c->kv_heads, v.dim = c->head_dim, v.status = c->d_status;
    for (v.page_shift = 4; (1 << v.page_shift) < c->page_size;) v.page_shift++;
    return FTMOE_OK;
}

int check_batch(const ftmoe_kv_batch *b, const kv::View &c, kv::Batch &v) {
    if (!b) return fail(FTMOE_ERR_INVALID_ARG, "null batch");
    if (b->batch < 0 || b->batch > 65535) return fail(FTMOE_ERR_INVALID_ARG, "batch=%d outside [0, 65535]", b->batch);
    if (b->tokens < 0 || b->max_q < 0 || b->max_kv < 0 || b->max_pages < 0)
        return fail(FTMOE_ERR_INVALID_ARG, "negative tokens, max_q, max_kv or max_pages");
    if (b->batch > 0 && (!b->d_block_table || !b->d_kv_lens || !b->d_cu_q))
        return fail(FTMOE_ERR_INVALID_ARG, "null block table, kv_lens or cu_q");
    if (b->table_stride < b->max_pages) return fail(FTMOE_ERR_INVALID_ARG, "table_stride below max_pages");
    if (((int64_t)b->max_pages << c.page_shift) < b->max_kv)
        return fail(FTMOE_ERR_INVALID_ARG, "max_kv=%d does not fit %d pages", b->max_kv, b->max_pages);
    if (b->max_kv > 1 << 30) return fail(FTMOE_ERR_INVALID_ARG, "max_kv=%d above 2^30", b->max_kv);
    v.table = b->d_block_table, v.table_stride = b->table_stride, v.kv_lens = b->d_kv_lens, v.cu_q = b->d_cu_q;
    v.batch = b->batch, v.tokens = b->tokens, v.max_q = b->max_q, v.max_kv = b->max_kv;
    if (v.max_q > v.tokens) v.max_q = v.tokens;
    return FTMOE_OK;
}

int check_rows(const ftmoe_rows *r, const char *name, int heads, int dim, kv::Rows &v) {
    if (!r || !r->d || !aligned16(r->d)) return fail(FTMOE_ERR_INVALID_ARG, "%s must be non-null and 16-byte aligned", name);
    if (!stride_ok(r->token) || !stride_ok(r->head))
        return fail(FTMOE_ERR_INVALID_ARG, "%s strides must be positive multiples of 8 elements", name);
    if (heads > 1 && r->head < dim) return fail(FTMOE_ERR_INVALID_ARG, "%s heads overlap", name);
    v.d = static_cast<uint16_t *>(r->d), v.token = r->token, v.head = r->head;
    return FTMOE_OK;
}

int attend_params(const ftmoe_kv_cache *kvc, const ftmoe_kv_batch *batch, int q_heads, int window, int causal,
                  kv::AttendParams &p) {
    int rc = check_cache(kvc, p.c);
    if (rc) return rc;
    if ((rc = check_batch(batch, p.c, p.bt))) return rc;
    if (p.c.dim != 64 && p.c.dim != 128)
        return fail(FTMOE_ERR_FORMAT, "attention takes head_dim 64 or 128, not %d", p.c.dim);
    if (q_heads <= 0 || q_heads % p.c.kv_heads || q_heads > 65535)
        return fail(FTMOE_ERR_INVALID_ARG, "q_heads=%d: a multiple of kv_heads=%d", q_heads, p.c.kv_heads);
    if (window < 0) return fail(FTMOE_ERR_INVALID_ARG, "window=%d", window);
    if (window && !causal) return fail(FTMOE_ERR_INVALID_ARG, "a window needs causal attention");
    if (q_heads / p.c.kv_heads > 128)
        return fail(FTMOE_ERR_FORMAT, "%d query heads a key head: at most 128", q_heads / p.c.kv_heads);
    p.q_heads = q_heads, p.group = q_heads / p.c.kv_heads, p.causal = causal != 0;
    p.window = window < p.bt.max_kv ? window : 0;  // a wider one hides no slot, and sums with it could pass 32 bits
    p.item_tokens = 2 * (128 / p.group);
    return FTMOE_OK;
}

int check_w4(int N, int K, int group) {
    if (N <= 0 || K <= 0) return fail(FTMOE_ERR_INVALID_ARG, "N=%d, K=%d must be positive", N, K);
    if (group != 32 && group != 64 && group != 128) return fail(FTMOE_ERR_FORMAT, "group=%d: 32, 64 or 128", group);
    if (K % group) return fail(FTMOE_ERR_INVALID_ARG, "K=%d is not a multiple of group=%d", K, group);
    if (N > 1 << 26 || K > 1 << 26) return fail(FTMOE_ERR_INVALID_ARG, "N=%d, K=%d above 2^26", N, K);
    return FTMOE_OK;
}

}  // namespace

int ftmoe_rope_append(const ftmoe_kv_cache *kvc, const ftmoe_kv_batch *batch, const ftmoe_rotary *rotary,
                      const ftmoe_rows *q, const ftmoe_rows *q_out, int32_t q_heads, const ftmoe_rows *k,
                      const ftmoe_rows *v, const int32_t *d_positions, void *stream) {
    NvtxRange range("ftmoe_rope_append");
    kv::AppendParams p{};
    int rc = check_cache(kvc, p.c);
    if (rc) return rc;
    if ((rc = check_batch(batch, p.c, p.bt))) return rc;
    if (!rotary) return fail(FTMOE_ERR_INVALID_ARG, "null rotary plan");
    if (rotary->rot_dim < 0 || rotary->rot_dim > p.c.dim || rotary->rot_dim % 16)
        return fail(FTMOE_ERR_INVALID_ARG, "rot_dim=%d: a multiple of 16, at most head_dim=%d", rotary->rot_dim, p.c.dim);
    if (rotary->rot_dim && (!rotary->d_freq || ((uintptr_t)rotary->d_freq & 7)))
        return fail(FTMOE_ERR_INVALID_ARG, "d_freq must be non-null and 8-byte aligned");
    if (!std::isfinite(rotary->factor)) return fail(FTMOE_ERR_INVALID_ARG, "rotary factor is not finite");
    if (q_heads < 0 || q_heads > 65535) return fail(FTMOE_ERR_INVALID_ARG, "q_heads=%d", q_heads);
    if (q_heads > 0) {
        if ((rc = check_rows(q, "q", q_heads, p.c.dim, p.q))) return rc;
        if ((rc = check_rows(q_out, "q_out", q_heads, p.c.dim, p.q_out))) return rc;
    }
    if ((rc = check_rows(k, "k", p.c.kv_heads, p.c.dim, p.k))) return rc;
    if ((rc = check_rows(v, "v", p.c.kv_heads, p.c.dim, p.v))) return rc;
    if (!d_positions) return fail(FTMOE_ERR_INVALID_ARG, "null positions");
    if (p.bt.tokens == 0 || p.bt.batch == 0) return FTMOE_OK;
    p.q_heads = q_heads, p.rot = rotary->rot_dim, p.interleaved = rotary->interleaved != 0, p.factor = rotary->factor;
    p.freq = reinterpret_cast<const float2 *>(rotary->d_freq);
    p.pos = d_positions;
    return cuda_rc(kv::launch_append(p, kvc->dtype == FTMOE_DT_BF16, static_cast<cudaStream_t>(stream)), "append kernel");
}

int ftmoe_paged_attention_workspace_bytes(const ftmoe_kv_cache *kvc, const ftmoe_kv_batch *batch, int32_t q_heads,
                                          int32_t window, int32_t causal, int32_t want_mass, size_t *bytes) {
    if (!bytes) return fail(FTMOE_ERR_INVALID_ARG, "null bytes");
    kv::AttendParams p{};
    int rc = attend_params(kvc, batch, q_heads, window, causal, p), sms = 0;
    if (rc) return rc;
    if ((rc = num_sms(sms))) return rc;
    float want = 0.f;
    p.mass = want_mass ? &want : nullptr;
    *bytes = kv::attend_workspace(p, sms, nullptr);
    return FTMOE_OK;
}

int ftmoe_paged_attention(const ftmoe_kv_cache *kvc, const ftmoe_kv_batch *batch, const ftmoe_rows *q, int32_t q_heads,
                          float scale, int32_t window, int32_t causal, const float *d_sinks, const ftmoe_rows *out,
                          float *d_lse, float *d_mass, int64_t mass_seq, int64_t mass_head, void *d_workspace,
                          size_t workspace_bytes, void *stream) {
    NvtxRange range("ftmoe_paged_attention");
    kv::AttendParams p{};
    int rc = attend_params(kvc, batch, q_heads, window, causal, p), sms = 0;
    if (rc) return rc;
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(FTMOE_ERR_INVALID_ARG, "scale must be positive and finite");
    if ((rc = check_rows(q, "q", q_heads, p.c.dim, p.q))) return rc;
    if ((rc = check_rows(out, "out", q_heads, p.c.dim, p.out))) return rc;
    if (p.out.d == p.q.d && ((p.bt.tokens > 1 && p.out.token != p.q.token) || (q_heads > 1 && p.out.head != p.q.head)))
        return fail(FTMOE_ERR_INVALID_ARG, "out over q needs q's strides");
    if (d_mass && (mass_head < p.bt.max_kv || mass_seq < 0))
        return fail(FTMOE_ERR_INVALID_ARG, "mass rows of %lld elements for max_kv=%d", (long long)mass_head, p.bt.max_kv);
    if (p.bt.tokens == 0 || p.bt.batch == 0 || p.bt.max_q == 0) return FTMOE_OK;
    if ((rc = num_sms(sms))) return rc;
    p.scale = scale, p.sinks = d_sinks, p.lse = d_lse, p.mass = d_mass, p.mass_seq = mass_seq, p.mass_head = mass_head;
    const size_t need = kv::attend_workspace(p, sms, static_cast<unsigned char *>(d_workspace));
    if (need && (!d_workspace || ((uintptr_t)d_workspace & 255) || workspace_bytes < need))
        return fail(FTMOE_ERR_INVALID_ARG, "workspace: %zu bytes at a 256-byte boundary needed, %zu given", need, workspace_bytes);
    return cuda_rc(kv::launch_attend(p, kvc->dtype == FTMOE_DT_BF16, sms, static_cast<cudaStream_t>(stream)),
                   "attention kernels");
}

int ftmoe_kv_evict(const ftmoe_kv_cache *kvc, const ftmoe_kv_batch *batch, const float *d_mass, int64_t mass_seq,
                   int64_t mass_head, int32_t budget, int32_t recent, const int32_t *d_new_table, int64_t new_stride,
                   int32_t *d_kept, float *d_new_mass, int32_t *d_new_lens, void *stream) {
    NvtxRange range("ftmoe_kv_evict");
    kv::EvictParams p{};
    int rc = check_cache(kvc, p.c), sms = 0;
    if (rc) return rc;
    if ((rc = check_batch(batch, p.c, p.bt))) return rc;
    if (budget < 1 || recent < 0 || recent > budget)
        return fail(FTMOE_ERR_INVALID_ARG, "budget=%d, recent=%d: 0 <= recent <= budget, budget >= 1", budget, recent);
    if (!d_mass || !d_new_table || !d_kept || !d_new_mass || !d_new_lens)
        return fail(FTMOE_ERR_INVALID_ARG, "null mass, new table, kept, new mass or new lens");
    if (mass_head < p.bt.max_kv || mass_seq < 0)
        return fail(FTMOE_ERR_INVALID_ARG, "mass rows of %lld elements for max_kv=%d", (long long)mass_head, p.bt.max_kv);
    const int64_t most = budget < p.bt.max_kv ? budget : p.bt.max_kv;
    if (new_stride << p.c.page_shift < most)
        return fail(FTMOE_ERR_INVALID_ARG, "new table rows of %lld pages for %lld slots", (long long)new_stride, (long long)most);
    if (p.bt.batch == 0) return FTMOE_OK;
    if ((rc = num_sms(sms))) return rc;
    p.mass = d_mass, p.mass_seq = mass_seq, p.mass_head = mass_head, p.budget = budget, p.recent = recent;
    p.new_table = d_new_table, p.new_stride = new_stride, p.kept = d_kept, p.new_mass = d_new_mass, p.new_lens = d_new_lens;
    return cuda_rc(kv::launch_evict(p, sms, static_cast<cudaStream_t>(stream)), "eviction kernels");
}

int ftmoe_w4_packed_bytes(int32_t N, int32_t K, int32_t group, int32_t has_zeros, size_t *bytes) {
    if (!bytes) return fail(FTMOE_ERR_INVALID_ARG, "null bytes");
    if (int rc = check_w4(N, K, group)) return rc;
    const w4::Geometry g = w4::geometry(N, K, group, has_zeros != 0);
    *bytes = (size_t)(g.code_bytes + g.meta_bytes);
    return FTMOE_OK;
}

int ftmoe_w4_pack(const void *d_codes, const void *d_scales, const void *d_zeros, int32_t N, int32_t K, int32_t group,
                  void *d_packed, size_t packed_bytes, void *stream) {
    if (int rc = check_w4(N, K, group)) return rc;
    const w4::Geometry g = w4::geometry(N, K, group, d_zeros != nullptr);
    if (!d_codes || !d_scales) return fail(FTMOE_ERR_INVALID_ARG, "null codes or scales");
    if (!d_packed || ((uintptr_t)d_packed & 255) || packed_bytes < (size_t)(g.code_bytes + g.meta_bytes))
        return fail(FTMOE_ERR_INVALID_ARG, "packed weights: %lld bytes at a 256-byte boundary needed, %zu given",
                    (long long)(g.code_bytes + g.meta_bytes), packed_bytes);
    return cuda_rc(w4::launch_pack(g, static_cast<const uint8_t *>(d_codes), static_cast<const uint16_t *>(d_scales),
                                   static_cast<const uint8_t *>(d_zeros), static_cast<unsigned char *>(d_packed),
                                   static_cast<cudaStream_t>(stream)),
                   "weight packing kernel");
}

int ftmoe_w4_matvec(const void *d_packed, int32_t N, int32_t K, int32_t group, int32_t has_zeros, int32_t dtype,
                    const void *d_x, int64_t x_stride, int32_t tokens, void *d_y, int64_t y_stride, void *stream) {
    NvtxRange range("ftmoe_w4_matvec");
    if (int rc = check_w4(N, K, group)) return rc;
    if (dtype != FTMOE_DT_BF16 && dtype != FTMOE_DT_F16) return fail(FTMOE_ERR_FORMAT, "dtype %d: bf16 or f16", dtype);
    if (tokens < 0) return fail(FTMOE_ERR_INVALID_ARG, "tokens=%d", tokens);
    if (tokens == 0) return FTMOE_OK;
    if (!d_packed || ((uintptr_t)d_packed & 255)) return fail(FTMOE_ERR_INVALID_ARG, "packed weights must be 256-byte aligned");
    if (!d_x || !aligned16(d_x) || x_stride < K || x_stride % 8)
        return fail(FTMOE_ERR_INVALID_ARG, "x must be 16-byte aligned with rows a multiple of 8 elements apart, at least K");
    if (!d_y || y_stride < N) return fail(FTMOE_ERR_INVALID_ARG, "null y, or rows closer than N");
    int sms = 0;
    if (int rc = num_sms(sms)) return rc;
    w4::MatvecParams p{};
    p.g = w4::geometry(N, K, group, has_zeros != 0);
    p.packed = static_cast<const unsigned char *>(d_packed);
    p.x = static_cast<const uint16_t *>(d_x), p.y = static_cast<uint16_t *>(d_y);
    p.x_stride = x_stride, p.y_stride = y_stride, p.tokens = tokens;
    return cuda_rc(w4::launch_matvec(p, dtype == FTMOE_DT_BF16, sms, static_cast<cudaStream_t>(stream)), "4-bit product kernel");
}

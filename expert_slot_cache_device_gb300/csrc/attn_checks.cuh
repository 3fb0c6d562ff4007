// What the host sides of the attention entry points share: error reports, device queries, checks
// of the arguments they have in common.
#pragma once

#include <atomic>
#include <cstdarg>
#include <cstdio>

#include <nvtx3/nvToolsExt.h>

#include "internal.cuh"
#include "kv.cuh"

namespace ftmoe {
namespace checks {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

inline int fail(int code, const char *fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    return report_error(code, msg);
}

inline int cuda_rc(cudaError_t e, const char *what) {
    if (e == cudaSuccess) return FTMOE_OK;
    cudaGetLastError();  // reported here: not again by the caller's next call
    return fail(FTMOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// SMs of the current device, asked for once a device.
inline int num_sms(int &n) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return FTMOE_OK;
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(n, std::memory_order_relaxed);
    return cuda_rc(e, "device query");
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
inline bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0; }

inline int check_batch(const ftmoe_kv_batch *b, int page_shift, kv::Batch &v) {
    if (!b) return fail(FTMOE_ERR_INVALID_ARG, "null batch");
    if (b->batch < 0 || b->batch > 65535) return fail(FTMOE_ERR_INVALID_ARG, "batch=%d outside [0, 65535]", b->batch);
    if (b->tokens < 0 || b->max_q < 0 || b->max_kv < 0 || b->max_pages < 0)
        return fail(FTMOE_ERR_INVALID_ARG, "negative tokens, max_q, max_kv or max_pages");
    if (b->batch > 0 && (!b->d_block_table || !b->d_kv_lens || !b->d_cu_q))
        return fail(FTMOE_ERR_INVALID_ARG, "null block table, kv_lens or cu_q");
    if (b->table_stride < b->max_pages) return fail(FTMOE_ERR_INVALID_ARG, "table_stride below max_pages");
    if (((int64_t)b->max_pages << page_shift) < b->max_kv)
        return fail(FTMOE_ERR_INVALID_ARG, "max_kv=%d does not fit %d pages", b->max_kv, b->max_pages);
    if (b->max_kv > 1 << 30) return fail(FTMOE_ERR_INVALID_ARG, "max_kv=%d above 2^30", b->max_kv);
    v.table = b->d_block_table, v.table_stride = b->table_stride, v.kv_lens = b->d_kv_lens, v.cu_q = b->d_cu_q;
    v.batch = b->batch, v.tokens = b->tokens, v.max_q = b->max_q, v.max_kv = b->max_kv;
    if (v.max_q > v.tokens) v.max_q = v.tokens;
    return FTMOE_OK;
}

inline int check_rows(const ftmoe_rows *r, const char *name, int heads, int dim, kv::Rows &v) {
    if (!r || !r->d || !aligned16(r->d)) return fail(FTMOE_ERR_INVALID_ARG, "%s must be non-null and 16-byte aligned", name);
    if (!stride_ok(r->token) || !stride_ok(r->head))
        return fail(FTMOE_ERR_INVALID_ARG, "%s strides must be positive multiples of 8 elements", name);
    if (heads > 1 && r->head < dim) return fail(FTMOE_ERR_INVALID_ARG, "%s heads overlap", name);
    v.d = static_cast<uint16_t *>(r->d), v.token = r->token, v.head = r->head;
    return FTMOE_OK;
}

}  // namespace checks
}  // namespace ftmoe

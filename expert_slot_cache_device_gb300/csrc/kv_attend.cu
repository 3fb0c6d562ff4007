// Which attention kernels a call runs, and its workspace.
#include "kv_attend.cuh"

namespace ftmoe {
namespace kv {
namespace {

// The single-token kernel takes calls whose rows a (sequence, key head) fit its 16.
bool is_step(const AttendParams &p) { return (int64_t)p.bt.max_q * p.group <= kStepRows; }

}  // namespace

size_t attend_workspace(AttendParams &p, int num_sms, unsigned char *base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char *at = base ? base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    p.part_o = nullptr, p.part_ml = nullptr, p.join = nullptr, p.lse2 = nullptr, p.logits = nullptr, p.mass_parts = nullptr, p.mass_split = 1;
    // a part that starts an item and one that goes on with one for each CTA
    const size_t ctas = is_step(p) ? step_ctas(p, num_sms) : chunk_ctas(p, num_sms);
    const size_t rows = 2 * ctas * (is_step(p) ? kStepRows : chunk_rows());
    if (is_step(p) ? step_parts(p, num_sms) : chunk_parts(p, num_sms)) {
        p.part_o = reinterpret_cast<float *>(take(rows * p.c.dim * 4));
        p.part_ml = reinterpret_cast<float2 *>(take(rows * 8));
        p.join = reinterpret_cast<int4 *>(take(ctas * 16));
    }
    if (p.mass) {
        p.lse2 = reinterpret_cast<float *>(take((size_t)p.bt.tokens * p.q_heads * 4));
        if (is_step(p)) {
            p.logit_rows = p.bt.max_q * p.group;
            p.logit_stride = ((int64_t)p.bt.max_kv + 127) & ~(int64_t)127;
            p.logits = reinterpret_cast<float *>(take((size_t)p.bt.batch * p.c.kv_heads * p.logit_rows * p.logit_stride * 4));
        } else if ((p.mass_split = mass_split(p, num_sms)) > 1) {
            p.logit_stride = ((int64_t)p.bt.max_kv + 127) & ~(int64_t)127;
            p.mass_parts = reinterpret_cast<float *>(take((size_t)p.mass_split * p.bt.batch * p.c.kv_heads * p.logit_stride * 4));
        }
    }
    return off;
}

cudaError_t launch_attend(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    if (is_step(p)) return launch_step(p, bf16, num_sms, st);
    const cudaError_t e = launch_chunk(p, bf16, num_sms, st);
    return e == cudaSuccess && p.mass ? launch_mass(p, bf16, num_sms, st) : e;
}

}  // namespace kv
}  // namespace ftmoe

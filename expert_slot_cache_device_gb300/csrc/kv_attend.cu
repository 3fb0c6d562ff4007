// Which attention kernels a call runs, and its workspace.
#include "kv_attend.cuh"

namespace ftmoe {
namespace kv {
namespace {

// The single-token kernel takes calls whose rows a (sequence, key head) fit its 16.
bool is_step(const AttendParams &p) { return (int64_t)p.bt.max_q * p.group <= kStepRows; }

// Rows of `heads` heads of `per` 16-byte chunks, one chunk a thread at a time.
__global__ void __launch_bounds__(256) copy_rows(const Rows from, const Rows to, int64_t chunks, int heads, int per) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < chunks; i += gridDim.x * 256ll) {
        const int64_t row = i / per, t = row / heads;
        const int c = (int)(i - row * per) * 8, h = (int)(row - t * heads);
        *reinterpret_cast<uint4 *>(to.d + t * to.token + h * to.head + c) = *reinterpret_cast<const uint4 *>(from.d + t * from.token + h * from.head + c);
    }
}

}  // namespace

size_t attend_workspace(AttendParams &p, int num_sms, unsigned char *base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        unsigned char *at = base ? base + off : nullptr;
        off += (bytes + 255) & ~(size_t)255;
        return at;
    };
    p.part_o = nullptr, p.part_ml = nullptr, p.join = nullptr, p.lse2 = nullptr, p.logits = nullptr, p.mass_parts = nullptr, p.mass_split = 1, p.q_copy = nullptr;
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
        } else {
            if ((p.mass_split = mass_split(p, num_sms)) > 1) {
                p.logit_stride = ((int64_t)p.bt.max_kv + 127) & ~(int64_t)127;
                p.mass_parts = reinterpret_cast<float *>(take((size_t)p.mass_split * p.bt.batch * p.c.kv_heads * p.logit_stride * 4));
            }
            p.q_copy = reinterpret_cast<uint16_t *>(take((size_t)p.bt.tokens * p.q_heads * p.c.dim * 2));
        }
    }
    return off;
}

cudaError_t launch_attend(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    if (is_step(p)) return launch_step(p, bf16, num_sms, st);
    AttendParams m = p;  // of the mass pass, which reads the queries after the outputs are written
    cudaError_t e = cudaSuccess;
    if (p.mass && p.out.d == p.q.d) {
        m.q = Rows{p.q_copy, (int64_t)p.q_heads * p.c.dim, p.c.dim};
        const int64_t chunks = (int64_t)p.bt.tokens * p.q_heads * (p.c.dim >> 3), blocks = (chunks + 255) / 256, most = 16 * num_sms;
        copy_rows<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(p.q, m.q, chunks, p.q_heads, p.c.dim >> 3);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if ((e = launch_chunk(p, bf16, num_sms, st)) != cudaSuccess || !p.mass) return e;
    return launch_mass(m, bf16, num_sms, st);
}

}  // namespace kv
}  // namespace ftmoe

// Which attention kernel a call runs, its workspace, and the mass pass of chunks: one warp a
// (sequence, key head, slot) adds 2^(s - lse) over the rows that see the slot, so each mass element
// has one writer and one order.
#include "kv_attend.cuh"

namespace ftmoe {
namespace kv {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

template <bool BF, int D>
__global__ void __launch_bounds__(128) mass_slots(const AttendParams p, const float *lse) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, j = blockIdx.x * 4 + (threadIdx.x >> 5), hk = blockIdx.y, b = blockIdx.z;
    const Seq s = seq_info(p.bt, b, p.c.status);
    if (j >= s.kv_len) return;
    const int first = s.kv_len - s.q_len;
    int lo = p.causal ? j - first : 0, hi = s.q_len;  // rows that see slot j
    if (p.window && j + p.window - first < hi) hi = j + p.window - first;
    if (lo < 0) lo = 0;
    if (first < 0 && lo < -first) lo = -first;
    if (lo >= hi) return;
    const int page = page_of(p.c, p.bt, b, j), row = j & ((1 << p.c.page_shift) - 1);
    if (page < 0) return;
    float k[E], sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; e++) k[e] = to_f<BF>(p.c.k[k_at(p.c, page, row, hk) + lane * E + e]);
    for (int i = lo; i < hi; i++)
        for (int h = hk * p.group; h < (hk + 1) * p.group; h++) {
            const int64_t t = s.q0 + i;
            float d = 0.f;
#pragma unroll
            for (int e = 0; e < E; e++) d += k[e] * to_f<BF>(p.q.d[t * p.q.token + h * p.q.head + lane * E + e]);
            const float z = lse[t * p.q_heads + h];
            if (z != -INFINITY) sum += ex2(warp_sum(d) * p.scale * kLog2e - z);
        }
    if (lane == 0) p.mass[b * p.mass_seq + hk * p.mass_head + j] += sum;
}

template <bool BF, int D>
cudaError_t launch_mass(const AttendParams &p, cudaStream_t st) {
    mass_slots<BF, D><<<dim3((p.bt.max_kv + 3) / 4, p.c.kv_heads, p.bt.batch), 128, 0, st>>>(p, p.lse2);
    return cudaGetLastError();
}

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
    p.part_o = nullptr, p.part_ml = nullptr, p.lse2 = nullptr, p.logits = nullptr;
    if (is_step(p)) {
        const size_t slots = 2 * (size_t)step_ctas(p, num_sms);
        p.part_o = reinterpret_cast<float *>(take(slots * kStepRows * p.c.dim * 4));
        p.part_ml = reinterpret_cast<float2 *>(take(slots * kStepRows * 8));
    } else {
        const size_t rows = chunk_part_rows(p, num_sms);
        p.part_o = reinterpret_cast<float *>(take(rows * p.c.dim * 4));
        p.part_ml = reinterpret_cast<float2 *>(take(rows * 8));
    }
    if (p.mass) {
        p.lse2 = reinterpret_cast<float *>(take((size_t)p.bt.tokens * p.q_heads * 4));
        if (is_step(p)) {
            p.logit_rows = p.bt.max_q * p.group;
            p.logit_stride = ((int64_t)p.bt.max_kv + 127) & ~(int64_t)127;
            p.logits = reinterpret_cast<float *>(take((size_t)p.bt.batch * p.c.kv_heads * p.logit_rows * p.logit_stride * 4));
        }
    }
    return off;
}

cudaError_t launch_attend(const AttendParams &p, bool bf16, int num_sms, cudaStream_t st) {
    if (is_step(p)) return launch_step(p, bf16, num_sms, st);
    cudaError_t e = launch_chunk(p, bf16, num_sms, st);
    if (e != cudaSuccess || !p.mass) return e;
    if (p.c.dim == 64) return bf16 ? launch_mass<true, 64>(p, st) : launch_mass<false, 64>(p, st);
    return bf16 ? launch_mass<true, 128>(p, st) : launch_mass<false, 128>(p, st);
}

}  // namespace kv
}  // namespace ftmoe

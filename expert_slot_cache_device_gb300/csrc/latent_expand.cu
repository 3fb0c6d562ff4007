// Expanded latent attention, one CTA a (token, head).
#include "kv_split.cuh"
#include "latent.cuh"

namespace ftmoe {
namespace latent {
namespace {

using kv::to_f;

constexpr int kThreads = 256, kTile = 64;

// out = sum_j exp(s_j) value_j / sum_j exp(s_j) of one row over n slots; key(j, e) and value(j, e) are elements.
template <bool BF, typename Key, typename Value>
__device__ void row_attend(const float *q, int kd, int vd, int n, float scale, uint16_t *out, float *lse, Key key, Value value) {
    __shared__ float s_p[kTile];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float c2 = scale * kv::kLog2e;
    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    for (int j0 = 0; j0 < n; j0 += kTile) {
        __syncthreads();
        for (int k = warp; k < kTile; k += kThreads / 32) {
            float s = 0.f;
            if (j0 + k < n)
                for (int e = lane; e < kd; e += 32) s += q[e] * key(j0 + k, e);
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
            if (lane == 0) s_p[k] = j0 + k < n ? s * c2 : -INFINITY;
        }
        __syncthreads();
        float top = m;
        for (int k = 0; k < kTile; k++) top = fmaxf(top, s_p[k]);
        const float base = top == -INFINITY ? 0.f : top, f = kv::ex2(m - base);
        m = top, l *= f, acc[0] *= f, acc[1] *= f;
        for (int k = 0; k < kTile && j0 + k < n; k++) {
            const float p = kv::ex2(s_p[k] - base);
            l += p;
            for (int i = 0; i < 2; i++)
                if (tid + i * kThreads < vd) acc[i] += p * value(j0 + k, tid + i * kThreads);
        }
    }
    for (int i = 0; i < 2; i++)
        if (tid + i * kThreads < vd) out[tid + i * kThreads] = kv::from_f<BF>(l == 0.f ? 0.f : acc[i] / l);
    if (tid == 0 && lse) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

template <bool BF>
__global__ void __launch_bounds__(kThreads) expand_plain(const ExpandParams p) {
    __shared__ float s_q[192];
    __shared__ int s_seq;
    const int t = blockIdx.x / p.heads, h = blockIdx.x - t * p.heads, tid = threadIdx.x, kd = p.nope + p.rope;
    if (tid == 0) s_seq = -1;
    __syncthreads();
    for (int b = tid; b < p.batch; b += kThreads) {
        const kv::Seq s = row_seq(p, b, p.status).s;
        if (t >= s.q0 && t < s.q0 + s.q_len) s_seq = b;
    }
    for (int e = tid; e < kd; e += kThreads) s_q[e] = to_f<BF>(p.q.d[t * p.q.token + h * p.q.head + e]);
    __syncthreads();
    const int b = s_seq;
    if (b < 0) return;
    const RowSeq r = row_seq(p, b, nullptr);
    const kv::Range seen = kv::visible(r.s, t - r.s.q0, t - r.s.q0 + 1, 0, p.causal);
    auto key = [&](int j, int e) -> float {
        const int64_t row = r.row0 + j;
        return to_f<BF>(e < p.nope ? p.k.d[row * p.k.token + h * p.k.head + e] : p.key[row * p.key_stride + e - p.nope]);
    };
    auto value = [&](int j, int e) -> float { return to_f<BF>(p.v.d[(int64_t)(r.row0 + j) * p.v.token + h * p.v.head + e]); };
    row_attend<BF>(s_q, kd, p.vdim, seen.hi, p.scale, p.out.d + t * p.out.token + h * p.out.head,
                   p.lse ? p.lse + (int64_t)t * p.heads + h : nullptr, key, value);
}

}  // namespace

size_t expand_workspace(ExpandParams &, int, unsigned char *) { return 0; }

cudaError_t launch_expand(const ExpandParams &p, bool bf16, int, cudaStream_t st) {
    (bf16 ? expand_plain<true> : expand_plain<false>)<<<(unsigned)((int64_t)p.tokens * p.heads), kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace latent
}  // namespace ftmoe

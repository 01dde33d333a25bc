// Causal attention over packed documents with a sliding window and sinks.
//
//   s_j = scale q . k_j over the keys the row sees, m = max s, l = sum exp(s_j - m),
//   out = sum exp(s_j - m) v_j / l, lse = m + log l.
// A row that sees nothing has out = 0 and lse = -inf.
#include "attention_common.cuh"

namespace cpt {

namespace {

// One warp computes one row of one head: lanes hold four elements each, keys
// come one at a time, the softmax keeps its running maximum and sum.
__device__ void row_forward(const AttentionParams &p, int64_t row, int head)
{
    const int lane = threadIdx.x & 31, at = lane * 4, D = p.D;
    const int kvh = head / (p.Hq / p.Hkv);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = -INFINITY, l = 0.0f;
    const int32_t g = token_of_row(p, row);
    if (g >= 0) {
        const float4 q = load4(row_of(p.q, row, p.Hq, head, D), at, D);
        const RowKeys r = keys_of_token(p, g);
        int32_t j = r.kb;
        while (true) {
            if (j == r.kb + r.ns) j = r.lo;
            if (j > g) break;
            const float s = warp_sum(dot4(q, load4(row_of(p.k, j, p.Hkv, kvh, D), at, D))) * p.scale;
            const float4 v = load4(row_of(p.v, j, p.Hkv, kvh, D), at, D);
            const float mn = fmaxf(m, s);
            const float w = mn == -INFINITY ? (s != s ? s : 0.0f) : expf(s - mn);
            const float c = mn == -INFINITY || m == -INFINITY ? 0.0f : expf(m - mn);
            l = __fmaf_rn(l, c, w);
            o = make_float4(o.x * c, o.y * c, o.z * c, o.w * c);
            axpy4(o, w, v);
            m = mn;
            ++j;
        }
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    store4(const_cast<uint16_t *>(row_of(p.out, row, p.Hq, head, D)), at, D,
           make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (lane == 0) p.lse[head * p.Tpad + row] = m + logf(l);
}

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) attention_rows_kernel(const __grid_constant__ AttentionParams p)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (i >= p.Tpad * p.Hq) return;
    row_forward(p, i % p.Tpad, static_cast<int>(i / p.Tpad));
}

}  // namespace

cudaError_t launch_attention(const AttentionParams &p, cudaStream_t stream)
{
    const int64_t rows = p.Tpad * p.Hq;
    if (rows == 0) return cudaSuccess;
    const int64_t grid = (rows + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    attention_rows_kernel<<<static_cast<unsigned>(grid), 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t read_attention_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

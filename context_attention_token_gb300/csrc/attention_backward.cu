// Gradient of the windowed attention.
//
//   p_ij = exp(scale q_i . k_j - lse_i), delta_i = do_i . o_i,
//   ds_ij = scale p_ij (do_i . v_j - delta_i),
//   dq_i = sum_j ds_ij k_j, and for the rows i of rank r alone
//   dk_j(r) = sum_i ds_ij q_i, dv_j(r) = sum_i p_ij do_i.
#include "attention_common.cuh"

namespace cpt {

namespace {

typedef AttentionBackwardParams Params;

// p and ds of one (row, key) pair, the same in every lane.
__device__ __forceinline__ void pair_grad(const Params &b, float4 q, float4 dout, float4 k, float4 v, float lse,
                                          float delta, float &p, float &ds)
{
    const float s = warp_sum(dot4(q, k)) * b.a.scale;
    const float dp = warp_sum(dot4(dout, v));
    p = lse == -INFINITY ? 0.0f : expf(s - lse);
    ds = p * (dp - delta) * b.a.scale;
}

__device__ void row_dq(const Params &b, int64_t row, int head)
{
    const AttentionParams &p = b.a;
    const int at = (threadIdx.x & 31) * 4, D = p.D;
    const int kvh = head / (p.Hq / p.Hkv);
    float4 dq = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int32_t g = token_of_row(p, row);
    if (g >= 0) {
        const float4 q = load4(row_of(p.q, row, p.Hq, head, D), at, D);
        const float4 dout = load4(row_of(b.dout, row, p.Hq, head, D), at, D);
        const float lse = p.lse[head * p.Tpad + row], delta = b.delta[head * p.Tpad + row];
        const RowKeys r = keys_of_token(p, g);
        int32_t j = r.kb;
        while (true) {
            if (j == r.kb + r.ns) j = r.lo;
            if (j > g) break;
            const float4 k = load4(row_of(p.k, j, p.Hkv, kvh, D), at, D);
            float w, ds;
            pair_grad(b, q, dout, k, load4(row_of(p.v, j, p.Hkv, kvh, D), at, D), lse, delta, w, ds);
            axpy4(dq, ds, k);
            ++j;
        }
    }
    store4(const_cast<uint16_t *>(row_of(b.dq, row, p.Hq, head, D)), at, D, dq);
}

// dK and dV of one raw key for one writer, over the rows of that rank.
__device__ void key_dkdv(const Params &b, int32_t j, int rank, int kvh)
{
    const AttentionParams &p = b.a;
    const int lane = threadIdx.x & 31, at = lane * 4, D = p.D, G = p.Hq / p.Hkv;
    const int32_t doc = find_doc(p.cu, p.n_docs, j);
    const int32_t kb = p.cu[doc], end = p.cu[doc + 1], pos0 = b.cup[doc] - kb;
    const float4 k = load4(row_of(p.k, j, p.Hkv, kvh, D), at, D);
    const float4 v = load4(row_of(p.v, j, p.Hkv, kvh, D), at, D);
    float4 dk = make_float4(0.0f, 0.0f, 0.0f, 0.0f), dv = dk;
    const int32_t last = j - kb < p.sinks ? end : static_cast<int32_t>(min((int64_t)end, (int64_t)j + p.window));
    for (int32_t i0 = j; i0 < last; i0 += 32) {
        int64_t row = -1;
        if (i0 + lane < last) {
            row = b.g2l[pos0 + i0 + lane];
            if (row / p.Tp != rank || !in_bounds(row < p.Tpad)) row = -1;
        }
        unsigned todo = __ballot_sync(0xFFFFFFFFu, row >= 0);
        while (todo) {
            const int from = __ffs(todo) - 1;
            todo &= todo - 1;
            const int64_t i = __shfl_sync(0xFFFFFFFFu, row, from);
            for (int h = kvh * G; h < (kvh + 1) * G; ++h) {
                const float4 q = load4(row_of(p.q, i, p.Hq, h, D), at, D);
                const float4 dout = load4(row_of(b.dout, i, p.Hq, h, D), at, D);
                float w, ds;
                pair_grad(b, q, dout, k, v, p.lse[h * p.Tpad + i], b.delta[h * p.Tpad + i], w, ds);
                axpy4(dk, ds, q);
                axpy4(dv, w, dout);
            }
        }
    }
    const int64_t pos = pos0 + j;
    store4(const_cast<uint16_t *>(row_of(b.dk[rank], pos, p.Hkv, kvh, D)), at, D, dk);
    store4(const_cast<uint16_t *>(row_of(b.dv[rank], pos, p.Hkv, kvh, D)), at, D, dv);
}

constexpr int kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) delta_kernel(const __grid_constant__ Params b)
{
    const AttentionParams &p = b.a;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (i >= p.Tpad * p.Hq) return;
    const int64_t row = i / p.Hq;
    const int head = static_cast<int>(i % p.Hq), lane = threadIdx.x & 31;
    const float d = warp_sum(dot4(load4(row_of(p.out, row, p.Hq, head, p.D), lane * 4, p.D),
                                  load4(row_of(b.dout, row, p.Hq, head, p.D), lane * 4, p.D)));
    if (lane == 0) b.delta[head * p.Tpad + row] = d;
}

__global__ void __launch_bounds__(32 * kWarps) dq_rows_kernel(const __grid_constant__ Params b)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (i >= b.a.Tpad * b.a.Hq) return;
    row_dq(b, i % b.a.Tpad, static_cast<int>(i / b.a.Tpad));
}

// One warp per (writer, padded global position, kv head); positions of
// padding are written as zeros.
__global__ void __launch_bounds__(32 * kWarps) dkdv_rows_kernel(const __grid_constant__ Params b)
{
    const AttentionParams &p = b.a;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (i >= p.Tpad * p.Hkv * p.P) return;
    const int32_t pos = static_cast<int32_t>(i % p.Tpad);
    const int kvh = static_cast<int>(i / p.Tpad % p.Hkv), rank = static_cast<int>(i / p.Tpad / p.Hkv);
    const int32_t doc = find_doc(b.cup, p.n_docs, pos);
    const int32_t j = pos - b.cup[doc] + p.cu[doc];
    if (j < p.cu[doc + 1]) {
        key_dkdv(b, j, rank, kvh);
    } else {
        const int at = (threadIdx.x & 31) * 4;
        const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        store4(const_cast<uint16_t *>(row_of(b.dk[rank], pos, p.Hkv, kvh, p.D)), at, p.D, zero);
        store4(const_cast<uint16_t *>(row_of(b.dv[rank], pos, p.Hkv, kvh, p.D)), at, p.D, zero);
    }
}

}  // namespace

cudaError_t launch_attention_backward(const AttentionBackwardParams &b, cudaStream_t stream)
{
    const AttentionParams &p = b.a;
    if (p.Tpad == 0) return cudaSuccess;
    const int64_t rows = (p.Tpad * p.Hq + kWarps - 1) / kWarps;
    const int64_t keys = (p.Tpad * p.Hkv * p.P + kWarps - 1) / kWarps;
    if (rows > 0x7FFFFFFF || keys > 0x7FFFFFFF) return cudaErrorInvalidValue;
    delta_kernel<<<static_cast<unsigned>(rows), 32 * kWarps, 0, stream>>>(b);
    dq_rows_kernel<<<static_cast<unsigned>(rows), 32 * kWarps, 0, stream>>>(b);
    dkdv_rows_kernel<<<static_cast<unsigned>(keys), 32 * kWarps, 0, stream>>>(b);
    return cudaGetLastError();
}

cudaError_t read_attention_backward_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

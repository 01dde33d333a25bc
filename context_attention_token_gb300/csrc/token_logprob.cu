// The logarithm of the probability that a row of logits gives to its target, and its gradient.
//
// Mathematics. With m the largest logit and l = log sum exp(scale (x - m)):
//   logp = scale (x_t - m) - l,  dx_j = dlogp scale ([j = t] - exp(scale (x_j - m) - l)).
// One pass over the row: every thread keeps the largest logit that it has seen and the sum of the weights
// relative to it, scaled anew when a batch of its loads holds a larger one; the pairs are joined at the end. m is
// subtracted from a logit before anything is rounded, so large logits lose nothing.
//
// HBM bounds both: the logits are read once (and the gradient written once).
#include "cpt_internal.h"
#include "token_rows.cuh"

#include <math_constants.h>

namespace cpt {

namespace {

constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest logit of some columns, and the sum of 2^(c (x - m)) over them.
struct Sum {
    float m, s;
};

// With m at -inf nothing is subtracted: every weight is 0 then, as it should be, and not NaN.
__device__ __forceinline__ float reference(float m) { return m == -CUDART_INF_F ? 0.0f : m; }

__device__ __forceinline__ Sum joined(Sum a, Sum b, float c)
{
    const float m = fmaxf(a.m, b.m), r = reference(m);
    Sum o;
    o.m = m;
    // a side that has seen nothing has s = 0 (or NaN, which stays)
    const float fa = a.m == m ? 1.0f : exp2_fast(__fmul_rn(__fsub_rn(a.m, r), c));
    const float fb = b.m == m ? 1.0f : exp2_fast(__fmul_rn(__fsub_rn(b.m, r), c));
    o.s = __fadd_rn(__fmul_rn(a.s, fa), __fmul_rn(b.s, fb));
    return o;
}

constexpr int kRowThreads = 512;
constexpr int kRowUnroll = 4;

template <bool BF16>
__device__ __forceinline__ void add_units(const uint4 (&raw)[kRowUnroll], const int64_t (&at)[kRowUnroll], int64_t vocab,
                                          float c, Sum &sum)
{
    constexpr int E = Unit<BF16>::E;
    float x[kRowUnroll][E];
    float m = sum.m;
#pragma unroll
    for (int k = 0; k < kRowUnroll; ++k) {
        Unit<BF16>::unpack(raw[k], x[k]);
        const int64_t left = vocab - at[k] * E;
        if (left < E) {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e >= left) x[k][e] = -CUDART_INF_F;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) m = fmaxf(m, x[k][e]);
    }
    const float r = reference(m);
    if (m != sum.m) sum.s = __fmul_rn(sum.s, exp2_fast(__fmul_rn(__fsub_rn(sum.m, r), c)));
    sum.m = m;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kRowUnroll; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) s = __fadd_rn(s, exp2_fast(__fmul_rn(__fsub_rn(x[k][e], r), c)));
    sum.s = __fadd_rn(sum.s, s);
}

// One CTA a token.
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) token_logprob_kernel(const __grid_constant__ LogprobParams p)
{
    constexpr int E = Unit<BF16>::E;
    __shared__ Sum room[32];
    const float c = __fmul_rn(p.scale, kLog2E);
    const int64_t units = (p.vocab + E - 1) / E;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t target = p.targets[t];
        const int64_t row = p.row_of_token == nullptr ? t : p.row_of_token[t];
        if (target < 0 || target >= p.vocab || !in_bounds(row >= 0 && row < p.rows, threadIdx.x == 0)) {
            if (threadIdx.x == 0) {
                p.logp[t] = 0.0f;
                p.stats[t] = make_float2(0.0f, 0.0f);
            }
            continue;
        }
        const uint4 *from = reinterpret_cast<const uint4 *>(p.logits) + row * p.units;
        float wanted = 0.0f;
        if (threadIdx.x == 0) {
            if (BF16) wanted = bf16_lo(reinterpret_cast<const uint16_t *>(from)[target]);
            else wanted = reinterpret_cast<const float *>(from)[target];
        }
        Sum sum = {-CUDART_INF_F, 0.0f};
        for (int64_t u = threadIdx.x; u < units; u += kRowThreads * kRowUnroll) {
            uint4 raw[kRowUnroll];
            int64_t at[kRowUnroll];
#pragma unroll
            for (int k = 0; k < kRowUnroll; ++k) {
                at[k] = u + k * kRowThreads;
                raw[k] = make_uint4(0, 0, 0, 0);
                if (at[k] < units) raw[k] = ld_once(from + at[k]);
            }
            add_units<BF16>(raw, at, p.vocab, c, sum);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            Sum other = {__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.s, d)};
            sum = joined(sum, other, c);
        }
        __syncthreads();   // the last token's sums have been read
        if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kRowThreads / 32; ++w) sum = joined(sum, room[w], c);
            const float l = logf(sum.s);
            p.logp[t] = __fsub_rn(__fmul_rn(__fsub_rn(wanted, sum.m), p.scale), l);
            p.stats[t] = make_float2(sum.m, l);
        }
    }
}

// ----------------------------------------------------------------- gradient

constexpr int kFlatThreads = 256;
constexpr int kFlatUnroll = 4;

// What a row's gradient needs besides its logits.
struct RowOf {
    float m, l2, factor;   // dx = factor ([j = t] - 2^(c (x - m) - l2))
    int64_t target;        // -1: the row is zeros
};

__device__ __forceinline__ RowOf row_of(const LogprobParams &p, int64_t row)
{
    RowOf r;
    r.target = -1;
    r.m = r.l2 = r.factor = 0.0f;
    const int64_t t = p.token_of_row == nullptr ? row : p.token_of_row[row];
    if (t < 0 || !in_bounds(t < p.T)) return r;
    const int64_t target = p.targets[t];
    if (target < 0 || target >= p.vocab) return r;
    const float d = p.logp[t];
    if (d == 0.0f) return r;
    const float2 st = p.stats[t];
    r.target = target;
    r.m = st.x;
    r.l2 = __fmul_rn(st.y, kLog2E);
    r.factor = __fmul_rn(d, p.scale);
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 gradient_unit(const uint4 &raw, const RowOf &r, int64_t unit, int64_t vocab, float c)
{
    constexpr int E = Unit<BF16>::E;
    float x[E];
    Unit<BF16>::unpack(raw, x);
    const int64_t first = unit * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float w = exp2_fast(__fmaf_rn(__fsub_rn(x[e], r.m), c, -r.l2));
        x[e] = __fmul_rn(-r.factor, w);
    }
    const int64_t to = r.target - first;
    if (to >= 0 && to < E) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e == to) x[e] = __fadd_rn(r.factor, x[e]);
    }
    if (first + E > vocab) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (first + e >= vocab) x[e] = 0.0f;
    }
    return Unit<BF16>::pack(x);
}

template <bool BF16>
__global__ void __launch_bounds__(kFlatThreads) token_logprob_backward_kernel(const __grid_constant__ LogprobParams p)
{
    const float c = __fmul_rn(p.scale, kLog2E);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kFlatThreads;
    const int64_t items = p.rows * p.units;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kFlatThreads + threadIdx.x;
    int64_t row = i / p.units, unit = i - row * p.units;
    for (; i < items; i += stride * kFlatUnroll) {
        uint4 raw[kFlatUnroll];
        RowOf of[kFlatUnroll];
        int64_t at[kFlatUnroll];
#pragma unroll
        for (int k = 0; k < kFlatUnroll; ++k) {
            const int64_t j = i + k * stride;
            at[k] = unit;
            of[k].target = -1;
            if (j < items) {
                of[k] = row_of(p, row);
                if (of[k].target >= 0) raw[k] = __ldcs(reinterpret_cast<const uint4 *>(p.logits) + j);
            }
            row += p.step_rows;
            unit += p.step_units;
            if (unit >= p.units) {
                unit -= p.units;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < kFlatUnroll; ++k) {
            const int64_t j = i + k * stride;
            if (j >= items) continue;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (of[k].target >= 0) v = gradient_unit<BF16>(raw[k], of[k], at[k], p.vocab, c);
            __stcs(reinterpret_cast<uint4 *>(p.dlogits) + j, v);
        }
    }
}

}  // namespace

cudaError_t launch_token_logprob(LogprobParams p, int dtype, cudaStream_t stream)
{
    if (p.T == 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>(p.T);
    if (dtype == kBf16) token_logprob_kernel<true><<<grid, kRowThreads, 0, stream>>>(p);
    else token_logprob_kernel<false><<<grid, kRowThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_token_logprob_backward(LogprobParams p, int dtype, cudaStream_t stream)
{
    const int64_t items = p.rows * p.units;
    if (items == 0) return cudaSuccess;
    const int64_t ctas = (items + kFlatThreads * kFlatUnroll - 1) / (kFlatThreads * kFlatUnroll);
    const int64_t most = 8 * static_cast<int64_t>(sm_count(-1));
    const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
    const int64_t stride = static_cast<int64_t>(grid) * kFlatThreads;
    p.step_rows = stride / p.units;
    p.step_units = stride % p.units;
    if (dtype == kBf16) token_logprob_backward_kernel<true><<<grid, kFlatThreads, 0, stream>>>(p);
    else token_logprob_backward_kernel<false><<<grid, kFlatThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t read_logprob_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

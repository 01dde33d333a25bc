// A clipped policy loss with a KL term over the documents of a plan, and its gradient.
//
// Mathematics, for a token that counts, with u = logp - logp_old, r = exp(u), A the document's advantage:
//   held = (A > 0 and r > 1 + high) or (A < 0 and r < 1 - low)
//   loss = held ? -A (1 + high or 1 - low) : -A r       gradient: held ? 0 : -A r
//   e = logp_ref - logp:  kl = exp(e) - e - 1           gradient: 1 - exp(e)
// and the document's mean of loss + kl_coef kl. On which side of a border u lies is settled exactly: u is held
// as two floats (the rounded difference and its error), and so are the borders' logarithms. kl comes from its
// series where the terms cancel.
//
// A document has one CTA. The gradient needs the number of tokens that count, so the mask is read first.
#include "cpt_internal.h"
#include "token_rows.cuh"

namespace cpt {

namespace {

constexpr int kThreads = 512;

// a - b and what its rounding left out.
__device__ __forceinline__ void exact_difference(float a, float b, float &d, float &rest)
{
    d = __fsub_rn(a, b);
    const float bb = __fsub_rn(a, d);
    rest = __fadd_rn(__fsub_rn(a, __fadd_rn(d, bb)), __fsub_rn(bb, b));
    if (!(fabsf(rest) < 3.0e38f)) rest = 0.0f;   // infinities and NaN are in d
}

// exp(x) - 1 - x
__device__ __forceinline__ float exp_less_line(float x)
{
    if (fabsf(x) < 0.5f) {
        float s = __fmaf_rn(x, 1.0f / 40320, 1.0f / 5040);
        s = __fmaf_rn(x, s, 1.0f / 720);
        s = __fmaf_rn(x, s, 1.0f / 120);
        s = __fmaf_rn(x, s, 1.0f / 24);
        s = __fmaf_rn(x, s, 1.0f / 6);
        s = __fmaf_rn(x, s, 0.5f);
        return __fmul_rn(__fmul_rn(x, x), s);
    }
    return __fsub_rn(expm1f(x), x);
}

// A sum of any number of terms, with what its roundings left out.
struct LongSum {
    float s = 0.0f, rest = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(s, x), back = __fsub_rn(t, s);
        rest = __fadd_rn(rest, __fadd_rn(__fsub_rn(s, __fsub_rn(t, back)), __fsub_rn(x, back)));
        s = t;
    }
    // infinities and NaN leave no rest
    __device__ __forceinline__ float value() const { return fabsf(rest) < 3.0e38f ? __fadd_rn(s, rest) : s; }
};

__global__ void __launch_bounds__(kThreads) policy_loss_kernel(const __grid_constant__ PolicyParams p)
{
    __shared__ float room[BlockSum::kRoom];
    BlockSum sum(room);
    for (int64_t d = blockIdx.x; d < p.n_docs; d += gridDim.x) {
        const int64_t lo = p.cu[d], hi = p.cu[d + 1];
        const float A = p.advantages[d];
        // counted in whole numbers, in two floats of 2^24 each: exact for any length
        float n[2] = {0.0f, 0.0f};
        if (p.mask == nullptr) {
            n[0] = static_cast<float>(hi - lo);
        } else {
            int mine = 0;
            for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) mine += p.mask[t] != 0;
            n[0] = static_cast<float>(mine & 0xFFF);
            n[1] = static_cast<float>(mine >> 12);
            sum(n);
            n[0] = __fmaf_rn(n[1], 4096.0f, n[0]);
        }
        const float share = __fdiv_rn(1.0f, fmaxf(n[0], 1.0f));
        const float weight = __fmul_rn(p.weights == nullptr ? p.weight : p.weights[d], share);
        LongSum loss, kl;
        int held_count = 0;
        for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) {
            float g = 0.0f;
            if (p.mask == nullptr || p.mask[t] != 0) {
                float u, rest;
                exact_difference(p.logp[t], p.old[t], u, rest);
                const bool above = __fadd_rn(__fsub_rn(u, p.high_hi), __fsub_rn(rest, p.high_lo)) > 0.0f;
                const bool below = __fadd_rn(__fsub_rn(u, p.low_hi), __fsub_rn(rest, p.low_lo)) < 0.0f;
                const bool held = (above && A > 0.0f) || (below && A < 0.0f);
                const float r = expf(u);
                const float ar = __fmul_rn(-A, __fmul_rn(r, __fadd_rn(1.0f, rest)));
                loss.add(held ? __fmul_rn(-A, above ? p.above : p.below) : ar);
                held_count += held;
                g = held ? 0.0f : ar;
                if (p.ref != nullptr) {
                    const float e = __fsub_rn(p.ref[t], p.logp[t]);
                    kl.add(exp_less_line(e));
                    g = __fmaf_rn(-p.kl, expm1f(e), g);
                }
                g = __fmul_rn(g, weight);
            }
            p.dlogp[t] = g;
        }
        float s[3] = {loss.value(), kl.value(), static_cast<float>(held_count)};
        sum(s);
        if (threadIdx.x == 0)
            p.terms[d] = make_float4(__fmul_rn(__fmaf_rn(p.kl, s[1], s[0]), share), __fmul_rn(s[1], share),
                                     __fmul_rn(s[2], share), n[0]);
    }
}

}  // namespace

cudaError_t launch_policy_loss(const PolicyParams &p, cudaStream_t stream)
{
    if (p.n_docs == 0) return cudaSuccess;
    policy_loss_kernel<<<static_cast<unsigned>(p.n_docs), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace cpt

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
// The gradient needs the number of tokens that count, so a document's mask is read first; its sums stay within a warp, a CTA or
// a cluster, so that one launch does.
#include "cpt_internal.h"
#include "token_rows.cuh"

#include <cooperative_groups.h>

#include <cstring>

namespace cpt {

namespace {

constexpr int kThreads = 512;
constexpr int kWarpTokens = 512;       // of a document that a warp takes
constexpr int kClusterTokens = 8192;   // of one that is worth a cluster

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

// What a thread finds in its tokens.
struct Found {
    LongSum loss, kl;
    int held = 0;
};

__device__ __forceinline__ void add_token(const PolicyParams &p, int64_t t, float A, float weight, Found &f)
{
    float g = 0.0f;
    if (p.mask == nullptr || p.mask[t] != 0) {
        const float logp = p.logp[t];
        float u, rest;
        exact_difference(logp, p.old[t], u, rest);
        const bool above = __fadd_rn(__fsub_rn(u, p.high_hi), __fsub_rn(rest, p.high_lo)) > 0.0f;
        const bool below = __fadd_rn(__fsub_rn(u, p.low_hi), __fsub_rn(rest, p.low_lo)) < 0.0f;
        const bool held = (above && A > 0.0f) || (below && A < 0.0f);
        const float r = expf(u);
        const float ar = __fmul_rn(-A, __fmul_rn(r, __fadd_rn(1.0f, rest)));
        f.loss.add(held ? __fmul_rn(-A, above ? p.above : p.below) : ar);
        f.held += held;
        g = held ? 0.0f : ar;
        if (p.ref != nullptr) {
            const float e = __fsub_rn(p.ref[t], logp);
            f.kl.add(exp_less_line(e));
            g = __fmaf_rn(-p.kl, expm1f(e), g);
        }
        g = __fmul_rn(g, weight);
    }
    p.dlogp[t] = g;
}

__device__ __forceinline__ float4 terms_of(const PolicyParams &p, float loss, float kl, float held, float n, float share)
{
    return make_float4(__fmul_rn(__fmaf_rn(p.kl, kl, loss), share), __fmul_rn(kl, share), __fmul_rn(held, share), n);
}

// Tokens of [lo, hi) that count, those of every `step`-th from lo + first on.
__device__ __forceinline__ int count_tokens(const PolicyParams &p, int64_t lo, int64_t hi, int first, int step)
{
    int n = 0;
#pragma unroll 8
    for (int64_t t = lo + first; t < hi; t += step) n += p.mask[t] != 0;
    return n;
}

// A cluster of S CTAs takes p.docs neighbouring documents: the short ones a warp each, then the others one after the
// other with all its threads.
template <int S>
__global__ void __launch_bounds__(kThreads) policy_loss_kernel(const __grid_constant__ PolicyParams p)
{
    namespace cg = cooperative_groups;
    __shared__ float room[BlockSum::kRoom];
    __shared__ float shares[2][8][5];   // of two documents in turn, every CTA's: counts (two floats), then sums
    BlockSum sum(room);
    const int rank = S == 1 ? 0 : static_cast<int>(blockIdx.x % S), lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.x / S) * p.docs;
    const int64_t last = min(first + p.docs, static_cast<int64_t>(p.n_docs));

    for (int64_t d = first + rank * (kThreads / 32) + (threadIdx.x >> 5); d < last; d += S * (kThreads / 32)) {
        const int64_t lo = p.cu[d], hi = p.cu[d + 1];
        if (hi - lo > kWarpTokens) continue;
        float n = static_cast<float>(hi - lo);
        if (p.mask != nullptr) n = static_cast<float>(__reduce_add_sync(0xFFFFFFFFu, count_tokens(p, lo, hi, lane, 32)));
        const float share = __fdiv_rn(1.0f, fmaxf(n, 1.0f));
        const float weight = __fmul_rn(p.weights == nullptr ? p.weight : p.weights[d], share);
        Found f;
        for (int64_t t = lo + lane; t < hi; t += 32) add_token(p, t, p.advantages[d], weight, f);
        float v[3] = {f.loss.value(), f.kl.value(), static_cast<float>(f.held)};
        lanes_sum<3>(v, 32);
        if (lane == 0) p.terms[d] = terms_of(p, v[0], v[1], v[2], n, share);
    }

    int turn = 0;
    for (int64_t d = first; d < last; ++d) {
        const int64_t lo = p.cu[d], hi = p.cu[d + 1];
        if (hi - lo <= kWarpTokens) continue;
        float(*mine)[5] = shares[turn];
        turn ^= 1;
        const int at = rank * kThreads + threadIdx.x;
        float n = static_cast<float>(hi - lo);
        if (p.mask != nullptr) {
            // whole numbers in two floats, of 4096 and of one: exact for any length
            const int c = count_tokens(p, lo, hi, at, S * kThreads);
            float v[2] = {static_cast<float>(c & 0xFFF), static_cast<float>(c >> 12)};
            sum(v);
            if constexpr (S > 1) {
                cg::cluster_group cluster = cg::this_cluster();
                if (threadIdx.x < S) {
                    float *to = cluster.map_shared_rank(&mine[rank][0], threadIdx.x);
                    to[0] = v[0];
                    to[1] = v[1];
                }
                cluster.sync();
                v[0] = v[1] = 0.0f;
                for (int i = 0; i < S; ++i) {
                    v[0] = __fadd_rn(v[0], mine[i][0]);
                    v[1] = __fadd_rn(v[1], mine[i][1]);
                }
            }
            n = __fmaf_rn(v[1], 4096.0f, v[0]);
        }
        const float share = __fdiv_rn(1.0f, fmaxf(n, 1.0f));
        const float weight = __fmul_rn(p.weights == nullptr ? p.weight : p.weights[d], share);
        const float A = p.advantages[d];
        Found f;
#pragma unroll 4
        for (int64_t t = lo + at; t < hi; t += S * kThreads) add_token(p, t, A, weight, f);
        float v[3] = {f.loss.value(), f.kl.value(), static_cast<float>(f.held)};
        sum(v);
        if constexpr (S > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (threadIdx.x == 0) {
                float *to = cluster.map_shared_rank(&mine[rank][2], 0);
                for (int i = 0; i < 3; ++i) to[i] = v[i];
            }
            // behind it the first CTA has all sums, and no CTA has ended that is still written to
            cluster.sync();
            if (rank == 0 && threadIdx.x == 0) {
                for (int j = 0; j < 3; ++j) {
                    v[j] = mine[0][2 + j];
                    for (int i = 1; i < S; ++i) v[j] = __fadd_rn(v[j], mine[i][2 + j]);
                }
            }
        }
        if (rank == 0 && threadIdx.x == 0) p.terms[d] = terms_of(p, v[0], v[1], v[2], n, share);
    }
}

}  // namespace

cudaError_t launch_policy_loss(PolicyParams p, cudaStream_t stream)
{
    if (p.n_docs == 0) return cudaSuccess;
    // a cluster of eight where a document is long; documents of a cluster: one while there is room for all
    const int split = p.longest > kClusterTokens ? 8 : 1;
    const int64_t room = 4 * static_cast<int64_t>(sm_count(-1));
    int64_t docs = (static_cast<int64_t>(p.n_docs) * split + room - 1) / room;
    const int64_t most = static_cast<int64_t>(split) * (kThreads / 32);
    p.docs = static_cast<int32_t>(docs < 1 ? 1 : docs > most ? most : docs);
    const int64_t ctas = (static_cast<int64_t>(p.n_docs) + p.docs - 1) / p.docs * split;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t config;
    memset(&config, 0, sizeof config);
    config.gridDim = dim3(static_cast<unsigned>(ctas));
    config.blockDim = dim3(kThreads);
    config.stream = stream;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {static_cast<unsigned>(split), 1, 1};
    config.attrs = &cluster;
    config.numAttrs = split > 1 ? 1 : 0;
    return split > 1 ? cudaLaunchKernelEx(&config, policy_loss_kernel<8>, p) : cudaLaunchKernelEx(&config, policy_loss_kernel<1>, p);
}

}  // namespace cpt

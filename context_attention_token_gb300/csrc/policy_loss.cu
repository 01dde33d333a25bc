// A clipped policy loss with a KL term over the documents of a plan, and its gradient.
//
// Mathematics, for a token that counts, with u = logp - logp_old, r = exp(u), A the document's advantage:
//   held = (A > 0 and r > 1 + high) or (A < 0 and r < 1 - low)
//   loss = held ? -A (1 + high or 1 - low) : -A r       gradient: held ? 0 : -A r
//   e = logp_ref - logp:  kl = exp(e) - e - 1           gradient: 1 - exp(e)
// and the document's mean of loss + kl_coef kl. An A, a kl_coef or a weight of 0 takes all of what it multiplies, exponentials
// beyond binary32 too. On which side of a border u lies is settled exactly: u is held
// as two floats (the rounded difference and its error), and so are the borders' logarithms. kl comes from its
// series where the terms cancel.
//
// The gradient's weight needs the number of tokens that count. So the gradients wait for it in registers (in dlogp, where a
// thread has more than kTokens), and a document's sums stay within a warp, a CTA or a cluster, so that one launch does.
// Latency bounds it: 512 tokens take 9 to 10 us, most of it the call's, 262139 tokens 10.8, where the bytes would take 0.5. Few long
// documents take longer, by the tokens of a thread: four of 65536 tokens 23 us, one of 262144 68.
#include "cpt_internal.h"
#include "token_rows.cuh"

#include <cooperative_groups.h>
#include <math_constants.h>

#include <cstring>

namespace cpt {

namespace {

constexpr int kThreads = 512;
constexpr int kTokens = 8;                            // of a thread at a time
constexpr int kWarpTokens = 128;                      // of a document that a warp takes
constexpr int kClusterTokens = kTokens * kThreads;    // a longer one is worth a cluster
// CTAs of a cluster: 262139 tokens in 83 documents take 23.1 us with one, 16.3 with 2, 10.3 with 4, and 20.5 with 8, where the
// documents no longer fit at once and a cluster takes two.
constexpr int kSplit = 4;

// a - b and what its rounding left out.
__device__ __forceinline__ void exact_difference(float a, float b, float &d, float &rest)
{
    d = __fsub_rn(a, b);
    const float bb = __fsub_rn(a, d);
    rest = __fadd_rn(__fsub_rn(a, __fadd_rn(d, bb)), __fsub_rn(bb, b));
    if (!(fabsf(rest) < 3.0e38f)) rest = 0.0f;   // infinities and NaN are in d
}

// exp(x) - 1 - x from y = exp(x) - 1; infinite at both infinities
__device__ __forceinline__ float exp_less_line(float x, float y)
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
    return y == CUDART_INF_F ? y : __fsub_rn(y, x);
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
    int held = 0, count = 0;
};

// K tokens from t on, every `step`-th below hi: into `f`, and the gradients before the weight into g.
template <int K>
__device__ __forceinline__ void add_tokens(const PolicyParams &p, int64_t t, int64_t step, int64_t hi, float A, Found &f, float (&g)[K])
{
    float logp[K], old[K], ref[K];
    bool on[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {   // all loads at once; what is masked is not used
        const int64_t at = t + k * step;
        on[k] = false;
        logp[k] = old[k] = ref[k] = 0.0f;
        if (at >= hi) continue;
        on[k] = p.mask == nullptr || p.mask[at] != 0;
        logp[k] = p.logp[at];
        old[k] = p.old[at];
        if (p.ref != nullptr) ref[k] = p.ref[at];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        g[k] = 0.0f;
        if (!on[k]) continue;
        float u, rest;
        exact_difference(logp[k], old[k], u, rest);
        const bool above = __fadd_rn(__fsub_rn(u, p.high_hi), __fsub_rn(rest, p.high_lo)) > 0.0f;
        const bool below = __fadd_rn(__fsub_rn(u, p.low_hi), __fsub_rn(rest, p.low_lo)) < 0.0f;
        const bool held = (above && A > 0.0f) || (below && A < 0.0f);
        const float r = expf(A == 0.0f && u > 0.0f ? 0.0f : u);   // of no advantage, not 0 times a ratio beyond binary32
        const float ar = __fmul_rn(-A, __fmul_rn(r, __fadd_rn(1.0f, rest)));
        f.loss.add(held ? __fmul_rn(-A, above ? p.above : p.below) : ar);
        f.held += held;
        ++f.count;
        g[k] = held ? 0.0f : ar;
        if (p.ref != nullptr) {
            const float e = __fsub_rn(ref[k], logp[k]), y = expm1f(e);
            f.kl.add(exp_less_line(e, y));
            g[k] = __fmaf_rn(-p.kl, p.kl != 0.0f ? y : 0.0f, g[k]);   // with 0 the KL is only reported, infinite or not
        }
    }
}

// A token's gradient times its document's weight. A gradient of 0 (a masked or held token) stays 0, and a weight of 0 leaves nothing
// of an infinite one.
__device__ __forceinline__ float weighted(float g, float weight)
{
    return g == 0.0f || (weight == 0.0f && fabsf(g) == CUDART_INF_F) ? 0.0f : __fmul_rn(g, weight);
}

__device__ __forceinline__ float4 terms_of(const PolicyParams &p, float loss, float kl, float held, float n, float share)
{
    const float all = p.kl != 0.0f ? __fmaf_rn(p.kl, kl, loss) : loss;
    return make_float4(__fmul_rn(all, share), __fmul_rn(kl, share), __fmul_rn(held, share), n);
}

// A cluster of S CTAs takes p.docs neighbouring documents: the short ones a warp each, then the others one after the
// other with all its threads.
template <int S>
__global__ void __launch_bounds__(kThreads) policy_loss_kernel(const __grid_constant__ PolicyParams p)
{
    namespace cg = cooperative_groups;
    constexpr int kSums = 5;                   // loss, kl, held; tokens, in units of one and of 4096: exact for any length
    __shared__ float room[TeamSum<128>::kRoom];
    __shared__ float shares[2][S][kSums];      // of two documents in turn, every CTA's
    TeamSum<128> sum(room, Team{static_cast<int>(threadIdx.x), kThreads, 1});
    const int rank = S == 1 ? 0 : static_cast<int>(blockIdx.x % S), lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.x / S) * p.docs;
    const int64_t last = min(first + p.docs, static_cast<int64_t>(p.n_docs));
    if constexpr (S > 1) cluster_begun();

    for (int64_t d = first + rank * (kThreads / 32) + (threadIdx.x >> 5); d < last; d += S * (kThreads / 32)) {
        const int64_t lo = p.cu[d], hi = p.cu[d + 1];
        if (hi - lo > kWarpTokens) continue;
        const float A = p.advantages[d], own = p.weights == nullptr ? p.weight : p.weights[d];
        Found f;
        float g[kWarpTokens / 32];
        add_tokens<kWarpTokens / 32>(p, lo + lane, 32, hi, A, f, g);
        float v[4] = {f.loss.value(), f.kl.value(), static_cast<float>(f.held), static_cast<float>(f.count)};
        lanes_sum<4>(v, 32);
        const float share = __fdiv_rn(1.0f, fmaxf(v[3], 1.0f)), weight = __fmul_rn(own, share);
#pragma unroll
        for (int k = 0; k < kWarpTokens / 32; ++k)
            if (lo + lane + k * 32 < hi) p.dlogp[lo + lane + k * 32] = weighted(g[k], weight);
        if (lane == 0) p.terms[d] = terms_of(p, v[0], v[1], v[2], v[3], share);
    }

    int turn = 0;
    if constexpr (S > 1) cluster_wait_begun();
    for (int64_t d = first; d < last; ++d) {
        const int64_t lo = p.cu[d], hi = p.cu[d + 1];
        if (hi - lo <= kWarpTokens) continue;
        const float A = p.advantages[d], own = p.weights == nullptr ? p.weight : p.weights[d];
        const int64_t t = lo + rank * kThreads + threadIdx.x, step = S * kThreads;
        const bool held_back = hi - lo <= kTokens * step;   // a thread's gradients wait in registers for the weight
        Found f;
        float g[kTokens];
        for (int64_t at = t; at < hi; at += kTokens * step) {
            add_tokens<kTokens>(p, at, step, hi, A, f, g);
            if (held_back) break;
#pragma unroll
            for (int k = 0; k < kTokens; ++k)
                if (at + k * step < hi) p.dlogp[at + k * step] = g[k];
        }
        float v[kSums] = {f.loss.value(), f.kl.value(), static_cast<float>(f.held), static_cast<float>(f.count & 0xFFF),
                          static_cast<float>(f.count >> 12)};
        sum(v);
        if constexpr (S > 1) {
            namespace cg = cooperative_groups;
            cg::cluster_group cluster = cg::this_cluster();
            float(*mine)[kSums] = shares[turn];
            turn ^= 1;
            if (threadIdx.x < S) {
                float *to = cluster.map_shared_rank(&mine[rank][0], threadIdx.x);
#pragma unroll
                for (int j = 0; j < kSums; ++j) to[j] = v[j];
            }
            // A place is written again two documents on, behind the barrier of the next, which every CTA reaches only
            // after it has read; and behind this one no CTA is written to any more that may have ended.
            cluster.sync();
#pragma unroll
            for (int j = 0; j < kSums; ++j) {
                v[j] = mine[0][j];
                for (int i = 1; i < S; ++i) v[j] = __fadd_rn(v[j], mine[i][j]);
            }
        }
        const float n = __fmaf_rn(v[4], 4096.0f, v[3]);
        const float share = __fdiv_rn(1.0f, fmaxf(n, 1.0f)), weight = __fmul_rn(own, share);
        if (held_back) {
#pragma unroll
            for (int k = 0; k < kTokens; ++k)
                if (t + k * step < hi) p.dlogp[t + k * step] = weighted(g[k], weight);
        } else {
#pragma unroll 4
            for (int64_t at = t; at < hi; at += step) p.dlogp[at] = weighted(p.dlogp[at], weight);
        }
        if (rank == 0 && threadIdx.x == 0) p.terms[d] = terms_of(p, v[0], v[1], v[2], n, share);
    }
}

}  // namespace

cudaError_t launch_policy_loss(PolicyParams p, cudaStream_t stream)
{
    if (p.n_docs == 0) return cudaSuccess;
    // a cluster where a document is long; documents of a cluster: one while there is room for all
    const int split = p.longest > kClusterTokens ? kSplit : 1;
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
    return split > 1 ? cudaLaunchKernelEx(&config, policy_loss_kernel<kSplit>, p) : cudaLaunchKernelEx(&config, policy_loss_kernel<1>, p);
}

}  // namespace cpt

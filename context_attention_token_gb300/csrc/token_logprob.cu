// The logarithm of the probability that a row of logits gives to its target, and its gradient.
//
// Mathematics. With m the largest logit and l = log sum exp(scale (x - m)):
//   logp = scale (x_t - m) - l,  dx_j = dlogp scale ([j = t] - exp(scale (x_j - m) - l)).
// One pass over the row: every thread keeps the largest logit that it has seen and the sum of the weights
// relative to it, scaled anew when a batch of its loads holds a larger one; the pairs are joined at the end. m is
// subtracted from a logit before anything is rounded, so large logits lose nothing.
//
// HBM bounds both: the logits are read once (and the gradient written once). 8191 x 157184 bf16 takes 359 us forward (7.2 TB/s)
// and 826 for its gradient (6.2 TB/s, 0.92 of a copy).
#include "cpt_internal.h"
#include "token_rows.cuh"

#include <cooperative_groups.h>
#include <math_constants.h>

#include <cstring>

namespace cpt {

namespace {

constexpr float kLog2E = 1.4426950408889634f;

// 2^x, off by 2^-22 of itself at most.
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

// The larger of two bf16 pairs, half by half; a NaN loses.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// A word without weight: -inf in every column.
template <bool BF16>
constexpr uint32_t kNoWeight = BF16 ? 0xFF80FF80u : 0xFF800000u;

// Adds N units to a sum.
template <bool BF16, int N>
__device__ __forceinline__ void add_units(const uint4 (&raw)[N], float c, Sum &sum)
{
    typedef UnitPairs<BF16> V;
    float m = sum.m;
    if constexpr (BF16) {
        uint32_t w = raw[0].x;
#pragma unroll
        for (int k = 0; k < N; ++k) w = max_bf16x2(max_bf16x2(w, raw[k].x), max_bf16x2(raw[k].y, max_bf16x2(raw[k].z, raw[k].w)));
        m = fmaxf(m, fmaxf(bf16_lo(w), bf16_hi(w)));
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(raw[k].x), __uint_as_float(raw[k].y)),
                               fmaxf(__uint_as_float(raw[k].z), __uint_as_float(raw[k].w))));
    }
    const float r = reference(m);
    if (m != sum.m) sum.s = __fmul_rn(sum.s, exp2_fast(__fmul_rn(__fsub_rn(sum.m, r), c)));
    sum.m = m;
    const F2 minus = pair_of(-r, -r), cc = pair_of(c, c);
    F2 s[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
#pragma unroll
    for (int k = 0; k < N; ++k) {
        F2 x[V::N];
        V::unpack(raw[k], x);
#pragma unroll
        for (int i = 0; i < V::N; ++i) {
            const float2 a = both(mul2(add2(x[i], minus), cc));
            s[i & 1] = add2(s[i & 1], pair_of(exp2_fast(a.x), exp2_fast(a.y)));
        }
    }
    const float2 t = both(add2(s[0], s[1]));
    sum.s = __fadd_rn(sum.s, __fadd_rn(t.x, t.y));
}

// The units from `u` on, every `step`-th below `end`, of a row of `vocab` columns.
template <bool BF16, int N>
__device__ __forceinline__ Sum sum_units(const uint4 *row, int64_t u, int64_t step, int64_t end, int64_t vocab, float c)
{
    constexpr int E = Unit<BF16>::E;
    constexpr uint32_t none = kNoWeight<BF16>;
    Sum sum = {-CUDART_INF_F, 0.0f};
    for (; u < end; u += step * N) {
        uint4 raw[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            raw[k] = make_uint4(none, none, none, none);
            if (u + k * step < end) raw[k] = ld_once(row + u + k * step);
        }
        // the row's last unit may hold columns past the vocabulary
        if ((u + (N - 1) * step + 1) * E > vocab) {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int64_t left = vocab - (u + k * step) * E;
                uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (BF16) {
                        if (2 * i + 1 >= left) w[i] = (w[i] & 0xFFFFu) | (none << 16);
                        if (2 * i >= left) w[i] = none;
                    } else if (i >= left) {
                        w[i] = none;
                    }
                }
                raw[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        add_units<BF16, N>(raw, c, sum);
    }
    return sum;
}

// The row of a token that has a target, else -1.
__device__ __forceinline__ int64_t scored_row(const LogprobParams &p, int64_t t, int64_t &target, bool count)
{
    target = p.targets[t];
    if (target < 0 || target >= p.vocab) return -1;
    const int64_t row = p.row_of_token == nullptr ? t : p.row_of_token[t];
    return in_bounds(row >= 0 && row < p.rows, count) ? row : -1;
}

template <bool BF16>
__device__ __forceinline__ float logit(const uint4 *row, int64_t column)
{
    if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t *>(row)[column]);
    else return reinterpret_cast<const float *>(row)[column];
}

__device__ __forceinline__ void put_logprob(const LogprobParams &p, int64_t t, float wanted, Sum sum)
{
    const float l = logf(sum.s);
    p.logp[t] = __fsub_rn(__fmul_rn(__fsub_rn(wanted, sum.m), p.scale), l);
    p.stats[t] = make_float2(sum.m, l);
}

__device__ __forceinline__ void put_none(const LogprobParams &p, int64_t t)
{
    p.logp[t] = 0.0f;
    p.stats[t] = make_float2(0.0f, 0.0f);
}

// Sum over the `group` lanes that share a row.
__device__ __forceinline__ Sum lanes_joined(Sum sum, int group, float c)
{
    for (int d = group >> 1; d > 0; d >>= 1) {
        const Sum other = {__shfl_xor_sync(0xFFFFFFFFu, sum.m, d), __shfl_xor_sync(0xFFFFFFFFu, sum.s, d)};
        sum = joined(sum, other, c);
    }
    return sum;
}

constexpr int kRowThreads = 256;
constexpr int kRowUnroll = 8;
constexpr int kShortUnroll = 4;
constexpr int kMostSplit = 4;      // CTAs of a long row
constexpr int kShortThreads = 256;
// Of rows that a part of a warp reads. No border that was measured: 8192 rows of 257 units take 18 us in parts of a warp, of
// 513 units 47 (float32) and 66 (bf16) and of 1024 bf16 68 in CTAs most of whose loads are empty. From some 4000 units on
// CTAs come within a fifth of HBM's rate.
constexpr int kShortUnits = 512;

// Long rows: p.split CTAs of a cluster a token, each a part of the row; their pairs are joined in the
// first one's shared memory.
template <bool BF16>
__global__ void __launch_bounds__(kRowThreads) token_logprob_kernel(const __grid_constant__ LogprobParams p)
{
    constexpr int E = Unit<BF16>::E;
    __shared__ Sum room[kRowThreads / 32], parts[kMostSplit];
    const float c = __fmul_rn(p.scale, kLog2E);
    const int64_t units = (p.vocab + E - 1) / E;
    const int part = static_cast<int>(blockIdx.x % p.split);
    const int64_t t = blockIdx.x / p.split;
    const int64_t begin = units * part / p.split, end = units * (part + 1) / p.split;
    int64_t target;
    const int64_t row = scored_row(p, t, target, threadIdx.x == 0 && part == 0);
    if (row < 0) {   // so in every CTA of the cluster
        if (threadIdx.x == 0 && part == 0) put_none(p, t);
        return;
    }
    if (p.split > 1) cluster_begun();
    const uint4 *from = reinterpret_cast<const uint4 *>(p.logits) + row * p.units;
    float wanted = 0.0f;
    if (threadIdx.x == 0 && part == 0) wanted = logit<BF16>(from, target);
    Sum sum = sum_units<BF16, kRowUnroll>(from, begin + threadIdx.x, kRowThreads, end, p.vocab, c);
    sum = lanes_joined(sum, 32, c);
    if ((threadIdx.x & 31) == 0) room[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x < 32) {
        sum = threadIdx.x < kRowThreads / 32 ? room[threadIdx.x] : Sum{-CUDART_INF_F, 0.0f};
        sum = lanes_joined(sum, 32, c);
    }
    if (p.split > 1) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        cluster_wait_begun();
        if (threadIdx.x == 0) *cluster.map_shared_rank(&parts[part], 0) = sum;
        cluster.sync();
        if (part != 0) return;
        if (threadIdx.x == 0)
            for (int i = 1; i < p.split; ++i) sum = joined(sum, parts[i], c);
    }
    if (threadIdx.x == 0) put_logprob(p, t, wanted, sum);
}

// Short rows: p.group lanes of a warp a token, the warp's tokens next to one another.
template <bool BF16>
__global__ void __launch_bounds__(kShortThreads) token_logprob_short_kernel(const __grid_constant__ LogprobParams p)
{
    constexpr int E = Unit<BF16>::E;
    const float c = __fmul_rn(p.scale, kLog2E);
    const int64_t units = (p.vocab + E - 1) / E;
    const int lane = threadIdx.x & (p.group - 1);
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kShortThreads + threadIdx.x) / p.group;
    int64_t target = -1, row = -1;
    if (t < p.T) row = scored_row(p, t, target, lane == 0);
    Sum sum = {-CUDART_INF_F, 0.0f};
    float wanted = 0.0f;
    if (row >= 0) {
        const uint4 *from = reinterpret_cast<const uint4 *>(p.logits) + row * p.units;
        if (lane == 0) wanted = logit<BF16>(from, target);
        sum = sum_units<BF16, kShortUnroll>(from, lane, p.group, units, p.vocab, c);
    }
    sum = lanes_joined(sum, p.group, c);
    if (lane != 0 || t >= p.T) return;
    if (row < 0) put_none(p, t);
    else put_logprob(p, t, wanted, sum);
}

// ----------------------------------------------------------------- gradient

constexpr int kTileThreads = 256;
constexpr int kTileUnroll = 4;
constexpr int kTileUnits = kTileThreads * kTileUnroll;

// What a row's gradient needs besides its logits: dx = factor ([j = t] - 2^(c (x - m) - l2)).
struct RowOf {
    float m, l2, factor;
    int32_t target;   // -1: the row is zeros
};

__device__ __forceinline__ RowOf row_of(const LogprobParams &p, int64_t row)
{
    RowOf r = {0.0f, 0.0f, 0.0f, -1};
    const int64_t t = p.token_of_row == nullptr ? row : p.token_of_row[row];
    if (t < 0 || !in_bounds(t < p.T)) return r;
    const int32_t target = p.targets[t];
    const float d = p.logp[t];
    const float2 st = p.stats[t];
    if (target < 0 || target >= p.vocab || d == 0.0f) return r;
    r.target = target;
    r.m = st.x;
    r.l2 = __fmul_rn(st.y, kLog2E);
    r.factor = __fmul_rn(d, p.scale);
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 gradient_unit(const uint4 &raw, const RowOf &r, int32_t first, int32_t vocab, float c)
{
    constexpr int E = Unit<BF16>::E;
    typedef UnitPairs<BF16> V;
    F2 x[V::N];
    V::unpack(raw, x);
    const F2 m = pair_of(-r.m, -r.m), cc = pair_of(c, c), l = pair_of(-r.l2, -r.l2), f = pair_of(-r.factor, -r.factor);
    float y[E];
#pragma unroll
    for (int i = 0; i < V::N; ++i) {
        const float2 a = both(fma2(add2(x[i], m), cc, l));
        const float2 w = both(mul2(pair_of(exp2_fast(a.x), exp2_fast(a.y)), f));
        y[2 * i] = w.x;
        y[2 * i + 1] = w.y;
    }
    // the unit of the target, the one at the vocabulary's end
    const uint32_t to = static_cast<uint32_t>(r.target - first);
    if (to < E || first + E > vocab) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (e == to) y[e] = __fadd_rn(r.factor, y[e]);
            if (first + e >= vocab) y[e] = 0.0f;
        }
    }
    return Unit<BF16>::pack(y);
}

// A CTA takes kTileUnits neighbouring units of the logits, of a part of a row or of several. What it needs of the rows is looked up
// first, once a row.
template <bool BF16>
__global__ void __launch_bounds__(kTileThreads) token_logprob_backward_kernel(const __grid_constant__ LogprobParams p)
{
    constexpr int E = Unit<BF16>::E;
    extern __shared__ __align__(16) uint8_t smem[];
    RowOf *rows = reinterpret_cast<RowOf *>(smem);
    const float c = __fmul_rn(p.scale, kLog2E);
    const int64_t items = p.rows * p.units, start = static_cast<int64_t>(blockIdx.x) * kTileUnits;
    const int64_t row0 = start / p.units;
    const uint32_t units = static_cast<uint32_t>(p.units), skip = static_cast<uint32_t>(start - row0 * p.units);
    const uint32_t here = static_cast<uint32_t>(min(items - start, static_cast<int64_t>(kTileUnits)));
    const uint32_t n = (skip + here - 1) / units + 1;
    for (uint32_t i = threadIdx.x; i < n; i += kTileThreads) rows[i] = row_of(p, row0 + i);
    __syncthreads();
    const uint4 *from = reinterpret_cast<const uint4 *>(p.logits) + start;
    uint4 *to = reinterpret_cast<uint4 *>(p.dlogits) + start;
    uint4 raw[kTileUnroll];
    RowOf of[kTileUnroll];
    uint32_t column[kTileUnroll];
#pragma unroll
    for (int k = 0; k < kTileUnroll; ++k) {
        const uint32_t i = threadIdx.x + k * kTileThreads;
        of[k].target = -1;
        if (i >= here) continue;
        const uint32_t q = (skip + i) / units;
        column[k] = (skip + i - q * units) * E;
        of[k] = rows[q];
        if (of[k].target >= 0) raw[k] = __ldcs(from + i);
    }
#pragma unroll
    for (int k = 0; k < kTileUnroll; ++k) {
        const uint32_t i = threadIdx.x + k * kTileThreads;
        if (i >= here) continue;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (of[k].target >= 0) v = gradient_unit<BF16>(raw[k], of[k], column[k], static_cast<int32_t>(p.vocab), c);
        __stcs(to + i, v);
    }
}

}  // namespace

cudaError_t launch_token_logprob(LogprobParams p, int dtype, cudaStream_t stream)
{
    if (p.T == 0) return cudaSuccess;
    const int per = dtype == kBf16 ? 8 : 4;
    const int64_t units = (p.vocab + per - 1) / per;
    if (units <= kShortUnits) {
        p.group = 1;
        while (p.group < 32 && p.group * 2 <= units) p.group *= 2;
        const int64_t ctas = (p.T * p.group + kShortThreads - 1) / kShortThreads;
        if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
        const unsigned grid = static_cast<unsigned>(ctas);
        if (dtype == kBf16) token_logprob_short_kernel<true><<<grid, kShortThreads, 0, stream>>>(p);
        else token_logprob_short_kernel<false><<<grid, kShortThreads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    // few tokens: a row's columns over the CTAs of a cluster, two CTAs an SM at most (64 rows of 157184 bf16 take 14.7
    // us with one CTA a row, 10.2 with two, four or eight).
    // 256 threads read 8191 such rows in 360 us, 512 in 381, 1024 in 501. (By all tokens, as those that have a target are
    // not known here: 60 of 8192 take 31 us.)
    const int64_t room = 2 * static_cast<int64_t>(sm_count(-1));
    p.split = 1;
    while (p.split < kMostSplit && p.T * p.split * 2 <= room && units >= p.split * 2 * kRowThreads) p.split *= 2;
    if (p.T * p.split > 0x7FFFFFFF) return cudaErrorInvalidValue;
    cudaLaunchConfig_t config;
    memset(&config, 0, sizeof config);
    config.gridDim = dim3(static_cast<unsigned>(p.T * p.split));
    config.blockDim = dim3(kRowThreads);
    config.stream = stream;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim = {static_cast<unsigned>(p.split), 1, 1};
    config.attrs = &cluster;
    config.numAttrs = p.split > 1 ? 1 : 0;
    return dtype == kBf16 ? cudaLaunchKernelEx(&config, token_logprob_kernel<true>, p)
                          : cudaLaunchKernelEx(&config, token_logprob_kernel<false>, p);
}

cudaError_t launch_token_logprob_backward(LogprobParams p, int dtype, cudaStream_t stream)
{
    const int64_t items = p.rows * p.units;
    if (items == 0) return cudaSuccess;
    const int64_t ctas = (items + kTileUnits - 1) / kTileUnits;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(ctas);
    // the most rows that a tile touches
    const size_t shared = sizeof(RowOf) * static_cast<size_t>((kTileUnits - 1) / p.units + 2);
    if (dtype == kBf16) token_logprob_backward_kernel<true><<<grid, kTileThreads, shared, stream>>>(p);
    else token_logprob_backward_kernel<false><<<grid, kTileThreads, shared, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t read_logprob_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

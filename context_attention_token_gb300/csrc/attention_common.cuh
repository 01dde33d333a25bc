// What the attention kernels share: which keys a row sees, and a warp's plain
// computation of one row of each output from the definitions.
#pragma once

#include "cpt_device.cuh"
#include "cpt_internal.h"

namespace cpt {

// The keys (raw tokens) a row sees: [kb, kb + ns) and [lo, g], the second
// after the first and possibly empty. A row of padding sees none (g < kb).
struct RowKeys {
    int32_t g;    // raw token of the row itself
    int32_t kb;   // first token of its document
    int32_t ns;   // first tokens that stay visible
    int32_t lo;   // first token of the window behind them
};

// Document that holds raw token g: the largest d with cu[d] <= g.
__device__ __forceinline__ int32_t find_doc(const int32_t *cu, int32_t n_docs, int32_t g)
{
    int32_t a = 0, b = n_docs - 1;
    while (a < b) {
        const int32_t m = a + (b - a + 1) / 2;
        if (cu[m] <= g) a = m;
        else b = m - 1;
    }
    return a;
}

__device__ __forceinline__ RowKeys keys_of_token(const AttentionParams &p, int32_t g)
{
    RowKeys r;
    r.g = g;
    r.kb = p.cu[find_doc(p.cu, p.n_docs, g)];
    const int32_t u = g - r.kb;   // position in the document
    r.ns = min(p.sinks, u + 1);
    r.lo = r.kb + max(r.ns, p.window > u ? 0 : u - p.window + 1);
    return r;
}

// The same as up to two spans [x, y) and [z, w) of tokens in ascending order,
// (0, 0) when empty, one span alone in the second place.
__device__ __forceinline__ int4 spans_of(const AttentionParams &p, int32_t g)
{
    const RowKeys k = keys_of_token(p, g);
    int4 r = make_int4(0, 0, 0, 0);
    if (k.ns > 0) {
        r.x = k.kb;
        r.y = k.kb + k.ns;
    }
    if (k.lo <= g) {
        r.z = k.lo;
        r.w = g + 1;
        if (r.y == r.z && k.ns > 0) {
            r.z = r.x;
            r.x = r.y = 0;
        }
    }
    return r;
}

// First key >= x of a row's spans; the largest int when there is none.
__device__ __forceinline__ int next_key(int4 r, int x)
{
    return x < r.y ? max(x, r.x) : (x < r.w ? max(x, r.z) : 0x7FFFFFFF);
}

// Raw token of a local row; -1 for padding (and for an entry that fails its check).
__device__ __forceinline__ int32_t token_of_row(const AttentionParams &p, int64_t row)
{
    const int32_t g = p.l2r[row];
    return g >= 0 && in_bounds(g < p.T) ? g : -1;
}

// Four neighbouring bf16 elements, widened (zeros at and past `D`).
__device__ __forceinline__ float4 load4(const void *row, int at, int D)
{
    if (at >= D) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const uint2 x = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + at);
    return make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y));
}

__device__ __forceinline__ void store4(void *row, int at, int D, float4 x)
{
    if (at >= D) return;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(row) + at) =
        make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    return x;
}

__device__ __forceinline__ float dot4(float4 a, float4 b)
{
    return __fmaf_rn(a.x, b.x, __fmaf_rn(a.y, b.y, __fmaf_rn(a.z, b.z, __fmul_rn(a.w, b.w))));
}

__device__ __forceinline__ void axpy4(float4 &y, float a, float4 x)
{
    y.x = __fmaf_rn(a, x.x, y.x);
    y.y = __fmaf_rn(a, x.y, y.y);
    y.z = __fmaf_rn(a, x.z, y.z);
    y.w = __fmaf_rn(a, x.w, y.w);
}

// For rows that are computed again: whether one of four elements that the tiled kernels left
// without a finite value is not NaN in `now` (it stays NaN once it is).
__device__ __forceinline__ bool any_open(float4 tiled, float4 now)
{
    return (!isfinite(tiled.x) && now.x == now.x) || (!isfinite(tiled.y) && now.y == now.y) ||
           (!isfinite(tiled.z) && now.z == now.z) || (!isfinite(tiled.w) && now.w == now.w);
}

__device__ __forceinline__ float4 finite_or_nan(float4 x)
{
    return make_float4(isfinite(x.x) ? x.x : NAN, isfinite(x.y) ? x.y : NAN, isfinite(x.z) ? x.z : NAN,
                       isfinite(x.w) ? x.w : NAN);
}

__device__ __forceinline__ void note_nan(float4 &to, float4 x)
{
    if (x.x != x.x) to.x = NAN;
    if (x.y != x.y) to.y = NAN;
    if (x.z != x.z) to.z = NAN;
    if (x.w != x.w) to.w = NAN;
}

__device__ __forceinline__ bool all_nan(float4 x) { return x.x != x.x && x.y != x.y && x.z != x.z && x.w != x.w; }

__device__ __forceinline__ bool all_finite(float4 x)
{
    return isfinite(x.x) && isfinite(x.y) && isfinite(x.z) && isfinite(x.w);
}

__device__ __forceinline__ const uint16_t *row_of(const void *base, int64_t row, int heads, int head, int D)
{
    return static_cast<const uint16_t *>(base) + (row * heads + head) * D;
}

}  // namespace cpt

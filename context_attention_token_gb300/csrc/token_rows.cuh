// Helpers of the kernels that work on token rows in units of 16 bytes: unpacking to
// binary32, the counter-based generator of dropout, sums over the threads of a row.
#pragma once

#include "cpt_device.cuh"
#include "cpt_internal.h"

namespace cpt {

// A unit of 16 bytes: E consecutive columns of a row, in binary32.
template <bool BF16>
struct Unit {
    static constexpr int E = BF16 ? 8 : 4;
    static __device__ __forceinline__ void unpack(const uint4 &v, float (&x)[E])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
    // one rounding, to nearest even, for bf16
    static __device__ __forceinline__ uint4 pack(const float (&x)[E])
    {
        uint4 v;
        if constexpr (BF16) {
            v.x = pack_bf16x2(x[0], x[1]);
            v.y = pack_bf16x2(x[2], x[3]);
            v.z = pack_bf16x2(x[4], x[5]);
            v.w = pack_bf16x2(x[6], x[7]);
        } else {
            v.x = __float_as_uint(x[0]);
            v.y = __float_as_uint(x[1]);
            v.z = __float_as_uint(x[2]);
            v.w = __float_as_uint(x[3]);
        }
        return v;
    }
};

// The same as pairs of columns, for arithmetic on two values at a time.
template <bool BF16>
struct UnitPairs {
    static constexpr int N = Unit<BF16>::E / 2;
    static __device__ __forceinline__ void unpack(const uint4 &v, F2 (&x)[N])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (BF16) x[i] = pair_of(w[i] << 16, w[i] & 0xFFFF0000u);
            else x[i] = pair_of(w[2 * i], w[2 * i + 1]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const F2 (&x)[N])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 f = both(x[i]);
            if constexpr (BF16) {
                w[i] = pack_bf16x2(f.x, f.y);
            } else {
                w[2 * i] = __float_as_uint(f.x);
                w[2 * i + 1] = __float_as_uint(f.y);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Philox-4x32 with ten rounds, from the published description (Salmon and others, "Parallel
// random numbers: as easy as 1, 2, 3", 2011). Ten is the authors' recommendation; they found
// seven enough for their tests. One call serves eight columns with 16 bits each.
__device__ __forceinline__ uint4 philox(uint32_t k0, uint32_t k1, uint4 c)
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
        const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
        c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                       static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

struct DropKey {
    uint32_t k0, k1, step;
    __device__ __forceinline__ void load(const DropRule &r)
    {
        if (r.rng == nullptr) return;
        const uint64_t seed = r.rng[0];
        k0 = static_cast<uint32_t>(seed);
        k1 = static_cast<uint32_t>(seed >> 32);
        step = static_cast<uint32_t>(r.rng[1]);
    }
};

// Which elements of unit `unit` of `token`'s row are kept; the others become 0, whatever they were. The factor
// is the caller's to multiply by.
template <bool BF16>
__device__ __forceinline__ void drop_unit(const DropRule &r, const DropKey &key, uint32_t token, uint32_t unit,
                                          F2 (&x)[Unit<BF16>::E / 2])
{
    const uint4 w = philox(key.k0, key.k1, make_uint4(BF16 ? unit : unit >> 1, token, key.step, r.site));
    uint32_t h[4] = {w.x, w.y, w.z, w.w};
    if (!BF16 && (unit & 1)) {   // a float32 unit is half a group of eight columns
        h[0] = h[2];
        h[1] = h[3];
    }
    const uint32_t below = r.kept << 16;   // kept is 0..65535 here, so a half compares as the top of a word
#pragma unroll
    for (int i = 0; i < Unit<BF16>::E / 2; ++i) {
        const float2 f = both(x[i]);
        x[i] = pair_of((h[i] << 16) < below ? f.x : 0.0f, h[i] < below ? f.y : 0.0f);
    }
}

// Sums of N values over the `group` lanes of a warp that share a row (a power of two), in a fixed order.
template <int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N], int group)
{
    for (int d = group >> 1; d > 0; d >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], d));
    }
}

// Sums over a CTA of whole warps, in a fixed order. There are two places for the warps' sums; one is written
// again only after every thread has passed the barrier of the other, so one barrier a sum is enough.
struct BlockSum {
    float *room;   // [2][32 * 4], shared, 16-byte aligned
    int turn = 0;
    __device__ explicit BlockSum(float *r) : room(r) {}

    // one value
    __device__ __forceinline__ void operator()(float (&v)[1])
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        float *at = room + turn * 128;
        turn ^= 1;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], d));
        if (lane == 0) at[warp] = v[0];
        __syncthreads();
        const int span = warps > 16 ? 32 : warps > 8 ? 16 : 8;   // every `span` lanes hold all of the warps' sums
        v[0] = (lane & (span - 1)) < warps ? at[lane & (span - 1)] : 0.0f;
        for (int d = span >> 1; d > 0; d >>= 1) v[0] = __fadd_rn(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], d));
    }

    // three values: lanes give away those that they do not keep, so that 6 shuffles do for 15
    __device__ __forceinline__ void operator()(float (&v)[3])
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        float *at = room + turn * 128;
        turn ^= 1;
        const bool odd = lane & 1, upper = lane & 2;
        float a = odd ? v[1] : v[0], c = odd ? 0.0f : v[2];
        a = __fadd_rn(a, __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[1], 1));
        c = __fadd_rn(c, __shfl_xor_sync(0xFFFFFFFFu, odd ? v[2] : 0.0f, 1));
        float s = upper ? c : a;
        s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, upper ? a : c, 2));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
        if (lane < 4) at[warp * 4 + lane] = s;   // lane i: value i
        __syncthreads();
        s = 0.0f;
        for (int i = lane; i < warps * 4; i += 32) s = __fadd_rn(s, at[i]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
#pragma unroll
        for (int i = 0; i < 3; ++i) v[i] = __shfl_sync(0xFFFFFFFFu, s, i);
    }
};

}  // namespace cpt

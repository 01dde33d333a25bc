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

// x of unit `unit` of `token`'s row: times the factor where it is kept, 0 elsewhere.
template <bool BF16>
__device__ __forceinline__ void drop_unit(const DropRule &r, const DropKey &key, uint32_t token, uint32_t unit,
                                          float (&x)[Unit<BF16>::E])
{
    const uint4 w = philox(key.k0, key.k1, make_uint4(BF16 ? unit : unit >> 1, token, key.step, r.site));
    uint32_t h[4] = {w.x, w.y, w.z, w.w};
    if (!BF16 && (unit & 1)) {   // a float32 unit is half a group of eight columns
        h[0] = h[2];
        h[1] = h[3];
    }
#pragma unroll
    for (int e = 0; e < Unit<BF16>::E; e += 2) {
        const uint32_t v = h[e / 2];
        x[e] = (v & 0xFFFFu) < r.kept ? __fmul_rn(x[e], r.factor) : 0.0f;
        x[e + 1] = (v >> 16) < r.kept ? __fmul_rn(x[e + 1], r.factor) : 0.0f;
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

// Sums of N values over a CTA of whole warps, in a fixed order. `room` holds two turns of kSumRoom floats, whatever
// N a call has; a turn is written again only after every thread has passed the barrier of the other, so one
// barrier a sum is enough.
constexpr int kSumRoom = 96;
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *room, int &turn)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    static_assert(N * 32 <= kSumRoom, "more sums than a turn holds");
    float *at = room + turn * kSumRoom;
    turn ^= 1;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], d));
    }
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) at[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane < warps ? at[i * 32 + lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], d));
    }
}

}  // namespace cpt

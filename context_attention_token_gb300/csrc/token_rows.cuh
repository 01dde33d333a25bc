// Helpers of the kernels that work on token rows in units of 16 bytes: unpacking to
// binary32, the counter-based generator of dropout, sums over the threads of a row.
#pragma once

#include "cpt_device.cuh"
#include "cpt_internal.h"
#include "pairs.cuh"

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
// The N counters of a call go through the rounds side by side, with one key schedule.
template <int N>
__device__ __forceinline__ void philox(uint32_t k0, uint32_t k1, uint4 (&c)[N])
{
#pragma unroll
    for (int i = 0; i < 10; ++i) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const uint64_t a = static_cast<uint64_t>(c[n].x) * 0xD2511F53u;
            const uint64_t b = static_cast<uint64_t>(c[n].z) * 0xCD9E8D57u;
            c[n] = make_uint4(static_cast<uint32_t>(b >> 32) ^ c[n].y ^ k0, static_cast<uint32_t>(b),
                              static_cast<uint32_t>(a >> 32) ^ c[n].w ^ k1, static_cast<uint32_t>(a));
        }
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
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

// The random bits of N units: a word for every two of a unit's columns.
template <bool BF16, int N>
__device__ __forceinline__ void unit_bits(const DropRule &r, const DropKey &key, const uint32_t (&token)[N],
                                          const uint32_t (&unit)[N], uint32_t (&bits)[N][Unit<BF16>::E / 2])
{
    uint4 w[N];
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = make_uint4(BF16 ? unit[n] : unit[n] >> 1, token[n], key.step, r.site);
    philox<N>(key.k0, key.k1, w);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if constexpr (BF16) {
            bits[n][0] = w[n].x;
            bits[n][1] = w[n].y;
            bits[n][2] = w[n].z;
            bits[n][3] = w[n].w;
        } else {   // a float32 unit is half a group of eight columns
            bits[n][0] = unit[n] & 1 ? w[n].z : w[n].x;
            bits[n][1] = unit[n] & 1 ? w[n].w : w[n].y;
        }
    }
}

// The bits of a thread's units lane, lane + group, ... of a token's row, with groups of whole warps. Two neighbouring
// lanes have the halves of the same group of eight float32 columns: each calls the generator for one of two units
// and they exchange what the other needs.
template <bool BF16, int U>
__device__ __forceinline__ void thread_bits(const DropRule &r, const DropKey &key, uint32_t token, int lane, int group,
                                            uint32_t (&bits)[U][Unit<BF16>::E / 2])
{
    constexpr int C = BF16 ? U : U / 2;   // calls
    static_assert(BF16 || U % 2 == 0, "pairs of units");
    const bool odd = lane & 1;
    uint4 w[C];
#pragma unroll
    for (int k = 0; k < C; ++k)
        w[k] = make_uint4(BF16 ? lane + k * group : (lane + (2 * k + odd) * group) >> 1, token, key.step, r.site);
    philox<C>(key.k0, key.k1, w);
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const uint4 v = w[k];
        if constexpr (BF16) {
            bits[k][0] = v.x;
            bits[k][1] = v.y;
            bits[k][2] = v.z;
            bits[k][3] = v.w;
        } else {
            const uint32_t a = __shfl_xor_sync(0xFFFFFFFFu, odd ? v.x : v.z, 1);
            const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, odd ? v.y : v.w, 1);
            bits[2 * k][0] = odd ? a : v.x;
            bits[2 * k][1] = odd ? b : v.y;
            bits[2 * k + 1][0] = odd ? v.z : a;
            bits[2 * k + 1][1] = odd ? v.w : b;
        }
    }
}

// x where an element is kept, `other` where it is dropped.
template <int N>
__device__ __forceinline__ void keep_or(const DropRule &r, const uint32_t (&bits)[N], F2 (&x)[N], const F2 (&other)[N])
{
    const uint32_t below = r.kept << 16;   // kept is 0..65535 here, so a half compares as the top of a word
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 f = both(x[i]), o = both(other[i]);
        x[i] = pair_of((bits[i] << 16) < below ? f.x : o.x, bits[i] < below ? f.y : o.y);
    }
}

template <int N>
__device__ __forceinline__ void keep_or_zero(const DropRule &r, const uint32_t (&bits)[N], F2 (&x)[N])
{
    F2 zero[N];
#pragma unroll
    for (int i = 0; i < N; ++i) zero[i] = pair_of(0.0f, 0.0f);
    keep_or<N>(r, bits, x, zero);
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

// Threads of a CTA that work on the same rows: whole warps, with a barrier of their own (1..15).
struct Team {
    int thread, threads, barrier;
    __device__ __forceinline__ int warp() const { return thread >> 5; }
    __device__ __forceinline__ int warps() const { return threads >> 5; }
    // Waits for all of the team; whether any has asked.
    __device__ __forceinline__ bool any(bool ask) const
    {
        uint32_t r;
        asm volatile(
            "{ .reg .pred q, s; setp.ne.u32 q, %1, 0; barrier.cta.red.or.pred s, %2, %3, q; selp.u32 %0, 1, 0, s; }"
            : "=r"(r)
            : "r"(static_cast<uint32_t>(ask)), "r"(barrier), "r"(threads)
            : "memory");
        return r != 0;
    }
};

// Shared memory of another CTA of the cluster may be written once that CTA has begun: every thread arrives at its own start
// and waits for all before the first such write, with its loads in between.
__device__ __forceinline__ void cluster_begun() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_begun() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

// Sums over a team, in a fixed order. There are two places for the warps' sums; one is written again only after every
// thread has passed the barrier of the other, so one barrier a sum is enough.
template <int TURN>   // floats of a place: 1, 2, 4 or 8 for a warp's 1, 2, up to 4 or up to 8 values
struct TeamSum {
    static constexpr int kRoom = 2 * TURN;   // floats
    float *room;                             // shared
    Team team;
    int turn = 0;
    bool stop = false;   // the vote of the last barrier: a thread has asked to stop
    bool ask = false;
    __device__ TeamSum(float *r, const Team &t) : room(r), team(t) {}

    // N values: lanes give away those that they do not keep, so that (for N = 6) 9 shuffles do for 30
    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
        constexpr int W = N == 1 ? 1 : N == 2 ? 2 : N <= 4 ? 4 : 8;
        static_assert(N <= 8, "at most eight values");
        const int lane = team.thread & 31, warp = team.warp(), warps = team.warps();
        float *at = room + turn * TURN;
        turn ^= 1;
        float a[W];
#pragma unroll
        for (int i = 0; i < W; ++i) a[i] = i < N ? v[i] : 0.0f;
#pragma unroll
        for (int bit = 1; bit < W; bit *= 2) {   // then a[i] is value 2 i + (the lane's bit) of before
#pragma unroll
            for (int i = 0; i < W / 2 / bit; ++i) {
                const float keep = lane & bit ? a[2 * i + 1] : a[2 * i], give = lane & bit ? a[2 * i] : a[2 * i + 1];
                a[i] = __fadd_rn(keep, __shfl_xor_sync(0xFFFFFFFFu, give, bit));
            }
        }
        float s = a[0];
#pragma unroll
        for (int d = W; d < 32; d *= 2) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
        if (lane < W) at[warp * W + lane] = s;   // lane i: value i
        stop = team.any(ask);
        if (W == 1 && warps <= 4) {
            s = at[0];
            for (int i = 1; i < warps; ++i) s = __fadd_rn(s, at[i]);
            v[0] = s;
            return;
        }
        s = 0.0f;
        for (int i = lane; i < warps * W; i += 32) s = __fadd_rn(s, at[i]);
#pragma unroll
        for (int d = W; d < 32; d *= 2) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, d));
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = W == 1 ? s : __shfl_sync(0xFFFFFFFFu, s, i);
    }
};

}  // namespace cpt

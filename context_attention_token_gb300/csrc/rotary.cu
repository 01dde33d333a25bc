// Rotary positions with several axes, applied while token rows move between
// global order and rank-local order.
//
// Mathematics. Pair i of a head follows axis a(i); token g turns it by the
// angle theta = pos[a(i)][g] * f_i:
//   (x, y) -> (x cos - y sin, x sin + y cos),
// the inverse with -theta (the gradient of a rotation is its inverse). The
// elements past the last pair are copied.
//
// Angles. A binary32 product pos * f loses the angle of a far position (at
// pos = 2^17 it is off by 2^-7 rad), and binary64 runs at 1/64 of the binary32
// rate. Only the angle modulo one turn matters, so f_i / 2 pi is held as a
// 64-bit fixed-point fraction F_i of a turn and pos * F_i is taken modulo
// 2^64: an exact reduction in one integer multiplication, whatever the
// position. Its top two bits (rounded) are the quadrant; the next 30 are an angle
// in [-pi/4, pi/4]. In binary32 that is off by up to 8e-8 rad (2^-26 of a turn: the
// conversion 2.4e-8, the constant 2.2e-8, the product 3e-8), which stands beside
// the 6e-8 of a result's own rounding. The Taylor polynomials of sine (to x^9,
// remainder 1.8e-9) and cosine (to x^10, remainder 1.2e-10) hold in binary32.
//
// Traffic. Every row is read once and written once, so HBM bounds it. All
// heads of a token share its angles: a CTA computes the sines and cosines of
// a tile of tokens into shared memory once, then streams the heads of all
// tensors past them, four vectors of every thread in flight. Measured: 262144 x
// 2 x 20 x 128 bf16 in rank-local order 843 us, 6.37 TB/s; 131071 padded tokens x
// 2 x 16 x 128 bf16 moved from global order 366 us, 5.87 TB/s (a copy: 6.67).
#include "cpt_device.cuh"
#include "cpt_internal.h"

namespace cpt {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;     // rows in flight per thread
// The table of a CTA's tile (16 tokens of 64 pairs). While it is made the CTA loads nothing, so more and
// smaller ones keep HBM busier, until each has too few rows: 131071 padded tokens of 2 x 16 heads of 128 bf16
// take 434, 393, 366, 356 us with tables of 32, 16, 8, 4 KB, 262144 tokens of 2 x 20 heads 925, 870, 843, 856 us,
// 20011 tokens of 8 heads of 72 binary32 26, 25, 25, 31 us.
constexpr int kTableBytes = 8 * 1024;

// Sine and cosine of `phase` / 2^64 turns.
__device__ __forceinline__ void sincos_turns(uint64_t phase, float &sn, float &cs)
{
    const uint32_t hi = static_cast<uint32_t>(phase >> 32);
    const uint32_t quad = (hi + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(hi - (quad << 30));   // [-2^29, 2^29) of 2^32
    const float x = __fmul_rn(static_cast<float>(rest), 1.46291807926715968e-9f);  // 2 pi / 2^32
    const float z = __fmul_rn(x, x);
    float s = __fmaf_rn(z, 2.75573192239858907e-6f, -1.98412698412698413e-4f);
    s = __fmaf_rn(z, s, 8.33333333333333333e-3f);
    s = __fmaf_rn(z, s, -1.66666666666666667e-1f);
    s = __fmaf_rn(__fmul_rn(z, x), s, x);
    float c = __fmaf_rn(z, -2.75573192239858907e-7f, 2.48015873015873016e-5f);
    c = __fmaf_rn(z, c, -1.38888888888888889e-3f);
    c = __fmaf_rn(z, c, 4.16666666666666667e-2f);
    c = __fmaf_rn(z, c, -0.5f);
    c = __fmaf_rn(z, c, 1.0f);
    const float a = (quad & 1) ? c : s, b = (quad & 1) ? s : c;
    sn = (quad & 2) ? -a : a;
    cs = ((quad + 1) & 2) ? -b : b;
}

// VB consecutive bytes of a row: E values of type T.
template <int VB>
struct Raw;
template <>
struct Raw<16> { typedef uint4 type; };
template <>
struct Raw<8> { typedef uint2 type; };
template <>
struct Raw<4> { typedef uint32_t type; };
template <>
struct Raw<2> { typedef uint16_t type; };

template <int VB, bool BF16>
struct Vec {
    static constexpr int E = VB / (BF16 ? 2 : 4);
    typedef typename Raw<VB>::type R;
    union U {
        R r;
        uint16_t h[VB / 2];
        float f[VB >= 4 ? VB / 4 : 1];
        __device__ U() {}
    };
    static __device__ __forceinline__ void unpack(const R &r, float *x)
    {
        U u;
        u.r = r;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (BF16) x[e] = __uint_as_float(static_cast<uint32_t>(u.h[e]) << 16);
            else x[e] = u.f[e];
        }
    }
    // one rounding, to nearest even, for bf16
    static __device__ __forceinline__ R pack(const float *x)
    {
        U u;
        if constexpr (BF16) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const uint32_t w = pack_bf16x2(x[e], E > 1 ? x[e + 1] : 0.0f);
                u.h[e] = static_cast<uint16_t>(w);
                if (E > 1) u.h[e + 1] = static_cast<uint16_t>(w >> 16);
            }
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) u.f[e] = x[e];
        }
        return u.r;
    }
};

// C consecutive values of the table, from a multiple of C.
template <int C>
__device__ __forceinline__ void load_table(const float *from, float (&x)[C])
{
    if constexpr (C % 4 == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(from + i);
            x[i] = v.x;
            x[i + 1] = v.y;
            x[i + 2] = v.z;
            x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = from[i];
    }
}

// A thread keeps one unit of a head (VB bytes of each half of its pairs, VB
// bytes of neighbouring pairs when they are interleaved, or VB bytes that are
// copied) and walks over the (token, head) items of the CTA's tile of tokens.
template <int VB, bool BF16, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryParams p)
{
    typedef Vec<VB, BF16> V;
    typedef typename V::R R;
    constexpr int E = V::E;
    constexpr int kElem = BF16 ? 2 : 4;
    constexpr int C = INTER ? E / 2 : E;          // pairs of a unit, of which n is a multiple
    extern __shared__ __align__(16) float table[];   // [tile][2][pairs]
    __shared__ int32_t src_row[kRotaryMaxTile];
    const int n = p.pairs;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * p.tile;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(p.tile), p.rows - first));

    for (int t = threadIdx.x; t < tokens; t += kThreads) {
        const int64_t d = first + t;
        int64_t s = d;
        if (p.row_map != nullptr) s = p.row_map[d];
        if (s >= 0 && !in_bounds(s < p.src_rows)) s = -1;
        if (p.pad_map != nullptr && p.pad_map[d] < 0) s = -1;
        src_row[t] = static_cast<int32_t>(s);
    }
    for (int i = threadIdx.x; i < tokens * n; i += kThreads) {
        const int t = i / n, j = i - t * n;
        int64_t raw = first + t;
        if (p.token_map != nullptr) raw = p.token_map[raw];
        float sn = 0.0f, cs = 1.0f;
        if (raw >= 0 && in_bounds(raw < p.T)) {
            const int64_t pos = p.positions[static_cast<int64_t>(p.axis[j]) * p.T + raw];
            sincos_turns(static_cast<uint64_t>(pos) * p.turn[j], sn, cs);
        }
        table[(2 * t) * n + j] = cs;
        table[(2 * t + 1) * n + j] = p.inverse ? -sn : sn;
    }
    __syncthreads();

    const int units = p.rot_units + p.copy_units;
    const int groups = kThreads / units;
    const int unit = threadIdx.x % units;
    const int group = threadIdx.x / units;
    if (group >= groups) return;
    const bool rot = unit < p.rot_units;
    // byte offset of this unit in a head, and its first pair
    const int at = rot ? unit * VB : (INTER ? unit * VB : (unit + p.rot_units) * VB);
    const int pair = INTER ? unit * E / 2 : unit * E;
    const int half = n * kElem;
    const uint32_t heads = static_cast<uint32_t>(p.heads_total);
    const uint32_t items = static_cast<uint32_t>(tokens) * heads;

    // token and head of the thread's next item, and the step to the one after
    uint32_t at_token = group / heads, at_head = group - at_token * heads;
    const uint32_t step_tokens = groups / heads, step_heads = groups - step_tokens * heads;

    for (uint32_t i0 = group; i0 < items; i0 += groups * kUnroll) {
        R lo[kUnroll], hi[kUnroll];
        uint8_t *out[kUnroll];
        int tok[kUnroll];
        bool zero[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const uint32_t i = i0 + k * groups;
            out[k] = nullptr;
            const uint32_t t = at_token;
            int h = static_cast<int>(at_head);
            at_token += step_tokens;
            at_head += step_heads;
            if (at_head >= heads) {
                at_head -= heads;
                ++at_token;
            }
            if (i >= items) continue;
            int w = 0;
            while (h >= p.heads[w]) h -= p.heads[w++];
            const int64_t s = src_row[t];
            const int64_t in_head = static_cast<int64_t>(h) * p.head_bytes + at;
            out[k] = p.dst[w] + (first + t) * p.row_bytes[w] + in_head;
            tok[k] = static_cast<int>(t);
            zero[k] = s < 0;
            if (s >= 0) {
                const uint8_t *src = p.src[w] + s * p.row_bytes[w] + in_head;
                lo[k] = __ldcs(reinterpret_cast<const R *>(src));
                if (!INTER && rot) hi[k] = __ldcs(reinterpret_cast<const R *>(src + half));
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (out[k] == nullptr) continue;
            R a = lo[k], b = hi[k];
            float x[E], y[E];
            if (zero[k]) {
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = 0.0f;
                a = b = V::pack(x);
            } else if (rot) {
                float cs[C], sn[C];
                load_table<C>(table + 2 * tok[k] * n + pair, cs);
                load_table<C>(table + (2 * tok[k] + 1) * n + pair, sn);
                V::unpack(a, x);
                if constexpr (INTER) {
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float c = cs[e / 2], s = sn[e / 2], u = x[e], v = x[e + 1];
                        x[e] = __fmaf_rn(u, c, -__fmul_rn(v, s));
                        x[e + 1] = __fmaf_rn(u, s, __fmul_rn(v, c));
                    }
                } else {
                    V::unpack(b, y);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float c = cs[e], s = sn[e], u = x[e], v = y[e];
                        x[e] = __fmaf_rn(u, c, -__fmul_rn(v, s));
                        y[e] = __fmaf_rn(u, s, __fmul_rn(v, c));
                    }
                    b = V::pack(y);
                }
                a = V::pack(x);
            }
            __stcs(reinterpret_cast<R *>(out[k]), a);
            if (!INTER && rot) __stcs(reinterpret_cast<R *>(out[k] + half), b);
        }
    }
}

template <int VB, bool BF16>
cudaError_t launch_vec(const RotaryParams &p, bool interleaved, unsigned grid, size_t smem, cudaStream_t stream)
{
    if (interleaved) {
        if constexpr (VB >= (BF16 ? 4 : 8)) rotary_kernel<VB, BF16, true><<<grid, kThreads, smem, stream>>>(p);
        else return cudaErrorInvalidValue;   // a pair is one vector at least
    } else {
        rotary_kernel<VB, BF16, false><<<grid, kThreads, smem, stream>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(RotaryParams p, int dtype, bool interleaved, cudaStream_t stream)
{
    if (p.rows == 0 || p.heads_total == 0) return cudaSuccess;
    const int elem = dtype == kBf16 ? 2 : 4;
    // the widest vector that starts of heads and ends of pairs are multiples of
    const int span = (interleaved ? 2 : 1) * p.pairs * elem;
    int vb = 16;
    while (span % vb != 0 || p.head_bytes % vb != 0) vb /= 2;
    const int rot_bytes = 2 * p.pairs * elem;
    p.rot_units = span / vb;
    p.copy_units = (p.head_bytes - rot_bytes) / vb;
    // a tile: its table within kTableBytes, at least a few hundred items of work for a CTA
    const int row_floats = 2 * (p.pairs > 0 ? p.pairs : 1);
    int64_t tile = kTableBytes / (4 * row_floats);
    if (tile > kRotaryMaxTile) tile = kRotaryMaxTile;
    const int64_t per_sm = (p.rows + 4 * (int64_t)sm_count(-1) - 1) / (4 * (int64_t)sm_count(-1));
    if (tile > per_sm) tile = per_sm;
    if (tile < 1) tile = 1;
    p.tile = static_cast<int32_t>(tile);
    const int64_t grid = (p.rows + tile - 1) / tile;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const size_t smem = static_cast<size_t>(tile) * row_floats * 4;
    const unsigned g = static_cast<unsigned>(grid);
    if (dtype == kBf16) {
        switch (vb) {
        case 16: return launch_vec<16, true>(p, interleaved, g, smem, stream);
        case 8: return launch_vec<8, true>(p, interleaved, g, smem, stream);
        case 4: return launch_vec<4, true>(p, interleaved, g, smem, stream);
        default: return launch_vec<2, true>(p, interleaved, g, smem, stream);
        }
    }
    switch (vb) {
    case 16: return launch_vec<16, false>(p, interleaved, g, smem, stream);
    case 8: return launch_vec<8, false>(p, interleaved, g, smem, stream);
    default: return launch_vec<4, false>(p, interleaved, g, smem, stream);
    }
}

cudaError_t read_rotary_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

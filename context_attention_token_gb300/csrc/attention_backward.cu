// Gradient of the windowed attention.
//
//   p_ij = exp(scale q_i . k_j - lse_i), delta_i = do_i . o_i,
//   ds_ij = scale p_ij (do_i . v_j - delta_i),
//   dq_i = sum_j ds_ij k_j, and for the rows i of rank r alone
//   dk_j(r) = sum_i ds_ij q_i, dv_j(r) = sum_i p_ij do_i.
//
// Two kernels for the sums, each with its own S and dP: dQ by rows, dK and dV by
// keys, so that every sum stays in tensor memory until it is whole (or, cut into
// parts, is added up in their order) and a repeated call gives the same bits.
// p and ds are rounded to bf16 once, for the matrix unit; it bounds both:
// 8192 x 16 x 128, whole triangle, takes 0.26 ms for dQ (the unit busy for 79 % of
// it) and 0.35 ms for dK and dV (71 %), 0.61 to 0.67 ms in all.
#include "attention_common.cuh"
#include "tcgen05.cuh"

#include <atomic>

namespace cpt {

namespace {

typedef AttentionBackwardParams Params;

// Waits that ran out (see cpt_kernel_wait_timeouts).
__device__ unsigned int g_wait_timeouts;

// p and ds of one (row, key) pair, the same in every lane.
__device__ __forceinline__ void pair_grad(const Params &b, float4 q, float4 dout, float4 k, float4 v, float lse,
                                          float delta, float &p, float &ds)
{
    const float s = warp_sum(dot4(q, k)) * b.a.scale;
    const float dp = warp_sum(dot4(dout, v));
    p = lse == -INFINITY ? 0.0f : expf(s - lse);
    ds = p * (dp - delta) * b.a.scale;
}

// A warp's computation of one row from the definition, for rows that an
// infinity or NaN behind a hidden key or row spoiled in the tiled kernels. A NaN in
// lse or delta is in every ds of the row, and what is NaN stays so: the keys
// end with the last element that can be anything else.
__device__ __noinline__ void row_dq(const Params &b, int64_t row, int head)
{
    const AttentionParams &p = b.a;
    const int at = (threadIdx.x & 31) * 4, D = p.D;
    const int kvh = head / (p.Hq / p.Hkv);
    float4 dq = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int32_t g = token_of_row(p, row);
    if (g >= 0) {
        const float4 q = load4(row_of(p.q, row, p.Hq, head, D), at, D);
        const float4 dout = load4(row_of(b.dout, row, p.Hq, head, D), at, D);
        const float lse = p.lse[head * p.Tpad + row], delta = b.delta[head * p.Tpad + row];
        const RowKeys r = keys_of_token(p, g);
        int32_t j = r.kb;
        if (lse != lse || delta != delta) {
            dq = make_float4(NAN, NAN, NAN, NAN);
            j = g + 1;
        }
        while (true) {
            if (j == r.kb + r.ns) j = r.lo;
            if (j > g) break;
            const float4 k = load4(row_of(p.k, j, p.Hkv, kvh, D), at, D);
            float w, ds;
            pair_grad(b, q, dout, k, load4(row_of(p.v, j, p.Hkv, kvh, D), at, D), lse, delta, w, ds);
            axpy4(dq, ds, k);
            if (!__any_sync(0xFFFFFFFFu, at < D && !all_nan(dq))) break;
            ++j;
        }
    }
    store4(const_cast<uint16_t *>(row_of(b.dq, row, p.Hq, head, D)), at, D, dq);
}

// Rows of a rank whose (padded) global position is below x, a position of
// document doc or its end.
__device__ __forceinline__ int64_t rows_below(const Params &b, int rank, int32_t doc, int64_t x)
{
    const AttentionParams &p = b.a;
    if (b.packed) return min(max(x - rank * p.Tp, (int64_t)0), p.Tp);
    const int64_t begin = b.cup[doc], m = (b.cup[doc + 1] - begin) / (2 * p.P), u = x - begin;
    return begin / p.P + min(max(u - rank * m, (int64_t)0), m) +
           min(max(u - (2 * p.P - 1 - rank) * m, (int64_t)0), m);
}

// dK and dV of one raw key for one writer, over the rows of that rank. What a NaN in the
// rows' lse or delta settles is looked up first, 128 rows at a time: lse makes
// both NaN throughout, delta dK, and dV where that row's dO holds one (which is in its delta).
// Other elements are right where the tiled kernel's are finite.
__device__ __noinline__ void key_dkdv(const Params &b, int32_t j, int rank, int kvh)
{
    const AttentionParams &p = b.a;
    const int lane = threadIdx.x & 31, at = lane * 4, D = p.D, G = p.Hq / p.Hkv;
    const int32_t doc = find_doc(p.cu, p.n_docs, j);
    const int32_t kb = p.cu[doc], end = p.cu[doc + 1], pos0 = b.cup[doc] - kb;
    const int64_t pos = pos0 + j;
    uint16_t *const dk_row = const_cast<uint16_t *>(row_of(b.dk[rank], pos, p.Hkv, kvh, D));
    uint16_t *const dv_row = const_cast<uint16_t *>(row_of(b.dv[rank], pos, p.Hkv, kvh, D));
    // the rows that see the key
    const int32_t last = j - kb < p.sinks ? end : static_cast<int32_t>(min((int64_t)end, (int64_t)j + p.window));
    const int64_t row0 = rank * p.Tp + rows_below(b, rank, doc, pos);
    const int64_t row1 = rank * p.Tp + rows_below(b, rank, doc, (int64_t)pos0 + last);
    float4 dk = load4(dk_row, at, D), dv = load4(dv_row, at, D), seen = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float4 all = make_float4(NAN, NAN, NAN, NAN), tiled = dv;
    const bool dk_finite = !__any_sync(0xFFFFFFFFu, !all_finite(dk));
    bool lse_nan = false, delta_nan = false, settled = false;
    for (int64_t i0 = row0; !settled && i0 < row1; i0 += 128)
        for (int h = kvh * G; !settled && h < (kvh + 1) * G; ++h) {
            float lse[4], delta[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int64_t i = i0 + 32 * u + lane, x = h * p.Tpad + i;
                lse[u] = i < row1 ? p.lse[x] : 0.0f;
                delta[u] = i < row1 ? b.delta[x] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) lse_nan |= lse[u] != lse[u];
            lse_nan = __any_sync(0xFFFFFFFFu, lse_nan);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                unsigned todo = __ballot_sync(0xFFFFFFFFu, delta[u] != delta[u]);
                delta_nan |= todo != 0;
                while (!lse_nan && todo && __any_sync(0xFFFFFFFFu, any_open(tiled, seen))) {
                    const int64_t i = i0 + 32 * u + __ffs(todo) - 1;
                    todo &= todo - 1;
                    note_nan(seen, load4(row_of(b.dout, i, p.Hq, h, D), at, D));
                }
            }
            settled = lse_nan || ((delta_nan || dk_finite) && !__any_sync(0xFFFFFFFFu, any_open(tiled, seen)));
        }
    if (settled) {
        if (lse_nan || delta_nan) dk = all;
        dv = lse_nan ? all : finite_or_nan(tiled);
    } else {
        const float4 k = load4(row_of(p.k, j, p.Hkv, kvh, D), at, D);
        const float4 v = load4(row_of(p.v, j, p.Hkv, kvh, D), at, D);
        dk = dv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int64_t i = row0; i < row1; ++i) {
            for (int h = kvh * G; h < (kvh + 1) * G; ++h) {
                const float4 q = load4(row_of(p.q, i, p.Hq, h, D), at, D);
                const float4 dout = load4(row_of(b.dout, i, p.Hq, h, D), at, D);
                float w, ds;
                pair_grad(b, q, dout, k, v, p.lse[h * p.Tpad + i], b.delta[h * p.Tpad + i], w, ds);
                axpy4(dk, ds, q);
                axpy4(dv, w, dout);
            }
            if (!__any_sync(0xFFFFFFFFu, at < D && !(all_nan(dk) && all_nan(dv)))) break;
        }
    }
    store4(dk_row, at, D, dk);
    store4(dv_row, at, D, dv);
}

// ----------------------------------------------------------------- preparation

constexpr int kPrepRows = 32;   // rows of one block: 8 lanes each
constexpr int kPrepHeads = 4;   // and heads, whose loads are in flight together

__device__ __forceinline__ float4 floats(uint32_t a, uint32_t b)
{
    return make_float4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b));
}

// Rows: delta and the base-2 log-sum-exp of every (head, row), the spans of
// keys that a row sees, zeros in the writers' padding positions. A row that
// sees nothing gets lse2 = +inf, which makes all its weights zero.
__device__ __forceinline__ void prepare_rows(const Params &b, int64_t block)
{
    const AttentionParams &p = b.a;
    const int groups = (p.Hq + kPrepHeads - 1) / kPrepHeads;
    const int head0 = static_cast<int>(block % groups) * kPrepHeads;
    const int64_t row = block / groups * kPrepRows + threadIdx.x / 8;
    const int lane = threadIdx.x & 7;
    const bool in = row < p.Tpad;
    const int32_t g = in ? token_of_row(p, row) : -1;
    float d[kPrepHeads];
#pragma unroll
    for (int h = 0; h < kPrepHeads; ++h) {
        d[h] = 0.0f;
        if (g < 0 || head0 + h >= p.Hq) continue;
        const uint16_t *o = row_of(p.out, row, p.Hq, head0 + h, p.D), *w = row_of(b.dout, row, p.Hq, head0 + h, p.D);
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // up to 128 elements
            const int at = 8 * lane + 64 * i;
            if (at < p.D) {
                const uint4 x = *reinterpret_cast<const uint4 *>(o + at), y = *reinterpret_cast<const uint4 *>(w + at);
                d[h] += dot4(floats(x.x, x.y), floats(y.x, y.y)) + dot4(floats(x.z, x.w), floats(y.z, y.w));
            }
        }
    }
    float mine = 0.0f;   // lane h keeps head h's
#pragma unroll
    for (int h = 0; h < kPrepHeads; ++h) {
#pragma unroll
        for (int s = 4; s > 0; s >>= 1) d[h] += __shfl_xor_sync(0xFFFFFFFFu, d[h], s);
        if (lane == h) mine = d[h];
    }
    if (!in) return;
    if (lane < kPrepHeads && head0 + lane < p.Hq) {
        const int64_t at = (head0 + lane) * p.Tpad + row;
        const float lse = g >= 0 ? p.lse[at] : -INFINITY;
        b.delta[at] = mine;
        b.lse2[at] = lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f;
    }
    // the rows that see nothing: the matrix kernels pass them over
    if (g < 0 || (p.window == 0 && p.sinks == 0)) {
        uint16_t *dq = const_cast<uint16_t *>(row_of(b.dq, row, p.Hq, head0, p.D));
        const int elements = min(kPrepHeads, p.Hq - head0) * p.D;   // neighbouring heads
        for (int i = 8 * lane; i < elements; i += 64) *reinterpret_cast<uint4 *>(dq + i) = make_uint4(0, 0, 0, 0);
    }
    if (head0 != 0) return;
    if (lane == 0) {
        int4 r = make_int4(0, 0, 0, 0);
        if (g >= 0) r = spans_of(p, g);
        b.spans[row] = r;
    }
    if (p.l2r[row] < 0) {
        const int64_t bytes = static_cast<int64_t>(p.Hkv) * p.D * 2, pos = b.l2g[row];
        if (in_bounds(pos >= 0 && pos < p.Tpad))
            for (int r = 0; r < p.P; ++r)
                for (int64_t i = 16 * lane; i < bytes; i += 128) {
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(b.dk[r]) + pos * bytes + i) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(b.dv[r]) + pos * bytes + i) = make_uint4(0, 0, 0, 0);
                }
    }
}

// Padded global position of a raw token.
__device__ __forceinline__ int32_t position_of_token(const Params &b, int32_t j)
{
    if (b.r2l == nullptr) return j;
    const int32_t row = b.r2l[j];
    return in_bounds(row >= 0 && row < b.a.Tpad) ? b.l2g[row] : -1;
}

// Tiles of 128 rows in a key tile's ranges: of the first, where the second
// begins (the last tile of the first may reach into it), of both.
__device__ __forceinline__ int3 row_tiles_of(int4 range)
{
    const int first = (range.y - range.x + kTile - 1) / kTile, from = max(range.z, range.x + first * kTile);
    return make_int3(first, from, first + (range.w > from ? (range.w - from + kTile - 1) / kTile : 0));
}

// ----------------------------------------------------------------- units of work
//
// A key tile takes as many row tiles as see it: few behind a window, all of a
// document under the whole triangle or where its sinks lie. Those with more
// than half of a CTA's share of all row tiles (kLeastPart at least) are cut into
// parts, which leave binary32 sums in the workspace; whichever part ends last
// adds them up in their order. So no CTA is left with a long tile alone, and
// small batches use more CTAs than they have key tiles.

// Parts of at least 2, 4, 8, 16, 32 row tiles: 4799 tokens in documents x 4(2) x 128, window 18, take 80, 73, 76,
// 87, 100 us, 4096 x 4(2) x 128, window 1000, 91, 90, 96, 92, 111 us, 65536 x 2(1) x 64, window 64, 179, 178,
// 179, 161, 192 us; larger batches do not cut that fine.
constexpr int kLeastPart = 4;

// Lists the units: {slot, part, parts, place of the first part's sums}. One warp,
// of the last block to have put its tile in the list.
__device__ void list_units(const Params &b, int slots, int sms)
{
    const int lane = threadIdx.x & 31, group = b.a.Hq / b.a.Hkv;
    const int front = __ldcg(&b.counters[0]), n = front + __ldcg(&b.counters[1]);
    const long long entries = __ldcg(reinterpret_cast<const long long *>(b.counters + 4)) * b.a.Hkv;
    const long long share = (entries + 2 * sms - 1) / (2 * sms);
    const int most = static_cast<int>(min(max(share, (long long)kLeastPart), 0x40000000ll));
    int units = 0, places = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        int slot = 0, parts = 0;
        if (i < n) {
            slot = __ldcg(&b.list[i < front ? i : slots - 1 - (i - front)]);
            parts = (row_tiles_of(__ldcg(&b.ranges[slot])).z * group + most - 1) / most;
        }
        const int need = parts > 1 ? parts : 0;
        int u = parts, q = need;   // inclusive sums over the warp
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int du = __shfl_up_sync(0xFFFFFFFFu, u, s), dq = __shfl_up_sync(0xFFFFFFFFu, q, s);
            if (lane >= s) {
                u += du;
                q += dq;
            }
        }
        for (int k = 0; k < parts; ++k)
            if (in_bounds(units + u - parts + k < b.unit_places))
                b.units[units + u - parts + k] = make_int4(slot, k, parts, places + q - need);
        units += __shfl_sync(0xFFFFFFFFu, u, 31);
        places += __shfl_sync(0xFFFFFFFFu, q, 31);
    }
    if (lane == 0) b.counters[6] = units;
}

// Key tiles of every rank: the local rows that may see one of the 128 keys, as
// up to two ranges (the window's, and the rest of the documents whose
// sinks lie in the tile); tiles that no row sees keep an empty one.
// The others go into a list, those with a range of sinks (the long ones) from
// its front, the rest from its back. The order of the list sets which CTA takes
// a tile and no result.
__device__ __forceinline__ void prepare_tile(const Params &b, int block, int tiles, int sms)
{
    const AttentionParams &p = b.a;
    __shared__ bool last;
    const int rank = block % p.P, tile = block / p.P;
    const int32_t k0 = tile * kTile, k1 = static_cast<int32_t>(min((int64_t)k0 + kTile, p.T)) - 1;
    if (threadIdx.x == 0) {
        const int32_t d0 = find_doc(p.cu, p.n_docs, k0), d1 = find_doc(p.cu, p.n_docs, k1);
        const int64_t pos0 = b.cup[d0] + (k0 - p.cu[d0]), pos1 = b.cup[d1] + (k1 - p.cu[d1]), end = b.cup[d1 + 1];
        int64_t w0 = 0, w1 = 0, s0 = 0, s1 = 0;
        if (p.window > 0) {
            w0 = rows_below(b, rank, d0, pos0);
            w1 = rows_below(b, rank, d1, min(pos1 + p.window, end));
        }
        const bool own_sinks = k0 - p.cu[d0] < p.sinks;
        if (p.sinks > 0 && (own_sinks || d1 > d0)) {
            s0 = rows_below(b, rank, d0, own_sinks ? pos0 : (int64_t)b.cup[d0 + 1]);
            s1 = rows_below(b, rank, d1, end);
        }
        const bool far = s1 > s0 && s1 > w1;
        if (w1 <= w0) {
            w0 = s0;
            w1 = s1;
            s0 = s1 = 0;
        } else if (s1 <= s0) {
            s0 = s1 = 0;
        } else if (s0 <= w1) {
            w1 = max(w1, s1);
            s0 = s1 = 0;
        }
        const int i = tile * p.P + rank;
        b.ranges[i] = make_int4((int)w0, (int)w1, (int)s0, (int)s1);
        if (w1 > w0) {
            // row tiles of all heads of a group
            const long long entries = static_cast<long long>(row_tiles_of(b.ranges[i]).z) * (p.Hq / p.Hkv);
            atomicAdd(reinterpret_cast<unsigned long long *>(b.counters + 4), static_cast<unsigned long long>(entries));
            if (far) b.list[atomicAdd(&b.counters[0], 1)] = i;
            else b.list[tiles * p.P - 1 - atomicAdd(&b.counters[1], 1)] = i;
        }
        __threadfence();
        last = atomicAdd(&b.counters[7], 1) == tiles * p.P - 1;
        __threadfence();
    }
    __syncthreads();
    if (last && threadIdx.x < 32) list_units(b, tiles * p.P, sms);
}

// Zeros in the gradients of key tiles that no row of the rank sees. One warp, which
// has nothing else to do while the matrix unit is busy; as a part of the
// preparation these writes took it from 0.07 to 0.2 ms (32768 x 20 x 128, 4 ranks).
__device__ void zero_unseen(const Params &b, int slots)
{
    const AttentionParams &p = b.a;
    const int lane = threadIdx.x & 31;
    const int64_t bytes = static_cast<int64_t>(p.Hkv) * p.D * 2;
    for (int i = blockIdx.x; i < slots; i += gridDim.x) {
        const int4 range = b.ranges[i];
        if (range.y > range.x) continue;
        const int32_t k0 = i / p.P * kTile;
        uint8_t *dk = static_cast<uint8_t *>(b.dk[i % p.P]), *dv = static_cast<uint8_t *>(b.dv[i % p.P]);
        for (int t0 = 0; t0 < kTile; t0 += 32) {
            const int32_t mine = k0 + t0 + lane < p.T ? position_of_token(b, k0 + t0 + lane) : -1;
            for (int t = 0; t < 32; ++t) {
                const int64_t pos = __shfl_sync(0xFFFFFFFFu, mine, t);
                if (pos < 0) continue;
                for (int64_t at = pos * bytes + 16 * lane; at < (pos + 1) * bytes; at += 512) {
                    st_once(dk + at, make_uint4(0, 0, 0, 0));
                    st_once(dv + at, make_uint4(0, 0, 0, 0));
                }
            }
        }
    }
}

// One launch for both, the tiles first, so that the units are listed while rows
// are still read.
__global__ void __launch_bounds__(8 * kPrepRows) prepare_kernel(const __grid_constant__ Params b, int tiles, int sms)
{
    next_grid_may_start();
    const int slots = tiles * b.a.P;
    if (static_cast<int64_t>(blockIdx.x) < slots) prepare_tile(b, blockIdx.x, tiles, sms);
    else prepare_rows(b, static_cast<int64_t>(blockIdx.x) - slots);
}

// ----------------------------------------------------------------- shared by both kernels

constexpr int kRing = 8;       // tile announcements in flight
constexpr int kThreads = 640;  // 4 warps that load and issue, 4 warpgroups that compute
constexpr uint32_t kFull = 1, kFirst = 2, kLast = 4, kStop = 8, kDirty = 16, kPart = 32;

template <int DP>
struct Shape {
    static constexpr int kSlabs = DP / 64;
    static constexpr uint32_t kTileBytes = kSlabs * kSlab;
};

struct Maps {
    CUtensorMap q, k, v, dout;
};

__device__ __forceinline__ void load_tile(const CUtensorMap *map, uint32_t to, int slabs, int head, int64_t row,
                                          uint64_t *bar)
{
    mbar_expect_tx(bar, slabs * kSlab);
    for (int i = 0; i < slabs; ++i) tma_slab(to + i * kSlab, map, 64 * i, head, static_cast<int>(row), bar);
}

// d (+)= A B with the weights of a tile, which lie as four quarters of 32 inner
// columns (one for each warpgroup), each over the first half of the columns of
// scores that it came from.
__device__ __forceinline__ void mma_quarters(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add)
{
    mma_weights<4, 2>(d, a, 32, b, 4096, shape, add);
}

// The same over the first or second 16 inner columns of every quarter.
template <int PART>
__device__ __forceinline__ void mma_half(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, bool add)
{
    mma_weights<4, 1>(d, a + 8 * PART, 32, b + 2048 * PART, 4096, shape, add);
}

// One arrival of a warp whose lanes have all written (or read) tensor memory.
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    tmem_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The bits of a 32 x 32 matrix, one row per lane, transposed.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x)
{
    const uint32_t lane = threadIdx.x & 31;
    uint32_t m = 0x0000FFFFu;
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, j);
        x = lane & j ? (x & ~m) | ((y & ~m) >> j) : (x & m) | ((y & m) << j);
        m ^= m << (j >> 1);
    }
    return x;
}

__device__ __forceinline__ uint32_t visible_bits(int4 r, int key, int word)
{
    return span_bits(r.x - key, r.y - key, word) | span_bits(r.z - key, r.w - key, word);
}

// ----------------------------------------------------------------- dQ
//
// An item is 128 query rows of one head; Q and dO stay in shared memory, the
// key tiles pass by as in the forward kernel. Per key tile three products,
//   S = Q K^T, dP = dO V^T, dQ += dS K,
// with dS = P (dP - delta), rounded to bf16 for the matrix unit, over S in
// tensor memory. S is there twice and issued a tile ahead, so that while four
// warpgroups (32 key columns each, one thread per row) make dS, the matrix unit
// has the last tile's dQ and the next S to do.
// Tensor memory: S, S, dP, dQ. Shared memory: Q, dO, 3 K, 2 V.

template <int DP>
struct DqShared {
    static constexpr int kK = 3, kV = 2;
    uint8_t q[Shape<DP>::kTileBytes], dout[Shape<DP>::kTileBytes];
    uint8_t k[kK][Shape<DP>::kTileBytes], v[kV][Shape<DP>::kTileBytes];
    uint64_t q_full, do_full;
    uint64_t k_full[kK], k_empty[kK], v_full[kV];
    uint64_t info_full[kRing], info_empty[kRing];
    uint64_t s_ready[2], dp_ready[2], dp_free;
    uint64_t ds_ready[2];              // by tile parity: a warp may be a tile ahead of another
    uint64_t acc_done, drained[2];
    int4 info[kRing];              // first key, flags, item
    uint32_t tmem, stop, spoiled;
};

struct DqItem {
    int rank, head;
    int64_t row0;
};

__device__ __forceinline__ DqItem dq_item(const AttentionParams &p, int64_t i, int64_t row_tiles)
{
    DqItem t;
    const int64_t per_head = row_tiles * p.P, h = i / per_head, j = i - h * per_head;
    t.head = static_cast<int>(h);
    t.rank = static_cast<int>(j % p.P);
    t.row0 = (row_tiles - 1 - j / p.P) * kTile;
    return t;
}

template <int DP, int STEPS>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ Params b, const __grid_constant__ Maps maps, int64_t items, int64_t row_tiles,
              int slots)
{
    typedef DqShared<DP> Sh;
    constexpr int kSlabs = Shape<DP>::kSlabs;
    const AttentionParams &p = b.a;
    extern __shared__ __align__(1024) uint8_t raw[];
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    const bool aligned = (smem_addr(raw) & 1023) == 0;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    if (warp == 3) tmem_alloc(&sh.tmem);
    if (threadIdx.x == 0) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.do_full, 1);
        for (int i = 0; i < Sh::kK; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < Sh::kV; ++i) mbar_init(&sh.v_full[i], 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh.info_full[i], 1);
            mbar_init(&sh.info_empty[i], 18);     // issuers, 16 warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_ready[i], 1);
            mbar_init(&sh.dp_ready[i], 1);
            mbar_init(&sh.ds_ready[i], 16);
        }
        mbar_init(&sh.dp_free, 16);
        mbar_init(&sh.acc_done, 1);
        mbar_init(&sh.drained[0], 1);
        mbar_init(&sh.drained[1], 1);
        sh.spoiled = 0;
        sh.stop = aligned ? 0 : 1;  // the swizzle needs 1024-byte tiles
        mbar_init_fence();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // from here on what the preparation has left is read; dK and dV need nothing of this kernel's
    wait_for_last_grid();
    next_grid_may_start();
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *stop = &sh.stop;
    const int steps = STEPS ? STEPS : (p.D + 15) / 16;
    // 128 x 64 + 512 x 104 of the 640 x 96 registers of the launch
    if (warp < 4) {
    fewer_registers<64>();
    if (warp == 0 && aligned) {
        // ------------------------------------------------------------- loader
        uint32_t n = 0;                           // tiles
        uint32_t nk = 0, nv = 0, nq = 0, no = 0;  // loads issued
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
            return ok;
        };
        auto announce = [&](int key, uint32_t flags, int64_t item) {
            const uint32_t s = n % kRing;
            if (wait(&sh.info_empty[s], (n / kRing & 1) ^ 1) && lane == 0) {
                sh.info[s] = make_int4(key, static_cast<int>(flags), static_cast<int>(item & 0xFFFFFFFF),
                                       static_cast<int>(item >> 32));
                mbar_arrive(&sh.info_full[s]);
            }
            return ok;
        };
        for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x) {
            const DqItem t = dq_item(p, it, row_tiles);
            const int64_t row = t.rank * p.Tp + t.row0;
            int4 r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = t.row0 + lane + 32 * i < p.Tp ? b.spans[row + lane + 32 * i] : make_int4(0, 0, 0, 0);
            auto next = [&](int x) {
                return __reduce_min_sync(0xFFFFFFFFu, min(min(next_key(r[0], x), next_key(r[1], x)),
                                                          min(next_key(r[2], x), next_key(r[3], x))));
            };
            const int kvh = t.head / (p.Hq / p.Hkv);
            int key = next(0);
            if (key == 0x7FFFFFFF) continue;   // no row sees a key
            // the last item's Q is free with its last S, its dO with its last dP; a V with its dP (by tile
            // parity: the next tile's may be ready too by the time this one's is asked for)
            // A wait by parity takes a phase that has not begun for one that is over, so the S before is waited
            // for first: with three tiles so far nothing else has waited for S(0), on whose barrier S(2)
            // comes (dP(0), without Q, may be there long before it).
            const uint32_t m = n - 1;
            if (n > 1 && !wait(&sh.s_ready[(m - 1) & 1], (m - 1) / 2 & 1)) break;
            if (n > 0 && !wait(&sh.s_ready[m & 1], m / 2 & 1)) break;
            if (lane == 0) load_tile(&maps.q, smem_addr(sh.q), kSlabs, t.head, row, &sh.q_full);
            ++nq;
            for (uint32_t first = kFirst; ok && key != 0x7FFFFFFF; first = 0) {
                const int end = key + kTile;
                bool full = true;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    full &= (r[i].x <= key && r[i].y >= end) || (r[i].z <= key && r[i].w >= end) ||
                            (r[i].y == 0 && r[i].w == 0);
                uint32_t flags = first;
                if (__all_sync(0xFFFFFFFFu, full)) flags |= kFull;
                const int after = next(end);
                if (after == 0x7FFFFFFF) flags |= kLast;
                const uint32_t ks = n % Sh::kK, vs = n % Sh::kV;
                // the issuer asks for a tile's K before the last item's dO is free
                if (!announce(key, flags, it)) break;
                if (!wait(&sh.k_empty[ks], (n / Sh::kK & 1) ^ 1)) break;
                if (lane == 0) load_tile(&maps.k, smem_addr(sh.k[ks]), kSlabs, kvh, key, &sh.k_full[ks]);
                ++nk;
                if (first) {
                    if (n > 0 && !wait(&sh.dp_ready[m & 1], m / 2 & 1)) break;
                    if (lane == 0) load_tile(&maps.dout, smem_addr(sh.dout), kSlabs, t.head, row, &sh.do_full);
                    ++no;
                }
                if (n >= Sh::kV && !wait(&sh.dp_ready[n & 1], (n - 2) / 2 & 1)) break;
                if (lane == 0) load_tile(&maps.v, smem_addr(sh.v[vs]), kSlabs, kvh, key, &sh.v_full[vs]);
                ++nv;
                ++n;
                key = after;
            }
        }
        if (ok) announce(0, kStop, 0);
        if (*stop != 0 && lane == 0) {   // copies in flight end before the CTA does
            for (uint32_t i = nk > Sh::kK ? nk - Sh::kK : 0; i < nk; ++i)
                mbar_wait_bounded(&sh.k_full[i % Sh::kK], i / Sh::kK & 1);
            for (uint32_t i = nv > Sh::kV ? nv - Sh::kV : 0; i < nv; ++i)
                mbar_wait_bounded(&sh.v_full[i % Sh::kV], i / Sh::kV & 1);
            if (nq > 0) mbar_wait_bounded(&sh.q_full, (nq - 1) & 1);
            if (no > 0) mbar_wait_bounded(&sh.do_full, (no - 1) & 1);
        }
    } else if (warp < 3 && aligned) {
        // ------------------------------------------------------------- issuers
        // One warp for S and dQ, one for dP: what one spends on barriers passes while the matrix unit
        // works for the other.
        const bool leader = lane == 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        const uint32_t s_shape = mma_shape(kTile, false), o_shape = mma_shape(16 * steps, true);
        if (warp == 1) {
            uint32_t ns = 0, items_seen = 0;   // tiles whose S is issued, items begun
            uint32_t flags[2] = {0, 0};        // of the tiles between S and dQ
            auto issue_s = [&]() {             // false at the end
                const uint32_t slot = ns % kRing, ks = ns % Sh::kK;
                if (!wait(&sh.info_full[slot], ns / kRing & 1)) return false;
                const uint32_t e = static_cast<uint32_t>(sh.info[slot].y);
                __syncwarp();
                if (leader) mbar_arrive(&sh.info_empty[slot]);
                if (e & kStop) return false;
                if ((e & kFirst) && !wait(&sh.q_full, items_seen++ & 1)) return false;
                if (!wait(&sh.k_full[ks], ns / Sh::kK & 1)) return false;
                mma_scores<STEPS>(tmem + 128 * (ns & 1), smem_addr(sh.q), smem_addr(sh.k[ks]), s_shape, steps);
                mma_commit(&sh.s_ready[ns & 1]);
                flags[ns & 1] = e;
                ++ns;
                return true;
            };
            bool more = issue_s() && issue_s();
            for (uint32_t i = 0; i < ns; ++i) {
                if (!wait(&sh.ds_ready[i & 1], i / 2 & 1)) break;
                tmem_fence_after();
                const uint32_t e = flags[i & 1], ks = i % Sh::kK;
                mma_quarters(tmem + 384, tmem + 128 * (i & 1), smem_addr(sh.k[ks]), o_shape, !(e & kFirst));
                if (e & kLast) mma_commit(&sh.acc_done);
                mma_commit(&sh.k_empty[ks]);
                if (more) more = issue_s();
            }
        } else {
            uint32_t items_seen = 0;
            for (uint32_t n = 0;; ++n) {
                const uint32_t slot = n % kRing, vs = n % Sh::kV;
                if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
                const uint32_t e = static_cast<uint32_t>(sh.info[slot].y);
                __syncwarp();
                if (leader) mbar_arrive(&sh.info_empty[slot]);
                if (e & kStop) break;
                if ((e & kFirst) && !wait(&sh.do_full, items_seen++ & 1)) break;
                if (!wait(&sh.v_full[vs], n / Sh::kV & 1)) break;
                // dP's columns are in registers long before dS is made of them
                if (n > 0 && !wait(&sh.dp_free, (n - 1) & 1)) break;
                tmem_fence_after();
                mma_scores<STEPS>(tmem + 256, smem_addr(sh.dout), smem_addr(sh.v[vs]), s_shape, steps);
                mma_commit(&sh.dp_ready[n & 1]);
            }
        }
        mma_commit(&sh.drained[warp - 1]);
        mbar_wait_bounded(&sh.drained[warp - 1], 0);
    } else if (warp == 3) {
        // ------------------------------------------------------------- tiles that no row sees
        zero_unseen(b, slots);
    }
    } else {
        more_registers<104>();
        // ------------------------------------------------------------- scores to dS
        const int y = warp / 4 - 1, t = threadIdx.x & (kTile - 1);
        const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const float c = p.scale * 1.4426950408889634f;
        int4 r = make_int4(0, 0, 0, 0);
        float lse2 = INFINITY, delta = 0.0f;
        int head = 0;
        int64_t row = 0;
        bool valid = false;
        uint32_t done = 0;
        bool spoiled = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        for (uint32_t n = 0; aligned; ++n) {
            const uint32_t slot = n % kRing;
            if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
            const int4 e = sh.info[slot];
            const uint32_t flags = static_cast<uint32_t>(e.y);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
            if (flags & kStop) break;
            if (flags & kFirst) {
                const DqItem d = dq_item(p, static_cast<int64_t>(e.w) << 32 | static_cast<uint32_t>(e.z), row_tiles);
                head = d.head;
                row = d.rank * p.Tp + d.row0 + t;
                valid = d.row0 + t < p.Tp;
                r = make_int4(0, 0, 0, 0);
                lse2 = INFINITY;
                delta = 0.0f;
                if (valid) {
                    r = b.spans[row];
                    lse2 = b.lse2[head * p.Tpad + row];
                    delta = b.delta[head * p.Tpad + row];
                }
            }
            if (!wait(&sh.s_ready[n & 1], n / 2 & 1) || !wait(&sh.dp_ready[n & 1], n / 2 & 1)) break;
            tmem_fence_after();
            const uint32_t s_at = at + 128 * (n & 1) + 32 * y;
            uint32_t s[32], dp[32], w[16];
            tmem_load32(s_at, s);
            tmem_load32(at + 256 + 32 * y, dp);
            tmem_wait_loads(s);
            tmem_wait_loads(dp);
            warp_arrive(&sh.dp_free);
            if (!(flags & kFull)) {
                const uint32_t bits = visible_bits(r, e.x, y);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (!(bits >> j & 1)) s[j] = 0xFF800000u;
            }
            const F2 c2 = pair_of(c, c), lse22 = pair_of(-lse2, -lse2), delta2 = pair_of(-delta, -delta);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float2 a = both(fma2(pair_of(s[2 * j], s[2 * j + 1]), c2, lse22));
                const F2 pr = pair_of(exp2_fast(a.x), exp2_fast(a.y));
                const float2 ds = both(mul2(pr, add2(pair_of(dp[2 * j], dp[2 * j + 1]), delta2)));
                w[j] = pack_bf16x2(ds.x, ds.y);
            }
            tmem_store16(s_at, w);
            tmem_wait_stores();
            warp_arrive(&sh.ds_ready[n & 1]);
            if (flags & kLast) {
                if (!wait(&sh.acc_done, done++ & 1)) break;
                tmem_fence_after();
                float bad = 0.0f;
                const bool write = valid && (r.y != 0 || r.w != 0);
                uint16_t *out = const_cast<uint16_t *>(row_of(b.dq, row, p.Hq, head, p.D));
                if (32 * y < p.D) store_block(at + 384, y, p.D, p.scale, write, out, write, bad);
                tmem_fence_before();
                spoiled |= write && bad != 0.0f;
            }
        }
        if (spoiled) sh.spoiled = 1;
    }
    __syncthreads();
    if (warp == 3) tmem_free(tmem);
    if (sh.stop != 0) {
        if (threadIdx.x == 0) atomicAdd(&g_wait_timeouts, 1u);
        return;
    }
    if (threadIdx.x == 0 && sh.spoiled != 0) b.counters[3] = 1;
}

// ----------------------------------------------------------------- dK and dV
//
// An item is 128 keys of one kv head for one writer; K and V stay in shared
// memory, the row tiles that see them (of every query head of the group) pass
// by. Scores are transposed, so that P and dS are first operands in tensor
// memory:
//   S' = K Q^T, dP' = V dO^T, dV += P' dO, dK += dS' Q,
// issued as dV(i) S(i+1) by one warp and dK(i) dP(i+1) by another: the matrix
// unit works on two products while four warpgroups (32 row columns each, one
// thread per key) make P, and on the other two while they make dS.
// Tensor memory: S', dP', dV, dK. Shared memory: K, V, 3 Q, 2 dO.
// With heads of up to 64 elements the sums need half the columns, S' is there
// twice, and S(i+1) goes before dV(i) instead of waiting for P(i). With longer
// heads P lies over the only S' and S(i+1) waits for dV(i): there the products
// begin with the first half of P (and dS), while the second is made.

template <int DP>
struct DkvShared {
    static constexpr int kQ = 3, kO = 2;
    static constexpr bool kTwice = DP == 64;          // S' twice
    static constexpr uint32_t kDp = kTwice ? 256 : 128, kDv = kTwice ? 384 : 256, kDk = kTwice ? 448 : 384;
    uint8_t k[Shape<DP>::kTileBytes], v[Shape<DP>::kTileBytes];
    uint8_t q[kQ][Shape<DP>::kTileBytes], dout[kO][Shape<DP>::kTileBytes];
    float lse2[2][kTile], delta[2][kTile];
    uint64_t kv_full, q_full[kQ], do_full[kO];
    uint64_t info_full[kRing], info_empty[kRing];
    uint64_t aux_full[2], aux_empty[2];
    uint64_t s_ready[2], dp_ready[2];  // S' and dV of the tile before, dP' and dK of it: by tile parity
    uint64_t half[2], weights[2][2];   // P, dS in tensor memory: the first half of every quarter; all, by tile
                                       // parity (with S' twice a warp may be a tile ahead of another)
    uint64_t dv_done[2];               // with S' twice: dV of a tile, by tile parity
    uint64_t acc_done[2], drained[2];
    int4 info[kRing];              // first row, flags and head, tile * P + rank
    uint32_t tmem, stop, spoiled;
};

static_assert(sizeof(DkvShared<128>) <= 232448 && sizeof(DqShared<128>) <= 232448, "shared memory of a block");

// A warp's columns of a part's sums go to the workspace; the warp that is the
// last of all parts to come by gets their total, in the order of the parts, back
// into its tensor memory. [place][dV, dK][column][key]
__device__ __noinline__ bool add_parts(const Params &b, int4 unit, int kvh, int warp, int of_k, int odd, uint32_t acc)
{
    const int lane = threadIdx.x & 31, D32 = (b.a.D + 31) / 32 * 32, key = (warp & 3) * 32 + lane;
    const int64_t tile = 2ll * D32 * kTile, place0 = static_cast<int64_t>(unit.w) * b.a.Hkv + kvh;
    auto at = [&](int part, int column) {
        return b.sums + (place0 + static_cast<int64_t>(part) * b.a.Hkv) * tile + (of_k * D32 + column) * kTile + key;
    };
    for (int i = odd; 32 * i < b.a.D; i += 2) {
        uint32_t o[32];
        tmem_load32(acc + 32 * i, o);
        tmem_wait_loads(o);
        float *to = at(unit.y, 32 * i);
#pragma unroll
        for (int j = 0; j < 32; ++j) __stcg(to + j * kTile, __uint_as_float(o[j]));
    }
    __threadfence();
    __syncwarp();
    int before = 0;
    if (lane == 0) before = atomicAdd(&b.arrived[place0 * 16 + warp], 1);
    before = __shfl_sync(0xFFFFFFFFu, before, 0);
    if (before != unit.z - 1) return false;
    __threadfence();
    for (int i = odd; 32 * i < b.a.D; i += 2) {
        float sum[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) sum[j] = 0.0f;
        for (int part = 0; part < unit.z; ++part) {
            const float *from = at(part, 32 * i);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[j] += __ldcg(from + j * kTile);
        }
        uint32_t o[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(sum[16 * h + j]);
            tmem_store16(acc + 32 * i + 16 * h, o);
        }
        tmem_wait_stores();
    }
    return true;
}

template <int DP, int STEPS>
__global__ void __launch_bounds__(kThreads, 1)
    dkdv_kernel(const __grid_constant__ Params b, const __grid_constant__ Maps maps)
{
    typedef DkvShared<DP> Sh;
    constexpr int kSlabs = Shape<DP>::kSlabs;
    const AttentionParams &p = b.a;
    extern __shared__ __align__(1024) uint8_t raw[];
    Sh &sh = *reinterpret_cast<Sh *>(raw);
    const bool aligned = (smem_addr(raw) & 1023) == 0;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;
    if (warp == 3) tmem_alloc(&sh.tmem);
    if (threadIdx.x == 0) {
        mbar_init(&sh.kv_full, 1);
        for (int i = 0; i < Sh::kQ; ++i) mbar_init(&sh.q_full[i], 1);
        for (int i = 0; i < Sh::kO; ++i) mbar_init(&sh.do_full[i], 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh.info_full[i], 1);
            mbar_init(&sh.info_empty[i], 19);     // issuers, statistics, 16 warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.aux_full[i], 32);
            mbar_init(&sh.aux_empty[i], 16);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_ready[i], 1);
            mbar_init(&sh.dp_ready[i], 1);
            mbar_init(&sh.half[i], 16);
            mbar_init(&sh.weights[i][0], 16);
            mbar_init(&sh.weights[i][1], 16);
            mbar_init(&sh.dv_done[i], 1);
            mbar_init(&sh.acc_done[i], 1);
            mbar_init(&sh.drained[i], 1);
        }
        sh.spoiled = 0;
        sh.stop = aligned ? 0 : 1;
        mbar_init_fence();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    // What the preparation has left is read from here on, without a wait for the grid before (dQ), beside which this
    // one runs. Blocks start only once every block of dQ has said next_grid_may_start, which each does behind its
    // own wait for the preparation: that grid has ended by then, and its writes are in L2, which all
    // SMs share. The fence, of every thread that reads, keeps it from older lines of its SM's own cache.
    __threadfence();
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *stop = &sh.stop;
    const int steps = STEPS ? STEPS : (p.D + 15) / 16, group = p.Hq / p.Hkv;
    const int64_t items = static_cast<int64_t>(b.counters[6]) * p.Hkv;
    // 128 x 64 + 512 x 104 of the 640 x 96 registers of the launch
    if (warp < 4) {
    fewer_registers<64>();
    if (warp == 0 && aligned) {
        // ------------------------------------------------------------- loader
        uint32_t n = 0;                        // tiles
        uint32_t nq = 0, nkv = 0;              // loads issued
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
            return ok;
        };
        auto announce = [&](int row, uint32_t flags, int slot, int unit) {
            const uint32_t s = n % kRing;
            if (wait(&sh.info_empty[s], (n / kRing & 1) ^ 1) && lane == 0) {
                sh.info[s] = make_int4(row, static_cast<int>(flags), slot, unit);
                mbar_arrive(&sh.info_full[s]);
            }
            return ok;
        };
        // Items are as long as the rows that see their keys are many, so each is taken when the CTA is
        // free for it (dealt out in turn, the CTAs ended up to a fifth apart; this one may have started
        // late). The number of the next one is asked for an item ahead.
        auto take = [&]() { return lane == 0 ? atomicAdd(&b.counters[2], 1) : 0; };
        int64_t it = __shfl_sync(0xFFFFFFFFu, take(), 0);
        while (ok && it < items) {
            const int ahead = take();
            const int index = static_cast<int>(it / p.Hkv), kvh = static_cast<int>(it - index * (int64_t)p.Hkv);
            const int4 unit = b.units[index];
            const int4 range = b.ranges[unit.x];
            const int rank = unit.x % p.P, key = unit.x / p.P * kTile;
            const int64_t base = rank * p.Tp;
            int4 r[4];
            auto load_spans = [&](int from) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t row = from + lane + 32 * i;
                    r[i] = row < p.Tp ? b.spans[base + row] : make_int4(0, 0, 0, 0);
                }
            };
            const int3 tiles = row_tiles_of(range);
            const int total = tiles.z * group;
            const int e0 = static_cast<int>(static_cast<int64_t>(total) * unit.y / unit.z);
            const int e1 = static_cast<int>(static_cast<int64_t>(total) * (unit.y + 1) / unit.z);
            int h = e0 / tiles.z, j = e0 - h * tiles.z;
            auto row_of_tile = [&](int j) {
                return j < tiles.x ? range.x + j * kTile : tiles.y + (j - tiles.x) * kTile;
            };
            load_spans(row_of_tile(j));
            for (int e = e0; ok && e < e1; ++e) {
                // whether all rows see all keys, and whether some are not rows of this rank
                bool full = true, dirty = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    full &= (r[i].x <= key && r[i].y >= key + kTile) || (r[i].z <= key && r[i].w >= key + kTile);
                    dirty |= r[i].y == 0 && r[i].w == 0;
                }
                const int head = kvh * group + h, row0 = row_of_tile(j);
                uint32_t flags = static_cast<uint32_t>(head) << 16;
                if (__all_sync(0xFFFFFFFFu, full)) flags |= kFull;
                if (__any_sync(0xFFFFFFFFu, dirty)) flags |= kDirty;
                if (e == e0) flags |= kFirst;
                if (unit.z > 1) flags |= kPart;
                if (++j == tiles.z) {
                    j = 0;
                    ++h;
                }
                if (e == e1 - 1) flags |= kLast;
                else load_spans(row_of_tile(j));   // while the barriers below are waited for
                // The Q of tile j is free with tile j + 1's dP', which its dK precedes. This is waited for
                // before the tile is announced, so that its own dP' cannot come between.
                const uint32_t qs = n % Sh::kQ;
                if (n >= Sh::kQ && !wait(&sh.dp_ready[n & 1], (n - 2) / 2 & 1)) break;
                if (!announce(row0, flags, unit.x, index)) break;
                if (e == e0) {
                    // the last item's last tile has its S' and dP'
                    const uint32_t m = n - 1;
                    if (n > 0 && !(wait(&sh.s_ready[m & 1], m / 2 & 1) && wait(&sh.dp_ready[m & 1], m / 2 & 1))) break;
                    if (lane == 0) {
                        mbar_expect_tx(&sh.kv_full, 2 * kSlabs * kSlab);
                        for (int i = 0; i < kSlabs; ++i) {
                            tma_slab(smem_addr(sh.k) + i * kSlab, &maps.k, 64 * i, kvh, key, &sh.kv_full);
                            tma_slab(smem_addr(sh.v) + i * kSlab, &maps.v, 64 * i, kvh, key, &sh.kv_full);
                        }
                    }
                    ++nkv;
                }
                if (lane == 0) load_tile(&maps.q, smem_addr(sh.q[qs]), kSlabs, head, base + row0, &sh.q_full[qs]);
                ++nq;
                ++n;
            }
            it = __shfl_sync(0xFFFFFFFFu, ahead, 0);
        }
        if (ok) announce(0, kStop, 0, 0);
        if (*stop != 0 && lane == 0) {   // copies in flight end before the CTA does
            for (uint32_t i = nq > Sh::kQ ? nq - Sh::kQ : 0; i < nq; ++i)
                mbar_wait_bounded(&sh.q_full[i % Sh::kQ], i / Sh::kQ & 1);
            if (nkv > 0) mbar_wait_bounded(&sh.kv_full, (nkv - 1) & 1);
        }
    } else if (warp < 3 && aligned) {
        // ------------------------------------------------------------- issuers
        // One warp for S' and dV, one for dP' and dK: the same loop, on other barriers and operands.
        const bool leader = lane == 0, first = warp == 1;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        const uint32_t s_shape = mma_shape(kTile, false), o_shape = mma_shape(16 * steps, true);
        const uint32_t scores_at = tmem + (first ? 0 : Sh::kDp), acc = tmem + (first ? Sh::kDv : Sh::kDk);
        const uint32_t key_at = first ? smem_addr(sh.k) : smem_addr(sh.v);
        uint32_t prev = 0, k = 0;   // flags of the last tile, items begun
        for (uint32_t n = 0;; ++n) {
            const uint32_t slot = n % kRing;
            if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
            const uint32_t e = static_cast<uint32_t>(sh.info[slot].y);
            __syncwarp();
            if (leader) mbar_arrive(&sh.info_empty[slot]);
            const uint32_t i = n - 1, qs = n % Sh::kQ, os = n % Sh::kO;
            const bool fresh = (e & kFirst) != 0, more = !(e & kStop);
            // before a new item's K and V, the last one's products
            auto operand = [&]() {
                return first ? wait(&sh.q_full[qs], n / Sh::kQ & 1) : wait(&sh.do_full[os], n / Sh::kO & 1);
            };
            const uint32_t with = first ? smem_addr(sh.dout[i % Sh::kO]) : smem_addr(sh.q[i % Sh::kQ]);
            const bool twice = Sh::kTwice && first;
            auto product = [&]() {
                // dV reads dO, for which P has not waited
                if (first && !wait(&sh.do_full[i % Sh::kO], i / Sh::kO & 1)) return false;
                const uint32_t weights = scores_at + (twice ? 128 * (i & 1) : 0);
                if (!Sh::kTwice) {
                    if (!wait(&sh.half[warp - 1], i & 1)) return false;
                    tmem_fence_after();
                    mma_half<0>(acc, weights, with, o_shape, !(prev & kFirst));
                    if (!wait(&sh.weights[warp - 1][i & 1], i / 2 & 1)) return false;
                    tmem_fence_after();
                    mma_half<1>(acc, weights, with, o_shape, true);
                } else {
                    if (!wait(&sh.weights[warp - 1][i & 1], i / 2 & 1)) return false;
                    tmem_fence_after();
                    mma_quarters(acc, weights, with, o_shape, !(prev & kFirst));
                }
                if (prev & kLast) mma_commit(&sh.acc_done[warp - 1]);
                return true;
            };
            const bool late = n > 0 && twice && more && !fresh;   // the product after the next scores
            if (more && !fresh && !operand()) break;
            if (n > 0 && !late && !product()) break;
            if (!more) break;
            if (fresh && !(wait(&sh.kv_full, k++ & 1) && operand())) break;
            mma_scores<STEPS>(scores_at + (twice ? 128 * (n & 1) : 0), key_at,
                       first ? smem_addr(sh.q[qs]) : smem_addr(sh.dout[os]), s_shape, steps);
            mma_commit(first ? &sh.s_ready[n & 1] : &sh.dp_ready[n & 1]);
            if (late) {
                if (!product()) break;
                mma_commit(&sh.dv_done[i & 1]);
            } else if (Sh::kTwice && first && n > 0) {
                mma_commit(&sh.dv_done[i & 1]);
            }
            prev = e;
        }
        mma_commit(&sh.drained[warp - 1]);
        mbar_wait_bounded(&sh.drained[warp - 1], 0);
    } else if (warp == 3 && aligned) {
        // ------------------------------------------------------------- statistics of the rows, dO
        // A loader of its own: dO has two places and waits longer for one than Q does.
        int64_t rank_row = 0;
        uint32_t n = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        for (;; ++n) {
            const uint32_t slot = n % kRing, s = n & 1, os = n % Sh::kO;
            if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
            const int4 e = sh.info[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
            if (e.y & kStop) break;
            if (e.y & kFirst) rank_row = e.z % p.P * p.Tp;
            const int head = e.y >> 16;
            const int64_t base = head * p.Tpad + rank_row;
            float lse2[4], delta[4];   // negated, as they are added
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = e.x + lane + 32 * i;
                lse2[i] = row < p.Tp ? -b.lse2[base + row] : -INFINITY;
                delta[i] = row < p.Tp ? -b.delta[base + row] : 0.0f;
            }
            // the dO of tile j is free with its dV (which tile j + 1's S' follows, or which is told of by
            // itself) and its dP'
            if (n >= Sh::kO && !wait(&sh.dp_ready[n & 1], (n - 2) / 2 & 1)) break;
            if (n >= Sh::kO && !(Sh::kTwice ? wait(&sh.dv_done[n & 1], (n - 2) / 2 & 1)
                                            : wait(&sh.s_ready[(n - 1) & 1], (n - 1) / 2 & 1)))
                break;
            if (lane == 0)
                load_tile(&maps.dout, smem_addr(sh.dout[os]), kSlabs, head, rank_row + e.x, &sh.do_full[os]);
            if (!wait(&sh.aux_empty[s], (n / 2 & 1) ^ 1)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sh.lse2[s][lane + 32 * i] = lse2[i];
                sh.delta[s][lane + 32 * i] = delta[i];
            }
            mbar_arrive(&sh.aux_full[s]);
        }
        if (*stop != 0 && lane == 0)
            for (uint32_t i = n > Sh::kO ? n - Sh::kO : 0; i < n; ++i)
                mbar_wait_bounded(&sh.do_full[i % Sh::kO], i / Sh::kO & 1);
    }
    } else {
        more_registers<104>();
        // ------------------------------------------------------------- scores to P and dS
        const int y = warp / 4 - 1, t = threadIdx.x & (kTile - 1);
        const uint32_t at = tmem + (static_cast<uint32_t>(warp & 3) << 21);
        const uint32_t s_base = at + 32 * y, dp_at = at + Sh::kDp + 32 * y;
        const float c = p.scale * 1.4426950408889634f;
        int rank = 0, key = 0;
        int64_t base = 0;
        uint32_t done = 0;
        bool spoiled = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        for (uint32_t n = 0; aligned; ++n) {
            const uint32_t slot = n % kRing, a = n & 1;
            if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
            const int4 e = sh.info[slot];
            const uint32_t flags = static_cast<uint32_t>(e.y);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
            if (flags & kStop) break;
            if (flags & kFirst) {
                rank = e.z % p.P;
                key = e.z / p.P * kTile;
                base = rank * p.Tp;
            }
            // bit j: whether this thread's key is seen by row 32 y + j
            uint32_t bits = 0xFFFFFFFFu;
            if (!(flags & kFull)) {
                const int64_t row = e.x + 32 * y + lane;
                const int4 r = row < p.Tp ? b.spans[base + row] : make_int4(0, 0, 0, 0);
                bits = transpose_bits(visible_bits(r, key, warp & 3));
            }
            if (!wait(&sh.aux_full[a], n / 2 & 1)) break;
            if (!wait(&sh.s_ready[n & 1], n / 2 & 1)) break;
            if (flags & kDirty) {
                // Rows that are not this rank's, or padding, may hold anything: a weight of zero does
                // not keep a NaN out of a product, so they become zeros.
                if (!wait(&sh.dp_ready[n & 1], n / 2 & 1)) break;
                const int64_t row = e.x + t;
                const int4 r = row < p.Tp ? b.spans[base + row] : make_int4(0, 0, 0, 0);
                if (y < 2 && r.y == 0 && r.w == 0) {
                    uint8_t *tile = y == 0 ? sh.dout[n % Sh::kO] : sh.q[n % Sh::kQ];
                    for (int i = 0; i < kSlabs; ++i)
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4 *>(tile + i * kSlab + t * 128 + j * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tmem_fence_after();
            const uint32_t s_at = s_base + (Sh::kTwice ? 128 * (n & 1) : 0);
            uint32_t s[32], dp[32], w[16];
            tmem_load32(s_at, s);
            tmem_wait_loads(s);
            if (!(flags & kFull)) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (!(bits >> j & 1)) s[j] = 0xFF800000u;
            }
            const F2 c2 = pair_of(c, c);
            const float4 *l4 = reinterpret_cast<const float4 *>(&sh.lse2[a][32 * y]);   // negated
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 l = l4[j];
                const float2 u = both(fma2(pair_of(s[4 * j], s[4 * j + 1]), c2, pair_of(l.x, l.y)));
                const float2 v = both(fma2(pair_of(s[4 * j + 2], s[4 * j + 3]), c2, pair_of(l.z, l.w)));
                const float pr[4] = {exp2_fast(u.x), exp2_fast(u.y), exp2_fast(v.x), exp2_fast(v.y)};
                w[2 * j] = pack_bf16x2(pr[0], pr[1]);
                w[2 * j + 1] = pack_bf16x2(pr[2], pr[3]);
#pragma unroll
                for (int h = 0; h < 4; ++h) s[4 * j + h] = __float_as_uint(pr[h]);
                if (!Sh::kTwice && j == 3) {
                    tmem_store8(s_at, w);
                    tmem_wait_stores();
                    warp_arrive(&sh.half[0]);
                }
            }
            if (Sh::kTwice) tmem_store16(s_at, w);
            else tmem_store8(s_at + 8, w + 8);
            tmem_wait_stores();
            warp_arrive(&sh.weights[0][n & 1]);
            if (!wait(&sh.dp_ready[n & 1], n / 2 & 1)) break;
            tmem_fence_after();
            tmem_load32(dp_at, dp);
            tmem_wait_loads(dp);
            if (!(flags & kFull)) {   // a row that is none may have left a NaN
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (!(bits >> j & 1)) dp[j] = 0;
            }
            const float4 *d4 = reinterpret_cast<const float4 *>(&sh.delta[a][32 * y]);   // negated
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 l = d4[j];
                const float2 u = both(mul2(pair_of(s[4 * j], s[4 * j + 1]),
                                           add2(pair_of(dp[4 * j], dp[4 * j + 1]), pair_of(l.x, l.y))));
                const float2 v = both(mul2(pair_of(s[4 * j + 2], s[4 * j + 3]),
                                           add2(pair_of(dp[4 * j + 2], dp[4 * j + 3]), pair_of(l.z, l.w))));
                w[2 * j] = pack_bf16x2(u.x, u.y);
                w[2 * j + 1] = pack_bf16x2(v.x, v.y);
                if (!Sh::kTwice && j == 3) {
                    tmem_store8(dp_at, w);
                    tmem_wait_stores();
                    warp_arrive(&sh.half[1]);
                }
            }
            if (Sh::kTwice) tmem_store16(dp_at, w);
            else tmem_store8(dp_at + 8, w + 8);
            tmem_wait_stores();
            warp_arrive(&sh.weights[1][n & 1]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.aux_empty[a]);
            if (flags & kLast) {
                const int32_t pos = key + t < p.T ? position_of_token(b, key + t) : -1;
                const int kvh = static_cast<int>(flags >> 16) / group;
                const int of_k = y >> 1;   // two warpgroups write dV, two dK, every other 32 columns
                if (!wait(&sh.acc_done[of_k], done++ & 1)) break;
                tmem_fence_after();
                const uint32_t acc = at + (of_k ? Sh::kDk : Sh::kDv);
                bool write = pos >= 0;
                if (flags & kPart) write = add_parts(b, b.units[e.w], kvh, warp - 4, of_k, y & 1, acc) && write;
                float bad = 0.0f;
                uint16_t *out = const_cast<uint16_t *>(row_of(of_k ? b.dk[rank] : b.dv[rank], pos, p.Hkv, kvh, p.D));
                if (__any_sync(0xFFFFFFFFu, write))
                    for (int i = y & 1; 32 * i < p.D; i += 2)
                        store_block(acc, i, p.D, of_k ? p.scale : 1.0f, true, out, write, bad);
                tmem_fence_before();
                spoiled |= write && bad != 0.0f;
            }
        }
        if (spoiled) sh.spoiled = 1;
    }
    __syncthreads();
    if (warp == 3) tmem_free(tmem);
    // The repair may start; earlier its blocks, and here idle blocks of this grid, would keep SMs that other
    // streams could use. One block's wait makes this grid end after the one of dQ.
    next_grid_may_start();
    if (blockIdx.x == 0) wait_for_last_grid();
    if (sh.stop != 0) {
        if (threadIdx.x == 0) atomicAdd(&g_wait_timeouts, 1u);
        return;
    }
    if (threadIdx.x == 0 && sh.spoiled != 0) b.counters[3] = 1;
}

// ----------------------------------------------------------------- repair
//
// Only where the kernels above have seen an infinity or NaN in an output: all
// rows that hold one are computed again from the definitions, without a
// multiplication by what is hidden. Without one the launch ends at once.

__device__ bool spoiled_row(const uint16_t *row, int D)
{
    const int at = (threadIdx.x & 31) * 4;
    bool bad = false;
    if (at < D)
        for (int i = 0; i < 4; ++i) bad |= (row[at + i] & 0x7F80) == 0x7F80;
    return __any_sync(0xFFFFFFFFu, bad);
}

__global__ void __launch_bounds__(256) repair_kernel(const __grid_constant__ Params b)
{
    wait_for_last_grid();
    if (b.counters[3] == 0) return;
    const AttentionParams &p = b.a;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / 32, warps = gridDim.x * 8ll;
    for (int64_t i = warp; i < p.Tpad * p.Hq; i += warps) {
        const int64_t row = i / p.Hq;
        const int head = static_cast<int>(i % p.Hq);
        if (p.l2r[row] >= 0 && spoiled_row(row_of(b.dq, row, p.Hq, head, p.D), p.D)) row_dq(b, row, head);
    }
    for (int64_t i = warp; i < p.T * p.Hkv * p.P; i += warps) {
        const int32_t key = static_cast<int32_t>(i / p.Hkv / p.P);
        const int rank = static_cast<int>(i / p.Hkv % p.P), kvh = static_cast<int>(i % p.Hkv);
        const int32_t pos = position_of_token(b, key);
        if (pos >= 0 && (spoiled_row(row_of(b.dk[rank], pos, p.Hkv, kvh, p.D), p.D) ||
                         spoiled_row(row_of(b.dv[rank], pos, p.Hkv, kvh, p.D), p.D)))
            key_dkdv(b, key, rank, kvh);
    }
}

// ----------------------------------------------------------------- launch

// A launch whose blocks may start before the last grid has ended, once all of
// that grid's blocks have said next_grid_may_start (or ended); what needs the
// last grid's results comes behind wait_for_last_grid. So dK and dV begin on the
// SMs that dQ has left, or never took; no block waits for one that has not
// started. (8192 x 16 x 128, whole triangle: 0.695 ms with the kernels one after
// the other, 0.640 so.)
template <class... Formal, class... Actual>
cudaError_t launch_after(void (*kernel)(Formal...), int64_t blocks, int threads, size_t shared, cudaStream_t stream,
                         Actual... args)
{
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(static_cast<unsigned>(blocks));
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = shared;
    c.stream = stream;
    c.attrs = &early;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, static_cast<Formal>(args)...);
}

template <int DP, int STEPS>
cudaError_t launch_tiled(const Params &b, const Maps &maps, int tiles, cudaStream_t stream)
{
    const AttentionParams &p = b.a;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> attr_set[64];
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(dq_kernel<DP, STEPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(DqShared<DP>));
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(dkdv_kernel<DP, STEPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(DkvShared<DP>));
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t sms = sm_count(dev), row_tiles = (p.Tp + kTile - 1) / kTile, items = row_tiles * p.P * p.Hq;
    e = launch_after(dq_kernel<DP, STEPS>, items < sms ? items : sms, kThreads, sizeof(DqShared<DP>), stream, b, maps,
                     items, row_tiles, static_cast<int>(tiles * p.P));
    if (e != cudaSuccess) return e;
    const int64_t most = static_cast<int64_t>(b.unit_places) * p.Hkv;
    return launch_after(dkdv_kernel<DP, STEPS>, most < sms ? most : sms, kThreads, sizeof(DkvShared<DP>), stream, b,
                        maps);
}

int64_t align256(int64_t x) { return (x + 255) & ~static_cast<int64_t>(255); }

// The workspace: delta and lse2 of every (head, row), the spans of every row, the
// ranges and the list of every (tile, rank), the units, and the counters and
// binary32 sums of the parts.
struct Space {
    int64_t lse2, spans, ranges, list, units, counters, counter_bytes, sums, total;
    int32_t unit_places;
};

Space space_of(int64_t T, int64_t Tpad, int P, int Hq, int Hkv, int D)
{
    const int64_t slots = (T + kTile - 1) / kTile * P, Tp = Tpad / P, sms = sm_count(-1);
    // Parts of one kv head: each tile that is cut has over `most` entries, so it makes at most twice its
    // entries / most parts, and `most` is at least a half of a CTA's share and kLeastPart.
    const int64_t entries = slots * ((Tp + kTile - 1) / kTile + 1) * (Hq / Hkv);
    int64_t parts = 4 * sms / Hkv + 2;
    if (parts > 2 * entries / kLeastPart) parts = 2 * entries / kLeastPart;
    Space s;
    int64_t at = align256(4 * Tpad * Hq);
    s.lse2 = at;
    at += align256(4 * Tpad * Hq);
    s.spans = at;
    at += align256(16 * Tpad);
    s.ranges = at;
    at += align256(16 * slots);
    s.list = at;
    at += align256(4 * slots);
    s.units = at;
    s.unit_places = static_cast<int32_t>(slots + parts);
    at += align256(16 * (slots + parts));
    s.counters = at;
    s.counter_bytes = 256 + 64 * parts * Hkv;
    at += align256(s.counter_bytes);
    s.sums = at;
    at += parts * Hkv * 2 * ((D + 31) / 32 * 32) * kTile * 4;
    s.total = at;
    return s;
}

}  // namespace

int64_t attention_backward_workspace(int64_t T, int64_t Tpad, int P, int Hq, int Hkv, int D)
{
    return space_of(T, Tpad, P, Hq, Hkv, D).total;
}

cudaError_t launch_attention_backward(AttentionBackwardParams b, void *workspace, cudaStream_t stream)
{
    const AttentionParams &p = b.a;
    if (p.Tpad == 0) return cudaSuccess;
    const int tiles = static_cast<int>((p.T + kTile - 1) / kTile);
    const int64_t slots = static_cast<int64_t>(tiles) * p.P;
    const Space s = space_of(p.T, p.Tpad, p.P, p.Hq, p.Hkv, p.D);
    uint8_t *w = static_cast<uint8_t *>(workspace);
    b.delta = reinterpret_cast<float *>(w);
    b.lse2 = reinterpret_cast<float *>(w + s.lse2);
    b.spans = reinterpret_cast<int4 *>(w + s.spans);
    b.ranges = reinterpret_cast<int4 *>(w + s.ranges);
    b.list = reinterpret_cast<int32_t *>(w + s.list);
    b.units = reinterpret_cast<int4 *>(w + s.units);
    b.unit_places = s.unit_places;
    b.counters = reinterpret_cast<int32_t *>(w + s.counters);
    b.arrived = b.counters + 64;
    b.sums = reinterpret_cast<float *>(w + s.sums);
    Maps maps;
    cudaError_t e = make_slab_map(&maps.q, p.q, p.D, p.Hq, p.Tpad);
    if (e == cudaSuccess) e = make_slab_map(&maps.k, p.k, p.D, p.Hkv, p.T);
    if (e == cudaSuccess) e = make_slab_map(&maps.v, p.v, p.D, p.Hkv, p.T);
    if (e == cudaSuccess) e = make_slab_map(&maps.dout, b.dout, p.D, p.Hq, p.Tpad);
    if (e != cudaSuccess) return e;
    const int64_t row_blocks = (p.Tpad + kPrepRows - 1) / kPrepRows * ((p.Hq + kPrepHeads - 1) / kPrepHeads);
    if (row_blocks + slots > 0x7FFFFFFF) return cudaErrorInvalidValue;
    if ((e = cudaMemsetAsync(b.counters, 0, s.counter_bytes, stream)) != cudaSuccess) return e;
    prepare_kernel<<<static_cast<unsigned>(row_blocks + slots), 8 * kPrepRows, 0, stream>>>(
        b, tiles, sm_count(-1));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // the common heads have kernels of their own (see mma_scores)
    if (p.D == 64) e = launch_tiled<64, 4>(b, maps, tiles, stream);
    else if (p.D == 128) e = launch_tiled<128, 8>(b, maps, tiles, stream);
    else e = p.D < 64 ? launch_tiled<64, 0>(b, maps, tiles, stream) : launch_tiled<128, 0>(b, maps, tiles, stream);
    if (e != cudaSuccess) return e;
    return launch_after(repair_kernel, 4 * sm_count(-1), 256, 0, stream, b);
}

cudaError_t read_attention_backward_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

cudaError_t read_attention_backward_wait_timeouts(unsigned int *count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace cpt

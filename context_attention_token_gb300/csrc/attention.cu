// Causal attention over packed documents with a sliding window and sinks.
//
//   s_j = scale q . k_j over the keys the row sees, m = max s, l = sum exp(s_j - m),
//   out = sum exp(s_j - m) v_j / l, lse = m + log l.
// A row that sees nothing has out = 0 and lse = -inf.
#include "attention_common.cuh"
#include "tcgen05.cuh"

#include <atomic>
#include <cfloat>

namespace cpt {

namespace {

// Waits that ran out (see cpt_kernel_wait_timeouts).
__device__ unsigned int g_wait_timeouts;

// One warp computes one row of one head from the definition: lanes hold four
// elements each, keys come one at a time, the softmax keeps its running
// maximum and sum. The tiled kernel multiplies hidden keys by a weight of zero,
// which an infinity or NaN in their V turns into NaN: it gives such rows to
// this function, which never touches a hidden key. A NaN stays one whatever comes
// behind it, so the keys end once every element that the tiled kernel left without a
// finite value is NaN (the others are right, as lse is where it is finite).
__device__ __noinline__ void row_forward(const AttentionParams &p, int64_t row, int head)
{
    const int lane = threadIdx.x & 31, at = lane * 4, D = p.D;
    const int kvh = head / (p.Hq / p.Hkv);
    uint16_t *out = const_cast<uint16_t *>(row_of(p.out, row, p.Hq, head, D));
    float *lse = p.lse + head * p.Tpad + row;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = -INFINITY, l = 0.0f;
    const int32_t g = token_of_row(p, row);
    if (g >= 0) {
        const float4 q = load4(row_of(p.q, row, p.Hq, head, D), at, D);
        const RowKeys r = keys_of_token(p, g);
        int32_t j = r.kb;
        while (true) {
            if (j == r.kb + r.ns) j = r.lo;
            if (j > g) break;
            const float s = warp_sum(dot4(q, load4(row_of(p.k, j, p.Hkv, kvh, D), at, D))) * p.scale;
            const float4 v = load4(row_of(p.v, j, p.Hkv, kvh, D), at, D);
            const float mn = fmaxf(m, s);
            const float w = mn == -INFINITY ? (s != s ? s : 0.0f) : expf(s - mn);
            const float c = mn == -INFINITY || m == -INFINITY ? 0.0f : expf(m - mn);
            l = __fmaf_rn(l, c, w);
            o = make_float4(o.x * c, o.y * c, o.z * c, o.w * c);
            axpy4(o, w, v);
            m = mn;
            if ((j & 15) == 0) {
                if (l != l) break;
                const float4 tiled = load4(out, at, D);
                if (isfinite(*lse) && !__any_sync(0xFFFFFFFFu, any_open(tiled, o))) {
                    store4(out, at, D, finite_or_nan(tiled));
                    return;
                }
            }
            ++j;
        }
    }
    const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    store4(out, at, D, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    if (lane == 0) *lse = m + logf(l);
}

// ----------------------------------------------------------------- tiled kernel
//
// A CTA works on items of two tiles of 128 query rows against one kv head: the
// same rows of two heads that share it, or neighbouring rows of one head (of one
// tile alone where there are few). It
// is persistent (one per SM) and split into roles that hand tiles on through
// barriers, so that loads, matrix instructions and softmax of different tiles
// run at the same time, across items too:
//   rows     (1 warp)   which keys every row of the next item sees;
//   loader   (1 warp)   the item's list of key tiles, its Q, K and V by TMA;
//   issuers  (2 warps)  the matrix instructions of one query tile each: S = Q K^T
//                       into tensor memory, then O += P V with P read from there;
//   softmax  (2 x 8 warps: two warpgroups per query tile, one thread per row and
//            64 of the keys) scores to weights in place, statistics, the division.
// Tensor memory: S of both tiles (the weights of 64 keys over the first half of
// their scores), O of both tiles: 4 x 128 columns.
//
// Key tiles start anywhere: the next one starts at the first key at or behind
// the last one's end that any row of the item sees. This covers windows,
// sinks, jumps between a rank's chunks and short documents in one rule, with
// at most one partly used tile per contiguous span.
//
// Bound by the matrix unit with heads of 128: 32768 x 8 x 128, window 4096, takes 0.34 ms on a cool GPU
// (1.52 PFLOP/s, the unit busy for 75 % of it) and 0.36 ms in a loop (1.43); by the masked tiles, the softmax and
// items of uneven length with documents: 65521 x 16(4) x 80, window 1000, 0.51 ms.

constexpr int kThreads = 640;  // 4 warps that load and issue, 4 warpgroups of softmax
constexpr int kRing = 8;       // key-tile announcements in flight
constexpr int kSteps = 8;      // barriers of the steps: more than a step can be ahead of whoever waits for it
constexpr uint32_t kNeed = 1, kFull = 4, kFirst = 16, kLast = 32, kStop = 64;   // kNeed, kFull: << query tile

// The largest weight of a row's first tile is 1 but for the rounding of its reference. That is off by half a step,
// which is tens of units from scores of 2^30 on: the weights may then all be infinite or all vanish, and
// past binary32 (scores of 2^127) the reference is infinite. A row whose sum is below this bound is computed
// again as one with an infinity is. (A row whose scores are all -inf is too: it has out = 0 and lse = -inf.)
constexpr float kLeastSum = 5.4210108624275222e-20f;   // 2^-64

template <int DP>
struct Shape {
    static constexpr int kSlabs = DP / 64;
    static constexpr uint32_t kTileBytes = kSlabs * kSlab;
    static constexpr int kStages = DP == 128 ? 4 : 8;      // K and V tiles
    static constexpr uint32_t kSmem = 1024 + (2 + kStages) * kTileBytes;
};

struct Shared {
    uint64_t q_full, q_empty;
    uint64_t kv_full[8];
    uint64_t info_full[kRing], info_empty[kRing];
    uint64_t rows_full[2], rows_empty[2];
    uint64_t step[2][kSteps];          // S of a tile is there and PV of the one before is done, tiles in turn
    uint64_t p_ready[2][2];            // the weights of the first 32 keys of both halves, of all
    uint64_t out_done[2][4];           // by item: while its rows are not taken, no third one after it is done
    uint64_t turn[2], drained[2];
    uint64_t join_full, join_empty;
    float join_ref[kTile], join_l[kTile];   // of the second tile's roles, by row
    uint64_t pair[2][4];               // two warps with the same rows meet, to exchange a number per row
    float given[2][2][2][kTile];       // ... by turns in two places

    int2 info[kRing];                  // first key, flags
    int4 rows[2][2][kTile];            // two visible spans of every row of an item
    uint32_t tmem;
    uint32_t stop, spoiled;
};

struct Maps {
    CUtensorMap q, k, v;
};

// Where an item lies.
struct Item {
    int rank, head;
    int64_t row0;        // first row, of the rank's
    bool pair;           // two heads, not two row tiles
};

__device__ __forceinline__ Item item_at(const AttentionParams &p, int64_t i, int64_t row_tiles, bool pair,
                                        int item_rows)
{
    // heads slowest, so that neighbouring CTAs share keys in L2; within a head the
    // later rows first, which see the most keys when the window is long
    Item t;
    t.pair = pair;
    const int64_t per_head = row_tiles * p.P;
    const int64_t h = i / per_head, j = i - h * per_head;
    t.head = static_cast<int>(pair ? 2 * h : h);
    t.rank = static_cast<int>(j % p.P);
    t.row0 = (row_tiles - 1 - j / p.P) * item_rows;
    return t;
}

// KEYS: an item is one tile of rows of one head, and the two tiles' roles take its
// key tiles in turn, without turns of their issuers; their sums are joined at its end.
template <int DP, int STEPS, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ AttentionParams p, const __grid_constant__ Maps maps, int64_t items,
                     int64_t row_tiles, bool pair)
{
    const bool same_rows = KEYS || pair;
    const int item_rows = same_rows ? kTile : 2 * kTile;
    typedef Shape<DP> Sh;
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    const uint32_t q_at = base, kv_at = base + 2 * Sh::kTileBytes;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0), lane = threadIdx.x & 31;

    if (warp == 3) tmem_alloc(&sh.tmem);
    if (threadIdx.x == 0) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 2);
        for (int i = 0; i < Sh::kStages; ++i) mbar_init(&sh.kv_full[i], 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sh.info_full[i], 1);
            mbar_init(&sh.info_empty[i], 18);    // issuers, 16 softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.rows_full[i], 32);
            mbar_init(&sh.rows_empty[i], 17);    // loader, 16 softmax warps
            for (int j = 0; j < kSteps; ++j) mbar_init(&sh.step[i][j], 1);
            mbar_init(&sh.p_ready[i][0], 8);
            mbar_init(&sh.p_ready[i][1], 8);
            for (int j = 0; j < 4; ++j) mbar_init(&sh.pair[i][j], 2);
            for (int j = 0; j < 4; ++j) mbar_init(&sh.out_done[i][j], 1);
            mbar_init(&sh.turn[i], 1);
            mbar_init(&sh.drained[i], 1);
        }
        mbar_init(&sh.join_full, 4);
        mbar_init(&sh.join_empty, 8);
        sh.stop = sh.spoiled = 0;
        mbar_init_fence();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile uint32_t *stop = &sh.stop;
    const int group = p.Hq / p.Hkv;
    const int steps = STEPS ? STEPS : (p.D + 15) / 16;

    // 128 x 64 + 512 x 104 of the 640 x 96 registers of the launch
    if (warp < 4) {
    fewer_registers<64>();
    if (warp == 0) {
        // ------------------------------------------------------------- loader
        uint32_t n = 0, c = 0, k = 0;   // announcements, ring loads, items
        bool ok = true;
        auto announce = [&](int key, uint32_t flags) {
            const uint32_t s = n % kRing;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(&sh.info_empty[s], (n / kRing & 1) ^ 1, stop));
            if (ok && lane == 0) {
                sh.info[s] = make_int2(key, static_cast<int>(flags));
                mbar_arrive(&sh.info_full[s]);
            }
            ++n;
            return ok;
        };
        // Ring places are K, V, K, V ...: tile j's K is free with step j, its V with step j + 1. The place
        // of load c was that of load c - kStages.
        auto load = [&](const CUtensorMap *map, int head, int key) {
            const uint32_t s = c % Sh::kStages;
            if (c >= Sh::kStages) {
                const uint32_t was = c - Sh::kStages, j = was / 2 + (was & 1);
                for (int x = 0; ok && x < 2; ++x)
                    ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(&sh.step[x][j % kSteps], j / kSteps & 1, stop));
            }
            if (!ok) return false;
            if (lane == 0) {
                mbar_expect_tx(&sh.kv_full[s], Sh::kTileBytes);
                for (int i = 0; i < Sh::kSlabs; ++i)
                    tma_slab(kv_at + s * Sh::kTileBytes + i * kSlab, map, 64 * i, head, key, &sh.kv_full[s]);
            }
            ++c;
            return true;
        };
        for (int64_t it = blockIdx.x; ok && it < items; it += gridDim.x, ++k) {
            const Item t = item_at(p, it, row_tiles, pair, item_rows);
            const int b = k & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(&sh.rows_full[b], k / 2 & 1, stop));
            if (!ok) break;
            int4 r[2][4];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) r[x][i] = sh.rows[b][same_rows ? 0 : x][lane + 32 * i];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.rows_empty[b]);
            ok = __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(&sh.q_empty, (k & 1) ^ 1, stop));
            if (!ok) break;
            if (lane == 0) {
                mbar_expect_tx(&sh.q_full, 2 * Sh::kTileBytes);
                for (int x = 0; x < 2; ++x)
                    for (int i = 0; i < Sh::kSlabs; ++i)
                        tma_slab(q_at + x * Sh::kTileBytes + i * kSlab, &maps.q, 64 * i, t.head + (pair ? x : 0),
                                 static_cast<int>(t.rank * p.Tp + t.row0 + (same_rows ? 0 : x * kTile)), &sh.q_full);
            }
            auto next = [&](int x) {
                int m = 0x7FFFFFFF;
#pragma unroll
                for (int i = 0; i < 4; ++i) m = min(m, min(next_key(r[0][i], x), next_key(r[1][i], x)));
                return __reduce_min_sync(0xFFFFFFFFu, m);
            };
            const int kvh = t.head / group;
            int key = next(0);
            uint32_t first = kFirst, whose = 0;
            if (key == 0x7FFFFFFF) announce(0, kFirst | kLast);
            while (ok && key != 0x7FFFFFFF) {
                const int end = key + kTile;   // below 2^31: a tile starts at a token
                bool need[2] = {false, false}, full[2] = {true, true};
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int4 v = r[x][i];
                        const bool any = (v.x < end && v.y > key) || (v.z < end && v.w > key);
                        const bool all = (v.x <= key && v.y >= end) || (v.z <= key && v.w >= end);
                        need[x] |= any;
                        full[x] &= all || (v.y == 0 && v.w == 0);
                    }
                uint32_t flags = first;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (__any_sync(0xFFFFFFFFu, need[x]) && (!KEYS || whose == x)) flags |= kNeed << x;
                    if (__all_sync(0xFFFFFFFFu, full[x])) flags |= kFull << x;
                }
                const int nk = next(end);
                if (nk == 0x7FFFFFFF) flags |= kLast;
                if (!announce(key, flags) || !load(&maps.k, kvh, key) || !load(&maps.v, kvh, key)) break;
                key = nk;
                first = 0;
                whose ^= 1;
            }
        }
        if (ok) announce(0, kStop);
        if (*stop != 0 && lane == 0) {   // copies in flight end before the CTA does
            for (uint32_t i = c > Sh::kStages ? c - Sh::kStages : 0; i < c; ++i)
                mbar_wait_bounded(&sh.kv_full[i % Sh::kStages], i / Sh::kStages & 1);
            if (k > 0) mbar_wait_bounded(&sh.q_full, (k - 1) & 1);
            mbar_wait_bounded(&sh.q_full, k & 1);
        }
    } else if (warp < 3) {
        // ------------------------------------------------------------- issuers
        // One warp for each query tile: what one spends on barriers passes while the matrix unit works
        // for the other (one warp for both left it idle for a quarter of the time). They take turns,
        // one tile's two products at a time: left to themselves they fall into step, and the
        // matrix unit then waits for both softmaxes.
        const int x = warp - 1;
        const bool leader = lane == 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        const uint32_t s_shape = mma_shape(kTile, false), o_shape = mma_shape(16 * steps, true);
        const uint32_t s_at = tmem + 128 * x, o_at = tmem + 256 + 128 * x, q = q_at + x * Sh::kTileBytes;
        uint32_t c = 0, items_seen = 0, ps = 0;
        uint32_t prev = 0, v = 0;   // flags of the last announcement, the ring place of its V
        bool started = false;
        for (uint32_t n = 0;; ++n) {
            const uint32_t slot = n % kRing;
            if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
            const uint32_t e = static_cast<uint32_t>(sh.info[slot].y);
            __syncwarp();
            if (leader) mbar_arrive(&sh.info_empty[slot]);
            const bool of_prev = (prev & (kNeed << x)) != 0, of_this = (e & (kNeed << x)) != 0;
            const uint32_t vs = v % Sh::kStages, ks = c % Sh::kStages;
            // what is waited for outside the turn; a new item's Q and K only after the last one's product
            auto operands = [&]() {
                return (!(e & kFirst) || wait(&sh.q_full, items_seen & 1)) &&
                       (!of_this || wait(&sh.kv_full[ks], c / Sh::kStages & 1));
            };
            if (of_prev && !(wait(&sh.kv_full[vs], v / Sh::kStages & 1) && wait(&sh.p_ready[x][0], ps & 1))) break;
            if (!(e & kFirst) && !operands()) break;
            if (!KEYS && !wait(&sh.turn[x], x == 0 ? (n & 1) ^ 1 : n & 1)) break;
            if (of_prev) {
                tmem_fence_after();
                mma_weights<2, 2>(o_at, s_at, 64, kv_at + vs * Sh::kTileBytes, 8192, o_shape, started);
                if (!wait(&sh.p_ready[x][1], ps & 1)) break;
                ++ps;
                tmem_fence_after();
                mma_weights<2, 2>(o_at, s_at + 16, 64, kv_at + vs * Sh::kTileBytes + 4096, 8192, o_shape, true);
                started = true;
            }
            if (prev & kLast) mma_commit(&sh.out_done[x][(items_seen - 1) & 3]);
            if ((e & kFirst) && !operands()) break;
            if (of_this)
                mma_scores<STEPS>(s_at, q, kv_at + ks * Sh::kTileBytes, s_shape, steps);
            if (!KEYS && leader) mbar_arrive(&sh.turn[1 - x]);
            if (e & kStop) break;
            if (e & kFirst) started = false;
            if (e & (3 * kNeed)) {
                mma_commit(&sh.step[x][c / 2 % kSteps]);
                v = c + 1;
                c += 2;
            }
            if (e & kLast) {
                mma_commit(&sh.q_empty);
                ++items_seen;
            }
            prev = e;
        }
        mma_commit(&sh.drained[x]);
        mbar_wait_bounded(&sh.drained[x], 0);
    } else {
        // ------------------------------------------------------------- rows
        // This warp alone waits for a whole item, which takes some 1.6 us for each key tile that its rows see, 0.8 s
        // for 2^26 tokens. (All others wait for a few tiles.)
        const uint32_t limit = 1 + static_cast<uint32_t>(p.T >> 25);
        uint32_t k = 0;
        for (int64_t it = blockIdx.x; it < items; it += gridDim.x, ++k) {
            const Item t = item_at(p, it, row_tiles, pair, item_rows);
            const int b = k & 1;
            if (!mbar_wait_or_stop(&sh.rows_empty[b], (k / 2 & 1) ^ 1, stop, limit)) break;
            for (int i = lane; i < item_rows; i += 32) {
                const int64_t row = t.row0 + i;
                const int32_t g = row < p.Tp ? token_of_row(p, t.rank * p.Tp + row) : -1;
                const int4 r = g >= 0 ? spans_of(p, g) : make_int4(0, 0, 0, 0);
                sh.rows[b][i / kTile][i % kTile] = r;
            }
            mbar_arrive(&sh.rows_full[b]);
        }
    }
    } else {
        more_registers<104>();
        // ------------------------------------------------------------- softmax
        const int x = (warp - 4) / 8, half = (warp / 4 - 1) & 1, t = threadIdx.x & (kTile - 1);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
        const uint32_t s_at = tmem + lanes + 128 * x + 64 * half, o_at = tmem + lanes + 256 + 128 * x;
        const float c = p.scale * 1.4426950408889634f;
        uint32_t k = 0, j_tile = 0, met = 0;   // items, tiles, exchanges
        int4 r = make_int4(0, 0, 0, 0);
        float ref = -INFINITY, l = 0.0f;       // the weights are 2^(score c - ref)
        bool spoiled = false, joined = false;  // joined: the second tile's roles have a part of this item
        int64_t it = blockIdx.x;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xFFFFFFFFu, mbar_wait_or_stop(bar, parity, stop));
        };
        // The number of the other warpgroup's thread for this row; false when the kernel stops.
        auto exchange = [&](float mine, float &other) {
            sh.given[met & 1][x][half][t] = mine;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pair[x][warp & 3]);
            if (!wait(&sh.pair[x][warp & 3], met & 1)) return false;
            other = sh.given[met & 1][x][half ^ 1][t];
            ++met;
            return true;
        };
        for (uint32_t n = 0;; ++n) {
            const uint32_t slot = n % kRing;
            if (!wait(&sh.info_full[slot], n / kRing & 1)) break;
            const int2 e = sh.info[slot];
            const uint32_t flags = static_cast<uint32_t>(e.y);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.info_empty[slot]);
            if (flags & kStop) break;
            if (flags & kFirst) {
                const int b = k & 1;
                if (!wait(&sh.rows_full[b], k / 2 & 1)) break;
                r = sh.rows[b][same_rows ? 0 : x][t];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.rows_empty[b]);
                ++k;
                ref = r.y != 0 || r.w != 0 ? -INFINITY : 0.0f;   // a row that sees nothing needs none
                l = 0.0f;
                joined = false;
            }
            if (KEYS) joined |= (flags & (kNeed << 1)) != 0;
            if (flags & (kNeed << x)) {
                // Which of 32 rows see which of 32 keys. Three of four such blocks of a masked tile are seen or
                // hidden as a whole; the warp finds that out before the scores are there, and masks no element
                // of the former and computes none of the latter (65521 packed tokens of 16(4) heads of 80:
                // 0.551 -> 0.517 ms).
                uint32_t bits[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                bool mixed[2] = {false, false}, none[2] = {false, false};
                if (!(flags & (kFull << x))) {
                    const int first = e.x + 64 * half;
                    const int a0 = r.x - first, a1 = r.y - first, b0 = r.z - first, b1 = r.w - first;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        bits[i] = span_bits(a0, a1, i) | span_bits(b0, b1, i);
                        mixed[i] = !__all_sync(0xFFFFFFFFu, bits[i] == 0xFFFFFFFFu);
                        none[i] = !__any_sync(0xFFFFFFFFu, bits[i] != 0);
                    }
                }
                // the last tile's PV is done too
                if (!wait(&sh.step[x][j_tile % kSteps], j_tile / kSteps & 1)) break;
                tmem_fence_after();
                auto hide = [&](int i, uint32_t (&s)[32]) {
                    if (!mixed[i]) return;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!(bits[i] >> j & 1)) s[j] = 0xFF800000u;
                };
                uint32_t s0[32], s1[32];
                tmem_load32(s_at, s0);
                tmem_load32(s_at + 32, s1);
                tmem_wait_loads(s0);
                tmem_wait_loads(s1);
                hide(0, s0);
                hide(1, s1);
                // A row's reference is the largest score of the first tile that it sees (times c); the
                // weights of later tiles may pass 1. So no tile but the first waits for a maximum. Weights
                // or sums that leave binary32 (scores 88 above the reference, in natural units; see also
                // kLeastSum) end as an infinity or NaN in the output, and the row is computed again below.
                if (__any_sync(0xFFFFFFFFu, ref == -INFINITY)) {
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        mx[j & 3] = fmaxf(mx[j & 3], fmaxf(__uint_as_float(s0[j]), __uint_as_float(s1[j])));
                    float other;
                    const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (!exchange(mine, other)) break;
                    if (ref == -INFINITY) ref = fmaxf(mine, other) * c;
                }
                const float mc = ref == -INFINITY ? 0.0f : ref;
                const F2 c2 = pair_of(c, c), mc2 = pair_of(-mc, -mc);
                F2 sum[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
                auto weigh = [&](int i, uint32_t (&s)[32]) {
                    uint32_t w[16];
                    if (none[i]) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = 0;
                        tmem_store16(s_at + 16 * i, w);
                        tmem_wait_stores();
                        tmem_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.p_ready[x][i]);
                        return;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 a = both(fma2(pair_of(s[2 * j], s[2 * j + 1]), c2, mc2));
                        const float x0 = exp2_fast(a.x), x1 = exp2_fast(a.y);
                        sum[j & 1] = add2(sum[j & 1], pair_of(x0, x1));
                        // weights are rounded to bf16 for the matrix instruction; their sum is not
                        w[j] = pack_bf16x2(x0, x1);
                    }
                    tmem_store16(s_at + 16 * i, w);
                    tmem_wait_stores();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_ready[x][i]);   // the product can begin with half
                };
                weigh(0, s0);
                weigh(1, s1);
                const float2 total = both(add2(sum[0], sum[1]));
                l += total.x + total.y;
            }
            if (flags & (3 * kNeed)) ++j_tile;
            if (flags & kLast) {
                const Item d = item_at(p, it, row_tiles, pair, item_rows);
                const int head = d.head + (pair ? x : 0);
                const int64_t in_rank = d.row0 + (same_rows ? 0 : x * kTile) + t;
                const int64_t row = d.rank * p.Tp + in_rank;
                const bool valid = in_rank < p.Tp, sees_any = r.y != 0 || r.w != 0;
                float other;
                if (!exchange(l, other)) break;
                l = half == 0 ? l + other : other + l;
                if (ref != -INFINITY && l < kLeastSum) l = INFINITY;   // not to be lost in the join
                if (KEYS && x == 1) {   // the first tile's roles write the row
                    if (half == 0) {
                        sh.join_ref[t] = ref;
                        sh.join_l[t] = l;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.join_full);
                    }
                    if (!wait(&sh.join_empty, (k - 1) & 1)) break;
                    it += gridDim.x;
                    continue;
                }
                if (KEYS) {
                    if (!wait(&sh.join_full, (k - 1) & 1)) break;
                    if (joined) {
                        // Each side's sums are relative to the first tile that it saw, and may be as large as
                        // binary32 goes: the factor of the lower reference comes in two parts, so that it does
                        // not vanish while its product with them still counts (below 2^-222 that is under
                        // 2^-95, of a sum of at least 1).
                        const float ref1 = sh.join_ref[t], l1 = sh.join_l[t], m = fmaxf(ref, ref1);
                        const float a = ref == -INFINITY ? 0.0f : exp2_fast(fmaxf(ref - m, -96.0f));
                        const float b = ref1 == -INFINITY ? 0.0f : exp2_fast(fmaxf(ref1 - m, -96.0f));
                        const float a2 = exp2_fast(fminf(ref - m + 96.0f, 0.0f));
                        const float b2 = exp2_fast(fminf(ref1 - m + 96.0f, 0.0f));
                        const bool again = l == INFINITY || l1 == INFINITY;   // and no NaN of a score
                        l = again ? INFINITY : l * a2 * a + l1 * b2 * b;
                        ref = m;
                        if (!wait(&sh.out_done[0][(k - 1) & 3], (k - 1) / 4 & 1) ||
                            !wait(&sh.out_done[1][(k - 1) & 3], (k - 1) / 4 & 1))
                            break;
                        tmem_fence_after();
                        for (int i = half; 32 * i < p.D; i += 2) {
                            uint32_t o0[32], o1[32], w[16];
                            tmem_load32(o_at + 32 * i, o0);
                            tmem_load32(o_at + 128 + 32 * i, o1);
                            tmem_wait_loads(o0);
                            tmem_wait_loads(o1);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
#pragma unroll
                                for (int j = 16 * h; j < 16 * h + 16; ++j)
                                    w[j - 16 * h] = __float_as_uint(__fmaf_rn(
                                        __uint_as_float(o0[j]) * a2, a, __uint_as_float(o1[j]) * b2 * b));
                                tmem_store16(o_at + 32 * i + 16 * h, w);
                            }
                            tmem_wait_stores();
                        }
                        tmem_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.join_empty);
                }
                // a sum past binary32 may go with a finite product, and one too small (see kLeastSum) with a
                // product of zero: both have to be seen in the output, and lse tells them from a NaN
                if (l < kLeastSum) l = INFINITY;
                const float inv = !sees_any ? 0.0f : l == INFINITY ? NAN : 1.0f / l;
                float bad = 0.0f;
                if (!wait(&sh.out_done[x][(k - 1) & 3], (k - 1) / 4 & 1)) break;
                tmem_fence_after();
                uint16_t *out = const_cast<uint16_t *>(row_of(p.out, row, p.Hq, head, p.D));
                for (int i = half; 32 * i < p.D; i += 2) store_block(o_at, i, p.D, inv, sees_any, out, valid, bad);
                if (valid && half == 0)
                    p.lse[head * p.Tpad + row] =
                        sees_any ? (fmaxf(ref, -FLT_MAX) + log2f(l)) * 0.69314718055994531f : -INFINITY;
                spoiled |= valid && bad != 0.0f;   // NaN
                it += gridDim.x;
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
    if (sh.spoiled == 0 || warp < 4) return;
    // Rows with an infinity or NaN once more, one warp to a row, when no role waits for another (by the
    // warps that kept their registers). A NaN in lse is that of a score that the row sees (as long as the
    // scale in base 2 is finite): such a row is NaN throughout, and stays as it is.
    const bool nan_is_final = p.scale * 1.4426950408889634f < INFINITY;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const Item d = item_at(p, it, row_tiles, pair, item_rows);
        for (int i = warp - 4; i < (KEYS ? kTile : 2 * kTile); i += kThreads / 32 - 4) {
            const int head = d.head + (pair ? i / kTile : 0);
            const int64_t in_rank = d.row0 + (pair ? i % kTile : i), row = d.rank * p.Tp + in_rank;
            if (in_rank >= p.Tp) continue;
            const float lse = p.lse[head * p.Tpad + row];
            if (nan_is_final && lse != lse) continue;
            const uint16_t *out = row_of(p.out, row, p.Hq, head, p.D);
            bool bad = false;
            if (4 * lane < p.D)
                for (int j = 0; j < 4; ++j) bad |= (out[4 * lane + j] & 0x7F80) == 0x7F80;
            if (__any_sync(0xFFFFFFFFu, bad)) row_forward(p, row, head);
        }
    }
}

// ----------------------------------------------------------------- launch

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeFn>(f);
}

}  // namespace

cudaError_t make_slab_map(CUtensorMap *map, const void *base, int D, int heads, int64_t rows)
{
    const EncodeFn encode = encode_fn();
    if (encode == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * (cuuint64_t)heads};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kTile}, ones[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
                              ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

namespace {

template <int DP, int STEPS>
cudaError_t launch_tiled(const AttentionParams &p, const Maps &maps, cudaStream_t stream)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> attr_set[64];
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(attention_kernel<DP, STEPS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<DP>::kSmem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(attention_kernel<DP, STEPS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<DP>::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
    }
    // Two heads of one kv head see the same keys and share every K and V tile. Where the items of two tiles
    // would be for half of the SMs at most, an item is one tile and its keys are shared out:
    // 8192 x 2 x 128, whole triangle, 90 -> 68 us, 9728 x 2 x 128, window 2048, 59 -> 45 us,
    // 4096 x 4(2) x 64, window 1000, 26 -> 23 us.
    const int64_t sms = sm_count(dev), one = (p.Tp + kTile - 1) / kTile * p.P * p.Hq;   // tiles of all heads
    const bool single = one <= sms, pair = !single && p.Hq / p.Hkv % 2 == 0;
    const int rows = single || pair ? kTile : 2 * kTile;
    const int64_t row_tiles = (p.Tp + rows - 1) / rows;
    const int64_t items = row_tiles * p.P * (pair ? p.Hq / 2 : p.Hq);
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
    if (single)
        attention_kernel<DP, STEPS, true><<<grid, kThreads, Shape<DP>::kSmem, stream>>>(p, maps, items, row_tiles, false);
    else
        attention_kernel<DP, STEPS, false><<<grid, kThreads, Shape<DP>::kSmem, stream>>>(p, maps, items, row_tiles, pair);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const AttentionParams &p, cudaStream_t stream)
{
    if (p.Tpad == 0) return cudaSuccess;
    Maps maps;
    cudaError_t e = make_slab_map(&maps.q, p.q, p.D, p.Hq, p.Tpad);
    if (e == cudaSuccess) e = make_slab_map(&maps.k, p.k, p.D, p.Hkv, p.T);
    if (e == cudaSuccess) e = make_slab_map(&maps.v, p.v, p.D, p.Hkv, p.T);
    if (e != cudaSuccess) return e;
    // the common heads have kernels of their own (see mma_scores)
    if (p.D == 64) return launch_tiled<64, 4>(p, maps, stream);
    if (p.D == 128) return launch_tiled<128, 8>(p, maps, stream);
    return p.D < 64 ? launch_tiled<64, 0>(p, maps, stream) : launch_tiled<128, 0>(p, maps, stream);
}

cudaError_t read_attention_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

cudaError_t read_attention_wait_timeouts(unsigned int *count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace cpt

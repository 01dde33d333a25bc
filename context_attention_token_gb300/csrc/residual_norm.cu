// The residual stream between two blocks, and its gradient.
//
// Mathematics, for one row of C columns:
//   hn = h r1, r1 = 1 / sqrt(mean(h^2) + eps);  b = hn w1 gate;  y = x + scale drop(b);
//   yn = y r2, r2 = 1 / sqrt(mean(y^2) + eps);  n = yn w2.
// With e = dn w2 the gradient of y is dY = dy + r2 (e - yn mean(e yn)), and dx = dY. With
// d = scale drop(dY): dgate = d hn w1, f = d gate w1, dw1 = sum f' hn over the rows (f' = d gate),
// dh = r1 (f - hn mean(f hn)), dw2 = sum dn yn.
// The statistics are computed again in the gradient: the sums of squares ride in the
// same reduction as the products, so storing them would save nothing.
//
// HBM bounds both: every row of every tensor is read or written once. A row belongs to a group
// of threads, a unit of 16 bytes (or two) each, held in registers from the load to the last store; the next row's
// loads are issued before this row's sums. Rows of up to 32 units take a part of a warp (sums by shuffles),
// longer ones a CTA.
//
// In the gradient a group takes neighbouring tokens and keeps its columns' part of dw1, dw2 and of the current
// document's dgate in registers; parts meet in the workspace and are added in a fixed order.
#include "cpt_internal.h"
#include "token_rows.cuh"

namespace cpt {

namespace {

constexpr int kSubThreads = 128;
constexpr int kGateToken = 1, kGateDocument = 2;

// How rows of so many units are dealt to threads.
struct Shape {
    int group;        // threads of a row
    int per_thread;   // units of a thread
    int threads;      // of a CTA
    int ctas_per_sm;  // of the gradient
    bool sub;         // several rows a warp or CTA
};

Shape shape_of(int units)
{
    Shape s;
    if (units <= 64) {
        s.sub = true;
        s.per_thread = units > 32 ? 2 : 1;
        s.group = 1;
        while (s.group * s.per_thread < units) s.group *= 2;
        s.threads = kSubThreads;
        s.ctas_per_sm = 6;
        return s;
    }
    s.sub = false;
    s.per_thread = units > 1024 ? 2 : 1;
    s.group = ((units + s.per_thread - 1) / s.per_thread + 31) / 32 * 32;
    s.threads = s.group;
    s.ctas_per_sm = s.group >= 512 ? 1 : 1024 / s.group < 8 ? 1024 / s.group : 8;
    return s;
}

// The document of a raw token: the last d with cu[d] <= t.
__device__ __forceinline__ int document_of(const int32_t *cu, int n, int64_t t)
{
    int lo = 0, hi = n;   // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Sums of N values over the threads of a row.
template <bool SUB, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int group, float *room, int &turn)
{
    if constexpr (SUB) lanes_sum<N>(v, group);
    else block_sum<N>(v, room, turn);
}

__device__ __forceinline__ float rsqrt_mean(float sum, float n, float eps)
{
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, n), eps));
}

template <int E>
__device__ __forceinline__ void load_floats(const float *from, float (&x)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(from + i);
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
    }
}

template <int E>
__device__ __forceinline__ void store_floats(float *to, const float (&x)[E])
{
#pragma unroll
    for (int i = 0; i < E; i += 4) *reinterpret_cast<float4 *>(to + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}

__device__ __forceinline__ uint4 load_unit(const uint8_t *base, int64_t at)
{
    return __ldcs(reinterpret_cast<const uint4 *>(base) + at);
}

__device__ __forceinline__ void store_unit(uint8_t *base, int64_t at, uint4 v)
{
    __stcs(reinterpret_cast<uint4 *>(base) + at, v);
}

// A row's data as it was loaded.
template <int U>
struct ForwardRaw {
    uint4 x[U], h[U], gate[U];
    int32_t token;
};

template <bool BF16, int U, bool SUB, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    __shared__ float room[SUB ? 1 : 2 * kSumRoom];
    int turn = 0;
    const int lane = SUB ? threadIdx.x % p.group : threadIdx.x;
    const int64_t which = SUB ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / p.group) + threadIdx.x / p.group
                              : blockIdx.x;
    const int64_t begin = which * p.per_group;
    const bool post = p.post != nullptr, pre = p.pre != nullptr, branch = p.h != nullptr;
    const bool drop = p.rule.rng != nullptr;
    const float C = static_cast<float>(p.row_elems);
    DropKey key;
    key.load(p.rule);
    float w1[U][E], w2[U][E];
    bool has[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int u = lane + k * p.group;
        has[k] = u < p.units;
        if (post && has[k]) load_floats<E>(p.post + static_cast<int64_t>(u) * E, w1[k]);
        if (pre && has[k]) load_floats<E>(p.pre + static_cast<int64_t>(u) * E, w2[k]);
    }
    // the document of the current token: doc_lo <= token < doc_hi
    int doc = 0;
    int32_t doc_lo = 0, doc_hi = -1;

    auto load = [&](int64_t row, ForwardRaw<U> &r) {
        r.token = -1;
        if (row >= p.rows) return;
        r.token = p.token_of_row == nullptr ? static_cast<int32_t>(row) : p.token_of_row[row];
        if (r.token >= 0 && !in_bounds(r.token < p.T, lane == 0)) r.token = -1;
        if (r.token < 0) return;
        const int64_t base = row * p.units + lane;
        int64_t gate_base = base;
        if (p.gate_kind == kGateDocument) {
            if (r.token < doc_lo || r.token >= doc_hi) {
                doc = document_of(p.cu, p.n_docs, r.token);
                doc_lo = p.cu[doc];
                doc_hi = p.cu[doc + 1];
            }
            gate_base = static_cast<int64_t>(doc) * p.units + lane;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has[k]) continue;
            r.x[k] = load_unit(p.x, base + k * p.group);
            if (branch) r.h[k] = load_unit(p.h, base + k * p.group);
            if (p.gate_kind == kGateToken) r.gate[k] = load_unit(p.gate, gate_base + k * p.group);
            else if (p.gate_kind == kGateDocument) r.gate[k] = reinterpret_cast<const uint4 *>(p.gate)[gate_base + k * p.group];
        }
    };

    ForwardRaw<U> next;
    load(begin, next);
    for (int64_t i = 0; i < p.per_group; ++i) {
        const int64_t row = begin + i;
        if (!SUB && row >= p.rows) break;   // the lanes of a warp go through the same sums
        const ForwardRaw<U> r = next;
        if (i + 1 < p.per_group) load(row + 1, next);
        const bool real = r.token >= 0;
        float u[U][E], y[U][E];
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < U; ++k) {
#pragma unroll
            for (int e = 0; e < E; ++e) u[k][e] = y[k][e] = 0.0f;
            if (!has[k] || !real) continue;
            Unit<BF16>::unpack(r.x[k], y[k]);
            if (!branch) continue;
            Unit<BF16>::unpack(r.h[k], u[k]);
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] = __fmaf_rn(u[k][e], u[k][e], s[0]);
        }
        if (post) {
            row_sum<SUB, 1>(s, p.group, room, turn);
            const float r1 = rsqrt_mean(s[0], C, p.eps);
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e) u[k][e] = __fmul_rn(__fmul_rn(u[k][e], r1), w1[k][e]);
        }
        s[0] = 0.0f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has[k]) continue;
            const int64_t at = row * p.units + lane + k * p.group;
            if (branch && real) {
                if (p.gate_kind != 0) {
                    float g[E];
                    Unit<BF16>::unpack(r.gate[k], g);
#pragma unroll
                    for (int e = 0; e < E; ++e) u[k][e] = __fmul_rn(u[k][e], g[e]);
                }
                if (drop) {
                    drop_unit<BF16>(p.rule, key, r.token, lane + k * p.group, u[k]);
#pragma unroll
                    for (int e = 0; e < E; ++e) y[k][e] = __fadd_rn(y[k][e], u[k][e]);
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) y[k][e] = __fmaf_rn(u[k][e], p.scale, y[k][e]);
                }
            }
            if (p.y != nullptr && row < p.rows) store_unit(p.y, at, Unit<BF16>::pack(y[k]));
#pragma unroll
            for (int e = 0; e < E; ++e) s[0] = __fmaf_rn(y[k][e], y[k][e], s[0]);
        }
        if (pre) {
            row_sum<SUB, 1>(s, p.group, room, turn);
            const float r2 = rsqrt_mean(s[0], C, p.eps);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (!has[k] || row >= p.rows) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) y[k][e] = real ? __fmul_rn(__fmul_rn(y[k][e], r2), w2[k][e]) : 0.0f;
                store_unit(p.n, row * p.units + lane + k * p.group, Unit<BF16>::pack(y[k]));
            }
        }
    }
}

// ----------------------------------------------------------------- gradient

template <int U>
struct BackwardRaw {
    uint4 dy[U], dn[U], y[U], h[U], gate[U];
    int64_t row;
};

template <bool BF16, int U, bool SUB, int MAXT>
__global__ void __launch_bounds__(MAXT) residual_norm_backward_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    __shared__ float room[SUB ? 1 : 2 * kSumRoom];
    int turn = 0;
    const int lane = SUB ? threadIdx.x % p.group : threadIdx.x;
    const int groups = SUB ? blockDim.x / p.group : 1;
    const int64_t which = static_cast<int64_t>(blockIdx.x) * groups + (SUB ? threadIdx.x / p.group : 0);
    const int64_t begin = which * p.per_group;
    const int64_t end = min(begin + p.per_group, p.T);
    const bool post = p.post != nullptr, pre = p.pre != nullptr, branch = p.n != nullptr;   // n: dh
    const bool drop = p.rule.rng != nullptr, need_h = post || p.gate_kind != 0;
    const float C = static_cast<float>(p.row_elems);
    DropKey key;
    key.load(p.rule);
    float w1[U][E], w2[U][E], sum1[U][E], sum2[U][E], sumg[U][E];
    bool has[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int u = lane + k * p.group;
        has[k] = u < p.units;
#pragma unroll
        for (int e = 0; e < E; ++e) w1[k][e] = w2[k][e] = sum1[k][e] = sum2[k][e] = sumg[k][e] = 0.0f;
        if (post && has[k]) load_floats<E>(p.post + static_cast<int64_t>(u) * E, w1[k]);
        if (pre && has[k]) load_floats<E>(p.pre + static_cast<int64_t>(u) * E, w2[k]);
    }

    // dgate of a document's tokens so far
    const bool by_document = p.gate_kind == kGateDocument;
    int doc = 0;
    int64_t doc_lo = 0, doc_hi = 0;
    auto enter_document = [&](int64_t t) {
        doc = document_of(p.cu, p.n_docs, t);
        doc_lo = p.cu[doc];
        doc_hi = p.cu[doc + 1];
    };
    auto leave_document = [&]() {
        // whole in this group: the result; begun earlier: part 0; goes on: part 1
        float *to = reinterpret_cast<float *>(p.dgate) + static_cast<int64_t>(doc) * p.row_elems;
        if (doc_lo < begin) to = p.part_gate + (which * 2) * p.row_elems;
        else if (doc_hi > end) to = p.part_gate + (which * 2 + 1) * p.row_elems;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (has[k]) store_floats<E>(to + static_cast<int64_t>(lane + k * p.group) * E, sumg[k]);
#pragma unroll
            for (int e = 0; e < E; ++e) sumg[k][e] = 0.0f;
        }
    };
    if (by_document && begin < end) enter_document(begin);

    auto load = [&](int64_t t, BackwardRaw<U> &r) {
        r.row = -1;
        if (t >= end) return;
        const int64_t row = p.row_of_token == nullptr ? t : p.row_of_token[t];
        if (!in_bounds(row >= 0 && row < p.rows, lane == 0)) return;
        r.row = row;
        const int64_t base = row * p.units + lane;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has[k]) continue;
            r.dy[k] = p.x != nullptr ? load_unit(p.x, base + k * p.group) : make_uint4(0, 0, 0, 0);
            if (pre) {
                r.dn[k] = load_unit(p.dn, base + k * p.group);
                r.y[k] = load_unit(p.y_in, base + k * p.group);
            }
            if (need_h) r.h[k] = load_unit(p.h, base + k * p.group);
            if (p.gate_kind == kGateToken) r.gate[k] = load_unit(p.gate, base + k * p.group);
        }
    };

    BackwardRaw<U> next;
    load(begin, next);
    for (int64_t i = 0; i < p.per_group; ++i) {
        const int64_t t = begin + i;
        if (!SUB && t >= end) break;
        const BackwardRaw<U> r = next;
        if (i + 1 < p.per_group) load(t + 1, next);
        const bool real = r.row >= 0;
        if (by_document && t < end && t >= doc_hi) {
            leave_document();
            enter_document(t);
        }
        float d[U][E], e1[U][E], hn[U][E];
        float s[3] = {0.0f, 0.0f, 0.0f};   // y^2, dn w2 y, h^2
#pragma unroll
        for (int k = 0; k < U; ++k) {
#pragma unroll
            for (int e = 0; e < E; ++e) d[k][e] = hn[k][e] = 0.0f;
            if (!has[k] || !real) continue;
            Unit<BF16>::unpack(r.dy[k], d[k]);
            if (pre) {
                float y[E], dn[E];
                Unit<BF16>::unpack(r.y[k], y);
                Unit<BF16>::unpack(r.dn[k], dn);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    s[0] = __fmaf_rn(y[e], y[e], s[0]);
                    s[1] = __fmaf_rn(__fmul_rn(dn[e], w2[k][e]), y[e], s[1]);
                }
            }
            if (need_h) {
                Unit<BF16>::unpack(r.h[k], hn[k]);
#pragma unroll
                for (int e = 0; e < E; ++e) s[2] = __fmaf_rn(hn[k][e], hn[k][e], s[2]);
            }
        }
        if (pre || post) row_sum<SUB, 3>(s, p.group, room, turn);
        const float r1 = rsqrt_mean(s[2], C, p.eps);
        if (pre) {
            const float r2 = rsqrt_mean(s[0], C, p.eps);
            const float mean = __fdiv_rn(__fmul_rn(s[1], r2), C);   // of dn w2 yn
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (!has[k] || !real) continue;
                float y[E], dn[E];
                Unit<BF16>::unpack(r.y[k], y);
                Unit<BF16>::unpack(r.dn[k], dn);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float yn = __fmul_rn(y[e], r2);
                    sum2[k][e] = __fmaf_rn(dn[e], yn, sum2[k][e]);
                    const float c = __fmaf_rn(-yn, mean, __fmul_rn(dn[e], w2[k][e]));
                    d[k][e] = __fmaf_rn(r2, c, d[k][e]);
                }
            }
        }
        float q[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < U; ++k) {
#pragma unroll
            for (int e = 0; e < E; ++e) e1[k][e] = 0.0f;
            if (!has[k] || !real) continue;
            const int64_t at = r.row * p.units + lane + k * p.group;
            store_unit(p.y, at, Unit<BF16>::pack(d[k]));
            if (!branch) continue;
            if (drop) {
                drop_unit<BF16>(p.rule, key, static_cast<uint32_t>(t), lane + k * p.group, d[k]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) d[k][e] = __fmul_rn(d[k][e], p.scale);
            }
            if (post) {
#pragma unroll
                for (int e = 0; e < E; ++e) hn[k][e] = __fmul_rn(hn[k][e], r1);
            }
            if (p.gate_kind != 0) {
                float g[E], z[E];
                if (by_document) Unit<BF16>::unpack(reinterpret_cast<const uint4 *>(p.gate)[static_cast<int64_t>(doc) * p.units + lane + k * p.group], g);
                else Unit<BF16>::unpack(r.gate[k], g);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    // what was dropped has no gradient, whatever it is multiplied by
                    const bool zero = d[k][e] == 0.0f;
                    z[e] = zero ? 0.0f : __fmul_rn(d[k][e], post ? __fmul_rn(hn[k][e], w1[k][e]) : hn[k][e]);
                    d[k][e] = zero ? 0.0f : __fmul_rn(d[k][e], g[e]);
                }
                if (by_document) {
#pragma unroll
                    for (int e = 0; e < E; ++e) sumg[k][e] = __fadd_rn(sumg[k][e], z[e]);
                } else {
                    store_unit(p.dgate, at, Unit<BF16>::pack(z));
                }
            }
            if (post) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    sum1[k][e] = __fmaf_rn(d[k][e], hn[k][e], sum1[k][e]);
                    e1[k][e] = __fmul_rn(d[k][e], w1[k][e]);
                    q[0] = __fmaf_rn(e1[k][e], hn[k][e], q[0]);
                }
            } else {
                store_unit(p.n, at, Unit<BF16>::pack(d[k]));
            }
        }
        if (post) {
            row_sum<SUB, 1>(q, p.group, room, turn);
            const float mean = __fdiv_rn(q[0], C);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (!has[k] || !real) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) d[k][e] = __fmul_rn(r1, __fmaf_rn(-hn[k][e], mean, e1[k][e]));
                store_unit(p.n, r.row * p.units + lane + k * p.group, Unit<BF16>::pack(d[k]));
            }
        }
    }
    if (by_document && begin < end) leave_document();

    // the CTA's part of the weights' gradients, its groups added in order
    __shared__ float join[SUB ? kSubThreads * U * E : 1];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (w == 0 ? !post : !pre) continue;
        float *to = (w == 0 ? p.part_post : p.part_pre) + static_cast<int64_t>(blockIdx.x) * p.row_elems;
        if constexpr (SUB) {
            const int row = p.group * U * E;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    join[(threadIdx.x / p.group) * row + (lane + k * p.group) * E + e] = w == 0 ? sum1[k][e] : sum2[k][e];
            __syncthreads();
            for (int c = threadIdx.x; c < p.row_elems; c += blockDim.x) {
                float v = join[c];
                for (int g = 1; g < groups; ++g) v = __fadd_rn(v, join[g * row + c]);
                to[c] = v;
            }
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (has[k]) store_floats<E>(to + static_cast<int64_t>(lane + k * p.group) * E, w == 0 ? sum1[k] : sum2[k]);
        }
    }

    // padding rows: every CTA zeroes its share
    if (p.token_of_row == nullptr || p.rows == p.T) return;
    const int64_t share = (p.rows + gridDim.x - 1) / gridDim.x;
    const int64_t last = min(static_cast<int64_t>(blockIdx.x + 1) * share, p.rows);
    for (int64_t row = blockIdx.x * share + (SUB ? threadIdx.x / p.group : 0); row < last; row += groups) {
        if (p.token_of_row[row] >= 0) continue;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has[k]) continue;
            const int64_t at = row * p.units + lane + k * p.group;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            store_unit(p.y, at, zero);
            if (branch) store_unit(p.n, at, zero);
            if (p.gate_kind == kGateToken) store_unit(p.dgate, at, zero);
        }
    }
}

// Adds the parts: blockIdx.y 0 and 1 the weights', one warp every 32nd part; the others the documents that
// reach over several groups, a warp each. 32 columns a block.
__global__ void __launch_bounds__(1024) residual_join_kernel(const __grid_constant__ ResidualParams p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    if (blockIdx.y < 2) {
        __shared__ float room[32][33];
        const float *from = blockIdx.y == 0 ? p.part_post : p.part_pre;
        float *to = blockIdx.y == 0 ? p.dpost : p.dpre;
        if (to == nullptr) return;
        float v = 0.0f;
        if (c < p.row_elems) {
#pragma unroll 8
            for (int i = warp; i < p.parts; i += 32) v = __fadd_rn(v, from[static_cast<int64_t>(i) * p.row_elems + c]);
        }
        room[warp][lane] = v;
        __syncthreads();
        v = room[lane][warp];   // this warp's column warp, part lane
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
        if (lane == 0 && blockIdx.x * 32 + warp < p.row_elems) to[blockIdx.x * 32 + warp] = v;
        return;
    }
    if (c >= p.row_elems) return;
    float *dgate = reinterpret_cast<float *>(p.dgate);
    const int64_t step = static_cast<int64_t>(gridDim.y - 2) * 32;
    for (int64_t d = (blockIdx.y - 2) * 32 + warp; d < p.n_docs; d += step) {
        const int64_t lo = p.cu[d], hi = p.cu[d + 1];
        if (lo >= hi) {
            dgate[d * p.row_elems + c] = 0.0f;
            continue;
        }
        const int64_t first = lo / p.per_group, last = (hi - 1) / p.per_group;
        if (first == last) continue;
        float v = p.part_gate[(first * 2 + 1) * p.row_elems + c];
#pragma unroll 8
        for (int64_t g = first + 1; g <= last; ++g) v = __fadd_rn(v, p.part_gate[g * 2 * p.row_elems + c]);
        dgate[d * p.row_elems + c] = v;
    }
}

template <bool BF16>
cudaError_t launch_forward(const ResidualParams &p, const Shape &s, unsigned grid, cudaStream_t stream)
{
    if (s.sub) {
        if (s.per_thread == 1) residual_norm_kernel<BF16, 1, true, kSubThreads><<<grid, s.threads, 0, stream>>>(p);
        else residual_norm_kernel<BF16, 2, true, kSubThreads><<<grid, s.threads, 0, stream>>>(p);
    } else if (s.per_thread == 1) {
        if (s.threads <= 512) residual_norm_kernel<BF16, 1, false, 512><<<grid, s.threads, 0, stream>>>(p);
        else residual_norm_kernel<BF16, 1, false, 1024><<<grid, s.threads, 0, stream>>>(p);
    } else {
        residual_norm_kernel<BF16, 2, false, 1024><<<grid, s.threads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_backward(const ResidualParams &p, const Shape &s, unsigned grid, cudaStream_t stream)
{
    if (s.sub) {
        if (s.per_thread == 1) residual_norm_backward_kernel<BF16, 1, true, kSubThreads><<<grid, s.threads, 0, stream>>>(p);
        else residual_norm_backward_kernel<BF16, 2, true, kSubThreads><<<grid, s.threads, 0, stream>>>(p);
    } else if (s.per_thread == 1) {
        if (s.threads <= 512) residual_norm_backward_kernel<BF16, 1, false, 512><<<grid, s.threads, 0, stream>>>(p);
        else residual_norm_backward_kernel<BF16, 1, false, 1024><<<grid, s.threads, 0, stream>>>(p);
    } else {
        residual_norm_backward_kernel<BF16, 2, false, 1024><<<grid, s.threads, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

int row_units(int64_t row_elems, int dtype) { return static_cast<int>(row_elems * (dtype == kBf16 ? 2 : 4) / 16); }

// Tokens of a group of the gradient, and its CTAs.
void deal(int64_t T, const Shape &s, int device, int64_t &per_group, int64_t &ctas)
{
    const int64_t groups = s.sub ? s.threads / s.group : 1;
    const int64_t most = static_cast<int64_t>(sm_count(device)) * s.ctas_per_sm * groups;
    per_group = (T + most - 1) / most;
    if (per_group < 1) per_group = 1;
    ctas = (T + per_group * groups - 1) / (per_group * groups);
}

}  // namespace

cudaError_t launch_residual_norm(ResidualParams p, int dtype, cudaStream_t stream)
{
    if (p.rows == 0) return cudaSuccess;
    p.units = row_units(p.row_elems, dtype);
    const Shape s = shape_of(p.units);
    const int64_t groups = s.sub ? s.threads / s.group : 1;
    p.group = s.group;
    // rows of a group: enough to fetch ahead, few enough that all SMs get some
    const int64_t even = p.rows / (static_cast<int64_t>(sm_count(-1)) * 8 * groups);
    p.per_group = even < 1 ? 1 : even > 16 ? 16 : even;
    const int64_t ctas = (p.rows + p.per_group * groups - 1) / (p.per_group * groups);
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(ctas);
    return dtype == kBf16 ? launch_forward<true>(p, s, grid, stream) : launch_forward<false>(p, s, grid, stream);
}

int64_t residual_backward_workspace(int64_t T, int64_t row_elems, int dtype, int device)
{
    const Shape s = shape_of(row_units(row_elems, dtype));
    int64_t per_group, ctas;
    deal(T, s, device, per_group, ctas);
    const int64_t groups = s.sub ? s.threads / s.group : 1;
    return (2 * ctas + 2 * ctas * groups) * row_elems * 4;
}

cudaError_t launch_residual_norm_backward(ResidualParams p, int dtype, void *workspace, int device, cudaStream_t stream)
{
    p.units = row_units(p.row_elems, dtype);
    const Shape s = shape_of(p.units);
    p.group = s.group;
    int64_t ctas;
    deal(p.T, s, device, p.per_group, ctas);
    p.parts = static_cast<int32_t>(ctas);
    p.part_post = static_cast<float *>(workspace);
    p.part_pre = p.part_post + ctas * p.row_elems;
    p.part_gate = p.part_pre + ctas * p.row_elems;
    if (p.T > 0) {
        const unsigned grid = static_cast<unsigned>(ctas);
        const cudaError_t e = dtype == kBf16 ? launch_backward<true>(p, s, grid, stream)
                                             : launch_backward<false>(p, s, grid, stream);
        if (e != cudaSuccess) return e;
    }
    const bool documents = p.gate_kind == kGateDocument && p.n_docs > 0;
    if (p.dpost == nullptr && p.dpre == nullptr && !documents) return cudaSuccess;
    int docs = 0;
    if (documents) docs = p.n_docs < 32 * 64 ? (p.n_docs + 31) / 32 : 64;
    const dim3 grid(static_cast<unsigned>((p.row_elems + 31) / 32), static_cast<unsigned>(2 + docs));
    residual_join_kernel<<<grid, 1024, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t read_residual_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

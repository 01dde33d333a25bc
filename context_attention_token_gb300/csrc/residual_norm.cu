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

#include <mutex>
#include <type_traits>

namespace cpt {

namespace {

constexpr int kShortThreads = 128;
constexpr int kForwardThreads = 640;    // of an SM's long rows: 96 registers each
constexpr int kBackwardThreads = 512;   // 128 registers each
constexpr int kMaxStages = 8;
constexpr int kMaxTeams = 10;              // of a forward CTA
constexpr int kSharedBytes = 228 * 1024;   // of an SM, 1 KB of each CTA the system's
constexpr int kOwnBytes = 1024 + 128 + kMaxTeams * (512 + kMaxStages * 12);   // of a CTA, besides rings and weights
constexpr int kGateToken = 1, kGateDocument = 2;

// How rows of so many units are dealt to threads.
struct Shape {
    int group;        // threads of a row
    int per_thread;   // units of a thread
    int threads;      // of a CTA
    int ctas_per_sm;
    bool shorter;     // several rows a CTA
    bool hold;        // the weights in shared memory
};

// Weights in shared memory: two rows of them, every thread's units whole.
int64_t weight_bytes(const Shape &s, int dtype) { return !s.hold ? 0 : 2 * s.per_thread * s.group * (dtype == kBf16 ? 8 : 4) * 4; }

// tensors: those that are read.
Shape shape_of(int units, int dtype, bool gradient, int tensors, bool by_document = false)
{
    Shape s;
    s.shorter = units <= 64;
    s.hold = false;
    if (s.shorter) {
        s.per_thread = units > 32 ? 2 : 1;
        s.group = 1;
        while (s.group * s.per_thread < units) s.group *= 2;
        s.threads = kShortThreads;
        s.ctas_per_sm = s.per_thread == 1 ? 4 : 2;
        return s;
    }
    const int eights = dtype == kBf16 ? units : (units + 1) / 2;   // groups of eight columns
    const int wide = gradient || eights <= 128 ? 2 : eights <= 192 ? 3 : 5;   // of a thread
    s.per_thread = dtype == kBf16 ? wide : 2 * wide;
    s.group = ((eights + wide - 1) / wide + 31) / 32 * 32;
    // one CTA an SM, of as many teams as registers, barriers and shared memory allow (a row each at least)
    s.ctas_per_sm = 1;
    const int threads = gradient ? kBackwardThreads : kForwardThreads;
    const int64_t row = s.per_thread * s.group * 16;   // bytes
    // (the widest float32 rows of the gradient leave no room for the weights: they are read anew each time)
    s.hold = true;
    s.hold = kSharedBytes - kOwnBytes - weight_bytes(s, dtype) >= row * (tensors + by_document);
    const int64_t left = (kSharedBytes - kOwnBytes - weight_bytes(s, dtype)) / (row * (tensors + by_document));
    const int teams = threads / s.group < kMaxTeams ? threads / s.group : kMaxTeams;
    s.threads = static_cast<int>(teams < left ? teams : left) * s.group;
    return s;
}

// Rows that a team's ring holds.
int stages_of(const Shape &s, int dtype, int tensors, bool by_document)
{
    const int64_t row = static_cast<int64_t>(s.threads / s.group) * s.per_thread * s.group * 16;
    const int64_t n = (kSharedBytes - kOwnBytes - weight_bytes(s, dtype) - (by_document ? row : 0)) / (row * tensors);
    return static_cast<int>(n > kMaxStages ? kMaxStages : n);
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

// 1 / sqrt(sum / C + eps), to 2 units in the last place of the function and one rounding of 1 / C.
__device__ __forceinline__ float rsqrt_mean(const ResidualParams &p, float sum)
{
    return rsqrtf(__fmaf_rn(sum, p.per_column, p.eps));
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

// A store under a predicate, without a branch that would keep apart what is computed on either side of it.
__device__ __forceinline__ void store_unit_if(bool there, uint8_t *base, int64_t at, uint4 v)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %0, 0; @p st.global.cs.v4.u32 [%1], {%2, %3, %4, %5}; }" ::"r"(
                     static_cast<uint32_t>(there)),
                 "l"(reinterpret_cast<uint4 *>(base) + at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ F2 twice(float x) { return pair_of(x, x); }

__device__ __forceinline__ float sum_of(F2 x)
{
    const float2 f = both(x);
    return __fadd_rn(f.x, f.y);
}

// What a call asks for, known to the compiler (F >= 0: bits 0 post norm, 1 pre norm, 2 dropout, from 3 on the kind of
// gate; there is a block's output) or read from the parameters (F = -1).
template <int F>
struct Asked {
    static __device__ __forceinline__ bool post(const ResidualParams &p) { return F < 0 ? p.post != nullptr : F & 1; }
    static __device__ __forceinline__ bool pre(const ResidualParams &p) { return F < 0 ? p.pre != nullptr : F & 2; }
    static __device__ __forceinline__ bool drop(const ResidualParams &p) { return F < 0 ? p.rule.rng != nullptr : F & 4; }
    static __device__ __forceinline__ int gate(const ResidualParams &p) { return F < 0 ? p.gate_kind : F >> 3; }
    static __device__ __forceinline__ bool block(bool there) { return F < 0 ? there : true; }
};

template <int U>
struct Has {
    bool at[U];   // whether unit lane + k * group is one of the row
};

// The weights of a unit, 0 past the row's end.
template <bool BF16>
__device__ __forceinline__ void load_weight(const float *w, bool there, int unit, F2 (&out)[Unit<BF16>::E / 2])
{
    constexpr int E = Unit<BF16>::E;
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 0.0f;
    if (w != nullptr && there) load_floats<E>(w + static_cast<int64_t>(unit) * E, f);
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pair_of(f[e], f[e + 1]);
}

template <bool BF16, int U>
__device__ __forceinline__ void load_weights(const float *w, const Has<U> &has, int lane, int group,
                                             F2 (&out)[U][Unit<BF16>::E / 2])
{
#pragma unroll
    for (int k = 0; k < U; ++k) load_weight<BF16>(w, has.at[k], lane + k * group, out[k]);
}

// Weights in registers.
template <bool BF16, int U>
struct HeldWeights {
    const F2 (&w)[U][Unit<BF16>::E / 2];
    __device__ __forceinline__ void operator()(int k, F2 (&out)[Unit<BF16>::E / 2]) const
    {
#pragma unroll
        for (int i = 0; i < Unit<BF16>::E / 2; ++i) out[i] = w[k][i];
    }
};

// Weights in shared memory.
template <bool BF16>
struct SharedWeights {
    const float *row;   // of this thread's unit 0
    int step;           // floats to its next unit
    __device__ __forceinline__ void operator()(int k, F2 (&out)[Unit<BF16>::E / 2]) const
    {
#pragma unroll
        for (int i = 0; i < Unit<BF16>::E / 2; i += 2) {
            const float4 v = *reinterpret_cast<const float4 *>(row + k * step + 2 * i);
            out[i] = pair_of(v.x, v.y);
            out[i + 1] = pair_of(v.z, v.w);
        }
    }
};

// One row of the forward call. x, h and gate give the data of a unit of it (0 past the row's end), bits all random bits,
// put_y and put_n take a unit's result and whether it is one of the row, sum adds over the row's threads.
template <bool BF16, int U, int F, class W1, class W2, class X, class H, class G, class Bits, class Sum, class PutY, class PutN>
__device__ __forceinline__ void forward_row(const ResidualParams &p, const Has<U> &has, W1 w1, W2 w2, X x, H h, G gate,
                                            Bits bits, Sum sum, PutY put_y, PutN put_n)
{
    typedef UnitPairs<BF16> V;
    typedef Asked<F> A;
    constexpr int N = V::N;
    F2 y[U][N], q = twice(0.0f);
    uint32_t rnd[U][N];
    float s[1];
    F2 factor = twice(p.rule.factor);
    if (A::post(p)) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            F2 u[N];
            V::unpack(h(k), u);
#pragma unroll
            for (int i = 0; i < N; ++i) q = fma2(u[i], u[i], q);
        }
    }
    // the generator needs no data: it runs while the sum is on its way
    if (A::drop(p)) bits(rnd);
    if (A::post(p)) {
        s[0] = sum_of(q);
        sum(s);
        factor = twice(__fmul_rn(rsqrt_mean(p, s[0]), p.rule.factor));
    }
    q = twice(0.0f);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        V::unpack(x(k), y[k]);
        if (A::block(p.h != nullptr)) {
            F2 u[N];   // h once more: kept over the sum it would cost registers that more rows at a time are worth
            V::unpack(h(k), u);
            if (A::post(p)) {
                F2 w[N];
                w1(k, w);
#pragma unroll
                for (int i = 0; i < N; ++i) u[i] = mul2(u[i], w[i]);
            }
            if (A::gate(p) != 0) {
                F2 g[N];
                V::unpack(gate(k), g);
#pragma unroll
                for (int i = 0; i < N; ++i) u[i] = mul2(u[i], g[i]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = fma2(u[i], factor, y[k][i]);
            if (A::drop(p)) keep_or<N>(p.rule, rnd[k], u, y[k]);
#pragma unroll
            for (int i = 0; i < N; ++i) y[k][i] = u[i];
            put_y(k, has.at[k], V::pack(y[k]));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) q = fma2(y[k][i], y[k][i], q);
    }
    if (!A::pre(p)) return;
    s[0] = sum_of(q);
    sum(s);
    const F2 r2 = twice(rsqrt_mean(p, s[0]));
#pragma unroll
    for (int k = 0; k < U; ++k) {
        F2 w[N];
        w2(k, w);
#pragma unroll
        for (int i = 0; i < N; ++i) y[k][i] = mul2(mul2(y[k][i], r2), w[i]);
        put_n(k, has.at[k], V::pack(y[k]));
    }
}

// What a thread adds up over its tokens.
template <bool BF16, int U>
struct Sums {
    F2 post[U][Unit<BF16>::E / 2], pre[U][Unit<BF16>::E / 2], gate[U][Unit<BF16>::E / 2];
};

// One token of the gradient; dy to gate give the data of a unit of its row (0 past the row's end). `enter` is called before
// the gate is asked for.
template <bool BF16, int U, int F, class W1, class W2, class DY, class DN, class Y, class H, class Enter, class G, class Bits,
          class Sum, class PutX, class PutH, class PutG>
__device__ __forceinline__ void backward_row(const ResidualParams &p, const Has<U> &has, W1 w1, W2 w2, Sums<BF16, U> &acc,
                                             DY dy, DN dn, Y y, H h, Enter enter, G gate, Bits bits, Sum sum, PutX put_x,
                                             PutH put_h, PutG put_gate)
{
    typedef UnitPairs<BF16> V;
    typedef Asked<F> A;
    constexpr int N = V::N;
    const bool post = A::post(p), pre = A::pre(p);
    uint32_t rnd[U][N];
    F2 q[3] = {twice(0.0f), twice(0.0f), twice(0.0f)};   // y^2, dn w2 y, h^2
#pragma unroll
    for (int k = 0; k < U; ++k) {
        if (pre) {
            F2 a[N], b[N], w[N];
            V::unpack(y(k), a);
            V::unpack(dn(k), b);
            w2(k, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                q[0] = fma2(a[i], a[i], q[0]);
                q[1] = fma2(mul2(b[i], w[i]), a[i], q[1]);
            }
        }
        if (post) {
            F2 a[N];
            V::unpack(h(k), a);
#pragma unroll
            for (int i = 0; i < N; ++i) q[2] = fma2(a[i], a[i], q[2]);
        }
    }
    // the generator needs no data: it runs while the sums are on their way
    if (A::drop(p)) bits(rnd);
    float s[3] = {sum_of(q[0]), sum_of(q[1]), sum_of(q[2])};
    if (pre || post) sum(s);
    if (A::gate(p) == kGateDocument) enter();
    const float r2 = pre ? rsqrt_mean(p, s[0]) : 0.0f, r1 = post ? rsqrt_mean(p, s[2]) : 1.0f;
    // dY = dy + r2 dn w2 - y r2^2 mean(dn w2 yn), yn = y r2
    const F2 back2 = twice(pre ? -__fmul_rn(__fmul_rn(r2, r2), __fmul_rn(__fmul_rn(s[1], r2), p.per_column)) : 0.0f);
    F2 e[U][N], t = twice(0.0f);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        F2 d[N];
        V::unpack(dy(k), d);
        if (pre) {
            F2 a[N], b[N], w[N];
            V::unpack(y(k), a);
            V::unpack(dn(k), b);
            w2(k, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                acc.pre[k][i] = fma2(mul2(a[i], b[i]), twice(r2), acc.pre[k][i]);
                d[i] = fma2(a[i], back2, fma2(mul2(b[i], w[i]), twice(r2), d[i]));
            }
        }
        put_x(k, has.at[k], V::pack(d));
        if (!A::block(p.n != nullptr)) continue;
        if (A::drop(p)) keep_or_zero<N>(p.rule, rnd[k], d);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = mul2(d[i], twice(p.rule.factor));
        F2 hn[N], w[N];
        if (post) w1(k, w);
        if (post || A::gate(p) != 0) {
            V::unpack(h(k), hn);
            if (post) {
#pragma unroll
                for (int i = 0; i < N; ++i) hn[i] = mul2(hn[i], twice(r1));
            }
        }
        if (A::gate(p) != 0) {
            F2 g[N], z[N];
            V::unpack(gate(k), g);
            // what was dropped has no gradient, whatever it is multiplied by (behind a norm, and with a gate that a whole
            // document shares, a row with an infinity is NaN throughout)
            const bool guard = A::drop(p) && !(post && A::gate(p) == kGateDocument);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                z[i] = mul2(d[i], post ? mul2(hn[i], w[i]) : hn[i]);
                d[i] = mul2(d[i], g[i]);
            }
            if (guard) {
                keep_or_zero<N>(p.rule, rnd[k], z);
                keep_or_zero<N>(p.rule, rnd[k], d);
            }
            if (A::gate(p) == kGateDocument) {
#pragma unroll
                for (int i = 0; i < N; ++i) acc.gate[k][i] = add2(acc.gate[k][i], z[i]);
            } else {
                put_gate(k, has.at[k], V::pack(z));
            }
        }
        if (post) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                acc.post[k][i] = fma2(d[i], hn[i], acc.post[k][i]);
                e[k][i] = mul2(d[i], w[i]);
                t = fma2(e[k][i], hn[i], t);
            }
        } else {
            put_h(k, has.at[k], V::pack(d));
        }
    }
    if (!post) return;
    float m[1] = {sum_of(t)};
    sum(m);
    // dh = r1 e - h r1^2 mean(e hn)
    const F2 back1 = twice(-__fmul_rn(__fmul_rn(r1, r1), __fmul_rn(m[0], p.per_column)));
#pragma unroll
    for (int k = 0; k < U; ++k) {
        F2 hn[N];
        V::unpack(h(k), hn);
#pragma unroll
        for (int i = 0; i < N; ++i) hn[i] = fma2(hn[i], back1, mul2(e[k][i], twice(r1)));
        put_h(k, has.at[k], V::pack(hn));
    }
}

// The document that tokens are in, looked for when it changes.
struct Document {
    int at = 0;
    int64_t lo = 0, hi = -1;   // its tokens
    __device__ __forceinline__ bool enter(const ResidualParams &p, int64_t token)
    {
        if (token >= lo && token < hi) return false;
        if (token == hi && at + 1 < p.n_docs && p.cu[at + 2] > token) ++at;   // the next one, mostly
        else at = document_of(p.cu, p.n_docs, token);
        lo = p.cu[at];
        hi = p.cu[at + 1];
        return true;
    }
};

// The sum over a token's gate gradients leaves for where it belongs: the result when the document lies in this
// group's tokens, part 0 when it began earlier, part 1 when it goes on.
template <bool BF16, int U>
__device__ __forceinline__ void leave_document(const ResidualParams &p, const Document &doc, int64_t which, int64_t begin,
                                               int64_t end, const Has<U> &has, int lane, Sums<BF16, U> &acc)
{
    constexpr int E = Unit<BF16>::E;
    float *to = reinterpret_cast<float *>(p.dgate) + static_cast<int64_t>(doc.at) * p.row_elems;
    if (doc.lo < begin) to = p.part_gate + which * 2 * p.row_elems;
    else if (doc.hi > end) to = p.part_gate + (which * 2 + 1) * p.row_elems;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        float f[E];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float2 v = both(acc.gate[k][i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
            acc.gate[k][i] = twice(0.0f);
        }
        if (has.at[k]) store_floats<E>(to + static_cast<int64_t>(lane + k * p.group) * E, f);
    }
}

template <int E>
__device__ __forceinline__ void spread(const F2 (&x)[E / 2], float (&f)[E])
{
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        const float2 v = both(x[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

// Padding rows of the outputs, this CTA's share of all rows.
template <int U>
__device__ __forceinline__ void zero_padding(const ResidualParams &p, const Has<U> &has, int lane, int first, int step)
{
    if (p.token_of_row == nullptr || p.rows == p.T) return;
    const int64_t share = (p.rows + gridDim.x - 1) / gridDim.x;
    const int64_t last = min(static_cast<int64_t>(blockIdx.x + 1) * share, p.rows);
    for (int64_t row = blockIdx.x * share + first; row < last; row += step) {
        if (p.token_of_row[row] >= 0) continue;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has.at[k]) continue;
            const int64_t at = row * p.units + lane + k * p.group;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            store_unit(p.y, at, zero);
            if (p.n != nullptr) store_unit(p.n, at, zero);
            if (p.gate_kind == kGateToken) store_unit(p.dgate, at, zero);
        }
    }
}

// ----------------------------------------------------------------- short rows: a part of a warp each

// A row's data as it was loaded.
template <int U>
struct ShortRaw {
    uint4 t[5][U];   // forward: x, h, gate; gradient: dy, dn, y, h, gate
    int64_t row;
    int32_t token;
};

template <bool BF16, int U>
__device__ __forceinline__ void short_bits(const ResidualParams &p, const DropKey &key, uint32_t token, int lane,
                                           uint32_t (&bits)[U][Unit<BF16>::E / 2])
{
    uint32_t tokens[U], units[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        tokens[k] = token;
        units[k] = lane + k * p.group;
    }
    unit_bits<BF16, U>(p.rule, key, tokens, units, bits);
}

template <bool BF16, int U>
__global__ void __launch_bounds__(kShortThreads) residual_norm_short_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    const int lane = threadIdx.x % p.group;
    const int64_t which = static_cast<int64_t>(blockIdx.x) * (kShortThreads / p.group) + threadIdx.x / p.group;
    const int64_t begin = which * p.per_group;
    DropKey key;
    key.load(p.rule);
    Has<U> has;
#pragma unroll
    for (int k = 0; k < U; ++k) has.at[k] = lane + k * p.group < p.units;
    F2 w1[U][E / 2], w2[U][E / 2];
    load_weights<BF16, U>(p.post, has, lane, p.group, w1);
    load_weights<BF16, U>(p.pre, has, lane, p.group, w2);
    Document doc;

    auto load = [&](int64_t row, ShortRaw<U> &r) {
        r.token = -1;
#pragma unroll
        for (int k = 0; k < U; ++k) r.t[0][k] = r.t[1][k] = r.t[2][k] = make_uint4(0, 0, 0, 0);
        if (row >= p.rows) return;
        r.token = p.token_of_row == nullptr ? static_cast<int32_t>(row) : p.token_of_row[row];
        if (r.token >= 0 && !in_bounds(r.token < p.T, lane == 0)) r.token = -1;
        if (r.token < 0) return;
        const int64_t base = row * p.units + lane;
        int64_t gate_base = base;
        if (p.gate_kind == kGateDocument) {
            doc.enter(p, r.token);
            gate_base = static_cast<int64_t>(doc.at) * p.units + lane;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has.at[k]) continue;
            r.t[0][k] = load_unit(p.x, base + k * p.group);
            if (p.h != nullptr) r.t[1][k] = load_unit(p.h, base + k * p.group);
            if (p.gate_kind == kGateToken) r.t[2][k] = load_unit(p.gate, base + k * p.group);
            else if (p.gate_kind == kGateDocument) r.t[2][k] = reinterpret_cast<const uint4 *>(p.gate)[gate_base + k * p.group];
        }
    };

    ShortRaw<U> next;
    load(begin, next);
    for (int64_t i = 0; i < p.per_group; ++i) {   // as often for every lane of a warp: they share the sums
        const int64_t row = begin + i;
        const ShortRaw<U> r = next;
        if (i + 1 < p.per_group) load(row + 1, next);
        const bool in = row < p.rows, real = r.token >= 0;
        const int64_t at = row * p.units + lane;
        forward_row<BF16, U, -1>(
            p, has, HeldWeights<BF16, U>{w1}, HeldWeights<BF16, U>{w2}, [&](int k) { return r.t[0][k]; },
            [&](int k) { return r.t[1][k]; }, [&](int k) { return r.t[2][k]; },
            [&](uint32_t(&bits)[U][E / 2]) { short_bits<BF16, U>(p, key, static_cast<uint32_t>(r.token), lane, bits); },
            [&](float(&v)[1]) { lanes_sum<1>(v, p.group); },
            [&](int k, bool there, uint4 v) { store_unit_if(in && there, p.y, at + k * p.group, real ? v : make_uint4(0, 0, 0, 0)); },
            [&](int k, bool there, uint4 v) { store_unit_if(in && there, p.n, at + k * p.group, real ? v : make_uint4(0, 0, 0, 0)); });
    }
}

template <bool BF16, int U>
__global__ void __launch_bounds__(kShortThreads, U == 1 ? 4 : 2) residual_norm_backward_short_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    const int lane = threadIdx.x % p.group, groups = kShortThreads / p.group;
    const int64_t which = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / p.group;
    const int64_t begin = which * p.per_group, end = min(begin + p.per_group, p.T);
    const bool need_h = p.post != nullptr || p.gate_kind != 0;
    DropKey key;
    key.load(p.rule);
    Has<U> has;
#pragma unroll
    for (int k = 0; k < U; ++k) has.at[k] = lane + k * p.group < p.units;
    F2 w1[U][E / 2], w2[U][E / 2];
    load_weights<BF16, U>(p.post, has, lane, p.group, w1);
    load_weights<BF16, U>(p.pre, has, lane, p.group, w2);
    Sums<BF16, U> acc;
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int i = 0; i < E / 2; ++i) acc.post[k][i] = acc.pre[k][i] = acc.gate[k][i] = twice(0.0f);
    Document doc;
    const bool by_document = p.gate_kind == kGateDocument;
    if (by_document && begin < end) doc.enter(p, begin);

    auto load = [&](int64_t t, ShortRaw<U> &r) {
        r.row = -1;
#pragma unroll
        for (int j = 0; j < 5; ++j)
#pragma unroll
            for (int k = 0; k < U; ++k) r.t[j][k] = make_uint4(0, 0, 0, 0);
        if (t >= end) return;
        const int64_t row = p.row_of_token == nullptr ? t : p.row_of_token[t];
        if (!in_bounds(row >= 0 && row < p.rows, lane == 0)) return;
        r.row = row;
        const int64_t base = row * p.units + lane;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has.at[k]) continue;
            if (p.x != nullptr) r.t[0][k] = load_unit(p.x, base + k * p.group);
            if (p.pre != nullptr) {
                r.t[1][k] = load_unit(p.dn, base + k * p.group);
                r.t[2][k] = load_unit(p.y_in, base + k * p.group);
            }
            if (need_h) r.t[3][k] = load_unit(p.h, base + k * p.group);
            if (p.gate_kind == kGateToken) r.t[4][k] = load_unit(p.gate, base + k * p.group);
        }
    };

    ShortRaw<U> next;
    load(begin, next);
    for (int64_t i = 0; i < p.per_group; ++i) {
        const int64_t t = begin + i;
        ShortRaw<U> r = next;
        if (i + 1 < p.per_group) load(t + 1, next);
        const bool real = r.row >= 0;
        if (by_document && real) {
            if (t >= doc.hi) {
                leave_document<BF16, U>(p, doc, which, begin, end, has, lane, acc);
                doc.enter(p, t);
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (has.at[k]) r.t[4][k] = reinterpret_cast<const uint4 *>(p.gate)[static_cast<int64_t>(doc.at) * p.units + lane + k * p.group];
        }
        const int64_t at = r.row * p.units + lane;
        backward_row<BF16, U, -1>(
            p, has, HeldWeights<BF16, U>{w1}, HeldWeights<BF16, U>{w2}, acc, [&](int k) { return r.t[0][k]; }, [&](int k) { return r.t[1][k]; },
            [&](int k) { return r.t[2][k]; }, [&](int k) { return r.t[3][k]; }, []() {},
            [&](int k) { return r.t[4][k]; },
            [&](uint32_t(&bits)[U][E / 2]) { short_bits<BF16, U>(p, key, static_cast<uint32_t>(t), lane, bits); },
            [&](auto &v) { lanes_sum(v, p.group); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, p.y, at + k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, p.n, at + k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, p.dgate, at + k * p.group, v); });
    }
    if (by_document && begin < end) leave_document<BF16, U>(p, doc, which, begin, end, has, lane, acc);

    // the CTA's part of the weights' gradients, its groups added in order
    __shared__ float join[kShortThreads * U * E];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (w == 0 ? p.post == nullptr : p.pre == nullptr) continue;
        float *to = (w == 0 ? p.part_post : p.part_pre) + static_cast<int64_t>(blockIdx.x) * p.row_elems;
        const int row = p.group * U * E;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float f[E];
            spread<E>(w == 0 ? acc.post[k] : acc.pre[k], f);
            store_floats<E>(join + (threadIdx.x / p.group) * row + (lane + k * p.group) * E, f);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < p.row_elems; c += kShortThreads) {
            float v = join[c];
            for (int g = 1; g < groups; ++g) v = __fadd_rn(v, join[g * row + c]);
            to[c] = v;
        }
    }
    zero_padding<U>(p, has, lane, threadIdx.x / p.group, groups);
}

// ----------------------------------------------------------------- long rows: a team of warps each

// A ring of rows in shared memory. A team's first warp has the bulk-copy engine fetch the row of every input tensor, a
// lane and one instruction for each.
struct Ring {
    uint8_t *smem;
    uint64_t *full;                // of every stage
    int32_t *index;                // of every stage: a forward call's token or a gradient's row (-1: none)
    int stages;
    uint32_t place, stage_bytes;   // bytes of a row's place (every thread's units whole) and of all tensors'
    int slot = 0;
    uint32_t phase = 0;

    // the current row of tensor 0
    __device__ __forceinline__ const uint4 *row() const { return reinterpret_cast<const uint4 *>(smem + slot * stage_bytes); }
    // What no copy writes: the ends of the places, behind the rows.
    __device__ __forceinline__ void zero_ends(const Team &team, int tensors, uint32_t row_bytes)
    {
        for (int i = 0; i < stages * tensors; ++i)
            for (uint32_t at = row_bytes + team.thread * 16; at < place; at += team.threads * 16)
                *reinterpret_cast<uint4 *>(smem + i * place + at) = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void advance()
    {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
};

__device__ unsigned int g_wait_timeouts;

// Runs `work(i, after)` for i = 0 .. count - 1 with the i-th row's data in the ring. It has to call after() once behind its
// first barrier, where every thread is done with the row before; `sum` votes there whether a wait has run
// out. index_of(i) looks the i-th row up (-1: it is not read), row_of(i, index) is its place in this lane's tensor, `base`.
template <class Sum, class Index, class RowOf, class Work>
__device__ __forceinline__ void walk(Ring &ring, Sum &sum, int64_t count, int tensors, uint32_t row_bytes, const uint8_t *base,
                                     Index index_of, RowOf row_of, Work work)
{
    const int lane = sum.team.thread & 31;
    const bool first = sum.team.thread < 32, several = ring.stages > 1;
    int64_t issued = 0;
    int put = 0;
    int32_t ahead = first ? index_of(0) : -1;   // looked up a row early
    auto issue = [&]() {   // by the first warp
        if (issued >= count) return;
        uint64_t *bar = &ring.full[put];
        if (lane == 0) {
            ring.index[put] = ahead;
            mbar_expect_tx(bar, ahead >= 0 ? static_cast<uint32_t>(tensors) * row_bytes : 0);
        }
        __syncwarp();
        if (lane < tensors && ahead >= 0)
            bulk_load(ring.smem + put * ring.stage_bytes + lane * ring.place, base + row_of(issued, ahead) * row_bytes, row_bytes, bar);
        ahead = index_of(++issued);
        if (++put == ring.stages) put = 0;
    };
    if (sum.team.thread == 0) {
        for (int c = 0; c < ring.stages; ++c) mbar_init(&ring.full[c], 1);
        mbar_init_fence();
    }
    __syncthreads();   // of all teams: what else was put into shared memory is there too
    if (first)
        for (int c = 0; c < ring.stages; ++c) issue();
    for (int64_t i = 0; i < count; ++i) {
        if (!mbar_wait_bounded(&ring.full[ring.slot], ring.phase)) sum.ask = true;
        work(i, [&]() {
            if (several && first && i > 0) issue();   // into the place of the row before
        });
        ring.advance();
        if (!several) {
            sum.stop = sum.team.any(sum.ask);
            if (first && !sum.stop) issue();
        }
        if (sum.stop) {   // by all: no copy may end in another CTA's shared memory
            if (first) {
                if (lane == 0) atomicAdd(&g_wait_timeouts, 1u);
                for (int64_t k = i + 1; k < issued; ++k) {
                    mbar_wait_bounded(&ring.full[ring.slot], ring.phase);
                    ring.advance();
                }
            }
            return;
        }
    }
}

// The weights of all teams in shared memory, every thread's units whole.
template <int F>
__device__ __forceinline__ void share_weights(const ResidualParams &p, float *to, int columns)
{
    for (int c = threadIdx.x; c < columns; c += blockDim.x) {
        if (Asked<F>::post(p)) to[c] = c < p.row_elems ? p.post[c] : 0.0f;
        if (Asked<F>::pre(p)) to[columns + c] = c < p.row_elems ? p.pre[c] : 0.0f;
    }
}

template <bool BF16, int U, int F>
__global__ void __launch_bounds__(kForwardThreads) residual_norm_long_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    typedef Asked<F> A;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float room[kMaxTeams][TeamSum<64>::kRoom];
    __shared__ __align__(8) uint64_t full[kMaxTeams][kMaxStages];
    __shared__ int32_t index[kMaxTeams][kMaxStages];
    const int mine = threadIdx.x / p.group, lane = threadIdx.x - mine * p.group, teams = blockDim.x / p.group;
    const Team team = {lane, p.group, mine + 1};
    const int64_t begin = (static_cast<int64_t>(blockIdx.x) * teams + mine) * p.per_group;
    const int64_t count = max(min(p.per_group, p.rows - begin), static_cast<int64_t>(0));
    DropKey key;
    key.load(p.rule);
    Has<U> has;
#pragma unroll
    for (int k = 0; k < U; ++k) has.at[k] = lane + k * p.group < p.units;
    float *weights = reinterpret_cast<float *>(smem);
    const int columns = U * p.group * E;
    share_weights<F>(p, weights, columns);
    const SharedWeights<BF16> w1 = {weights + lane * E, p.group * E}, w2 = {weights + columns + lane * E, p.group * E};
    Document doc;
    TeamSum<64> sum(room[mine], team);
    const uint32_t place = U * p.group * 16u, row_bytes = p.units * 16u, stage = place * p.tensors;
    Ring ring = {smem + 2 * columns * sizeof(float) + static_cast<size_t>(mine) * p.stages * stage, full[mine], index[mine],
                 p.stages, place, stage};
    ring.zero_ends(team, p.tensors, row_bytes);

    auto token_of = [&](int64_t i) {
        int32_t t = -1;
        if (i < count) t = p.token_of_row == nullptr ? static_cast<int32_t>(begin + i) : p.token_of_row[begin + i];
        return t >= 0 && in_bounds(t < p.T) ? t : -1;
    };
    // the rows are neighbours, padding is not read
    auto row_of = [&](int64_t i, int32_t) { return begin + i; };
    const int tensor = lane & 31;
    const uint8_t *base = tensor == 0 ? p.x : tensor == 1 && A::block(p.h != nullptr) ? p.h : p.gate;
    uint8_t *y = p.y, *n = p.n;
    walk(ring, sum, count, p.tensors, row_bytes, base, token_of, row_of, [&](int64_t i, auto after) {
        const int32_t token = ring.index[ring.slot];
        const bool real = token >= 0;
        const uint4 *data = ring.row() + lane;
        const int64_t at = (begin + i) * row_bytes + lane * 16;   // of this thread's first unit, in bytes
        uint4 gate[U];                                            // of the row's document
        if (A::gate(p) == kGateDocument) {
            if (real) doc.enter(p, token);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                gate[k] = make_uint4(0, 0, 0, 0);
                if (real && has.at[k])
                    gate[k] = reinterpret_cast<const uint4 *>(p.gate)[static_cast<int64_t>(doc.at) * p.units + lane + k * p.group];
            }
        }
        if (!real) {
#pragma unroll
            for (int k = 0; k < U; ++k) {
                store_unit_if(has.at[k] && y != nullptr, y + at, k * p.group, make_uint4(0, 0, 0, 0));
                store_unit_if(has.at[k] && n != nullptr, n + at, k * p.group, make_uint4(0, 0, 0, 0));
            }
        }
        bool waiting = true;
        forward_row<BF16, U, F>(
            p, has, w1, w2, [&](int k) { return data[k * p.group]; }, [&](int k) { return data[(U + k) * p.group]; },
            [&](int k) { return A::gate(p) == kGateToken ? data[(2 * U + k) * p.group] : gate[k]; },
            [&](uint32_t(&bits)[U][E / 2]) { thread_bits<BF16, U>(p.rule, key, static_cast<uint32_t>(token), lane, p.group, bits); },
            [&](float(&v)[1]) {
                sum(v);
                if (waiting) after();
                waiting = false;
            },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, y + at, k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, n + at, k * p.group, v); });
        if (waiting) {   // no norm, no sum
            sum.stop = team.any(sum.ask);
            after();
        }
    });
}

template <bool BF16, int U, int F>
__global__ void __launch_bounds__(kBackwardThreads) residual_norm_backward_long_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    typedef Asked<F> A;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float room[kMaxTeams][TeamSum<64>::kRoom];
    __shared__ __align__(8) uint64_t full[kMaxTeams][kMaxStages];
    __shared__ int32_t index[kMaxTeams][kMaxStages];
    const int mine = threadIdx.x / p.group, lane = threadIdx.x - mine * p.group, teams = blockDim.x / p.group;
    const Team team = {lane, p.group, mine + 1};
    const int64_t which = static_cast<int64_t>(blockIdx.x) * teams + mine;
    const int64_t begin = which * p.per_group, end = max(min(begin + p.per_group, p.T), begin), count = end - begin;
    const bool need_h = A::post(p) || A::gate(p) != 0, pre = A::pre(p), by_document = A::gate(p) == kGateDocument;
    DropKey key;
    key.load(p.rule);
    Has<U> has;
#pragma unroll
    for (int k = 0; k < U; ++k) has.at[k] = lane + k * p.group < p.units;
    Sums<BF16, U> acc;
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
        for (int i = 0; i < E / 2; ++i) acc.post[k][i] = acc.pre[k][i] = acc.gate[k][i] = twice(0.0f);
    Document doc;
    TeamSum<64> sum(room[mine], team);
    const uint32_t place = U * p.group * 16u, row_bytes = p.units * 16u, stage = place * p.tensors;
    // no weights are held for a call whose rows leave no room (a generic one)
    const bool hold = F >= 0 || p.hold;
    float *weights = reinterpret_cast<float *>(smem);
    const int columns = hold ? U * p.group * E : 0;
    share_weights<F>(p, weights, columns);
    auto w1 = [&](int k, F2(&out)[E / 2]) {
        if (hold) SharedWeights<BF16>{weights + lane * E, p.group * E}(k, out);
        else load_weight<BF16>(p.post, has.at[k], lane + k * p.group, out);
    };
    auto w2 = [&](int k, F2(&out)[E / 2]) {
        if (hold) SharedWeights<BF16>{weights + columns + lane * E, p.group * E}(k, out);
        else load_weight<BF16>(p.pre, has.at[k], lane + k * p.group, out);
    };
    // a team's own: a document's gate, each thread's part written and read by itself, and the ring
    uint8_t *own = smem + 2 * columns * sizeof(float);
    uint4 *own_gate = reinterpret_cast<uint4 *>(own + mine * place) + lane;
    if (by_document) own += teams * place;
    Ring ring = {own + static_cast<size_t>(mine) * p.stages * stage, full[mine], index[mine], p.stages, place, stage};
    ring.zero_ends(team, p.tensors, row_bytes);
    // places of the tensors in a stage, in units
    const int step = U * p.group;
    const int at_dn = p.x != nullptr ? step : 0, at_y = at_dn + (pre ? step : 0), at_h = at_y + (pre ? step : 0),
              at_gate = at_h + (need_h ? step : 0);
    // this lane's tensor
    int left = lane & 31;
    const uint8_t *base = nullptr;
    for (const uint8_t *b : {p.x, pre ? p.dn : nullptr, pre ? p.y_in : nullptr, need_h ? p.h : nullptr,
                             A::gate(p) == kGateToken ? p.gate : nullptr})
        if (b != nullptr && left-- == 0) base = b;

    auto index_of = [&](int64_t i) {
        int64_t row = -1;
        if (i < count) row = p.row_of_token == nullptr ? begin + i : p.row_of_token[begin + i];
        return static_cast<int32_t>(row >= 0 && in_bounds(row < p.rows) ? row : -1);
    };
    auto row_of = [&](int64_t, int32_t row) { return static_cast<int64_t>(row); };
    walk(ring, sum, count, p.tensors, row_bytes, base, index_of, row_of, [&](int64_t i, auto after) {
        const int32_t row = ring.index[ring.slot];
        if (row < 0) {   // an index that a check refused
            sum.stop = team.any(sum.ask);
            after();
            return;
        }
        const int64_t t = begin + i, at = static_cast<int64_t>(row) * row_bytes + lane * 16;
        const uint4 *data = ring.row() + lane;
        bool waiting = true;
        backward_row<BF16, U, F>(
            p, has, w1, w2, acc, [&](int k) { return p.x != nullptr ? data[k * p.group] : make_uint4(0, 0, 0, 0); },
            [&](int k) { return data[at_dn + k * p.group]; }, [&](int k) { return data[at_y + k * p.group]; },
            [&](int k) { return data[at_h + k * p.group]; },
            [&]() {
                if (t < doc.hi) return;
                if (doc.hi >= 0) leave_document<BF16, U>(p, doc, which, begin, end, has, lane, acc);
                doc.enter(p, t);
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    uint4 g = make_uint4(0, 0, 0, 0);
                    if (has.at[k]) g = reinterpret_cast<const uint4 *>(p.gate)[static_cast<int64_t>(doc.at) * p.units + lane + k * p.group];
                    own_gate[k * p.group] = g;
                }
            },
            [&](int k) { return by_document ? own_gate[k * p.group] : data[at_gate + k * p.group]; },
            [&](uint32_t(&bits)[U][E / 2]) { thread_bits<BF16, U>(p.rule, key, static_cast<uint32_t>(t), lane, p.group, bits); },
            [&](auto &v) {
                sum(v);
                if (waiting) after();
                waiting = false;
            },
            [&](int k, bool there, uint4 v) { store_unit_if(there, p.y + at, k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(there, p.n + at, k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(there, p.dgate + at, k * p.group, v); });
        if (waiting) {   // no norm, no sum
            sum.stop = team.any(sum.ask);
            after();
        }
    });
    if (by_document && doc.hi >= 0) leave_document<BF16, U>(p, doc, which, begin, end, has, lane, acc);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (w == 0 ? !A::post(p) : !A::pre(p)) continue;
        float *to = (w == 0 ? p.part_post : p.part_pre) + which * p.row_elems;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float f[E];
            spread<E>(w == 0 ? acc.post[k] : acc.pre[k], f);
            if (has.at[k]) store_floats<E>(to + static_cast<int64_t>(lane + k * p.group) * E, f);
        }
    }
    zero_padding<U>(p, has, lane, mine, teams);
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

int row_units(int64_t row_elems, int dtype) { return static_cast<int>(row_elems * (dtype == kBf16 ? 2 : 4) / 16); }

size_t shared_bytes(const ResidualParams &p, const Shape &s, int dtype, bool gate)
{
    const size_t row = static_cast<size_t>(s.threads / s.group) * s.per_thread * s.group * 16;
    return weight_bytes(s, dtype) + (gate ? row : 0) + row * p.stages * p.tensors;
}

// A kernel's limit of dynamic shared memory, raised once on each device.
template <auto kernel>
cudaError_t allow_shared(int device)
{
    static std::mutex mu;
    static bool done[64] = {false};
    std::lock_guard<std::mutex> lock(mu);
    if (device >= 0 && device < 64 && done[device]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedBytes - kOwnBytes);
    if (e == cudaSuccess && device >= 0 && device < 64) done[device] = true;
    return e;
}

// The kernel of its own for what is asked most: both norms, with any gate; the pre norm alone, without one. Each with
// and without dropout. The others share one that looks at its parameters (262144 x 2560 bf16, both norms, dropout:
// TIMES us).
template <class Launch>
cudaError_t with_asked(const ResidualParams &p, bool block, Launch launch)
{
    const int f = (p.post != nullptr) + 2 * (p.pre != nullptr) + 4 * (p.rule.rng != nullptr) + 8 * p.gate_kind;
    switch (block ? f : -1) {
    case 2: return launch(std::integral_constant<int, 2>());
    case 3: return launch(std::integral_constant<int, 3>());
    case 6: return launch(std::integral_constant<int, 6>());
    case 7: return launch(std::integral_constant<int, 7>());
    case 11: return launch(std::integral_constant<int, 11>());
    case 15: return launch(std::integral_constant<int, 15>());
    case 19: return launch(std::integral_constant<int, 19>());
    case 23: return launch(std::integral_constant<int, 23>());
    default: return launch(std::integral_constant<int, -1>());
    }
}

// A kernel as a type.
template <void (*K)(ResidualParams)>
struct Kernel {
    static constexpr auto value = K;
};

template <bool BF16>
cudaError_t launch_forward(const ResidualParams &p, const Shape &s, unsigned grid, int device, cudaStream_t stream)
{
    if (s.shorter) {
        if (s.per_thread == 1) residual_norm_short_kernel<BF16, 1><<<grid, s.threads, 0, stream>>>(p);
        else residual_norm_short_kernel<BF16, 2><<<grid, s.threads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    constexpr int U = BF16 ? 1 : 2;   // units of eight columns
    auto run = [&](auto kernel) {
        const cudaError_t e = allow_shared<decltype(kernel)::value>(device);
        if (e != cudaSuccess) return e;
        decltype(kernel)::value<<<grid, s.threads, shared_bytes(p, s, BF16 ? kBf16 : kF32, false), stream>>>(p);
        return cudaGetLastError();
    };
    return with_asked(p, p.h != nullptr, [&](auto f) {
        constexpr int F = decltype(f)::value;
        if (s.per_thread == 2 * U) return run(Kernel<residual_norm_long_kernel<BF16, 2 * U, F>>());
        if (s.per_thread == 3 * U) return run(Kernel<residual_norm_long_kernel<BF16, 3 * U, F>>());
        return run(Kernel<residual_norm_long_kernel<BF16, 5 * U, F>>());
    });
}

template <bool BF16>
cudaError_t launch_backward(const ResidualParams &p, const Shape &s, unsigned grid, int device, cudaStream_t stream)
{
    if (s.shorter) {
        if (s.per_thread == 1) residual_norm_backward_short_kernel<BF16, 1><<<grid, s.threads, 0, stream>>>(p);
        else residual_norm_backward_short_kernel<BF16, 2><<<grid, s.threads, 0, stream>>>(p);
        return cudaGetLastError();
    }
    constexpr int U = BF16 ? 1 : 2;   // units of eight columns
    auto run = [&](auto kernel) {
        const cudaError_t e = allow_shared<decltype(kernel)::value>(device);
        if (e != cudaSuccess) return e;
        decltype(kernel)::value<<<grid, s.threads, shared_bytes(p, s, BF16 ? kBf16 : kF32, p.gate_kind == kGateDocument), stream>>>(p);
        return cudaGetLastError();
    };
    if (!s.hold) return run(Kernel<residual_norm_backward_long_kernel<BF16, 2 * U, -1>>());
    return with_asked(p, p.n != nullptr, [&](auto f) { return run(Kernel<residual_norm_backward_long_kernel<BF16, 2 * U, decltype(f)::value>>()); });
}

// Tokens of a group of the gradient, and its CTAs.
void deal(int64_t T, const Shape &s, int device, int64_t &per_group, int64_t &ctas)
{
    const int64_t groups = s.threads / s.group;
    const int64_t most = static_cast<int64_t>(sm_count(device)) * s.ctas_per_sm * groups;
    per_group = (T + most - 1) / most;
    if (per_group < 1) per_group = 1;
    ctas = (T + per_group * groups - 1) / (per_group * groups);
}

}  // namespace

cudaError_t launch_residual_norm(ResidualParams p, int dtype, int device, cudaStream_t stream)
{
    if (p.rows == 0) return cudaSuccess;
    p.units = row_units(p.row_elems, dtype);
    p.per_column = 1.0f / static_cast<float>(p.row_elems);
    p.tensors = 1 + (p.h != nullptr) + (p.gate_kind == kGateToken);
    const Shape s = shape_of(p.units, dtype, false, p.tensors);
    p.group = s.group;
    int64_t ctas;
    if (s.shorter) {
        // rows of a group: enough to fetch ahead, few enough that all SMs get some
        const int64_t groups = s.threads / s.group;
        const int64_t even = p.rows / (static_cast<int64_t>(sm_count(device)) * 8 * groups);
        p.per_group = even < 1 ? 1 : even > 16 ? 16 : even;
        ctas = (p.rows + p.per_group * groups - 1) / (p.per_group * groups);
    } else {
        deal(p.rows, s, device, p.per_group, ctas);
        p.stages = stages_of(s, dtype, p.tensors, false);
    }
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(ctas);
    return dtype == kBf16 ? launch_forward<true>(p, s, grid, device, stream) : launch_forward<false>(p, s, grid, device, stream);
}

int64_t residual_backward_workspace(int64_t T, int64_t row_elems, int dtype, int device)
{
    // enough for any options: those that read least have the most CTAs
    const Shape s = shape_of(row_units(row_elems, dtype), dtype, true, 1);
    const int64_t groups = s.threads / s.group;
    int64_t most = static_cast<int64_t>(sm_count(device)) * s.ctas_per_sm * groups;
    if (most > T) most = T;
    return (most + groups - 1) / groups * groups * 4 * row_elems * 4;
}

cudaError_t launch_residual_norm_backward(ResidualParams p, int dtype, void *workspace, int device, cudaStream_t stream)
{
    p.units = row_units(p.row_elems, dtype);
    p.per_column = 1.0f / static_cast<float>(p.row_elems);
    const bool need_h = p.post != nullptr || p.gate_kind != 0;
    p.tensors = (p.x != nullptr) + 2 * (p.pre != nullptr) + need_h + (p.gate_kind == kGateToken);
    const Shape s = shape_of(p.units, dtype, true, p.tensors, p.gate_kind == kGateDocument);
    p.group = s.group;
    p.hold = s.hold;
    int64_t ctas;
    deal(p.T, s, device, p.per_group, ctas);
    // the weights' parts: a CTA's of short rows, a team's of long ones
    p.parts = static_cast<int32_t>(s.shorter ? ctas : ctas * (s.threads / s.group));
    p.part_post = static_cast<float *>(workspace);
    p.part_pre = p.part_post + static_cast<int64_t>(p.parts) * p.row_elems;
    p.part_gate = p.part_pre + static_cast<int64_t>(p.parts) * p.row_elems;
    if (p.T > 0) {
        p.stages = s.shorter ? 0 : stages_of(s, dtype, p.tensors, p.gate_kind == kGateDocument);
        const unsigned grid = static_cast<unsigned>(ctas);
        const cudaError_t e = dtype == kBf16 ? launch_backward<true>(p, s, grid, device, stream)
                                             : launch_backward<false>(p, s, grid, device, stream);
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

cudaError_t read_residual_wait_timeouts(unsigned int *count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

cudaError_t read_residual_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

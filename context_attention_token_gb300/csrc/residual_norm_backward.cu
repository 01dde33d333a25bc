// The gradient of the residual stream between two blocks. Mathematics, layout and reasons: residual_norm.cuh.
//
// A group of threads takes neighbouring tokens and keeps its columns' part of dw1, dw2 and of the current document's dgate in
// registers (which is why a thread of long rows has 16 columns here and up to 40 forward); parts meet in the workspace
// and are added in a fixed order.
//
// 131071 x 2560 bf16 with both norms, a document's gate and dropout takes 915 us (4.4 TB/s, 0.65 of a copy): some 58
// instructions a column at 15 warps an SM bound it; without a gate 131072 rows take 770 us (0.77). 20011 x 1132 float32 with a token's
// gate takes 138 us (5.2 TB/s).
#include "residual_norm.cuh"

#include <math_constants.h>

namespace cpt {

namespace {

// What a thread adds up over its tokens. With a gate that a document shares, gate holds sum d hn over the document's tokens so far:
// w1 times it is dgate, and gate times it the document's part of dw1. So one product a column and token does for both.
template <bool BF16, int U>
struct Sums {
    F2 post[U][Unit<BF16>::E / 2], pre[U][Unit<BF16>::E / 2], gate[U][Unit<BF16>::E / 2];
};

// One token of the gradient; dy to gate give the data of a unit of its row (0 past the row's end), set_h changes that of h.
// `enter` is called before the gate is asked for. Where `real` is false there is no token: its data are zeros, and it adds
// nothing to any sum (a statistic of zeros, which is infinite without an eps, is not used).
template <bool LONG, bool BF16, int U, int F, class W1, class W2, class DY, class DN, class Y, class H, class SetH, class Enter, class G,
          class Bits, class Sum, class PutX, class PutH, class PutG>
__device__ __forceinline__ void backward_row(const ResidualParams &p, bool real, const Has<U> &has, W1 w1, W2 w2,
                                             Sums<BF16, U> &acc, DY dy, DN dn, Y y, H h, SetH set_h, Enter enter, G gate, Bits bits,
                                             Sum sum, PutX put_x, PutH put_h, PutG put_gate)
{
    typedef UnitPairs<BF16> V;
    typedef Asked<F> A;
    constexpr int N = V::N;
    constexpr bool IN_PLACE = LONG && F >= 0 && (F & 1);
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
    if ((pre || post) && sum(s)) return;
    if (A::gate(p) == kGateDocument) enter();
    const float r2 = pre && real ? rsqrt_mean(p, s[0]) : 0.0f, r1 = !post ? 1.0f : real ? rsqrt_mean(p, s[2]) : 0.0f;
    // What was dropped has no gradient and adds nothing to a sum, whatever it is multiplied by: h is 0 there. Behind a norm only a row
    // whose squares have no finite sum holds what 0 would not take; such a row is changed where it stands, if it stands in
    // shared memory.
    if (IN_PLACE && A::drop(p) && !(s[2] < CUDART_INF_F)) {
#pragma unroll
        for (int k = 0; k < U; ++k) {
            F2 a[N];
            V::unpack(h(k), a);
            keep_or_zero<N>(p.rule, rnd[k], a);
            set_h(k, V::pack(a));
        }
    }
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
            if (!IN_PLACE && A::drop(p)) keep_or_zero<N>(p.rule, rnd[k], hn);
        }
        const bool by_document = A::gate(p) == kGateDocument;
        if (A::gate(p) != 0) {
            F2 g[N];
            V::unpack(gate(k), g);
            if (by_document) {   // its weights come in when the document is left
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    acc.gate[k][i] = fma2(d[i], hn[i], acc.gate[k][i]);
                    d[i] = mul2(d[i], g[i]);
                }
                if (A::drop(p)) keep_or_zero<N>(p.rule, rnd[k], d);
            } else {
                F2 z[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    z[i] = mul2(d[i], post ? mul2(hn[i], w[i]) : hn[i]);
                    d[i] = mul2(d[i], g[i]);
                }
                if (A::drop(p)) {
                    keep_or_zero<N>(p.rule, rnd[k], z);
                    keep_or_zero<N>(p.rule, rnd[k], d);
                }
                put_gate(k, has.at[k], V::pack(z));
            }
        }
        if (post) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!by_document) acc.post[k][i] = fma2(d[i], hn[i], acc.post[k][i]);
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
        if (!IN_PLACE && A::drop(p) && !(s[2] < CUDART_INF_F)) keep_or_zero<N>(p.rule, rnd[k], hn);
#pragma unroll
        for (int i = 0; i < N; ++i) hn[i] = fma2(hn[i], back1, mul2(e[k][i], twice(r1)));
        put_h(k, has.at[k], V::pack(hn));
    }
}

// The sums over a document's tokens leave: dgate for where it belongs (the result when the document lies in this group's
// tokens, part 0 when it began earlier, part 1 when it goes on), the document's part of dw1 to the others'.
template <bool BF16, int U, int F, class W1>
__device__ __forceinline__ void leave_document(const ResidualParams &p, const Document &doc, int64_t which, int32_t begin,
                                               int32_t end, const Has<U> &has, int lane, W1 w1, Sums<BF16, U> &acc)
{
    constexpr int E = Unit<BF16>::E;
    float *to = reinterpret_cast<float *>(p.dgate) + static_cast<int64_t>(doc.at) * p.row_elems;
    if (doc.lo < begin) to = p.part_gate + which * 2 * p.row_elems;
    else if (doc.hi > end) to = p.part_gate + (which * 2 + 1) * p.row_elems;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        F2 z[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            z[i] = acc.gate[k][i];
            acc.gate[k][i] = twice(0.0f);
        }
        if (Asked<F>::post(p)) {
            F2 w[E / 2], g[E / 2];
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (has.at[k]) raw = reinterpret_cast<const uint4 *>(p.gate)[static_cast<int64_t>(doc.at) * p.units + lane + k * p.group];
            UnitPairs<BF16>::unpack(raw, g);
            w1(k, w);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 sums = both(z[i]), gates = both(g[i]);   // no sum, no part: an infinite gate of dropped columns
                acc.post[k][i] = fma2(z[i], pair_of(sums.x == 0.0f ? 0.0f : gates.x, sums.y == 0.0f ? 0.0f : gates.y), acc.post[k][i]);
                z[i] = mul2(z[i], w[i]);
            }
        }
        float f[E];
        spread<E>(z, f);
        if (has.at[k]) store_floats<E>(to + static_cast<int64_t>(lane + k * p.group) * E, f);
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

template <bool BF16, int U, int F>
__global__ void __launch_bounds__(kShortThreads, short_ctas(U, F)) residual_norm_backward_short_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    typedef Asked<F> A;
    const int lane = threadIdx.x % p.group, groups = kShortThreads / p.group;
    const int64_t which = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / p.group;
    const int32_t begin = static_cast<int32_t>(min(which * p.per_group, p.T));
    const int32_t end = static_cast<int32_t>(min(begin + p.per_group, p.T)), count = end - begin;
    const bool need_h = A::post(p) || A::gate(p) != 0;
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
    const bool by_document = A::gate(p) == kGateDocument;
    if (by_document && begin < end) doc.enter(p, begin);

    auto load = [&](int32_t i, ShortRaw<U> &r) {   // token begin + i, if it is this group's
        r.row = -1;
#pragma unroll
        for (int j = 0; j < 5; ++j)
#pragma unroll
            for (int k = 0; k < U; ++k) r.t[j][k] = make_uint4(0, 0, 0, 0);
        if (i >= count) return;
        const int32_t t = begin + i;
        const int64_t row = p.row_of_token == nullptr ? t : p.row_of_token[t];
        if (!in_bounds(row >= 0 && row < p.rows, lane == 0)) return;
        r.row = row;
        const int64_t base = row * p.units + lane;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has.at[k]) continue;
            if (p.x != nullptr) r.t[0][k] = load_unit(p.x, base + k * p.group);
            if (A::pre(p)) {
                r.t[1][k] = load_unit(p.dn, base + k * p.group);
                r.t[2][k] = load_unit(p.y_in, base + k * p.group);
            }
            if (need_h) r.t[3][k] = load_unit(p.h, base + k * p.group);
            if (A::gate(p) == kGateToken) r.t[4][k] = load_unit(p.gate, base + k * p.group);
        }
    };

    ShortRaw<U> next;
    load(0, next);
    for (int32_t i = 0; i < p.per_group; ++i) {   // as often for every lane of a warp: they share the sums
        const int32_t t = i < count ? begin + i : 0;
        ShortRaw<U> r = next;
        load(i + 1, next);
        const bool real = r.row >= 0;
        if (by_document && real) {
            if (t >= doc.hi) {
                leave_document<BF16, U, F>(p, doc, which, begin, end, has, lane, HeldWeights<BF16, U>{w1}, acc);
                doc.enter(p, t);
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (has.at[k]) r.t[4][k] = reinterpret_cast<const uint4 *>(p.gate)[static_cast<int64_t>(doc.at) * p.units + lane + k * p.group];
        }
        const int64_t at = r.row * p.units + lane;
        backward_row<false, BF16, U, F>(
            p, real, has, HeldWeights<BF16, U>{w1}, HeldWeights<BF16, U>{w2}, acc, [&](int k) { return r.t[0][k]; }, [&](int k) { return r.t[1][k]; },
            [&](int k) { return r.t[2][k]; }, [&](int k) { return r.t[3][k]; },
            [](int, uint4) {}, []() {},
            [&](int k) { return r.t[4][k]; },
            [&](uint32_t(&bits)[U][E / 2]) { short_bits<BF16, U>(p, key, static_cast<uint32_t>(t), lane, bits); },
            [&](auto &v) {
                lanes_sum(v, p.group);
                return false;
            },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, p.y, at + k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, p.n, at + k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, p.dgate, at + k * p.group, v); });
    }
    if (by_document && begin < end) leave_document<BF16, U, F>(p, doc, which, begin, end, has, lane, HeldWeights<BF16, U>{w1}, acc);

    // the CTA's part of the weights' gradients, its groups added in order
    __shared__ float join[kShortThreads * U * E];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (w == 0 ? !A::post(p) : !A::pre(p)) continue;
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
    const int32_t which = blockIdx.x * teams + mine;
    // there are fewer than 2^31 tokens
    const int32_t begin = static_cast<int32_t>(min(which * p.per_group, p.T));
    const int32_t end = static_cast<int32_t>(min(begin + p.per_group, p.T)), count = end - begin;
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

    auto index_of = [&](int32_t i) {
        int32_t row = -1;
        if (i < count) row = p.row_of_token == nullptr ? begin + i : p.row_of_token[begin + i];
        return row >= 0 && in_bounds(row < p.rows) ? row : -1;
    };
    auto row_of = [&](int32_t, int32_t row) { return static_cast<int64_t>(row); };
    walk<F >= 0 ? kVote : kMinimum>(ring, sum, count, p.tensors, row_bytes, p.stall, base, index_of, row_of, [&](int32_t i, int32_t row, auto after) {
        if (row < 0) {   // an index that a check refused, or a wait that has run out
            sum.stop = team.any(sum.ask);
            after();
            return;
        }
        const int32_t t = begin + i;
        const int64_t at = static_cast<int64_t>(row) * row_bytes + lane * 16;
        uint4 *data = ring.row() + lane;   // a thread's units are its own
        bool waiting = true;
        backward_row<true, BF16, U, F>(
            p, true, has, w1, w2, acc, [&](int k) { return p.x != nullptr ? data[k * p.group] : make_uint4(0, 0, 0, 0); },
            [&](int k) { return data[at_dn + k * p.group]; }, [&](int k) { return data[at_y + k * p.group]; },
            [&](int k) { return data[at_h + k * p.group]; },
            [&](int k, uint4 v) {
                data[at_h + k * p.group] = v;
                fence_proxy_async_smem();   // a copy writes here next
            },
            [&]() {
                if (t < doc.hi) return;
                if (doc.hi >= 0) leave_document<BF16, U, F>(p, doc, which, begin, end, has, lane, w1, acc);
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
                return sum.stop;
            },
            [&](int k, bool there, uint4 v) { store_unit_if(there, p.y + at, k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(there, p.n + at, k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(there, p.dgate + at, k * p.group, v); });
        if (waiting) {   // no norm, no sum
            sum.stop = team.any(sum.ask);
            after();
        }
    });
    if (by_document && doc.hi >= 0) leave_document<BF16, U, F>(p, doc, which, begin, end, has, lane, w1, acc);
    // the CTA's part of the weights' gradients, its teams added in order; a team's ring has room for a row of sums (a
    // norm's gradient reads two tensors at least)
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (w == 0 ? !A::post(p) : !A::pre(p)) continue;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < U; ++k) {
            float f[E];
            spread<E>(w == 0 ? acc.post[k] : acc.pre[k], f);
            store_floats<E>(reinterpret_cast<float *>(ring.smem) + (lane + k * p.group) * E, f);
        }
        __syncthreads();
        float *to = (w == 0 ? p.part_post : p.part_pre) + static_cast<int64_t>(blockIdx.x) * p.row_elems;
        for (int c = threadIdx.x; c < p.row_elems; c += blockDim.x) {
            const uint8_t *from = own + c * sizeof(float);
            float v = *reinterpret_cast<const float *>(from);
            for (int g = 1; g < teams; ++g) v = __fadd_rn(v, *reinterpret_cast<const float *>(from + static_cast<size_t>(g) * p.stages * stage));
            to[c] = v;
        }
    }
    zero_padding<U>(p, has, lane, mine, teams);
}

// The sum of v over the block's 32 warps, of column `warp` in every lane.
__device__ __forceinline__ float across_warps(float (*room)[33], float v)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    room[warp][lane] = v;
    __syncthreads();
    v = room[lane][warp];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

constexpr int kWideDocument = 8;   // groups beyond its first that a warp still adds alone

// Adds the parts, in a fixed order, 32 columns a block: blockIdx.y 0 and 1 the weights', a warp every 32nd part; the
// others the documents that reach over several groups.
__global__ void __launch_bounds__(1024) residual_join_kernel(const __grid_constant__ ResidualParams p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    __shared__ float room[32][33];
    if (blockIdx.y < 2) {
        const float *from = blockIdx.y == 0 ? p.part_post : p.part_pre;
        float *to = blockIdx.y == 0 ? p.dpost : p.dpre;
        if (to == nullptr) return;
        float v = 0.0f;
        if (c < p.row_elems) {
#pragma unroll 8
            for (int i = warp; i < p.parts; i += 32) v = __fadd_rn(v, from[static_cast<int64_t>(i) * p.row_elems + c]);
        }
        v = across_warps(room, v);
        if (lane == 0 && blockIdx.x * 32 + warp < p.row_elems) to[blockIdx.x * 32 + warp] = v;
        return;
    }
    // a warp a document, but for those that reach over many groups: these all warps share out
    __shared__ int32_t wide[32];
    float *dgate = reinterpret_cast<float *>(p.dgate);
    const bool there = c < p.row_elems;
    for (int64_t d0 = (blockIdx.y - 2) * 32; d0 < p.n_docs; d0 += static_cast<int64_t>(gridDim.y - 2) * 32) {
        const int64_t d = d0 + warp;
        int64_t first = 0, last = 0;
        bool empty = false;
        if (d < p.n_docs) {
            const int64_t lo = p.cu[d], hi = p.cu[d + 1];
            empty = lo >= hi;
            first = lo / p.per_group;
            last = empty ? first : (hi - 1) / p.per_group;
        }
        if (lane == 0) wide[warp] = last - first > kWideDocument;
        if (empty && there) dgate[d * p.row_elems + c] = 0.0f;
        if (last > first && last - first <= kWideDocument && there) {
            float v = p.part_gate[(first * 2 + 1) * p.row_elems + c];
#pragma unroll 8
            for (int64_t g = first + 1; g <= last; ++g) v = __fadd_rn(v, p.part_gate[g * 2 * p.row_elems + c]);
            dgate[d * p.row_elems + c] = v;
        }
        __syncthreads();
        for (int w = 0; w < 32; ++w) {
            if (!wide[w]) continue;
            const int64_t from = p.cu[d0 + w] / p.per_group, to = (p.cu[d0 + w + 1] - 1) / p.per_group;
            float v = 0.0f;
            if (there) {
                if (warp == 0) v = p.part_gate[(from * 2 + 1) * p.row_elems + c];
#pragma unroll 8
                for (int64_t g = from + 1 + warp; g <= to; g += 32) v = __fadd_rn(v, p.part_gate[g * 2 * p.row_elems + c]);
            }
            v = across_warps(room, v);
            if (lane == 0 && blockIdx.x * 32 + warp < p.row_elems) dgate[(d0 + w) * p.row_elems + blockIdx.x * 32 + warp] = v;
        }
        __syncthreads();
    }
}

template <bool BF16>
cudaError_t launch_backward(const ResidualParams &p, const Shape &s, int f, unsigned grid, int device, cudaStream_t stream)
{
    if (s.shorter) {
        return with_asked<false>(f, [&](auto g) {
            constexpr int F = decltype(g)::value;
            if (s.per_thread == 1) residual_norm_backward_short_kernel<BF16, 1, F><<<grid, s.threads, 0, stream>>>(p);
            else residual_norm_backward_short_kernel<BF16, 2, F><<<grid, s.threads, 0, stream>>>(p);
            return cudaGetLastError();
        });
    }
    constexpr int U = BF16 ? 1 : 2;   // units of eight columns
    auto run = [&](auto kernel) {
        const cudaError_t e = allow_shared<decltype(kernel)::value>(device);
        if (e != cudaSuccess) return e;
        decltype(kernel)::value<<<grid, s.threads, shared_bytes(p, s, BF16 ? kBf16 : kF32, p.gate_kind == kGateDocument), stream>>>(p);
        return cudaGetLastError();
    };
    if (!s.hold) return run(Kernel<residual_norm_backward_long_kernel<BF16, 2 * U, -1>>());
    return with_asked<true>(f, [&](auto g) { return run(Kernel<residual_norm_backward_long_kernel<BF16, 2 * U, decltype(g)::value>>()); });
}

}  // namespace

int64_t residual_backward_workspace(int64_t T, int64_t row_elems, int dtype, int device)
{
    // enough for any options, so the largest of the shapes that a call can have: more tensors leave room for fewer teams, but
    // for fewer weights too, so neither end is the largest by itself. (A document's gate is read outside the ring: four tensors.)
    int64_t most = 0;
    for (int tensors = 1; tensors <= 5; ++tensors) {
        for (const bool by_document : {false, true}) {
            if (by_document && tensors == 5) continue;
            // (f: the most CTAs an SM)
            const Shape s = shape_of(row_units(row_elems, dtype), dtype, true, tensors, by_document, 2);
            int64_t per_group, ctas;
            deal(T, s, device, per_group, ctas);
            const int64_t rows = 2 * ctas + (by_document ? 2 * ctas * (s.threads / s.group) : 0);
            if (rows > most) most = rows;
        }
    }
    return most * row_elems * 4;
}

cudaError_t launch_residual_norm_backward(ResidualParams p, int dtype, void *workspace, int device, cudaStream_t stream)
{
    p.units = row_units(p.row_elems, dtype);
    p.per_column = 1.0f / static_cast<float>(p.row_elems);
    const bool need_h = p.post != nullptr || p.gate_kind != 0;
    p.tensors = (p.x != nullptr) + 2 * (p.pre != nullptr) + need_h + (p.gate_kind == kGateToken);
    const int f = asked(p, p.n != nullptr);
    const Shape s = shape_of(p.units, dtype, true, p.tensors, p.gate_kind == kGateDocument, f);
    p.group = s.group;
    p.hold = s.hold;
    int64_t ctas;
    deal(p.T, s, device, p.per_group, ctas);
    p.parts = static_cast<int32_t>(ctas);
    p.part_post = static_cast<float *>(workspace);
    p.part_pre = p.part_post + static_cast<int64_t>(p.parts) * p.row_elems;
    p.part_gate = p.part_pre + static_cast<int64_t>(p.parts) * p.row_elems;
    if (p.T > 0) {
        p.stages = s.shorter ? 0 : stages_of(s, dtype, p.tensors, p.gate_kind == kGateDocument);
        const unsigned grid = static_cast<unsigned>(ctas);
        const cudaError_t e = dtype == kBf16 ? launch_backward<true>(p, s, f, grid, device, stream)
                                             : launch_backward<false>(p, s, f, grid, device, stream);
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

cudaError_t read_residual_backward_wait_timeouts(unsigned int *count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_wait_timeouts, sizeof(unsigned int));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(unsigned int));
    }
    return e;
}

cudaError_t read_residual_backward_bounds_violations(unsigned int *count, bool reset)
{
    return read_bounds_counter(count, reset);
}

}  // namespace cpt

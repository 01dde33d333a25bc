// The residual stream between two blocks, forward: y = x + scale drop(norm(h) gate), n = norm(y). Mathematics, layout and
// reasons: residual_norm.cuh.
//
// 262144 x 2560 bf16 with both norms and dropout takes 866 us (6.20 TB/s, 0.91 of a copy). What bounds it: HBM, with issue slots half busy.
#include "residual_norm.cuh"

namespace cpt {

namespace {

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
        if (sum(s)) return;
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
    if (sum(s)) return;
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

template <bool BF16, int U, int F>
__global__ void __launch_bounds__(kShortThreads) residual_norm_short_kernel(const __grid_constant__ ResidualParams p)
{
    constexpr int E = Unit<BF16>::E;
    typedef Asked<F> A;
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
        if (A::gate(p) == kGateDocument) {
            doc.enter(p, r.token);
            gate_base = static_cast<int64_t>(doc.at) * p.units + lane;
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (!has.at[k]) continue;
            r.t[0][k] = load_unit(p.x, base + k * p.group);
            if (A::block(p.h != nullptr)) r.t[1][k] = load_unit(p.h, base + k * p.group);
            if (A::gate(p) == kGateToken) r.t[2][k] = load_unit(p.gate, base + k * p.group);
            else if (A::gate(p) == kGateDocument) r.t[2][k] = reinterpret_cast<const uint4 *>(p.gate)[gate_base + k * p.group];
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
        forward_row<BF16, U, F>(
            p, has, HeldWeights<BF16, U>{w1}, HeldWeights<BF16, U>{w2}, [&](int k) { return r.t[0][k]; },
            [&](int k) { return r.t[1][k]; }, [&](int k) { return r.t[2][k]; },
            [&](uint32_t(&bits)[U][E / 2]) { short_bits<BF16, U>(p, key, static_cast<uint32_t>(r.token), lane, bits); },
            [&](float(&v)[1]) {
                lanes_sum<1>(v, p.group);
                return false;
            },
            [&](int k, bool there, uint4 v) { store_unit_if(in && there, p.y, at + k * p.group, real ? v : make_uint4(0, 0, 0, 0)); },
            [&](int k, bool there, uint4 v) { store_unit_if(in && there, p.n, at + k * p.group, real ? v : make_uint4(0, 0, 0, 0)); });
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
    walk<kApart>(ring, sum, count, p.tensors, row_bytes, p.stall, base, token_of, row_of, [&](int64_t i, int32_t token, auto after) {
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
        if (token == -1) {   // padding
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
                return sum.stop;
            },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, y + at, k * p.group, v); },
            [&](int k, bool there, uint4 v) { store_unit_if(real && there, n + at, k * p.group, v); });
        if (waiting) {   // no norm, no sum
            sum.stop = team.any(sum.ask);
            after();
        }
    });
}

template <bool BF16>
cudaError_t launch_forward(const ResidualParams &p, const Shape &s, int f, unsigned grid, int device, cudaStream_t stream)
{
    if (s.shorter) {
        return with_asked<false>(f, [&](auto g) {
            constexpr int F = decltype(g)::value;
            if (s.per_thread == 1) residual_norm_short_kernel<BF16, 1, F><<<grid, s.threads, 0, stream>>>(p);
            else residual_norm_short_kernel<BF16, 2, F><<<grid, s.threads, 0, stream>>>(p);
            return cudaGetLastError();
        });
    }
    constexpr int U = BF16 ? 1 : 2;   // units of eight columns
    auto run = [&](auto kernel) {
        const cudaError_t e = allow_shared<decltype(kernel)::value>(device);
        if (e != cudaSuccess) return e;
        decltype(kernel)::value<<<grid, s.threads, shared_bytes(p, s, BF16 ? kBf16 : kF32, false), stream>>>(p);
        return cudaGetLastError();
    };
    return with_asked<true>(f, [&](auto g) {
        constexpr int F = decltype(g)::value;
        if (s.per_thread == 2 * U) return run(Kernel<residual_norm_long_kernel<BF16, 2 * U, F>>());
        if (s.per_thread == 3 * U) return run(Kernel<residual_norm_long_kernel<BF16, 3 * U, F>>());
        return run(Kernel<residual_norm_long_kernel<BF16, 5 * U, F>>());
    });
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
    const int f = asked(p, p.h != nullptr);
    return dtype == kBf16 ? launch_forward<true>(p, s, f, grid, device, stream) : launch_forward<false>(p, s, f, grid, device, stream);
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

// Dropout whose mask is a function of the token and the column.
//
// Mathematics. Element (g, c) is kept when its 16 bits of the generator are below `kept` and
// then multiplied by 2^16 / kept. Sixteen bits hold a probability to 2^-17; the factor is that of the
// probability held, so the expectation is exact. One generator call serves the eight columns of a
// 16-byte unit of bf16.
//
// HBM bounds it: every row is read and written once, units one after the other, four of every
// thread in flight.
#include "cpt_internal.h"
#include "token_rows.cuh"

namespace cpt {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <bool BF16>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutParams p)
{
    constexpr int N = UnitPairs<BF16>::N;
    const F2 factor = pair_of(p.rule.factor, p.rule.factor);
    DropKey key;
    key.load(p.rule);
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads;
    int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    int64_t row = i / p.units;
    uint32_t unit = static_cast<uint32_t>(i - row * p.units);
    const int64_t items = p.rows * p.units;
    for (; i < items; i += stride * kUnroll) {
        uint4 raw[kUnroll];
        int32_t token[kUnroll];
        uint32_t at[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t j = i + k * stride;
            token[k] = -1;
            at[k] = unit;
            if (j < items) {
                raw[k] = __ldcs(reinterpret_cast<const uint4 *>(p.src) + j);
                token[k] = p.token_of_row == nullptr ? static_cast<int32_t>(row) : p.token_of_row[row];
            }
            row += p.step_rows;
            unit += p.step_units;
            if (unit >= static_cast<uint32_t>(p.units)) {
                unit -= p.units;
                ++row;
            }
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t j = i + k * stride;
            if (j >= items) continue;
            uint4 out = raw[k];
            if (token[k] < 0) {   // padding
                out = make_uint4(0, 0, 0, 0);
            } else if (p.rule.rng != nullptr) {
                F2 x[N];
                UnitPairs<BF16>::unpack(raw[k], x);
                uint32_t bits[N];
                unit_bits<BF16>(p.rule, key, static_cast<uint32_t>(token[k]), at[k], bits);
                keep_or_zero<N>(p.rule, bits, x);
#pragma unroll
                for (int n = 0; n < N; ++n) x[n] = mul2(x[n], factor);
                out = UnitPairs<BF16>::pack(x);
            }
            __stcs(reinterpret_cast<uint4 *>(p.dst) + j, out);
        }
    }
}

}  // namespace

cudaError_t launch_dropout(DropoutParams p, int dtype, cudaStream_t stream)
{
    const int64_t items = p.rows * p.units;
    if (items == 0) return cudaSuccess;
    const int64_t ctas = (items + kThreads * kUnroll - 1) / (kThreads * kUnroll);
    const int64_t most = 8 * static_cast<int64_t>(sm_count(-1));
    const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
    const int64_t stride = static_cast<int64_t>(grid) * kThreads;
    p.step_rows = stride / p.units;
    p.step_units = static_cast<int32_t>(stride % p.units);
    if (dtype == kBf16) dropout_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else dropout_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace cpt

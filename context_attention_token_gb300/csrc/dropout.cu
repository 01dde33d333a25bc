// Dropout whose mask is a function of the token and the column.
//
// Mathematics. Element (g, c) is kept when its 16 bits of the generator are below `kept` and
// then multiplied by 2^16 / kept. Sixteen bits hold a probability to 2^-17; the factor is that of the
// probability held, so the expectation is exact. One generator call serves the eight columns of a
// 16-byte unit of bf16.
//
// HBM bounds it: every row is read and written once. A CTA takes a tile of neighbouring units, four of every
// thread in flight. 131071 x 2048 bf16 (padded) takes 172 us, 6.25 TB/s, 0.92 of a copy; with a loop over the grid 181, with a
// key schedule for every unit 195.
#include "cpt_internal.h"
#include "token_rows.cuh"

namespace cpt {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kTile = kThreads * kUnroll;   // units of a CTA, neighbours

template <bool BF16>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutParams p)
{
    constexpr int N = UnitPairs<BF16>::N;
    const F2 factor = pair_of(p.rule.factor, p.rule.factor);
    DropKey key;
    key.load(p.rule);
    const int64_t start = static_cast<int64_t>(blockIdx.x) * kTile;
    const uint32_t here = static_cast<uint32_t>(min(p.rows * p.units - start, static_cast<int64_t>(kTile)));
    const uint4 *from = reinterpret_cast<const uint4 *>(p.src) + start;
    uint4 *to = reinterpret_cast<uint4 *>(p.dst) + start;
    uint4 raw[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const uint32_t i = threadIdx.x + k * kThreads;
        if (i < here) raw[k] = __ldcs(from + i);
    }
    const int64_t row0 = start / p.units;
    const uint32_t units = static_cast<uint32_t>(p.units), skip = static_cast<uint32_t>(start - row0 * p.units);
    uint32_t token[kUnroll], unit[kUnroll], bits[kUnroll][N];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const uint32_t i = min(threadIdx.x + k * kThreads, here - 1);
        const uint32_t q = (skip + i) / units;
        unit[k] = skip + i - q * units;
        token[k] = static_cast<uint32_t>(p.token_of_row == nullptr ? row0 + q : p.token_of_row[row0 + q]);
    }
    if (p.rule.rng != nullptr) unit_bits<BF16, kUnroll>(p.rule, key, token, unit, bits);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
        const uint32_t i = threadIdx.x + k * kThreads;
        if (i >= here) continue;
        uint4 out = raw[k];
        if (p.rule.rng != nullptr) {
            F2 x[N];
            UnitPairs<BF16>::unpack(raw[k], x);
            keep_or_zero<N>(p.rule, bits[k], x);
#pragma unroll
            for (int n = 0; n < N; ++n) x[n] = mul2(x[n], factor);
            out = UnitPairs<BF16>::pack(x);
        }
        if (static_cast<int32_t>(token[k]) < 0) out = make_uint4(0, 0, 0, 0);   // padding
        __stcs(to + i, out);
    }
}

}  // namespace

cudaError_t launch_dropout(const DropoutParams &p, int dtype, cudaStream_t stream)
{
    const int64_t items = p.rows * p.units;
    if (items == 0) return cudaSuccess;
    const int64_t ctas = (items + kTile - 1) / kTile;
    if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(ctas);
    if (dtype == kBf16) dropout_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else dropout_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace cpt

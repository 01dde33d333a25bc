// Tensor memory, tcgen05 matrix instructions, tiled TMA loads and bounded
// barrier waits: the pieces of the attention kernels, in inline PTX.
//
// Conventions of these kernels. Tiles are bf16 with 128-byte swizzled rows
// of 64 elements ("slabs" of 128 rows, 16 KB); a head of more than 64 elements
// is two slabs. The first operand has 128 rows; it comes from shared memory
// (its inner dimension contiguous) or from tensor memory. The second has its
// inner dimension contiguous (scores) or its outer one (products with V, K, Q
// and dO, which are read as they lie).
#pragma once

#include <cuda.h>

#include "cpt_device.cuh"

namespace cpt {

constexpr int kTile = 128;                 // rows of every tile
constexpr uint32_t kSlab = 128 * 128;      // bytes of 128 rows x 64 bf16

// ----------------------------------------------------------------- descriptors

// Shared-memory operand with 128-byte swizzle whose inner dimension is
// contiguous: groups of 8 rows are 1024 bytes apart. The address is made opaque:
// with nvcc 13.0 a tile at a constant shared address got wrong bits once sums
// with it were folded into constants.
constexpr uint32_t kInnerUpper = 64u | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t inner_lower(uint32_t addr)
{
    asm volatile("" : "+r"(addr));
    return (addr >> 4) | (1u << 16);
}

// The same bytes read across: the outer dimension contiguous in blocks of 64
// one slab apart, groups of 8 inner rows 1024 bytes apart.
constexpr uint32_t kOuterUpper = kInnerUpper;

__device__ __forceinline__ uint32_t outer_lower(uint32_t addr)
{
    asm volatile("" : "+r"(addr));
    return (addr >> 4) | ((kSlab >> 4) << 16);
}

// bf16 x bf16 into binary32, 128 rows, n columns (a multiple of 16).
__device__ __forceinline__ uint32_t mma_shape(uint32_t n, bool b_outer)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_outer ? 1u << 16 : 0u) | ((n >> 3) << 17) | (8u << 24);
}

// ----------------------------------------------------------------- matrix instructions

// The whole warp runs the issuing code, so that addresses and descriptors stay
// in uniform registers; one lane issues, elected (the same one every time) for a
// run of instructions. With a predicate on each instruction instead an
// instruction took 88 cycles to issue next to the softmax, against 74 so.

__device__ __forceinline__ bool elect_lane()
{
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

// Descriptors come as two words: the lower one moves with the address, the
// upper one is constant.

__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t upper,
                                         uint32_t shape, bool add)
{
    asm volatile(
        "{ .reg .pred p; .reg .b64 a, b; mov.b64 a, {%1, %3}; mov.b64 b, {%2, %3};\n"
        "setp.ne.b32 p, %5, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(upper), "r"(shape), "r"(add ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t upper,
                                         uint32_t shape, bool add)
{
    asm volatile(
        "{ .reg .pred p; .reg .b64 b; mov.b64 b, {%2, %3};\n"
        "setp.ne.b32 p, %5, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(upper), "r"(shape), "r"(add ? 1u : 0u)
        : "memory");
}

// A product of 128 x 128 x 16 takes 64 cycles, and a warp can run ahead of the
// matrix unit by about two of them. So that they follow one another without
// gaps while the softmax takes its share of the issue slots, loops are unrolled
// and descriptors advance by constants (with address arithmetic in the loop an
// instruction took 100 cycles to issue, with a loop of four 75), and commits,
// which cost some 20 cycles each, are few: one commit stands for everything that
// its warp issued before it.

// Rows x columns of scores: both operands from shared memory, `steps` (at most
// 8) inner steps of 16, four to a slab. STEPS, unless 0, is their number: code
// for others in the same kernel costs it 2 to 6 %.
template <int STEPS>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, int steps)
{
    const uint32_t da = inner_lower(a), db = inner_lower(b);
    if (elect_lane()) {
#pragma unroll
        for (int k = 0; k < (STEPS ? STEPS : 8); ++k) {
            const uint32_t at = ((k >> 2) * kSlab + (k & 3) * 32) >> 4;
            if (STEPS || k < steps) mma_smem(d, da + at, db + at, kInnerUpper, shape, k > 0);
        }
    }
}

// d (+)= A B over RUNS x STEPS inner steps of 16: A from tensor memory, 8 columns
// a step, B read across. A run begins a_gap columns and b_gap bytes behind the
// one before.
template <int RUNS, int STEPS>
__device__ __forceinline__ void mma_weights(uint32_t d, uint32_t a, uint32_t a_gap, uint32_t b, uint32_t b_gap,
                                            uint32_t shape, bool add)
{
    const uint32_t db = outer_lower(b);
    if (elect_lane()) {
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
#pragma unroll
            for (int k = 0; k < STEPS; ++k)
                mma_tmem(d, a + r * a_gap + 8 * k, db + r * (b_gap >> 4) + k * (2048 >> 4), kOuterUpper, shape,
                         r > 0 || k > 0 || add);
    }
}

// An arrival on `bar` once every matrix instruction issued so far by this
// thread has completed (and an arrival on behalf of its reads of shared memory).
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    if (elect_lane())
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                     : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ----------------------------------------------------------------- tensor memory

// All 512 columns, by one warp; the kernels that call this run one CTA per SM.
__device__ __forceinline__ void tmem_alloc(uint32_t *to)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(to)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t addr)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
}

#define CPT_R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define CPT_R16(a, i) CPT_R4(a, i), CPT_R4(a, i + 4), CPT_R4(a, i + 8), CPT_R4(a, i + 12)
#define CPT_RR4(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3])
#define CPT_RR16(a, i) CPT_RR4(a, i), CPT_RR4(a, i + 4), CPT_RR4(a, i + 8), CPT_RR4(a, i + 12)
#define CPT_IN4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
#define CPT_IN16(a, i) CPT_IN4(a, i), CPT_IN4(a, i + 4), CPT_IN4(a, i + 8), CPT_IN4(a, i + 12)

// 32 neighbouring columns of this thread's lane. The values are there
// only after tmem_wait_loads has taken the array.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : CPT_R16(r, 0), CPT_R16(r, 16)
        : "r"(addr));
}

__device__ __forceinline__ void tmem_wait_loads(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : CPT_RR16(r, 0), CPT_RR16(r, 16)::"memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        CPT_IN16(r, 0)
        : "memory");
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), CPT_IN4(r, 0),
        CPT_IN4(r, 4)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ----------------------------------------------------------------- TMA

// A box of 64 elements of one head in 128 neighbouring rows; rows and elements
// outside the tensor arrive as zeros.
__device__ __forceinline__ void tma_slab(uint32_t to, const CUtensorMap *map, int at, int head, int row,
                                         uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(to),
        "l"(map), "r"(at), "r"(head), "r"(row), "r"(smem_addr(bar))
        : "memory");
}

// ----------------------------------------------------------------- barriers

__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Waits of a kernel whose roles wait on one another: each gives up after
// about a second (`limit` times that, at most 128), or as soon as another has given
// up (*stop, in shared memory). The role then leaves its loop; the CTA ends without further work.
__device__ __forceinline__ bool mbar_wait_slow(uint64_t *bar, uint32_t parity, volatile uint32_t *stop, uint32_t limit)
{
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0; it < (limit << 24); ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*stop != 0) return false;
        if (global_timer_ns() - t0 > limit * 1000000000ull) break;
    }
    *stop = 1;
    return false;
}

__device__ __forceinline__ bool mbar_wait_or_stop(uint64_t *bar, uint32_t parity, volatile uint32_t *stop,
                                                  uint32_t limit = 1)
{
    if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_slow(bar, parity, stop, limit);
}

// ----------------------------------------------------------------- grids in order

// See launch_after. All memory operations of the last grid are visible behind the
// wait; without that launch both end at once.
__device__ __forceinline__ void wait_for_last_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void next_grid_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ----------------------------------------------------------------- arithmetic

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;   // relative error 2^-22, exact zero for -inf
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two binary32 values in one register pair, and their arithmetic (round to
// nearest): one issue slot for two elements.
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 pair_of(uint32_t a, uint32_t b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ F2 pair_of(float a, float b) { return pair_of(__float_as_uint(a), __float_as_uint(b)); }

__device__ __forceinline__ float2 both(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// Registers of a warpgroup: given back, or taken from what others gave back.
template <int N>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The bits of columns [lo, hi) of a 128-column tile in its 32-column word w.
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int w)
{
    const int a = min(max(lo - 32 * w, 0), 32), b = min(max(hi - 32 * w, 0), 32);
    return static_cast<uint32_t>((1ull << b) - 1) & ~static_cast<uint32_t>((1ull << a) - 1);
}

// ----------------------------------------------------------------- rows out
//
// Every lane holds one row of an accumulator. Written as they are, 16 bytes of 32
// rows at a time, rows cost 32 wavefronts an instruction (5000 cycles for a
// tile of 128 x 128). So four lanes exchange their 16-byte units first and
// write 64 neighbouring bytes of a row together.

// Columns [32 block, 32 block + 32) below D of this warp's 32 rows: scaled,
// rounded to bf16 and written where `write` holds; zeros where `live` does not.
// `bad` becomes NaN once a value is not finite.
__device__ __forceinline__ void store_block(uint32_t tmem, int block, int D, float scale, bool live, uint16_t *row,
                                            bool write, float &bad)
{
    const int lane = threadIdx.x & 31;
    uint32_t o[32];
    tmem_load32(tmem + 32 * block, o);
    tmem_wait_loads(o);
    uint4 u[4];
    const F2 zero = pair_of(0.0f, 0.0f), by = pair_of(scale, scale);
    F2 odd[4] = {zero, zero, zero, zero};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const F2 x = mul2(pair_of(o[8 * i + 2 * j], o[8 * i + 2 * j + 1]), by);
            odd[i] = fma2(x, zero, odd[i]);
            const float2 v = both(x);
            w[j] = live ? pack_bf16x2(v.x, v.y) : 0;
        }
        u[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = both(odd[i]);
        if (32 * block + 8 * i < D) sum += v.x + v.y;
    }
    if (live) bad += sum;
    auto swap = [&](uint4 &low, uint4 &high, int bit) {   // lanes without the bit keep `low`, the others `high`
        const bool upper = (lane & bit) != 0;
        uint4 s = upper ? low : high;
        s.x = __shfl_xor_sync(0xFFFFFFFFu, s.x, bit);
        s.y = __shfl_xor_sync(0xFFFFFFFFu, s.y, bit);
        s.z = __shfl_xor_sync(0xFFFFFFFFu, s.z, bit);
        s.w = __shfl_xor_sync(0xFFFFFFFFu, s.w, bit);
        if (upper) low = s;
        else high = s;
    };
    swap(u[0], u[1], 1);
    swap(u[2], u[3], 1);
    swap(u[0], u[2], 2);
    swap(u[1], u[3], 2);
    const int at = 32 * block + 8 * (lane & 3);
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // unit lane & 3 of row k of the four
        const int from = (lane & ~3) + k;
        const unsigned long long to = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(row), from);
        const bool ok = __shfl_sync(0xFFFFFFFFu, write ? 1 : 0, from) != 0;
        if (ok && at < D) *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(to) + at) = u[k];
    }
}

}  // namespace cpt

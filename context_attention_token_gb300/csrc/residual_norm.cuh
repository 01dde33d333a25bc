// The residual stream between two blocks, and its gradient: what both directions share.
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
// HBM is the floor of both, every row of every tensor read or written once; issue slots come close to it, since the generator of
// dropout alone costs some 70 instructions for 8 columns. So arithmetic is on pairs of columns, and what is the same for a
// row is spread over many columns of a thread.
//
// Rows of up to 64 units of 16 bytes take a part of a warp each (sums by shuffles), loads one row ahead in registers.
// Longer ones take a team of a few warps with a barrier of its own; its rows come through a ring in shared memory,
// filled by the bulk-copy engine, and the weights stand there once for all teams of the SM's only CTA. Measured for 262144 x 2560
// bf16 with both norms and dropout: CTAs of 320 threads that load into registers 2543 us, a ring for each 1336, a CTA's weights
// from the cache and two rows at a time 1069, teams of 64 threads with 40 columns each 907, stores under predicates 864
// (866 to 869 since a row that could not be waited for is not stored).
#pragma once

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

// CTAs of short rows that an SM holds, in the gradient: those that ask for little have few sums.
constexpr int short_ctas(int per_thread, int f) { return (f == 2 || f == 34 ? 6 : 4) / per_thread; }

// Weights in shared memory: two rows of them, every thread's units whole.
inline int64_t weight_bytes(const Shape &s, int dtype) { return !s.hold ? 0 : 2 * s.per_thread * s.group * (dtype == kBf16 ? 8 : 4) * 4; }

// tensors: those that are read; f: what is asked (below).
inline Shape shape_of(int units, int dtype, bool gradient, int tensors, bool by_document = false, int f = 2)
{
    Shape s;
    s.shorter = units <= 64;
    s.hold = false;
    if (s.shorter) {
        s.per_thread = units > 32 ? 2 : 1;
        s.group = 1;
        while (s.group * s.per_thread < units) s.group *= 2;
        s.threads = kShortThreads;
        s.ctas_per_sm = short_ctas(s.per_thread, f);
        return s;
    }
    const int eights = dtype == kBf16 ? units : (units + 1) / 2;   // groups of eight columns
    // (of a thread; 2560 columns are 64 threads of 5 exactly, 2048 and 4096 leave a fifth of them idle: 131072 x 4096 bf16 takes 1.35 times
    // its bytes' time, 2048 columns 1.12, 2560 1.10)
    const int wide = gradient || eights <= 128 ? 2 : eights <= 192 ? 3 : 5;
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
inline int stages_of(const Shape &s, int dtype, int tensors, bool by_document)
{
    const int64_t row = static_cast<int64_t>(s.threads / s.group) * s.per_thread * s.group * 16;
    const int64_t n = (kSharedBytes - kOwnBytes - weight_bytes(s, dtype) - (by_document ? row : 0)) / (row * tensors);
    return static_cast<int>(n > kMaxStages ? kMaxStages : n);
}

// The document of a raw token: the last d with cu[d] <= t.
__device__ __forceinline__ int document_of(const int32_t *cu, int n, int32_t t)
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

// What a call asks for, known to the compiler (F >= 0: bits 0 post norm, 1 pre norm, 2 dropout, 3 and 4 the kind of
// gate, 5 no block's output) or read from the parameters (F = -1).
template <int F>
struct Asked {
    static __device__ __forceinline__ bool post(const ResidualParams &p) { return F < 0 ? p.post != nullptr : F & 1; }
    static __device__ __forceinline__ bool pre(const ResidualParams &p) { return F < 0 ? p.pre != nullptr : F & 2; }
    static __device__ __forceinline__ bool drop(const ResidualParams &p) { return F < 0 ? p.rule.rng != nullptr : F & 4; }
    static __device__ __forceinline__ int gate(const ResidualParams &p) { return F < 0 ? p.gate_kind : F >> 3 & 3; }
    static __device__ __forceinline__ bool block(bool there) { return F < 0 ? there : !(F & 32); }
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

// The document that tokens are in, looked for when it changes.
struct Document {
    int at = 0;
    int32_t lo = 0, hi = -1;   // its tokens
    __device__ __forceinline__ bool enter(const ResidualParams &p, int32_t token)
    {
        if (token >= lo && token < hi) return false;
        if (token == hi && at + 1 < p.n_docs && p.cu[at + 2] > token) ++at;   // the next one, mostly
        else at = document_of(p.cu, p.n_docs, token);
        lo = p.cu[at];
        hi = p.cu[at + 1];
        return true;
    }
};

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
    __device__ __forceinline__ uint4 *row() const { return reinterpret_cast<uint4 *>(smem + slot * stage_bytes); }
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

static __device__ unsigned int g_wait_timeouts;   // of this translation unit

constexpr int32_t kUnknown = -2;   // a row's index for a thread whose wait has run out: it uses and stores nothing of the row

// How a warp's lanes come to the same index, kUnknown where one lane's wait has run out, whatever the others saw. Needed where
// `work` parts by the index around full-warp shuffles, as the gradient's does: a lane would wait for ever for one that went the
// other way. The forward call's parts by it in stores only, and a vote costs the forward kernel that looks at its
// parameters 3 to 5 %. The gradient's kernels of their own are best with a vote (131072 x 2048 bf16, both norms, dropout: 557 us, 581 with
// the minimum), the shared one with the minimum, which is uniform (131072 x 2560 bf16, a post norm and dropout: 1188 us, 1423 with a
// vote; both before the dh of dropped infinities was looked after, which takes 50 more).
enum Together { kApart, kVote, kMinimum };

// Runs `work(i, index, after)` for i = 0 .. count - 1 with the i-th row's data in the ring. It has to call after() once behind its
// first barrier, where every thread is done with the row before; `sum` votes there whether a wait has run
// out, and then nothing that depends on other threads' data may be stored. (Int: 64 bits forward, where 32 make the compiler's
// schedule 4 % slower; 32 in the gradient, which is short of registers.) index_of(i) looks the i-th row up (-1: it is not read),
// row_of(i, index) is its place in this lane's tensor, `base`.
template <Together TOGETHER, class Int, class Sum, class Index, class RowOf, class Work>
__device__ __forceinline__ void walk(Ring &ring, Sum &sum, Int count, int tensors, uint32_t row_bytes, uint32_t stall,
                                     const uint8_t *base, Index index_of, RowOf row_of, Work work)
{
    const int lane = sum.team.thread & 31;
    const bool first = sum.team.thread < 32, several = ring.stages > 1;
    Int issued = 0;
    int put = 0;
    int32_t ahead = first ? index_of(0) : -1;   // looked up a row early
    auto issue = [&]() {   // by the first warp
        if (issued >= count) return;
        uint64_t *bar = &ring.full[put];
        if (lane == 0) {
            ring.index[put] = ahead;
            mbar_expect_tx(bar, ahead >= 0 ? static_cast<uint32_t>(tensors) * row_bytes + stall : 0);
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
    for (Int i = 0; i < count; ++i) {
        bool come = mbar_wait_bounded(&ring.full[ring.slot], ring.phase);
        if (TOGETHER == kVote) come = __all_sync(0xFFFFFFFFu, come);
        if (!come) sum.ask = true;
        int32_t at = come ? ring.index[ring.slot] : kUnknown;
        if (TOGETHER == kMinimum) at = __reduce_min_sync(0xFFFFFFFFu, at);
        work(i, at, [&]() {
            if (several && first && i > 0) issue();   // into the place of the row before
        });
        if (!several) {
            sum.stop = sum.team.any(sum.ask);
            if (first && !sum.stop) issue();
        }
        if (sum.stop) {   // by all: no copy may end in another CTA's shared memory
            if (first) {
                if (lane == 0) atomicAdd(&g_wait_timeouts, 1u);
                // (one wait that runs out here has given every copy in flight its second)
                for (Int k = i; k < issued && mbar_wait_bounded(&ring.full[ring.slot], ring.phase); ++k) ring.advance();
            }
            return;
        }
        ring.advance();
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

// ----------------------------------------------------------------- launching

inline int row_units(int64_t row_elems, int dtype) { return static_cast<int>(row_elems * (dtype == kBf16 ? 2 : 4) / 16); }

inline size_t shared_bytes(const ResidualParams &p, const Shape &s, int dtype, bool gate)
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

// What a call asks for, as Asked has it, or -1 for what has no kernel of its own.
inline int asked(const ResidualParams &p, bool block)
{
    return block ? (p.post != nullptr) + 2 * (p.pre != nullptr) + 4 * (p.rule.rng != nullptr) + 8 * p.gate_kind : 34;
}

// Kernels of their own for both norms, with any gate (long rows only); for the pre norm alone, without one; each with and
// without dropout; for the first norm of a model. The others (a gate without a post norm, no pre norm, short rows with a
// gate) share one that looks at its parameters and spills.
// (262144 x 2560 bf16 with both norms and dropout: 866 us with its own kernel, 1184 with the shared one; gradient of 131071 x 2560
// bf16, a document's gate too, 915 and 1707; of 20011 x 1132 float32 with a token's gate 138 and 208. What has none: the pre norm
// with a document's gate and dropout, 262144 x 2560 bf16, takes 1269 us where its bytes take 791, its gradient of 131072 rows 1239 for 593.)
template <bool GATES, class Launch>
cudaError_t with_asked(int f, Launch launch)
{
    switch (f) {
    case 2: return launch(std::integral_constant<int, 2>());
    case 3: return launch(std::integral_constant<int, 3>());
    case 6: return launch(std::integral_constant<int, 6>());
    case 7: return launch(std::integral_constant<int, 7>());
    case 34: return launch(std::integral_constant<int, 34>());
    default: break;
    }
    if constexpr (GATES) {
        switch (f) {
        case 11: return launch(std::integral_constant<int, 11>());
        case 15: return launch(std::integral_constant<int, 15>());
        case 19: return launch(std::integral_constant<int, 19>());
        case 23: return launch(std::integral_constant<int, 23>());
        default: break;
        }
    }
    return launch(std::integral_constant<int, -1>());
}

// A kernel as a type.
template <void (*K)(ResidualParams)>
struct Kernel {
    static constexpr auto value = K;
};

// Rows of a group, and the CTAs.
inline void deal(int64_t T, const Shape &s, int device, int64_t &per_group, int64_t &ctas)
{
    const int64_t groups = s.threads / s.group;
    const int64_t most = static_cast<int64_t>(sm_count(device)) * s.ctas_per_sm * groups;
    per_group = (T + most - 1) / most;
    if (per_group < 1) per_group = 1;
    ctas = (T + per_group * groups - 1) / (per_group * groups);
}

}  // namespace

}  // namespace cpt

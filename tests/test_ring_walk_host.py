"""The walk over a ring of rows in shared memory, its source run by threads of the host.

Every thread of a team waits for a row's copy by itself, for a bounded time. Full-warp shuffles follow, so lanes of a warp that
part over whether a copy has come would wait for one another for ever. Here a wait runs out for chosen lanes while the others'
copy comes: every warp has to go on as one, and the team has to stop at the barrier behind.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = r"""
#include <barrier>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline

constexpr int kThreads = 64, kCount = 12;
struct Warp {
    std::barrier<> meet{32};
    int32_t values[32];
};
struct Place { uint32_t a, b, c, d; };
typedef Place uint4;
static uint4 make_uint4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return {a, b, c, d}; }

static std::barrier<> cta(kThreads);
static Warp warps[2];
static thread_local int self;
static thread_local int waits;
static int fail_warp, fail_lanes, fail_row;   // whose wait runs out, and which one
static bool team_votes[kThreads];

static void __syncthreads() { cta.arrive_and_wait(); }
static void __syncwarp() { warps[self / 32].meet.arrive_and_wait(); }
static bool __all_sync(uint32_t, bool v)
{
    Warp &w = warps[self / 32];
    w.values[self % 32] = v;
    w.meet.arrive_and_wait();
    for (int32_t x : w.values) v = v && x;
    w.meet.arrive_and_wait();
    return v;
}
static int32_t __reduce_min_sync(uint32_t, int32_t v)
{
    Warp &w = warps[self / 32];
    w.values[self % 32] = v;
    w.meet.arrive_and_wait();
    for (int32_t x : w.values) v = x < v ? x : v;
    w.meet.arrive_and_wait();
    return v;
}
static unsigned atomicAdd(unsigned *p, unsigned v) { return __atomic_fetch_add(p, v, __ATOMIC_SEQ_CST); }

struct Team {
    int thread, threads, barrier;
    bool any(bool ask) const
    {
        team_votes[thread] = ask;
        cta.arrive_and_wait();
        bool r = false;
        for (bool x : team_votes) r = r || x;
        cta.arrive_and_wait();
        return r;
    }
};
// A barrier counts its completed phases; copies come at once, so a phase is complete when its bytes have been announced.
static void mbar_init(uint64_t *bar, int) { __atomic_store_n(bar, 0, __ATOMIC_RELEASE); }
static void mbar_init_fence() {}
static void mbar_expect_tx(uint64_t *bar, uint32_t) { __atomic_fetch_add(bar, 1, __ATOMIC_RELEASE); }
static void bulk_load(void *, const void *, uint32_t, uint64_t *) {}
static bool mbar_wait_bounded(uint64_t *bar, uint32_t parity)
{
    const bool fails = self / 32 == fail_warp && (fail_lanes >> (self % 32) & 1) && waits == fail_row;
    ++waits;
    if (fails) return false;
    for (int i = 0; i < 10000000; ++i) {
        if ((__atomic_load_n(bar, __ATOMIC_ACQUIRE) & 1) != parity) return true;
        std::this_thread::yield();
    }
    return false;
}
static unsigned g_wait_timeouts;

//RING

struct Sum {
    Team team;
    bool stop = false, ask = false;
};

int main(int argc, char **argv)
{
    const int stages = atoi(argv[1]);
    fail_warp = atoi(argv[2]);
    fail_lanes = static_cast<int>(strtoul(argv[3], nullptr, 0));
    fail_row = atoi(argv[4]);
    static uint8_t smem[8 * 64], base[kCount * 16 + 16];
    static uint64_t full[8];
    static int32_t index[8];
    static int seen[kThreads][kCount];
    for (auto &t : seen) for (int &x : t) x = -9;
    std::vector<std::thread> threads;
    for (int t = 0; t < kThreads; ++t)
        threads.emplace_back([&, t] {
            self = t;
            Sum sum = {Team{t, kThreads, 1}};
            Ring ring = {smem, full, index, stages, 16, 16};
            walk<TOGETHER>(ring, sum, kCount, 1, 16u, 0u, base, [](int i) { return i < kCount ? i : -1; }, [](int i, int32_t) { return i; },
                 [&](int i, int32_t row, auto after) {
                     seen[t][i] = row;
                     sum.stop = sum.team.any(sum.ask);
                     after();
                 });
        });
    for (auto &t : threads) t.join();
    for (int w = 0; w < 2; ++w)
        for (int i = 0; i < kCount; ++i)
            for (int l = 1; l < 32; ++l)
                if (seen[w * 32 + l][i] != seen[w * 32][i]) return printf("warp %d parts at row %d\n", w, i), 2;
    for (int t = 0; t < kThreads; ++t)
        for (int i = 0; i < kCount; ++i) {
            const bool lost = t / 32 == fail_warp && fail_lanes != 0 && i == fail_row;
            const int want = fail_lanes != 0 && i > fail_row ? -9 : lost ? kUnknown : i;
            if (seen[t][i] != want) return printf("thread %d, row %d: %d, not %d\n", t, i, seen[t][i], want), 3;
        }
    if (g_wait_timeouts != (fail_lanes != 0)) return printf("%u give-ups\n", g_wait_timeouts), 4;
    puts("ok");
    return 0;
}
"""


@pytest.fixture(scope="module", params=["kVote", "kMinimum"])
def program(request):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    with open(os.path.join(ROOT, "context_attention_token_gb300", "csrc", "residual_norm.cuh")) as f:
        source = f.read()
    ring = re.search(r"^struct Ring \{.*?^\};\n", source, re.S | re.M).group()
    walk = re.search(r"^constexpr int32_t kUnknown.*?^\}\n", source, re.S | re.M).group()
    work = os.path.join(ROOT, "_build", "ring_walk")
    os.makedirs(work, exist_ok=True)
    src, exe = os.path.join(work, "walk.cpp"), os.path.join(work, "walk")
    with open(src, "w") as f:
        f.write(PROGRAM.replace("//RING", ring + walk))
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", f"-DTOGETHER={request.param}", src, "-o", exe], check=True)
    return exe


@pytest.mark.parametrize("stages", [1, 2, 5])
@pytest.mark.parametrize("warp,lanes,row", [(0, 0, 0), (0, 0x20, 0), (1, 0x1, 3), (0, 0x1, 4), (1, 0xFFFF0000, 11), (0, 0xFFFFFFFF, 7)])
def test_a_warp_goes_on_as_one(program, stages, warp, lanes, row):
    out = subprocess.run([program, str(stages), str(warp), str(lanes), str(row)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout

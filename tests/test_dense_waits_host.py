"""The dense kernels' waiting and leaving, without a GPU: the device functions that decide
when a role may leave are taken from their source file, compiled for the host against
barriers and a clock that the test drives, and run."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunked_hierarchical_sparse_b200", "csrc")
DENSE = ("k_dense_fwd_tc.cu", "k_dense_bwd_tc.cu", "k_dense_cache.cu")


def source(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return f.read()


def function(name, file="dense_tc.cuh"):
    """The text of a device function, from its return type to its closing brace."""
    src = source(file)
    m = re.search(r"__device__ __forceinline__ [^;{}]*\b" + name + r"\(", src)
    assert m, f"{file} has no function {name}"
    i = src.index("{", m.end())
    depth = 0
    for j in range(i, len(src)):
        depth += {"{": 1, "}": -1}.get(src[j], 0)
        if depth == 0:
            return src[m.start():j + 1]
    raise AssertionError(name)


# One lane of a warp; time passes only while a wait is polled.  A barrier's phase n is
# complete from when[n] on.
STUBS = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>
using std::max;
#define __device__
#define __forceinline__ inline
typedef unsigned long long ull;
static uint64_t now = 0, tick = 1000;
struct Model { std::vector<uint64_t> when; int arrived = 0; };
static Model model[64];
static uint64_t bars[64];
static int done_phases(uint64_t *b) {
    int n = 0;
    for (uint64_t w : model[b - bars].when) n += w <= now;
    return n;
}
static bool mbar_test(uint64_t *b, uint32_t parity) { return (done_phases(b) & 1) != (int)parity; }
static bool mbar_try(uint64_t *b, uint32_t parity) {
    now += tick;
    return mbar_test(b, parity);
}
static uint64_t globaltimer() { return now; }
static bool mbar_wait(uint64_t *b, uint32_t parity, uint64_t limit) {
    for (const uint64_t t0 = now; !mbar_try(b, parity);)
        if (now - t0 > limit) return false;
    return true;
}
static void mbar_arrive_lane0(uint64_t *b, int lane) { if (lane == 0) ++model[b - bars].arrived; }
static bool __all_sync(unsigned, bool x) { return x; }
static bool __any_sync(unsigned, bool x) { return x; }
static void __syncwarp() {}
static void fence_proxy_async_smem() {}
struct uint4 { unsigned x, y, z, w; };
static uint4 make_uint4(unsigned x, unsigned y, unsigned z, unsigned w) { return {x, y, z, w}; }
static const uint64_t kDrainWaitNs = 2000000000ull;
"""


def run_host(tmp_path, code):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(STUBS + code)
    subprocess.run(["g++", "-std=c++17", "-O1", "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=60).stdout.split()


@pytest.mark.parametrize("stages,issued", [(5, 0), (5, 1), (5, 3), (5, 5), (5, 6), (5, 17), (10, 4), (1, 1), (1, 4), (2, 7)])
def test_a_loader_leaves_after_its_last_loads(tmp_path, stages, issued):
    """The last loads land long after they were issued; nothing else waits for them."""
    out = run_host(tmp_path, function("land") + f"""
int main() {{
    uint64_t last = 0;
    for (int i = 0; i < {issued}; ++i) {{  // the last round of the ring is still in flight
        const uint64_t t = i < {issued} - {stages} ? 0 : 5000000 + 1000 * ((i * 7) % {stages});
        model[i % {stages}].when.push_back(t);
        last = max(last, t);
    }}
    land(bars, {issued}, {stages});
    printf("%d\\n", now >= last);
}}""")
    assert out == ["1"]


@pytest.mark.parametrize("file", DENSE)
def test_loads_and_products_are_awaited_whoever_gave_up(file):
    """Another role's wait may run out after a loader has issued everything: no drain may depend
    on how the loader itself, or the MMA thread, fared."""
    src = source(file)
    assert not re.search(r"if \(!ok[^\n]*\n?[^\n]*(?:kDrainWaitNs|mma_commit\(done\)|land\(|finish_mma\()", src)
    loads = len(re.findall(r"mbar_arrive_expect_tx\(", src))
    assert len(re.findall(r"\bland\(", src)) == loads
    assert len(re.findall(r"\bfinish_mma\(", src)) == len(re.findall(r"tmem_alloc\(", src))


@pytest.mark.parametrize("file,bars", [("k_attend_tc.cu", ["B.q_full[", "B.kv_full[", "mma_done"]),
                                       ("k_bwd_tc.cu", ["qd_full[", "kv_full,", "mma_done"]),
                                       ("k_select_tc.cu", ["q_full", "b_full[", "mma_done"])])
def test_the_sparse_kernels_await_their_loads_too(file, bars):
    """Each barrier that a copy or a product completes is awaited at the end, outside of any `if (!ok)`."""
    src = source(file)
    for bar in bars:
        at = [m.start() for m in re.finditer(r"mbar_wait\(&?" + re.escape(bar) + r"[^;]*kDrainWaitNs", src)]
        assert len(at) == 1, bar
        # the blocks that enclose the wait, innermost first
        depth, i, heads = 0, at[0], []
        while i > 0 and len(heads) < 4:
            i -= 1
            depth += {"}": 1, "{": -1}.get(src[i], 0)
            if depth < 0:
                heads.append(src[src.rindex("\n", 0, i) + 1:i].strip())
                depth = 0
        line = src[src.rindex("\n", 0, at[0]) + 1:at[0]]
        assert not any("!ok" in h for h in heads + [line]), (bar, heads)


# Requests at the given times, then (at `last`) the final one; the MMA thread makes a step every `step` ns.
CLEAR = r"""
static volatile int job[3], gave_up;
static uint64_t step, last = 0;  // (0: no final request)
static bool step_try(uint64_t *b, uint32_t parity) {
    const bool done = mbar_try(b, parity);
    job[2] = step ? (int)(now / step) : 0;
    job[0] = last && now >= last ? -1 : 1;
    return done;
}
#define mbar_try step_try
%s
#undef mbar_try
static int serve(std::vector<uint64_t> when, int row, uint8_t *ring) {  // requests answered; stops at the end or when it gives up
    model[0].when = when;
    if (last) model[0].when.push_back(last);
    int answered = -1;
    for (int lane = 0; lane < 32; ++lane) {
        now = 0; tick = 1000000;
        model[1].arrived = 0;
        job[1] = row; job[2] = 0;
        clear_role(ring, 32768, 2, bars, bars + 1, job, &gave_up, 2000000000ull, lane);
        if (lane == 0) answered = model[1].arrived;
    }
    return answered;
}
int main() { %s }"""


def test_the_clearing_role_outlasts_a_long_kernel(tmp_path):
    """Requests a minute and more after the kernel began, and as far apart, are answered."""
    out = run_host(tmp_path, CLEAR % (function("clear_role"), """
    static uint8_t ring[2 * 32768];
    memset(ring, 7, sizeof ring);
    step = 1000000000;
    last = 300000000000ull;
    printf("%d ", serve({61000000000ull, 200000000000ull}, 50, ring));
    int cleared = 0, kept = 0;
    for (int h = 0; h < 2; ++h)
        for (int r = 0; r < 128; ++r)
            for (int c = 0; c < 128; ++c) (r < 50 ? kept : cleared) += ring[32768 + h * 16384 + r * 128 + c] == (r < 50 ? 7 : 0);
    for (int i = 0; i < 32768; ++i) kept += ring[i] == 7;
    printf("%d %d\\n", cleared, kept);"""))
    assert out == ["2", str(2 * 78 * 128), str(2 * 50 * 128 + 32768)]


def test_the_clearing_role_leaves(tmp_path):
    """When the MMA thread makes no step for long; at once when another role gave up."""
    out = run_host(tmp_path, CLEAR % (function("clear_role"), """
    static uint8_t ring[2 * 32768];
    step = 0;
    printf("%d ", serve({}, 50, ring));
    printf("%llu ", (ull)(now / 1000000000));
    step = 1000000000;
    gave_up = 1;
    printf("%d ", serve({}, 50, ring));
    printf("%d\\n", now < 10000000);"""))
    assert out[0] == "0" and 30 < int(out[1]) < 100 and out[2:] == ["0", "1"]

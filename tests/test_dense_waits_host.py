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

"""The bounded waits of the tree attention, run on the CPU: their source, with a thread for every lane of a warp and
barriers of the test's own for the votes.  On the GPU a vote that some lane does not come to never ends."""
import os
import re
import shutil
import subprocess

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_207_gb300", "csrc", "pa_tree_tc.cu")

HARNESS = r"""
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <thread>
#include <vector>
#define __device__
#define __noinline__
#define __forceinline__ inline

thread_local int lane;
std::mutex lock;
std::condition_variable bell;
int voters, phase;
bool verdict, result;
std::atomic<int> stuck{0};

// the warp's vote: false (and counted) when some lane does not come
bool __all_sync(unsigned, bool x) {
    std::unique_lock<std::mutex> hold(lock);
    if (voters == 0) verdict = true;
    verdict = verdict && x;
    const int mine = phase;
    if (++voters == 32) {
        voters = 0;
        ++phase;
        result = verdict;
        bell.notify_all();
        return result;
    }
    if (!bell.wait_for(hold, std::chrono::seconds(5), [&] { return phase != mine; })) {
        ++stuck;
        return false;
    }
    return result;
}
bool __any_sync(unsigned m, bool x) { return !__all_sync(m, !x); }

// what each lane's looks find: false `ready[lane]` times, then true (below 0: never)
int ready[32];
thread_local int looks;
std::atomic<uint64_t> clock_ns{0};
bool mbar_try_wait(uint32_t, uint32_t) { return ready[lane] >= 0 && looks++ >= ready[lane]; }
uint64_t global_timer_ns() { return clock_ns += 1000000; }
extern "C" inline void unused() {}

%s

int main(int argc, char** argv) {
    for (int i = 0; i < 32; ++i) ready[i] = atoi(argv[1 + i]);
    int yes = 0;
    std::mutex count;
    std::vector<std::thread> lanes;
    for (int i = 0; i < 32; ++i)
        lanes.emplace_back([&, i] {
            lane = i;
            looks = 0;
            const bool ok = warp_wait(0, 0%s);
            std::lock_guard<std::mutex> hold(count);
            yes += ok;
        });
    for (auto& t : lanes) t.join();
    printf("%%d %%d\n", yes, stuck.load());
}
"""


def _source():
    text = open(SOURCE).read()
    limit = re.search(r"constexpr uint64_t kWaitNs = [^;]+;", text).group(0)
    start = text.index("__device__ __noinline__ bool warp_wait_long")
    end = text.index("\n}\n", text.index("bool warp_wait(", start)) + 3
    return limit + "\n" + text[start:end]


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    where = tmp_path_factory.mktemp("waits")
    source = _source()
    more = ", kWaitNs" if re.search(r"bool warp_wait\([^)]*limit", source) else ""
    (where / "waits.cpp").write_text(HARNESS % (source, more))
    subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", str(where / "waits.cpp"), "-o", str(where / "waits")], check=True,
                   capture_output=True)

    def call(ready):
        out = subprocess.run([str(where / "waits"), *map(str, ready)], check=True, capture_output=True, text=True, timeout=60).stdout
        return tuple(map(int, out.split()))

    return call


@pytest.mark.parametrize("ready,yes", [
    ([0] * 32, 32),
    ([3] * 32, 32),
    ([0] * 5 + [1] * 27, 32),                    # a phase that ends while the lanes look
    ([1] * 31 + [0], 32),
    ([7] * 16 + [200] * 16, 32),
    ([-1] * 32, 0),                              # one that never ends: all give up
    ([0] * 31 + [-1], 0),
], ids=["ready", "later", "first lanes", "last lane", "halves", "never", "never for one"])
def test_all_lanes_vote_and_agree(run, ready, yes):
    assert run(ready) == (yes, 0)

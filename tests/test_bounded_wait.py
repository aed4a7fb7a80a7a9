"""The bounded wait of a warp (csrc/rssm_wait.h), compiled for the host: 32 threads stand in for the lanes, and each
sees the barrier's phase end and the limit pass at a time of its own.  Whatever they see, all lanes return the
same, and none is left behind at a vote."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "checkpoint_input_replay_rssm_b200", "csrc")

PROGRAM = r"""
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <random>
#include <thread>
#include <vector>
#include "rssm_wait.h"

constexpr int kLanes = 32;
// A vote of all lanes, as the hardware's: it returns once every lane is there.
struct Warp {
    std::mutex m;
    std::condition_variable cv;
    int here = 0, yes = 0, last_yes = 0;
    long round = 0;
    int vote(bool x) {
        std::unique_lock<std::mutex> l(m);
        const long mine = round;
        yes += x;
        if (++here == kLanes) {
            last_yes = yes;
            here = yes = 0;
            ++round;
            cv.notify_all();
        } else {
            cv.wait(l, [&] { return round != mine; });
        }
        return last_yes;
    }
};

int main() {
    std::mt19937 r(5);
    int outcomes[2] = {0, 0};
    for (int trial = 0; trial < 300; ++trial) {
        const int kind = trial % 3;  // phase first for all; limit first for some; both in any order
        int ready_at[kLanes], late_at[kLanes], got[kLanes], asked_after[kLanes] = {0};
        for (int i = 0; i < kLanes; ++i) {
            ready_at[i] = r() % 6;
            late_at[i] = kind == 0 ? 1000 : kind == 1 ? (int)(r() % 8 == 0 ? r() % 6 : 1000) : (int)(r() % 12);
        }
        if (kind == 1) ready_at[r() % kLanes] = 1 << 30;  // some lane never sees it
        if (kind == 1) late_at[r() % kLanes] = 3;
        Warp w;
        std::vector<std::thread> t;
        for (int i = 0; i < kLanes; ++i)
            t.emplace_back([&, i] {
                int polls = 0, checks = 0;
                bool seen = false;
                got[i] = rssm::wait_together(
                    [&] {
                        asked_after[i] += seen;
                        return seen = polls++ >= ready_at[i];
                    },
                    [&] { return checks++ >= late_at[i]; }, [&](bool x) { return w.vote(x) == kLanes; },
                    [&](bool x) { return w.vote(x) > 0; });
            });
        for (auto &x : t) x.join();
        for (int i = 0; i < kLanes; ++i) {
            if (got[i] != got[0]) return std::printf("trial %d: lanes disagree\n", trial), 1;
            if (asked_after[i]) return std::printf("trial %d: a phase was polled again after it had ended\n", trial), 1;
        }
        if (kind == 0 && !got[0]) return std::printf("trial %d: gave up without a reason\n", trial), 1;
        if (kind == 1 && got[0]) return std::printf("trial %d: a lane's phase never ended\n", trial), 1;
        ++outcomes[got[0]];
    }
    std::printf("%d %d\n", outcomes[0], outcomes[1]);
    return 0;
}
"""


def test_lanes_of_a_warp_leave_a_wait_together(tmp_path):
    src, exe = tmp_path / "wait.cpp", tmp_path / "wait"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stdout
    gave_up, went_on = map(int, done.stdout.split())
    assert gave_up >= 100 and went_on >= 100


@pytest.mark.parametrize("name", ["rssm_gdn_chunk.cu", "rssm_kv4_attend_tiles.cu"])
def test_roles_wait_a_warp_at_a_time(name):
    """In the kernels whose warps have roles, no wait is left to a lane: each wait_for is the warp's."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert "warp_wait(bar + which, parity, sfail)" in text
    assert "bar_try(" not in text

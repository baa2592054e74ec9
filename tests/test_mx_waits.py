"""The warp-wide bounded wait of the microscaled products (csrc/q4_wait.cuh),
compiled for the host with 32 threads as the lanes: whatever the lanes see,
they come back together with one answer."""
from __future__ import annotations

import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_gemv_b200", "csrc")

PROGRAM = r"""
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <random>
#include <thread>
#include <vector>
#include "q4_wait.cuh"

constexpr int kLanes = 32;

// A vote of all lanes; it hangs if one stays away, as the warp's does.
struct Vote {
    std::mutex m;
    std::condition_variable c;
    int in = 0, round = 0;
    bool all = true, last = true;
    bool operator()(bool b) {
        std::unique_lock<std::mutex> l(m);
        all = all && b;
        const int mine = round;
        if (++in == kLanes) {
            last = all;
            all = true;
            in = 0;
            ++round;
            c.notify_all();
        } else {
            c.wait(l, [&] { return round != mine; });
        }
        return last;
    }
};

int main(int argc, char** argv) {
    const bool together = argc > 1;
    std::mt19937 rng(7);
    int parted = 0, yes = 0, no = 0;
    for (int trial = 0; trial < 60; ++trial) {
        // the look from which on a lane sees the phase complete, and the limit
        // or the error flag: near each other, and different in every lane
        int ready_at[kLanes], expired_at[kLanes];
        for (int i = 0; i < kLanes; ++i) {
            ready_at[i] = trial % 5 == 0 ? 1 << 30 : 64 * (1 + static_cast<int>(rng() % 3));
            expired_at[i] = trial % 5 == 1 ? 1 << 30 : 1 + static_cast<int>(rng() % 4);
        }
        Vote vote;
        bool result[kLanes];
        std::vector<std::thread> lanes;
        for (int i = 0; i < kLanes; ++i)
            lanes.emplace_back([&, i] {
                int looks = 0, asked = 0;
                const auto ready = [&] { return ++looks > ready_at[i]; };
                const auto expired = [&] { return ++asked >= expired_at[i]; };
                if (together)
                    result[i] = q4::wait_together([&] { return vote(ready()); }, [&] { return !vote(!expired()); });
                else  // each lane for itself
                    result[i] = q4::wait_together(ready, expired);
            });
        for (auto& t : lanes) t.join();
        bool same = true;
        for (int i = 1; i < kLanes; ++i) same = same && result[i] == result[0];
        if (!same) ++parted;
        else if (result[0]) ++yes;
        else ++no;
    }
    std::printf("%d %d %d\n", parted, yes, no);
    return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    src, exe = d / "wait.cpp", d / "wait"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)


def _run(*cmd):
    res = subprocess.run(cmd, capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr
    return [int(v) for v in res.stdout.split()]


def test_lanes_come_back_together(program):
    parted, yes, no = _run(program, "together")
    assert parted == 0 and yes > 0 and no > 0


def test_the_trials_part_lanes_that_wait_each_for_itself(program):
    parted, _, _ = _run(program)
    assert parted > 0


def test_the_products_wait_as_warps():
    """wait_bar, which every role of both kernels waits with, asks only by votes."""
    text = open(os.path.join(CSRC, "q4_mx_tc.cuh")).read()
    body = text[text.index("bool try_wait_all("):text.index("struct Ring")]
    assert "vote.sync.all.pred q, p, 0xFFFFFFFF" in body and "__any_sync(0xFFFFFFFFu" in body
    assert "mbar_try_wait(" not in body and "mbar_wait(" not in body

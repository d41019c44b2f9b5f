"""The feeding warp of the paged tcgen05 kernel waits for every copy that it started before the CTA gives its shared memory
back, wherever a wait of it gave up (csrc/paged_feed.h, compiled for the host)."""
import os
import shutil
import subprocess

import pytest

import local_linear_attention_flashlla_gb300 as lla

CSRC = os.path.join(os.path.dirname(lla.__file__), "csrc")

PROGRAM = r"""
#include "paged_feed.h"
#include <cstdio>
#include <cstdlib>
#include <set>
#include <utility>

// mbarriers as the warp sees them: a stage's `full` phases, counted; nothing is ever consumed by force, a stage counts as
// empty unless this wait is the one that gives up.
template <int NS>
struct Fake {
    int until_failure;                                   // waits that succeed
    int copies[2][NS] = {}, landed[2][NS] = {};          // per stage: copies started, copies known to have landed
    bool wait_empty(int kv, int stage, int parity) {
        if (until_failure-- == 0) return false;
        // a stage that was filled c times is empty again in its phase c - 1: the parity waited for is its last one's
        if (((copies[kv][stage] - 1) & 1) != parity) std::exit(2);
        landed[kv][stage] = copies[kv][stage];           // consumed, so landed
        return true;
    }
    void copy(int kv, int stage) { ++copies[kv][stage]; }
    void wait_full(int kv, int stage, int parity) {
        if (((copies[kv][stage] - 1) & 1) != parity) std::exit(3);
        landed[kv][stage] = copies[kv][stage];
    }
};

template <int NS>
void check() {
    for (int waits = 0; waits <= 8 * NS + 2; ++waits) {
        Fake<NS> f{waits};
        lla::paged::RingCount<NS> n;
        int blocks = 0;
        while (n.feed_block(f)) ++blocks;
        if (blocks != waits / 2) std::exit(4);
        n.drain(f);
        for (int kv = 0; kv < 2; ++kv)
            for (int s = 0; s < NS; ++s)
                if (f.landed[kv][s] != f.copies[kv][s]) {
                    std::printf("stages %d, wait %d gave up: ring %d stage %d still in flight\n", NS, waits, kv, s);
                    std::exit(1);
                }
    }
}

int main() {
    check<2>();
    check<4>();
    return 0;
}
"""


def test_no_copy_is_left_in_flight(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "feed.cpp", tmp_path / "feed"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Wno-unknown-pragmas", "-I" + CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True)
    assert r.returncode == 0, r.stdout

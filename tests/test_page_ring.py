"""The few-row attention kernel's ring of pages (csrc/page_ring.h), on the CPU: what is drained after a wait
that ran out.  A warp's walk is run with a wait that fails at every place in turn, for walks of every length
around the ring's, and each page copied is either taken by a wait or drained: none is left landing."""
import subprocess

from bit_gemv_sherry_b200 import build

PROGRAM = r"""
#include <cstdio>
#include <set>
#include <utility>
#include "page_ring.h"

template <int S>
int walk(int pages, int fails_at) {
    sherry::PageRing<S> ring;
    std::set<int> landing;           // pages copied and not seen landing
    int slot_of[64], next = 0;
    auto copy = [&]() {
        if (next >= pages) return;
        slot_of[next] = ring.to;
        for (int j : landing) if (slot_of[j] == ring.to) std::printf("slot of page %d used again\n", j);
        landing.insert(next++);
        ring.copy();
    };
    for (int i = 0; i < S; i++) copy();
    for (int i = 0; i < pages; i++) {          // the walk goes on over all of its pages
        if (!ring.dead) {
            const int s = ring.at;
            const unsigned phase = ring.lap;
            if (s != i % S || phase != ((unsigned)(i / S) & 1u)) return std::printf("page %d: slot %d phase %u\n", i, s, phase), 1;
            ring.take(i != fails_at);
            if (!ring.dead) landing.erase(i);
        }
        if (!ring.dead) copy();
    }
    ring.drain([&](int s, unsigned phase) {
        bool found = false;
        for (int j : landing)
            if (slot_of[j] == s && phase == ((unsigned)(j / S) & 1u)) { landing.erase(j); found = true; break; }
        if (!found) std::printf("drained slot %d phase %u, which nothing lands in\n", s, phase), landing.insert(1000);
    });
    if (!landing.empty()) return std::printf("S %d, %d pages, wait %d fails: %zu left landing\n", S, pages, fails_at, landing.size()), 1;
    return ring.dead != (fails_at < pages);
}

int main() {
    int bad = 0;
    for (int pages = 0; pages < 20; pages++)
        for (int f = 0; f <= pages; f++) bad += walk<2>(pages, f) + walk<3>(pages, f);
    return bad != 0;
}
"""


def test_every_copied_page_is_taken_or_drained(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-Werror", "-I", build.CSRC, "-o", str(exe), str(src)])
    run = subprocess.run([str(exe)], capture_output=True, text=True)
    assert run.returncode == 0 and run.stdout == "", run.stdout

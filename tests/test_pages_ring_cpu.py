"""The ring between the prompt kernel's copies and its operand warps (csrc/ring.h), walked on the host: copies that land in any
order, consumers of any speed, mbarriers that know a phase's parity only."""

from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <algorithm>
#include <cstdio>
#include <random>
#include "ring.h"
template <int SLOTS>
int walk(unsigned seed, int blocks) {
    std::mt19937 rng(seed);
    auto chance = [&](int n) { return (int)(rng() % n) == 0; };
    const int items = 2 * blocks, land = 1 + rng() % 40;
    int slow[4], done[4] = {0, 0, 0, 0};  // four warps: 0, 1 take the even items, 2, 3 the odd ones
    for (int &x : slow) x = 1 + rng() % 40;
    int landed[SLOTS] = {}, arrivals[SLOTS] = {};  // uses that have landed; arrivals at the slot's other barrier, two a use
    bool flying[SLOTS] = {};
    int issued = 0;
    er::RingWalk<SLOTS> at[4] = {er::RingWalk<SLOTS>(0), er::RingWalk<SLOTS>(0), er::RingWalk<SLOTS>(1), er::RingWalk<SLOTS>(1)};
    auto least = [&] { return std::min(std::min(done[0], done[1]), std::min(done[2], done[3])); };
    for (long step = 0; least() < blocks; ++step) {
        if (step > 4000000) return 2;  // stuck
        const int s = issued % SLOTS;
        if (issued < items && arrivals[s] / 2 == issued / SLOTS && chance(2)) {
            flying[s] = true;
            ++issued;
        }
        for (int i = 0; i < SLOTS; ++i)
            if (flying[i] && chance(land)) {
                flying[i] = false;
                ++landed[i];
            }
        for (int w = 0; w < 4; ++w) {
            const int j = done[w], item = 2 * j + w / 2;
            // what it makes goes into two stages: block j - 1's, which it has passed, was free once all had made block j - 3's
            if (j >= blocks || least() < j - 2 || !chance(slow[w])) continue;
            auto passes = [](int phase, int par) { return (phase & 1) != par; };  // phase: the current, not complete one
            if (!at[w].ready([&](int slot, int par) { return passes(arrivals[slot] / 2, par); },
                             [&](int slot, int par) { return passes(landed[slot], par); }))
                continue;
            if (at[w].slot != item % SLOTS || landed[at[w].slot] != item / SLOTS + 1) return 1;  // not there
            ++arrivals[at[w].slot];
            ++done[w];
            at[w].step();
        }
    }
    return 0;
}
int main() {
    for (unsigned seed = 0; seed < 400; ++seed)
        for (int blocks : {1, 2, 3, 4, 7, 100})
            if (int r = SLOTS_FN(seed, blocks)) {
                std::printf("seed %u, %d blocks: %s\n", seed, blocks, r == 1 ? "an item was taken before it had landed" : "stuck");
                return 1;
            }
    return 0;
}
"""


def test_no_item_is_taken_before_it_has_landed(tmp_path):
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(SOURCE)
    csrc = os.path.join(ROOT, "block_quantized_token_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-DSLOTS_FN=walk<3>", "-I", csrc, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout

"""How the grouped products share out their tiles (uw_plan.h), compiled for the
host and checked for every k step of every tile over many sizes."""
import ctypes
import os
import subprocess

import pytest

from decode_gemm_bf16_b200 import build as uwbuild

SOURCE = r"""
#include <stdint.h>
#include <vector>
#include "uw_plan.h"
using namespace uw;

extern "C" void plan_of(uint32_t tiles, uint32_t P, uint32_t kt, uint32_t acc_w, int cut_parts, uint32_t* out) {
    const Plan pl = make_plan(tiles, P, kt, acc_w, cut_parts != 0);
    out[0] = pl.whole; out[1] = pl.units; out[2] = pl.ps; out[3] = pl.parts; out[4] = pl.rest;
}

// 0: the plan is sound, else which rule it breaks.
extern "C" int check_plan(uint32_t tiles, uint32_t P, uint32_t kt, uint32_t acc_w, int cut_parts) {
    const Plan pl = make_plan(tiles, P, kt, acc_w, cut_parts != 0);
    if (pl.whole > tiles) return 1;
    const uint32_t cut = tiles - pl.whole;
    std::vector<uint32_t> whole(pl.whole, 0);
    std::vector<uint8_t> step((size_t)cut * kt, 0);
    std::vector<int64_t> published(P, -1);                // tile whose sums a worker publishes
    std::vector<int64_t> joiner(cut, -1), last(cut, -1), parts(cut, 0);
    for (uint32_t b = 0; b < P; b++) {
        Seg s;
        for (uint32_t i = 0; segment(pl, b, i, s); i++) {
            if (s.tile >= tiles || s.kt0 < 0 || s.kt0 >= s.kt1 || s.kt1 > (int)kt) return 2;   // out of range, or empty
            const uint32_t to = last_joined(pl, s, b);
            if (s.tile < pl.whole) {
                if (s.kt0 != 0 || s.kt1 != (int)kt || publishes(s) || to != b) return 3;
                whole[s.tile]++;
                continue;
            }
            const uint32_t c = s.tile - pl.whole;
            parts[c]++;
            for (int k = s.kt0; k < s.kt1; k++)
                if (step[(size_t)c * kt + k]++) return 4;                                     // twice
            if (publishes(s)) {
                if (published[b] >= 0 || i != 0) return 5;                                    // one slot a worker; before any wait
                published[b] = s.tile;
                if (to != b) return 6;
            } else {
                if (joiner[c] >= 0) return 7;                                                 // two joiners
                joiner[c] = b;
                last[c] = to;
                if (to >= P) return 8;                                                        // a worker that is not there
            }
        }
    }
    for (uint32_t t = 0; t < pl.whole; t++)
        if (whole[t] != 1) return 9;
    for (uint8_t n : step)
        if (n != 1) return 10;
    for (uint32_t c = 0; c < cut; c++) {
        if (joiner[c] < 0) return 11;
        int64_t seen = 1;
        for (int64_t b = joiner[c] + join_stride(pl); b <= last[c]; b += join_stride(pl), seen++)
            if (published[b] != (int64_t)pl.whole + c) return 12;                             // nobody would write that tag
        if (seen != parts[c]) return 13;                                                      // sums left out
    }
    return 0;
}

extern "C" int warp_of_slot(int slot) { return slot_warp(slot); }

// The first (tiles, kt) in the ranges whose plan is not sound.
extern "C" int sweep(uint32_t tiles0, uint32_t tiles1, uint32_t P, uint32_t kt0, uint32_t kt1, uint32_t acc_w, int cut_parts,
                     uint32_t* bad) {
    for (uint32_t t = tiles0; t < tiles1; t++)
        for (uint32_t kt = kt0; kt < kt1; kt++) {
            const int r = check_plan(t, P, kt, acc_w, cut_parts);
            if (r) { bad[0] = t; bad[1] = kt; return r; }
        }
    return 0;
}
"""


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I", uwbuild.CSRC, str(src), "-o", str(lib)])
    return ctypes.CDLL(str(lib))


def _plan(L, *a):
    out = (ctypes.c_uint32 * 5)()
    L.plan_of(*a, out)
    return dict(zip(("whole", "units", "ps", "parts", "rest"), out))


@pytest.mark.parametrize("P", [74, 66, 1, 2, 3, 37])
@pytest.mark.parametrize("acc_w", [16, 128, 192, 224, 256])
def test_parts_are_sound(L, P, acc_w):
    bad = (ctypes.c_uint32 * 2)()
    assert L.sweep(0, 3 * P + 2, P, 1, 70, acc_w, 1, bad) == 0, list(bad)
    assert L.sweep(0, P + 2, P, 250, 260, acc_w, 1, bad) == 0, list(bad)


@pytest.mark.parametrize("P", [148, 132, 1, 2, 3])
def test_ranges_are_sound(L, P):
    bad = (ctypes.c_uint32 * 2)()
    assert L.sweep(0, 3 * P + 2, P, 1, 70, 16, 0, bad) == 0, list(bad)
    assert L.sweep(0, P + 2, P, 250, 260, 16, 0, bad) == 0, list(bad)


@pytest.mark.parametrize("tiles,kt,acc_w", [
    (112 * 2, 32, 224),    # 225 .. 448 rows (tiles of 112) of 14336 x 4096 in 4 bits: two tiles left over
    (16 * 14, 32, 224),    # 1457 .. 1568 rows of 4096 x 4096
    (1, 32, 256),          # 256 rows of 256 x 2048 in BF16: one tile
    (75, 64, 256),         # 256 rows of 19200 x 4096: one left over
    (2, 28, 192),          # both sides in 4 bits
    (112 * 2, 32, 192)])
def test_parts_stay_below_the_k_steps(L, tiles, kt, acc_w):
    """Few tiles left over and few k steps: as many parts as workers would leave parts without any."""
    assert L.check_plan(tiles, 74, kt, acc_w, 1) == 0
    p = _plan(L, tiles, 74, kt, acc_w, 1)
    assert 1 < p["parts"] <= kt // 2 and p["rest"] == tiles % 74


def test_both_sides_of_the_limits(L):
    # parts: kt acc_w (parts - 1) > 4300 parts
    assert _plan(L, 37, 74, 33, 256, 1)["parts"] == 0 and _plan(L, 37, 74, 34, 256, 1)["parts"] == 2
    # parts of fewer than two k steps are not made, whatever the accumulator
    assert _plan(L, 1, 74, 3, 1 << 20, 1)["parts"] == 0 and _plan(L, 1, 74, 4, 1 << 20, 1)["parts"] == 2
    # ranges: kt (P - rest) / P from 24 without a whole round, from 10 behind one
    assert _plan(L, 74, 148, 48, 16, 0)["ps"] == 0 and _plan(L, 74, 148, 50, 16, 0)["ps"] == 148
    assert _plan(L, 222, 148, 20, 16, 0)["ps"] == 0 and _plan(L, 222, 148, 22, 16, 0)["ps"] == 148
    # nothing is cut in whole rounds
    for cut in (0, 1):
        p = _plan(L, 296, 148, 256, 256, cut)
        assert p["whole"] == 296 and not p["ps"] and not p["parts"]


def _seen_before(warp_of_stage, S, stages=200):
    """Whether every wait for a slot is made by a warp that has seen the slot's phase before (a wait on a parity cannot
    tell a phase from the last but one)."""
    return all(warp_of_stage(q) == warp_of_stage(q - S) for q in range(S, stages))


@pytest.mark.parametrize("S", range(2, 13))
def test_a_slot_keeps_its_warp(L, S):
    assert _seen_before(lambda q: L.warp_of_slot(q % S), S)
    assert {L.warp_of_slot(q % S) for q in range(S)} == {0, 1}
    assert _seen_before(lambda q: q % 2, S) == (S % 2 == 0)   # stages in turn: wrong for every odd ring

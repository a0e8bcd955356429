// uw_plan.h -- how the grouped products share out their tiles: whole-number
// arithmetic alone, so that the kernel and a program on the host compile the
// same lines.
//
// Whole tiles are dealt out in rounds, one a worker (a CTA or a pair of CTAs).
// What is left over is cut along k where that pays, either
//   * in equal contiguous ranges of k steps, one a worker (`ps` workers), or
//   * (parts > 0) every one of the last `rest` tiles in `parts` equal parts,
//     worker part * rest + i taking a part of tile i.
// What holds for every plan: each k step of each tile belongs to one segment,
// no segment is empty, a worker publishes partial sums at most once, and a cut
// tile is joined by the worker with its first k steps alone, from workers
// after it that all publish.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define UW_HD __host__ __device__ __forceinline__
#else
#define UW_HD inline
#endif

namespace uw {

struct Plan {
    uint32_t whole;          // tiles dealt out whole (the first ones)
    uint32_t units;          // k steps of the cut tiles (contiguous ranges; the caller checks that units * P < 2^32)
    uint32_t ps;             // of the P workers, those that share them
    uint32_t P;
    uint32_t kt;             // k steps of a tile
    uint32_t parts, rest;
};

struct Seg {
    uint32_t tile;
    int kt0, kt1;
};

// `acc_w`: columns of a tile's accumulator.  `cut_parts`: see pick_parts.
UW_HD Plan make_plan(uint32_t tiles, uint32_t P, uint32_t kt, uint32_t acc_w, bool cut_parts) {
    Plan pl;
    const uint32_t rounds = tiles / P, rest = tiles - rounds * P;
    pl.P = P;
    pl.kt = kt;
    pl.units = pl.ps = pl.parts = pl.rest = 0;
    pl.whole = tiles;
    if (cut_parts) {
        // A part holds two k steps or more: an empty one would join where it has to publish, and one step costs more to
        // join than it saves.
        const uint32_t most = kt / 2, free = rest ? P / rest : 0, parts = free < most ? free : most;
        // joining parts takes about 4.5 us (8600 cycles) of the first one's time: worth it when that is less than the
        // k steps (2 cycles a column and step) that the others take off it.  (Limits of 3500, 4300 and 7000: 512 rows of
        // four experts of 2048 x 2048 in BF16 16.2, 14.8, 14.8 us; 256 rows of 14336 x 4096 in 4 bits 32.8, 32.8, 37.5.)
        if (parts > 1 && (uint64_t)kt * acc_w * (parts - 1) > 4300ull * parts) {
            pl.parts = parts;
            pl.rest = rest;
            pl.whole = tiles - rest;
        }
    } else if (rest && (uint64_t)kt * (P - rest) > (uint64_t)(rounds ? 10 : 24) * P) {
        // Ranges take kt (P - rest) / P steps off the longest worker and cost it a joining: worth it from 10 steps on,
        // 24 where no whole round comes first (then all memory bandwidth is close to used without them).  Whole tiles
        // against ranges, 64 rows in BF16: 12800 x 4096 (21 steps) 24.1 and 26.9 us, 16384 x 8192 (17) 49.0 and 52.6,
        // 9600 x 4096 (32) 21.5 and 22.7; one row in 4 bits: 14336 x 4096 (8) 13.8 and 14.8, 7000 x 4096 (20) 12.9
        // and 12.3, 9600 x 8192 (32) 18.9 and 16.7; behind a whole round: 18000 x 4096 (2) 14.1 and 15.5, 30000 x 4096
        // (13) 20.3 and 19.4.
        pl.whole = rounds > 1 ? (rounds - 1) * P : 0;
        pl.units = (tiles - pl.whole) * kt;
        // a range shorter than two k steps costs more to join than it saves
        const uint32_t most = (pl.units + 1) / 2;
        pl.ps = P < most ? P : most;
    }
    return pl;
}

// Units of worker b's range start here; owner of a unit.
UW_HD uint32_t unit_begin(uint32_t b, const Plan& pl) { return b * pl.units / pl.ps; }
UW_HD uint32_t unit_owner(uint32_t u, const Plan& pl) { return ((u + 1) * pl.ps - 1) / pl.units; }

// Segment i of worker b: its range or part of the cut tiles first (joining them
// then overlaps the whole tiles), then its whole tiles.
UW_HD bool segment(const Plan& pl, uint32_t b, uint32_t i, Seg& s) {
    const uint32_t kt = pl.kt;
    if (b < pl.ps) {
        const uint32_t u0 = unit_begin(b, pl), ue = unit_begin(b + 1, pl), t0 = u0 / kt;
        const uint32_t n = ue > u0 ? (ue - 1) / kt - t0 + 1 : 0;
        if (i < n) {
            const uint32_t tile0 = (t0 + i) * kt, end = tile0 + kt < ue ? tile0 + kt : ue;
            s.tile = pl.whole + t0 + i;
            s.kt0 = i ? 0 : (int)(u0 - tile0);
            s.kt1 = (int)(end - tile0);
            return true;
        }
        i -= n;
    } else if (b < pl.parts * pl.rest) {
        if (i == 0) {
            const uint32_t part = b / pl.rest;
            s.tile = pl.whole + b - part * pl.rest;
            s.kt0 = (int)(part * kt / pl.parts);
            s.kt1 = (int)((part + 1) * kt / pl.parts);
            return true;
        }
        i--;
    }
    s.tile = b + i * pl.P;
    s.kt0 = 0;
    s.kt1 = (int)kt;
    return s.tile < pl.whole;
}

// What becomes of a segment's sums: a cut tile's later ranges go to the
// workspace, and the worker with its first range adds them: those of workers
// b + join_stride(), ... up to last_joined() (b itself: nothing to add).
UW_HD bool publishes(const Seg& s) { return s.kt0 > 0; }
UW_HD uint32_t join_stride(const Plan& pl) { return pl.parts ? pl.rest : 1; }
UW_HD uint32_t last_joined(const Plan& pl, const Seg& s, uint32_t b) {
    if (s.kt0 > 0 || s.kt1 == (int)pl.kt) return b;
    return pl.parts ? b + (pl.parts - 1) * pl.rest : unit_owner((s.tile - pl.whole + 1) * pl.kt - 1, pl);
}

// Two warps share the work on a ring's slots.  A slot always has the same warp:
// a wait on a parity tells a phase from the one before alone, so whoever waits
// for a slot has to have seen its last phase too.  (Taking stages in turn, as
// it was, changes a slot's warp on every wrap of a ring of odd length.)
UW_HD int slot_warp(int slot) { return slot & 1; }

}  // namespace uw

// Tiles of a launch that runs one product per group of rows (the experts' products).
//
// offsets[g] .. offsets[g + 1] are group g's rows; they lie on the device, so the
// host knows only how many rows and groups there are.  A launch has as many
// workgroups as any division of the rows can need tiles; each finds its tile by a
// prefix sum over the groups' tile counts (one wave's worth of groups at a time,
// every wave for itself, so without a barrier) and the rest leave.  Where the
// sum ends is known only then, and the XCD ranges of the tile order are laid over
// the live tiles, not over the launch.
//
// Offsets that the host could not check stay harmless: each is clamped to the rows and
// raised to the largest before it, so groups never overlap and never leave the operands.
#pragma once

#include <cmath>

#include "common.h"

namespace ssg {

namespace group {

// Inclusive scans over a wave's 64 lanes (values >= 0; 0 comes in from outside).
template <class F>
__device__ __forceinline__ int scan(int v, F f) {
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));  // row_shr:1
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));  // row_bcast:15
    v = f(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return v;
}
__device__ __forceinline__ int scan_max(int v) {
    return scan(v, [](int a, int b) { return a > b ? a : b; });
}
__device__ __forceinline__ int scan_sum(int v) {
    return scan(v, [](int a, int b) { return a + b; });
}
__device__ __forceinline__ int clamped(int v, int rows) { return v < 0 ? 0 : v > rows ? rows : v; }

// Lane l's group of the 64 from g0 on: its rows [lo, hi).  reached: the end of the groups before
// (updated).  (An int of rows: the host keeps them below 2^31.)
__device__ __forceinline__ void span(const int32_t *offsets, int groups, int rows, int g0, int &reached, int &lo,
                                     int &hi) {
    const int lane = threadIdx.x & 63, g = g0 + lane;
    const int end = g < groups ? clamped(offsets[g + 1], rows) : 0;
    hi = max(scan_max(end), reached);
    lo = __builtin_amdgcn_update_dpp(reached, hi, 0x138, 0xf, 0xf, false);  // wave_shr:1, lane 0: reached
    reached = __builtin_amdgcn_readlane(hi, 63);
}

struct Tile {
    int group, row, rows, tile_n;  // group < 0: none; row: its first row, rows: of the group from there on
};

// The `block`-th tile of BM rows (and of tiles_n columns), GM tile rows of a group at a time.
template <int BM>
__device__ __forceinline__ Tile find_tile(int block, const int32_t *offsets, int groups, int rows, int tiles_n,
                                          int GM) {
    const int first = clamped(offsets[0], rows);
    int reached = first, total = 0, lo, hi, sum = 0, count = 0;
    for (int g0 = 0; g0 < groups; g0 += 64) {
        span(offsets, groups, rows, g0, reached, lo, hi);
        count = (hi - lo + BM - 1) / BM;
        sum = total + scan_sum(count);
        total = __builtin_amdgcn_readlane(sum, 63);
    }
    Tile t{-1, 0, 0, 0};
    if (block >= total * tiles_n) return t;
    const int b = xcd_remap(block, total * tiles_n);
    int g0 = 0;
    if (groups > 64) {
        reached = first, total = 0;
        for (;; g0 += 64) {
            span(offsets, groups, rows, g0, reached, lo, hi);
            count = (hi - lo + BM - 1) / BM;
            sum = total + scan_sum(count);
            total = __builtin_amdgcn_readlane(sum, 63);
            if (b < total * tiles_n) break;
        }
    }
    const int at = __builtin_ctzll(__ballot(b < sum * tiles_n));
    const int n = __builtin_amdgcn_readlane(count, at);
    const int j = b - (__builtin_amdgcn_readlane(sum, at) - n) * tiles_n;
    const int super = j / (GM * tiles_n), gm = min(n - super * GM, GM), in = j % (GM * tiles_n);
    const int tile_m = super * GM + in % gm;
    t.group = g0 + at;
    t.tile_n = in / gm;
    t.row = __builtin_amdgcn_readlane(lo, at) + tile_m * BM;
    t.rows = __builtin_amdgcn_readlane(hi, at) - t.row;
    return t;
}

// The k-th group (sorted: the k-th longest of its 64, ties in their order): its number and its rows
// [lo, hi).
__device__ __forceinline__ int nth_group(const int32_t *offsets, int groups, int rows, int k, bool sorted, int &lo,
                                         int &hi) {
    int reached = clamped(offsets[0], rows), l, h;
    for (int g0 = 0;; g0 += 64) {
        span(offsets, groups, rows, g0, reached, l, h);
        if (k >= g0 + 64) continue;
        int at = k - g0;
        if (sorted) {
            const int lane = threadIdx.x & 63, len = h - l, n = min(groups - g0, 64);
            int before = 0;  // groups that come before this lane's
            for (int j = 0; j < n; ++j) {
                const int other = __builtin_amdgcn_readlane(len, j);
                before += other > len || (other == len && j < lane) ? 1 : 0;
            }
            at = __builtin_ctzll(__ballot(before == k - g0 && lane < n));
        }
        lo = __builtin_amdgcn_readlane(l, at);
        hi = __builtin_amdgcn_readlane(h, at);
        return g0 + at;
    }
}

}  // namespace group

// A tile's cost in a launch: `per_cu` workgroups share a CU, so `tiles` of them take
// rounds = tiles / (256 per_cu), each of tile + stages * stage us (the stage times measured with one
// workgroup on a CU or with a full one), after a start that does not depend on them.  The figures are
// fitted to launches of random sizes on MI355X (80 for each product of grouped.hip, 110 of mxfp4.hip,
// all candidates timed); the choice by least cost is 4 to 5 % off the best tile of each in the mean.
struct TileCost {
    int bm, bn, per_cu;
    float start, tile, stage;
    float us(double tiles, double stages) const {
        double rounds = tiles / (256.0 * per_cu);
        if (rounds <= 3.0) rounds = double(int64_t(rounds) + (rounds > double(int64_t(rounds)) ? 1 : 0));
        else rounds += 0.5;
        const double share = tiles / 256.0 < 1.0 ? 1.0 : tiles / 256.0 < per_cu ? tiles / 256.0 : per_cu;
        return float(start + (rounds < 1.0 ? 1.0 : rounds) * (tile + stages * stage * share));
    }
};

// M rows in `groups` groups, whose lengths the host does not know: how many an even choice would reach,
// and the tile rows that they will need about, with half a tile empty at the end of each.
struct GroupRowsGuess {
    int64_t M, groups;
    double live;
    GroupRowsGuess(int64_t M_, int64_t groups_)
        : M(M_), groups(groups_), live(double(groups_) * (1.0 - std::exp(-double(M_) / double(groups_)))) {}
    double tiles(int bm) const {
        if (groups == 1) return double((M + bm - 1) / bm);
        const double rows = double(M) / bm + 0.5 * live;
        return rows > live ? rows : live;
    }
};

// The cheapest of N tiles (or of the first `some`): tiles(bm, bn) says how many a launch has.
template <int N, class F>
int cheapest(const TileCost (&c)[N], double stages, F tiles, int some = N) {
    int best = 0;
    float least = 0.0f;
    for (int i = 0; i < some; ++i) {
        const float us = c[i].us(tiles(c[i].bm, c[i].bn), stages);
        if (i == 0 || us < least) best = i, least = us;
    }
    return best;
}

// Whether an output's stores go past the L2: large ones, which no one finds there again (12000 rows of 4
// experts, 2008 x 1288, 87.7 us, cached 93.2; 4-bit 4000 x 4096 x 1024 16.1 and 17.4).  A small one may stay.
inline bool streams(int64_t bytes) { return bytes >= int64_t(8) << 20; }

// Workgroups that any division of M rows into `groups` groups can need.
inline int64_t group_tiles(int64_t M, int64_t groups, int64_t bm, int64_t tiles_n) {
    const int64_t full = M / bm + (groups < M ? groups : M);
    return full * tiles_n;
}

}  // namespace ssg

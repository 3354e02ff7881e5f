// Tile configurations of the GEMM skeleton and the rules that choose among them.
#pragma once

#include "gemm_core.h"

namespace ssg {

// Tile shapes (measured on MI355X at the ViT / BERT / ViT-Base shapes):
//   Big    256 x 256, 8 waves of 64 tokens x 128 channels, one workgroup per
//          CU -- best once there are about as many tiles as CUs and K is long
//          enough to amortise the prologue.  On the fp16 2:4 tile and the
//          dense tiles only waves 0..3 issue the loads, so each SIMD keeps
//          one wave whose matrix work no load waits behind (fp16 2:4 ViT-L
//          qkv 27.5 -> 26.3 us, fc1 31.5 -> 30.8; dense fp16 28.9 -> 28.1
//          and 37.3 -> 36.2; with two of the eight waves loading, no gain;
//          the int8 2:4 tile would spill, and the int8 Small2 tile with two
//          of four waves loading ran the headline 46.0 -> 48.7 us);
//   Mid    128 x 256, 4 waves, 2 stages (two workgroups per CU) -- short-K
//          int8 GEMMs with one to two such tiles per CU;
//   Small  128 x 128, 4 waves, 3 stages (two workgroups per CU) -- long-K
//          int8 GEMMs with more than 256 (dense: 576) such tiles, and the
//          8-way K splits of few-tile fp16 GEMMs;
//   SmallP the same tile with 4 more waves that only load (one workgroup
//          per CU) and, for the sparse kinds, metadata blocks of 4 (fp16) or
//          2 (int8) stages -- narrow outputs (N = 1024) that would leave CUs
//          idle with big tiles: every fp16 GEMM without enough Big tiles
//          (other than the few-tile ones of T64 / T32 below), and the long-K
//          int8 ones up to 256 tiles (dense: 576).  Against Small,
//          graph-timed on cold input sets: fp16 2:4 4096 x 1024 x 4096
//          (M x N x K) 42.3 -> 38.9 us, 4096 x 768 x 3072 31.5 -> 28.4,
//          6144 x 1024 x 4096 (384 tiles) 67.6 -> 63.4, 6144 x 1536 x 4096
//          (576) 96.8 -> 87.0; dense fp16 4096 x 1024 x 4096 43.1 -> 41.5;
//          int8 2:4 4096 x 768 x 3072 17.5 -> 16.5 us, but 6144 x 1024 x
//          4096 37.0 -> 39.0.  The int8 2:4 tile (unsplit, K a multiple of
//          256) takes stages twice as deep in K, 256 k with the metadata in
//          the stage (int8 2:4 4096 x 1024 x 4096 23.5 -> 20.8 us, 4096 x
//          768 x 3072 16.6 -> 16.0, 3072 x 1024 x 4096 20.7 -> 19.8); the
//          fp16 tiles run slower so (4096 x 1024 x 4096 37.7 -> 43.6), and
//          the dense ones, with two such stages, too.  Neither part pays alone (fp16 2:4 4096 x 1024
//          x 4096: metadata blocks 46.6-46.9 us, loader waves 45-46, both
//          41.5, Small 44.7-45.2 in that session): the metadata blocks cut
//          the cache lines the loads touch (a copy of the kernel without
//          fragment reads and matrix instructions ran 40.1 -> 34.8 us), and
//          only with the loads moved off the compute waves does the full
//          kernel follow;
//   Small2 128 x 128, 4 waves, 2 stages (three int8 workgroups per CU) --
//          short-K int8 GEMMs whose Mid tiles would fill the chip more than
//          twice or less than once, and the dense int8 GEMMs at short K;
//   T64    64 x 64 and T64N 64 x 128, 4 waves of 32 x 32 / 32 x 64, 3 stages
//          (the sparse fp16 T64N with 4 loader waves and 4-stage metadata
//          blocks: 512 x 3072 x 1024 9.6 -> 9.1 us, 512 x 4096 x 1024
//          10.6 -> 10.0, 2048 x 1024 x 4096 32.0 -> 27.7; the dense one runs
//          slower so, 10.4 -> 11.0 us at 512 x 3072 x 1024)
//          -- GEMMs with at most 128 tiles of 128 x 128 (half the CUs; int8
//          with K <= 1024: 192), e.g. one GPU's share of a token-sharded
//          layer (M = 512).  With so few
//          tiles each workgroup's K loop runs alone on its CU, limited by
//          what its four waves can pull into LDS per stage; smaller tiles
//          put more CUs to work and each moves less (int8 2:4 512 x 1024 x
//          1024: 9.2 us on 128 x 128, 5.8 on 64 x 64; 512 x 4096 x 1024:
//          19.6 -> 12.6 us; fp16 2:4 512 x 1024 x 1024: 10.7 us -> 9.0 on
//          64 x 128).  A deeper ring (4-6 stages) on 128 x 128 gained nothing
//          there.  The fp16 kinds keep 64 x 128 once 64 x 64 tiles would
//          outnumber the CUs (dense fp16 512 x 1024 x 3072: 10.1 us on
//          64 x 128, 11.1 on 64 x 64); int8, with half as many K stages,
//          takes 64 x 64 throughout;
//   T32    32 x 32, one wave, 4 stages -- the smallest GEMMs (at most 512
//          such tiles and fewer than 64 K stages).  Against 64-row tiles in
//          one sweep (its first, 3-stage rotated form): fp16 2:4 256 x 512 x
//          512 5.2 -> 4.4 us, 384 x 1024 x 1024 7.3 -> 6.4; int8 2:4 128 x
//          4096 x 4096 12.3 -> 10.5; at 1024 tiles (1024 x 1024 outputs) the
//          64-row tiles are ahead again.  The 4-stage ring from stage 0
//          (ROT below) took 256 x 512 x 512 to 3.8 us.
// K-loop start (ROT), measured with both variants timed in one process over
// alternating rounds, on input sets rotated through more than twice the
// 256 MB Infinity Cache: every dense kind and the sparse Big and Mid tiles run
// 3-10 % faster from stage 0 (ViT-L qkv / fc1 / fc2, 4096x8192x1024,
// 4096x2048x4096), while the sparse 128 x 128 tiles run 4-10 % faster rotated
// (fp16 ViT-L fc2 42.1 vs 46.2 us, int8 4096x8192x1024 43.7 vs 47.7 us; the
// short-K int8 one is within noise either way).  So ROT = sparse kind on a
// 128 x 128 tile, and on the sparse 64 x 128 tile (fp16 2:4 512 x 1024 x 4096
// 9.8 vs 10.2 us); the 64 x 64 and 32 x 32 tiles run faster from stage 0 (int8
// 2:4 512 x 1024 x 3072 6.6 vs 6.9 us on 64 x 64; 32 x 32 with a 4-stage ring:
// fp16 2:4 512 x 1024 x 1024 5.7 vs 6.5 us, int8 2:4 512 x 4096 x 1024 9.1 vs
// 10.6 us against the rotated 3-stage form).
template <bool NTS, int NLD = 0>
using CfgBig = Cfg<4, 2, 2, 4, 3, 8, NTS, false, 0, false, NLD>;
template <bool NTS>
using CfgBigDense = Cfg<4, 2, 2, 4, 2, 8, NTS, false, 0, false, 4>;
template <bool NTS>
using CfgMid = Cfg<2, 2, 2, 4, 2, 8, NTS, false>;
template <bool NTS, bool ROT>
using CfgSmall = Cfg<2, 2, 2, 2, 3, 8, NTS, ROT>;
template <bool NTS, bool ROT, int MP>
using CfgSmallP = Cfg<2, 2, 2, 2, 3, 8, NTS, ROT, MP, true>;
template <bool NTS, bool ROT>
using CfgSmallPD2 = Cfg<2, 2, 2, 2, 3, 8, NTS, ROT, 0, true, 0, 2>;
template <bool NTS, bool ROT>
using CfgSmall2 = Cfg<2, 2, 2, 2, 2, 8, NTS, ROT>;
template <bool NTS, bool ROT>
using CfgT64 = Cfg<2, 2, 1, 1, 3, 8, NTS, ROT>;
template <bool NTS, bool ROT>
using CfgT64N = Cfg<2, 2, 1, 2, 3, 8, NTS, ROT>;
template <bool NTS, bool ROT>
using CfgT64NP = Cfg<2, 2, 1, 2, 3, 8, NTS, ROT, 4, true>;
template <bool NTS>
using CfgT32 = Cfg<1, 1, 1, 1, 4, 8, NTS, false>;

enum Shape { SHAPE_BIG, SHAPE_MID, SHAPE_SMALL, SHAPE_SMALLP, SHAPE_SMALL2, SHAPE_T64, SHAPE_T64N, SHAPE_T32 };

inline long tiles(int M, int N, int bm, int bn) { return long((M + bm - 1) / bm) * long((N + bn - 1) / bn); }

// tile rows x columns of a shape
inline void tile_dims(Shape sh, int &bm, int &bn) {
    bm = sh == SHAPE_BIG ? 256 : (sh == SHAPE_T64 || sh == SHAPE_T64N) ? 64 : sh == SHAPE_T32 ? 32 : 128;
    bn = (sh == SHAPE_BIG || sh == SHAPE_MID) ? 256 : sh == SHAPE_T64 ? 64 : sh == SHAPE_T32 ? 32 : 128;
}

// few output tiles: at most `limit` tiles of 128 x 128 (128 = half the CUs)
inline bool few_tiles(int M, int N, long limit = 128) { return tiles(M, N, 128, 128) <= limit; }

// The smallest GEMMs (at most 512 tiles of 32 x 32, fewer than 64 K stages):
// one-wave 32 x 32 tiles.  Past 64 K stages such shapes split K on 64 x 64
// tiles instead, which is faster there (fp16 2:4 512 x 4096 x 1024: 15.6 us
// split vs 21.7 on 32 x 32).
inline bool tiny(int M, int N, int stages) { return stages < 64 && tiles(M, N, 32, 32) <= 512; }

// f16 kinds: big tiles when they still give >= 3/4 of a tile per CU; 64-row
// tiles for few-tile GEMMs.
inline Shape pick_f16(int M, int N, int K) {
    if (few_tiles(M, N)) {
        if (tiny(M, N, K / 64)) return SHAPE_T32;
        return tiles(M, N, 64, 64) <= 256 ? SHAPE_T64 : SHAPE_T64N;
    }
    return tiles(M, N, 256, 256) >= 192 ? SHAPE_BIG : SHAPE_SMALLP;
}

// int8 kinds.  Short K (<= 1024): the per-tile prologue and the output
// stream weigh most, so the choice follows how evenly the tiles fill the
// chip's workgroup slots (ViT-Base fc1 12608x768x3072: 1188 Mid tiles, Small2
// 45 us vs Mid 47.6; ViT-L qkv / fc1: 384 / 512 Mid tiles, Mid best; ViT-L
// proj: 128 Mid tiles, Small2 10.4 us vs Mid 14.0).  The dense kind keeps
// 2 x 96 KiB of stages for a Mid tile, i.e. one workgroup per CU, so it
// takes Small2 unless Big tiles fill the chip one to two times (ViT-L fc1).
// Long K: as the f16 kinds.
inline Shape pick_i8(int M, int N, int K, bool dense) {
    // (short K: up to 192 tiles; 1024 x 1024 x 3072 2:4 9.9 -> 9.1 us, dense
    // 9.9 -> 8.1; at 256 tiles within 5 %, and with K = 4096 at 192 tiles the
    // 128-row tiles stay ahead, 20.4 vs 24.7 us)
    if (few_tiles(M, N, K <= 1024 ? 192 : 128)) return tiny(M, N, K / 128) ? SHAPE_T32 : SHAPE_T64;
    if (K <= 1024) {
        if (dense) {
            const long big = tiles(M, N, 256, 256);
            return (big >= 256 && big <= 512) ? SHAPE_BIG : SHAPE_SMALL2;
        }
        const long mid = tiles(M, N, 128, 256);
        return (mid >= 256 && mid <= 512) ? SHAPE_MID : SHAPE_SMALL2;
    }
    if (tiles(M, N, 256, 256) >= 192) return SHAPE_BIG;
    return tiles(M, N, 128, 128) <= (dense ? 576 : 256) ? SHAPE_SMALLP : SHAPE_SMALL;
}

}  // namespace ssg

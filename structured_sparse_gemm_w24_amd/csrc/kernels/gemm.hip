// Dense and 2:4-sparse GEMMs for gfx950 on the skeleton of gemm_core.h (one
// skeleton, four kinds): the launchers.
#include "gemm_core.h"
#include "gemm_tiles.h"
#include "launch.h"

namespace ssg {

template <int KIND, int EPI, class CF>
static hipError_t launch(const void *A, const void *Wv, const uint32_t *meta, const float *scale,
                         const float *bias, void *C, int M, int N, int K, hipStream_t st, int splits = 1) {
    using LY = Layout<KIND, CF>;
    const int nb = ((M + LY::BM - 1) / LY::BM) * ((N + LY::BN - 1) / LY::BN);
    const int stages = K * (KindTraits<KIND>::kI8 ? 1 : 2) / (128 * CF::DK) / splits;
    hipLaunchKernelGGL((gemm_kernel<KIND, EPI, CF, NoExtra>), dim3(nb, splits), dim3(LY::NT), 0, st,
                       static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(Wv), meta, scale, bias, C, M, N,
                       K, stages, NoExtra{});
    return hipGetLastError();
}

template <int KIND, int EPI, bool NTS, bool DENSE>
static hipError_t launch_shape(Shape sh, const void *A, const void *Wv, const uint32_t *meta, const float *scale,
                               const float *bias, void *C, int M, int N, int K, hipStream_t st, int splits = 1) {
    if (sh == SHAPE_BIG) {
        if constexpr (DENSE) return launch<KIND, EPI, CfgBigDense<NTS>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
        else return launch<KIND, EPI, CfgBig<NTS, KIND == W24_F16 ? 4 : 0>>(A, Wv, meta, scale, bias, C, M, N, K, st,
                                                                          splits);
    }
    if (sh == SHAPE_MID) return launch<KIND, EPI, CfgMid<NTS>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
    constexpr bool ROT = KindTraits<KIND>::kSparse;
    if (sh == SHAPE_T64) {
        // split launches of the sparse kinds start rotated (fp16 2:4 512 x 4096
        // x 1024, 2 splits: 18.5 vs 19.4 us), unsplit ones from stage 0
        constexpr bool ROT64 = EPI == EPI_PART && KindTraits<KIND>::kSparse;
        return launch<KIND, EPI, CfgT64<NTS, ROT64>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
    }
    if (sh == SHAPE_T32) return launch<KIND, EPI, CfgT32<NTS>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
    if (sh == SHAPE_SMALLP) {
        // the int8 2:4 tile takes stages of 256 k when K allows (unsplit launches)
        if constexpr (KIND == W24_I8 && EPI != EPI_PART)
            if (K % 256 == 0)
                return launch<KIND, EPI, CfgSmallPD2<NTS, ROT>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
        constexpr int MP = !KindTraits<KIND>::kSparse ? 0 : KindTraits<KIND>::kI8 ? 2 : 4;
        return launch<KIND, EPI, CfgSmallP<NTS, ROT, MP>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
    }
    if constexpr (!KindTraits<KIND>::kI8) {  // (only the fp16 kinds pick T64N)
        if (sh == SHAPE_T64N) {
            if constexpr (KindTraits<KIND>::kSparse)
                return launch<KIND, EPI, CfgT64NP<NTS, ROT>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
            else return launch<KIND, EPI, CfgT64N<NTS, ROT>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
        }
    }
    if constexpr (KindTraits<KIND>::kI8)  // (only the int8 kinds pick Small2)
        if (sh == SHAPE_SMALL2)
            return launch<KIND, EPI, CfgSmall2<NTS, KindTraits<KIND>::kSparse>>(A, Wv, meta, scale, bias, C, M, N, K,
                                                                                st, splits);
    return launch<KIND, EPI, CfgSmall<NTS, KindTraits<KIND>::kSparse>>(A, Wv, meta, scale, bias, C, M, N, K, st, splits);
}

hipError_t launch_dense_f16(const void *A, const void *Wt, void *C, int M, int N, int K, hipStream_t st) {
    return launch_shape<DENSE_F16, EPI_F16, true, true>(pick_f16(M, N, K), A, Wt, nullptr, nullptr, nullptr, C, M, N, K,
                                                         st);
}

hipError_t launch_w24_f16(const void *A, const void *vals, const uint32_t *meta, void *C, int M, int N, int K,
                          hipStream_t st) {
    return launch_shape<W24_F16, EPI_F16, true, false>(pick_f16(M, N, K), A, vals, meta, nullptr, nullptr, C, M, N, K,
                                                        st);
}

// int8 kinds: out selects the epilogue (OUT_I32 raw accumulators; OUT_F32,
// OUT_F16 and OUT_I8 apply scale and the optional bias).  Every output kind
// keeps the int8 tile choice: with short K the main loop's operand traffic,
// not the output stream, sets most of the time (measured on the ViT-Base
// fc1 shape: fp32 / fp16 / int8 outputs 46.5 / 43.2 / 41.6 us).
template <int KIND, bool DENSE>
static hipError_t launch_i8(const void *A, const void *Wv, const uint32_t *meta, const float *scale,
                            const float *bias, void *C, int out, int M, int N, int K, hipStream_t st) {
    const Shape sh = pick_i8(M, N, K, DENSE);
    switch (out) {
        case OUT_I32:
            return launch_shape<KIND, EPI_I32, true, DENSE>(sh, A, Wv, meta, nullptr, nullptr, C, M, N, K, st);
        case OUT_F32:
            return launch_shape<KIND, EPI_F32_SCALE, true, DENSE>(sh, A, Wv, meta, scale, bias, C, M, N, K, st);
        case OUT_F16:
            return launch_shape<KIND, EPI_F16_SCALE, true, DENSE>(sh, A, Wv, meta, scale, bias, C, M, N, K, st);
        default:
            return launch_shape<KIND, EPI_I8_SCALE, true, DENSE>(sh, A, Wv, meta, scale, bias, C, M, N, K, st);
    }
}

hipError_t launch_dense_i8(const void *A, const void *Wt, const float *scale, const float *bias, void *C, int out,
                           int M, int N, int K, hipStream_t st) {
    return launch_i8<DENSE_I8, true>(A, Wt, nullptr, scale, bias, C, out, M, N, K, st);
}

hipError_t launch_w24_i8(const void *A, const void *vals, const uint32_t *meta, const float *scale, const float *bias,
                         void *C, int out, int M, int N, int K, hipStream_t st) {
    return launch_i8<W24_I8, false>(A, vals, meta, scale, bias, C, out, M, N, K, st);
}

}  // namespace ssg

namespace ssg {

// ---- split K.  The partial launches run the tile choice of the unsplit
// kinds with gridDim.y = splits and the EPI_PART epilogue (plain stores: the
// reduce launch reads the partials back right away).
// The tile of a split launch of the fp16 kinds.  Split launches read each
// weight once per tile row, cold from HBM, so where the split reaches one
// workgroup per CU with bigger tiles, those win (graph-timed, a fresh weight
// per call): fp16 2:4 512 x 4096 x 1024 16.9 us as 128 x 128 x 8 splits, 16.3
// as 64 x 128 x 4, 18.4 as 64 x 64 x 2; 512 x 8192 x 1024 21.9 / 23.2 / 30.6.
// A function of the shape and the split count alone, so an explicit split
// count gets a fixed tile too.
static Shape split_shape_f16(int M, int N, int K, int splits) {
    const Shape sh = pick_f16(M, N, K);
    if (sh != SHAPE_T64 && sh != SHAPE_T64N && sh != SHAPE_T32) return sh;
    const int S = K / 64;
    if (splits == 8 && M >= 128 && tiles(M, N, 128, 128) * 8 >= 256 && S / 8 >= 8) return SHAPE_SMALL;
    if (splits == 4 && tiles(M, N, 64, 128) * 4 >= 256 && S / 4 >= 8) return SHAPE_T64N;
    return sh;
}

hipError_t launch_gemm_partials(int kind, const void *A, const void *W, const uint32_t *meta, void *ws, int M,
                                int N, int K, int splits, hipStream_t st) {
    switch (kind) {
        case DENSE_F16:
            return launch_shape<DENSE_F16, EPI_PART, false, true>(split_shape_f16(M, N, K, splits), A, W, nullptr,
                                                                   nullptr, nullptr, ws, M, N, K, st, splits);
        case W24_F16:
            return launch_shape<W24_F16, EPI_PART, false, false>(split_shape_f16(M, N, K, splits), A, W, meta, nullptr,
                                                                  nullptr, ws, M, N, K, st, splits);
        case DENSE_I8:
            return launch_shape<DENSE_I8, EPI_PART, false, true>(pick_i8(M, N, K, true), A, W, nullptr, nullptr,
                                                                  nullptr, ws, M, N, K, st, splits);
        default:
            return launch_shape<W24_I8, EPI_PART, false, false>(pick_i8(M, N, K, false), A, W, meta, nullptr, nullptr,
                                                                 ws, M, N, K, st, splits);
    }
}

// Tile rows x columns the launchers pick for a kind and shape.
void tile_choice(int kind, int M, int N, int K, int *bm, int *bn) {
    const bool i8 = kind == DENSE_I8 || kind == W24_I8;
    const bool dense = kind == DENSE_F16 || kind == DENSE_I8;
    tile_dims(i8 ? pick_i8(M, N, K, dense) : pick_f16(M, N, K), *bm, *bn);
}

// Splitting K pays when a GEMM has few output tiles and a long K loop (one
// GPU's share of a token-sharded layer, e.g. 512 x 4096 x 1024): each tile's
// K loop is a chain of dependent stage loads, and cutting it into ranges run
// side by side shortens the chain, at the price of a second launch and the
// partials' round trip through memory (8 * M * N bytes per split).  Few-tile
// GEMMs already run on 64-row tiles (more workgroups, shorter chains per
// stage), so the split only pays from 64 K stages on.  Measured on MI355X
// with graph-timed replays on those tiles: fp16 2:4 512 x 4096 x 1024 (64
// stages, 128 tiles) 20.6 us unsplit, 15.6 with 2 splits; 128 x 4096 x 4096
// 20.2 -> 16.3; int8 2:4 512 x 8192 x 1024 21.1 -> 15.6; but with 32 stages
// (int8 512 x 4096 x 1024, fp16 256 x 2048 x 2048) 2 splits are no faster,
// and with more than 128 tiles every split loses (fp16 1024 x 4096 x 1024:
// 21.9 -> 26.5 us).  Within those bounds the splits double while tiles x
// splits stays within one workgroup per CU and every split keeps at least 8
// stages.
int suggest_splits(int kind, int M, int N, int K) {
    constexpr int kCUs = 256;
    if (M <= 0 || N <= 0 || K <= 0) return 1;
    const bool i8 = kind == DENSE_I8 || kind == W24_I8;
    const bool dense = kind == DENSE_F16 || kind == DENSE_I8;
    const Shape sh = i8 ? pick_i8(M, N, K, dense) : pick_f16(M, N, K);
    int bm, bn;
    tile_dims(sh, bm, bn);
    const long t = tiles(M, N, bm, bn);
    const int S = gemm_k_stages(kind, K);
    if (S < 64 || t > 128) return 1;
    if (!i8) {  // bigger tiles with more splits first (see split_shape_f16)
        for (int q : {8, 4})
            if (S % q == 0 && split_shape_f16(M, N, K, q) != sh) return q;
    }
    int p = 1;
    while (p < 16 && t * 2 * p <= kCUs && S % (2 * p) == 0 && S / (2 * p) >= 8) p *= 2;
    return p;
}

}  // namespace ssg

// Microscaled 4-bit floating point (E2M1 values, blocks of 32 along K that share a
// power-of-two scale; the MXFP4 format of the OCP Microscaling specification, v1.0):
// quantisation, its inverse, and products of packed operands.
//
//   scale byte = max(0, floor(log2 max|x|) - 2 + 127), the block's scale 2^(byte - 127);
//   code = nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 to |x| / scale, ties to the even code,
//          past 6: 6; bit 3 is the sign.  A block with an infinity or NaN has byte 255 and
//          stands for NaN.
//   C[m][n] = sum_k a[m][k] w[n][k], fp32 sums, rounded once.
//
// A lane of the scaled matrix instruction (32 x 32 x 64) holds 32 consecutive k of one
// row, which is one block: its 16 code bytes as they lie in memory, and one scale byte.
// So packed rows go to LDS as the other kinds' rows do, and the scales, 8 bytes a row and
// stage, beside them.
#include "elem.h"
#include "gemm_core.h"
#include "gemm_tiles.h"
#include "group_place.h"
#include "launch.h"
#include "mx_codes.h"

namespace ssg {

namespace {

// The piece `at` behind the first one of a workgroup, which is piece c0 of row m0 (one 64-bit division a
// workgroup).
struct Place {
    int64_t m;
    int c;
};
__device__ __forceinline__ Place piece_at(int64_t m0, uint32_t c0, uint32_t at, uint32_t pieces) {
    const uint32_t c = c0 + at, q = c / pieces;
    return {m0 + q, int(c - q * pieces) * 8};
}

// Pieces of eight values: four threads share a block, sixteen a word of four scales.  Each thread takes
// two, 256 apart, and has both loads under way before the first is used (8192 x 4096 fp16 16.5 us = 5.1
// TB/s, and 13.8 back; converted by way of fp32 bf16 took 17.8, one piece a thread 19.5, four 20.1).
constexpr int U = 2;
template <class T, bool TAIL>
__global__ void __launch_bounds__(256)
mx_quantize_kernel(const T *__restrict__ x, int64_t ldx, uint32_t *__restrict__ codes, uint32_t *__restrict__ scales,
                   int64_t M, int64_t K, int pieces) {  // pieces of a row: a multiple of 16
    constexpr int V = Elem<T>::V;
    const int64_t all = M * pieces, first = int64_t(blockIdx.x) * (256 * U), m0 = first / pieces;
    const uint32_t c0 = uint32_t(first - m0 * pieces);
    typename Elem<T>::Vec v[U][8 / V];
    int64_t col[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = u * 256 + threadIdx.x;
        if (first + at >= all) break;
        const Place p = piece_at(m0, c0, uint32_t(at), uint32_t(pieces));
        col[u] = p.c;
#pragma unroll
        for (int j = 0; j < 8 / V; ++j) v[u][j] = fetch_raw<T, TAIL>(x + p.m * ldx, p.c + j * V, K);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256 + threadIdx.x;
        if (i >= all) return;  // (a row's pieces are a multiple of 16: whole groups of lanes leave)
        Top<T> most;
#pragma unroll
        for (int j = 0; j < 8 / V; ++j) {
            v[u][j] = settle<T, TAIL>(v[u][j], col[u] + j * V, K);
            most.add(v[u][j]);
        }
        uint32_t top = most.bits();
        top = max(top, dpp<0xb1>(top));  // (quad permutations: lanes ^ 1, ^ 2)
        top = max(top, dpp<0x4e>(top));
        const uint32_t byte = scale_byte(top);
        codes[i] = codes_of<T>(v[u], byte);
        uint32_t word = byte << (8 * ((threadIdx.x >> 2) & 3));
        word |= dpp<0x124>(word);  // (row rotations by 4 and 8: all four quads of the row)
        word |= dpp<0x128>(word);
        if ((threadIdx.x & 15) == 0) scales[i >> 4] = word;
    }
}

template <class T, bool TAIL>
__global__ void __launch_bounds__(256)
mx_dequantize_kernel(const uint32_t *__restrict__ codes, const uint8_t *__restrict__ scales, T *__restrict__ out,
                     int64_t ldo, int64_t M, int64_t K, int pieces) {
    const int64_t all = M * pieces, first = int64_t(blockIdx.x) * (256 * U), m0 = first / pieces;
    const uint32_t c0 = uint32_t(first - m0 * pieces);
    uint32_t word[U], byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = first + u * 256 + threadIdx.x;
        if (i >= all) break;
        byte[u] = scales[i >> 2], word[u] = codes[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = u * 256 + threadIdx.x;
        if (first + at >= all) return;
        const Place p = piece_at(m0, c0, uint32_t(at), uint32_t(pieces));
        const int64_t m = p.m, c = p.c;
        const uint32_t b = byte[u], v = word[u];
        const float s = b == 255 ? __builtin_nanf("") : scale_of(b);
        typedef float f2 __attribute__((ext_vector_type(2)));
        const f2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 0);
        const f2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 1);
        const f2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 2);
        const f2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v, 1.0f, 3);
        const float f[8] = {p0.x * s, p0.y * s, p1.x * s, p1.y * s, p2.x * s, p2.y * s, p3.x * s, p3.y * s};
        constexpr int V = Elem<T>::V;
#pragma unroll
        for (int j = 0; j < 8; j += V) {
            float g[V];
#pragma unroll
            for (int q = 0; q < V; ++q) g[q] = f[j + q];
            if (c + j < K) store_vec<T, false, TAIL>(out + m * ldo, c + j, K, g);
        }
    }
}

// ---- products
template <bool GROUPED, int OB>
struct MxProduct {
    static constexpr bool kAfter = false, kEpilogue = false, kTransA = false, kTransW = false, kPlace = true;
    const int32_t *offsets;
    int groups;
    const uint8_t *sa, *sw;
    int64_t a_row, ldc;  // bytes of a packed row; elements between C's rows
    // Stores past the L2: large outputs whose rows are whole 64 bytes (others leave parts of cache lines in
    // every piece, which then go to memory one by one: 7648 x 3000 x 533 25.4 us, cached 23.2; but 16384 x
    // 4096 x 1024 61.6 and 65.3)
    bool stream;

    template <class CF, int BM, int BN>
    __device__ __forceinline__ bool place(int block, const uint8_t *&A, const uint8_t *&W, void *&C, int &M, int N,
                                          int K, int &, int &n0) {
        const int tiles_n = (N + BN - 1) / BN;
        int row, rows;
        if constexpr (GROUPED) {
            const group::Tile t = group::find_tile<BM>(block, offsets, groups, M, tiles_n, CF::GM);
            if (t.group < 0) return false;
            row = t.row, rows = t.rows, n0 = t.tile_n * BN;
            W += int64_t(t.group) * N * a_row;
            sw += int64_t(t.group) * N * (K / 32);
        } else {
            const int tiles_m = (M + BM - 1) / BM;
            const int b = xcd_remap(block, tiles_m * tiles_n);
            const int super = b / (CF::GM * tiles_n), gm = min(tiles_m - super * CF::GM, CF::GM);
            const int in = b % (CF::GM * tiles_n);
            row = (super * CF::GM + in % gm) * BM, rows = M - row, n0 = in / gm * BN;
        }
        A += row * a_row;
        sa += int64_t(row) * (K / 32);
        C = static_cast<uint8_t *>(C) + row * ldc * OB;
        M = rows;
        return true;
    }
};

template <int EPI, class CF, bool GROUPED>
hipError_t gemm_cfg(const Mxfp4Gemm &g, int K, hipStream_t st) {
    using LY = Layout<MX_F4, CF>;
    constexpr int OB = EPI == EPI_F32 ? 4 : 2;
    const bool whole = g.ldo * OB % 64 == 0 && reinterpret_cast<uintptr_t>(g.out) % 64 == 0;
    const MxProduct<GROUPED, OB> ex{g.offsets, g.experts, g.a_scales, g.w_scales, K / 2, g.ldo,
                                    whole && streams(g.M * g.N * OB)};
    const int64_t tiles_n = (g.N + LY::BN - 1) / LY::BN;
    const int64_t blocks =
        GROUPED ? group_tiles(g.M, g.experts, LY::BM, tiles_n) : (g.M + LY::BM - 1) / LY::BM * tiles_n;
    hipLaunchKernelGGL((gemm_kernel<MX_F4, EPI, CF, MxProduct<GROUPED, OB>>), dim3(unsigned(blocks)), dim3(LY::NT), 0,
                       st, g.a, g.w, nullptr, nullptr, nullptr, g.out, int(g.M), int(g.N), K, (K + 255) / 256, ex);
    return hipGetLastError();
}

// Tiles: the largest keep a whole stage's fragments in registers (CfgDeep: 8192^3 261 us, the same tile
// without 313, eight waves of two a SIMD 329); 128 x 128 ones share a CU in pairs, one's epilogue under
// the other's main loop, which short K likes (6000 x 4096 x 1024 22.3 us, 256 x 256 26.7).
using Mx32x32 = Cfg<1, 1, 1, 1, 4, 8, true, false, 0, true>;
using Mx64x64 = CfgDeep<1, 1, 8, true>;
using Mx64x128 = CfgDeep<1, 2, 8, true>;
using Mx128x128 = CfgDeep<2, 2, 8, true>;
using Mx192x256 = CfgDeep<3, 4, 8, true>;
using Mx256x256 = CfgDeep<4, 4, 4, true>;
constexpr TileCost kMxTiles[] = {{32, 32, 6, 4.5f, 2.2f, 0.10f},   {64, 64, 4, 4.3f, 1.7f, 0.21f},
                                 {64, 128, 2, 3.7f, 2.2f, 0.36f},  {128, 128, 2, 3.6f, 3.2f, 0.49f},
                                 {192, 256, 1, 1.4f, 7.5f, 1.13f}, {256, 256, 1, 2.3f, 8.8f, 1.31f}};

// (experts 0: one product)
int mx_tile(int64_t M, int64_t experts, int64_t N, int64_t K) {
    const GroupRowsGuess guess(M, experts ? experts : 1);
    auto count = [&](int bm, int bn) { return guess.tiles(bm) * double((N + bn - 1) / bn); };
    return cheapest(kMxTiles, double((K + 255) / 256), count);
}

template <int EPI, bool GROUPED>
hipError_t gemm_any(const Mxfp4Gemm &g, hipStream_t st) {
    const int K = int(mxfp4_padded(g.K));
    switch (mx_tile(g.M, GROUPED ? g.experts : 0, g.N, g.K)) {
        case 0: return gemm_cfg<EPI, Mx32x32, GROUPED>(g, K, st);
        case 1: return gemm_cfg<EPI, Mx64x64, GROUPED>(g, K, st);
        case 2: return gemm_cfg<EPI, Mx64x128, GROUPED>(g, K, st);
        case 3: return gemm_cfg<EPI, Mx128x128, GROUPED>(g, K, st);
        case 4: return gemm_cfg<EPI, Mx192x256, GROUPED>(g, K, st);
        default: return gemm_cfg<EPI, Mx256x256, GROUPED>(g, K, st);
    }
}

template <int EPI>
hipError_t gemm_epi(const Mxfp4Gemm &g, hipStream_t st) {
    return g.offsets ? gemm_any<EPI, true>(g, st) : gemm_any<EPI, false>(g, st);
}

template <class T>
hipError_t quantize(const void *x, int64_t ldx, uint8_t *codes, uint8_t *scales, int64_t M, int64_t K,
                    hipStream_t st) {
    const int pieces = int(mxfp4_padded(K) / 8);
    const dim3 grid(unsigned((M * pieces + 256 * U - 1) / (256 * U)));
    auto k = K % Elem<T>::V == 0 ? mx_quantize_kernel<T, false> : mx_quantize_kernel<T, true>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, st, static_cast<const T *>(x), ldx, reinterpret_cast<uint32_t *>(codes),
                       reinterpret_cast<uint32_t *>(scales), M, K, pieces);
    return hipGetLastError();
}

template <class T>
hipError_t dequantize(const uint8_t *codes, const uint8_t *scales, void *out, int64_t ldo, int64_t M, int64_t K,
                      hipStream_t st) {
    const int pieces = int(mxfp4_padded(K) / 8);
    const dim3 grid(unsigned((M * pieces + 256 * U - 1) / (256 * U)));
    auto k = K % Elem<T>::V == 0 ? mx_dequantize_kernel<T, false> : mx_dequantize_kernel<T, true>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, st, reinterpret_cast<const uint32_t *>(codes), scales,
                       static_cast<T *>(out), ldo, M, K, pieces);
    return hipGetLastError();
}

}  // namespace

// One launch for few rows (mxfp4_few.hip): its tiles of 32 rows, and what one costs in us for each unit of
// 256 k of a wave's, for a unit of a CU's share of all tiles, and for eight of a CU's waves.
struct FewCost {
    int bn, waves;
    float start, unit, load, waves8;
};
// with up to 8 rows a tile, and with more
constexpr FewCost kFewTiles[2][3] = {
    {{32, 4, 2.8f, 0.85f, 0.21f, 0.70f}, {32, 8, 2.4f, 1.05f, 0.20f, 1.35f}, {64, 4, 2.65f, 1.25f, 0.44f, 0.80f}},
    {{32, 4, 2.8f, 2.20f, 0.35f, 0.70f}, {32, 8, 2.4f, 2.60f, 0.41f, 1.35f}, {64, 4, 2.65f, 2.75f, 0.48f, 0.80f}}};

// The choice between one launch and two (quantisation and product: 1.76 times the product's estimate less
// 4.6) by least estimate, fitted as TileCost's to launches in graphs.  Up to 16 units, where the estimates of
// both are close, two count 1 us more: the second launch costs the host 3 us (32 rows of 32 experts, 2048 x 1024,
// a call 13.1 us, in one launch 10.5; in a graph 10.9 and 10.5).  Past that one launch may be far off its
// estimate (157 x 288 x 6100 27.3 us, two 13.3).  Over 224 random calls of 1 to 362 rows the choice takes in
// graphs 1.019 times the best of all four, called 1.022 times; without the microsecond 1.021 and 1.032, with it
// for any K 1.028 and 1.030, always two launches 1.33 and 1.26.  A packed operand goes the same way, so that
// the product of quantised rows is the same bit for bit.  (Past the fit, and with more than 2000 units of full
// tiles, always two: 334 rows of 22 experts, 7040 x 500, 16.2 us and 29.5.)
int mxfp4_few_kind(int64_t M, int64_t experts, int64_t N, int64_t K) {
    if (M > 512) return -1;
    const GroupRowsGuess guess(M, experts ? experts : 1);
    const double tiles = guess.tiles(32), units = double((K + 255) / 256);
    const bool full = double(M) > 8.0 * tiles;
    auto columns = [&](int bn) { return double((N + bn - 1) / bn); };
    if (full && tiles * columns(32) * units > 2000.0) return -1;
    const TileCost &two = kMxTiles[mx_tile(M, experts, N, K)];
    double least = 1.76 * two.us(guess.tiles(two.bm) * columns(two.bn), units) - (units <= 16.0 ? 3.6 : 4.6);
    int best = -1;
    for (int i = 0; i < 3; ++i) {
        const FewCost &c = kFewTiles[full][i];
        const double all = tiles * columns(c.bn), each = double((int64_t(units) + c.waves - 1) / c.waves);
        const double us = c.start + (experts ? 0.45 : 0.0) + each * c.unit + all * units / 256.0 * c.load +
                          all * c.waves / 2048.0 * c.waves8;
        if (us < least) best = i, least = us;
    }
    return best;
}

int mxfp4_tile(int64_t M, int64_t experts, int64_t N, int64_t K) { return mx_tile(M, experts, N, K); }

int64_t mxfp4_blocks(int64_t M, int64_t experts, int64_t N, int64_t K) {
    const int few = mxfp4_few_kind(M, experts, N, K);
    const TileCost &t = kMxTiles[mx_tile(M, experts, N, K)];
    const int bm = few < 0 ? t.bm : 32, bn = few < 0 ? t.bn : kFewTiles[0][few].bn;
    const int64_t tiles_n = (N + bn - 1) / bn;
    return experts ? group_tiles(M, experts, bm, tiles_n) : (M + bm - 1) / bm * tiles_n;
}

hipError_t launch_mxfp4_quantize(int dtype, const void *x, int64_t ldx, uint8_t *codes, uint8_t *scales, int64_t M,
                                 int64_t K, hipStream_t st) {
    if (dtype == DT_F16) return quantize<_Float16>(x, ldx, codes, scales, M, K, st);
    if (dtype == DT_BF16) return quantize<__bf16>(x, ldx, codes, scales, M, K, st);
    return quantize<float>(x, ldx, codes, scales, M, K, st);
}

hipError_t launch_mxfp4_dequantize(int dtype, const uint8_t *codes, const uint8_t *scales, void *out, int64_t ldo,
                                   int64_t M, int64_t K, hipStream_t st) {
    if (dtype == DT_F16) return dequantize<_Float16>(codes, scales, out, ldo, M, K, st);
    if (dtype == DT_BF16) return dequantize<__bf16>(codes, scales, out, ldo, M, K, st);
    return dequantize<float>(codes, scales, out, ldo, M, K, st);
}

hipError_t launch_mxfp4_gemm(const Mxfp4Gemm &g, hipStream_t st) {
    if (mxfp4_few_kind(g.M, g.offsets ? g.experts : 0, g.N, g.K) >= 0) return launch_mxfp4_few(g, -1, 0, st);
    if (g.dtype == DT_F16) return gemm_epi<EPI_F16>(g, st);
    if (g.dtype == DT_BF16) return gemm_epi<EPI_BF16>(g, st);
    return gemm_epi<EPI_F32>(g, st);
}

}  // namespace ssg

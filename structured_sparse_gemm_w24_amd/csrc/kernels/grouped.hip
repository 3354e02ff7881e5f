// Products grouped by expert: rows offsets[e] .. offsets[e + 1] of x meet expert e's weight.
//
//   out[m] = w[e] . x[m]                 (forward, w[e] [N][K])
//   dx[m]  = w[e]^T . dy[m]
//   dw[e]  = sum over e's rows of dy[m] x[m]^T
//
// All three run on the GEMM skeleton (gemm_core.h), whose place() hook finds a
// workgroup's tile (group_place.h).  dx reads w[e] as it lies, summed along its
// rows, and dw both dy and x, through transposing LDS reads; a group's last rows
// end its buffer, so that the rows of the next expert never enter a sum.  dw's
// groups have K loops of different lengths in one launch; with few tiles of many rows
// each group's rows are split over several workgroups, whose fp32 sums a second launch
// adds in order.
//
// Measured: 16384 rows of 16 experts, 4096 x 1024, forward fp16 151 to 162 us by card (850 to 910 TFLOP/s),
// gradients bf16 315 (870); with all rows at one of many experts dw is slow (16384 of 64, 1024 x 1024, 374 us, even 73);
// bound by the start and end of loops of 16 stages, the gradients by their transposing LDS reads.
#include "elem.h"
#include "gemm_core.h"
#include "gemm_tiles.h"
#include "group_place.h"
#include "launch.h"

namespace ssg {

namespace {

// forward (TW false) and dx (TW true): tiles of a group's rows.
template <bool TW>
struct GroupRows {
    static constexpr bool kAfter = false, kEpilogue = false, kTransA = false, kTransW = TW, kPlace = true;
    const int32_t *offsets;
    int groups;
    int64_t a_row, ldc, w_bytes;  // bytes between A's rows, elements between C's, bytes of a weight
    int ldw, rows_w;              // (TW)
    bool stream;                  // stores past the L2: large outputs

    template <class CF, int BM, int BN>
    __device__ __forceinline__ bool place(int block, const uint8_t *&A, const uint8_t *&W, void *&C, int &M, int N,
                                          int, int &, int &n0) const {
        const group::Tile t = group::find_tile<BM>(block, offsets, groups, M, (N + BN - 1) / BN, CF::GM);
        if (t.group < 0) return false;
        A += t.row * a_row;
        W += t.group * w_bytes;
        C = static_cast<uint16_t *>(C) + t.row * ldc;
        M = t.rows;
        n0 = t.tile_n * BN;
        return true;
    }
};

// dw: every tile of every expert; M and N are the weight's sides.  splits > 1: the launch repeats for
// each share of a group's K stages and writes its sums, fp32, to slices of all experts' weights.
template <int OB>
struct GroupWeights {
    static constexpr bool kAfter = false, kEpilogue = false, kTransA = true, kTransW = true, kPlace = true, stream = true;
    const int32_t *offsets;
    int groups, rows, splits;
    bool sorted;
    int64_t a_row, ldc;  // (a_row: unused)
    int lda, ldw;
    int rows_a, rows_w;        // (unused: the stages' buffers take bytes_a and bytes_w)
    int64_t bytes_a, bytes_w;  // of the group's rows, from the tile's first column on

    template <class CF, int BM, int BN>
    __device__ __forceinline__ bool place(int block, const uint8_t *&A, const uint8_t *&W, void *&C, int &M, int N,
                                          int, int &stages, int &n0) {
        const int tiles_n = (N + BN - 1) / BN, each = (M + BM - 1) / BM * tiles_n;
        // (every expert's tiles are spread over the XCDs: a popular expert is no XCD's alone)
        const int share = block / (each * groups), tile = block - share * (each * groups);
        const int j = xcd_remap(tile % each, each);
        int lo, hi;
        const int g = group::nth_group(offsets, groups, rows, tile / each, sorted, lo, hi);
        if (lo == hi && splits == 1) {
            // an expert without rows: its zeros as one run, a share for each of its workgroups (as tiles,
            // rows of any width leave parts of cache lines: 58 experts, mostly empty, 872 x 2936 118 us)
            const int64_t pieces = int64_t(M) * N * OB / 16, n = (pieces + each - 1) / each;
            const int64_t first = (tile % each) * n, last = min(first + n, pieces);
            u32x4 *const out = static_cast<u32x4 *>(C) + g * pieces;
            for (int64_t i = first + threadIdx.x; i < last; i += blockDim.x)
                __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, out + i);
            return false;
        }
        const int all = (hi - lo + 63) / 64, per = (all + splits - 1) / splits, from = min(share * per, all);
        stages = min(per, all - from);
        lo += from * 64;
        const int m0 = j / tiles_n * BM;
        n0 = j % tiles_n * BN;
        A += (int64_t(lo) * lda + m0) * 2;
        W += int64_t(lo) * ldw * 2;
        C = static_cast<uint8_t *>(C) + ((int64_t(share) * groups + g) * M + m0) * ldc * OB;
        bytes_a = (int64_t(hi - lo - 1) * lda + M - m0) * 2;
        bytes_w = (int64_t(hi - lo - 1) * ldw + N) * 2;
        M -= m0;
        return true;
    }
};

// Sums the splits' slices in order: eight weights a thread.
template <class T>
__global__ void __launch_bounds__(256)
group_sum_kernel(const float *__restrict__ part, int splits, int64_t size, T *__restrict__ out) {
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
    if (i >= size) return;
    float v[8] = {};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const floatx4 a = *reinterpret_cast<const floatx4 *>(part + s * size + i);
        const floatx4 b = *reinterpret_cast<const floatx4 *>(part + s * size + i + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += a[j], v[4 + j] += b[j];
    }
    typename Elem<T>::Vec t;
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = T(v[j]);
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, t), reinterpret_cast<u32x4 *>(out + i));
}

template <int KIND, class CF, class Extra, int EPI = KIND == DENSE_F16 ? EPI_F16 : EPI_BF16>
hipError_t launch_cfg(const void *A, const void *W, void *C, const Extra &ex, int64_t blocks, int M, int N, int K,
                      hipStream_t st) {
    using LY = Layout<KIND, CF>;
    hipLaunchKernelGGL((gemm_kernel<KIND, EPI, CF, Extra>), dim3(unsigned(blocks)), dim3(LY::NT), 0, st,
                       static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(W), nullptr, nullptr, nullptr, C,
                       M, N, K, (K + 63) / 64, ex);
    return hipGetLastError();
}

// Tiles: with few of them the smallest, whose loads have waves of their own (a chain of K stages, each
// waiting for memory: 2324 rows of 8 groups, 72 x 1560, 8.7 us, 64 x 64 without loader waves 10.9,
// 64 x 128 12.9); the forward's largest keep a stage's fragments in registers (side by side in a sweep of
// tiles on one card: 16384 rows of 16, 4096 x 1024, 141 us, with eight waves instead 145; 8192 of 8, 2048 x
// 2048, 192 x 256 77, 256 x 256 95); dx needs loader waves at nearly every size, as its transposing reads keep
// the others busy (8192 rows of 8, 2048 x 2048: 87 us on 192 x 128 with, 123 on 192 x 256 without).
using Cfg32x64 = Cfg<1, 2, 1, 1, 4, 8, true, false, 0, true>;
using Cfg64x64 = Cfg<2, 2, 1, 1, 3, 8, true, false>;
using Cfg64x64P = Cfg<2, 2, 1, 1, 4, 8, true, false, 0, true>;
using Cfg64x128 = Cfg<2, 2, 1, 2, 3, 8, true, false>;
using Cfg64x128P = Cfg<2, 2, 1, 2, 3, 8, true, false, 0, true>;
using Cfg128x128 = CfgDeep<2, 2, 8, true>;
using Cfg128x128P = Cfg<2, 2, 2, 2, 4, 8, true, false, 0, true>;
using Cfg192x128P = Cfg<2, 2, 3, 2, 4, 8, true, false, 0, true>;
using Cfg256x128P = Cfg<2, 2, 4, 2, 3, 8, true, false, 0, true>;
using Cfg192x256 = CfgDeep<3, 4, 4, true>;
using Cfg256x256 = CfgDeep<4, 4, 4, true>;
constexpr TileCost kFwdTiles[] = {{32, 64, 3, 3.9f, 0.8f, 0.19f},  {64, 64, 3, 4.7f, 0.1f, 0.29f},
                                  {64, 128, 2, 4.5f, 0.6f, 0.45f}, {128, 128, 2, 2.9f, 1.9f, 0.59f},
                                  {192, 128, 1, 0.1f, 4.8f, 0.70f}, {192, 256, 1, 0.7f, 6.6f, 1.07f},
                                  {256, 256, 1, 2.4f, 6.6f, 1.25f}};
constexpr TileCost kDxTiles[] = {{32, 64, 3, 3.7f, 0.7f, 0.22f},   {64, 64, 2, 3.6f, 1.3f, 0.31f},
                                 {64, 128, 1, 2.4f, 1.1f, 0.46f},  {128, 128, 1, 0.0f, 4.3f, 0.58f},
                                 {128, 128, 2, 4.6f, 0.9f, 0.77f}, {192, 128, 1, 0.0f, 5.6f, 0.67f},
                                 {256, 256, 1, 0.0f, 6.7f, 1.75f}};
constexpr TileCost kDwTiles[] = {{32, 64, 3, 3.1f, 1.2f, 0.21f},   {64, 128, 1, 3.9f, 0.9f, 0.45f},
                                 {128, 128, 2, 2.2f, 1.8f, 1.01f}, {128, 128, 1, 3.0f, 2.2f, 0.66f},
                                 {256, 128, 1, 3.6f, 3.6f, 1.04f}, {256, 256, 1, 1.9f, 4.5f, 2.41f}};

template <int KIND, class CF, bool TW>
hipError_t rows_cfg(const Grouped &a, const void *A, int64_t lda, void *C, int64_t ldc, int N, int K, hipStream_t st) {
    using LY = Layout<KIND, CF>;
    const GroupRows<TW> ex{a.offsets, a.experts, lda * 2, ldc, int64_t(N) * K * 2, N, K, streams(a.M * N * 2)};
    const int64_t blocks = group_tiles(a.M, a.experts, LY::BM, (N + LY::BN - 1) / LY::BN);
    return launch_cfg<KIND, CF>(A, a.w, C, ex, blocks, int(a.M), N, K, st);
}

// Entry of kFwdTiles, kDxTiles (TW) and kDwTiles for a product.
template <bool TW>
int rows_tile(int64_t M, int64_t experts, int64_t N, int64_t K) {
    const GroupRowsGuess guess(M, experts);
    auto count = [&](int bm, int bn) { return guess.tiles(bm) * double((N + bn - 1) / bn); };
    const double stages = double((K + 63) / 64);
    if constexpr (TW) return cheapest(kDxTiles, stages, count);
    else return cheapest(kFwdTiles, stages, count);
}
// dw's tile and splits: the least of the tiles' cost, with each group's stages in up to 32 shares of
// four at least, and for more than one share the second launch and the slices' way through memory
// (16384 rows of one expert, 1024 x 1024: 113 us in one share; below 256 MiB of slices).  Shares are for few
// tiles: the largest is never the cheapest with more than one (of 5 million random calls), and not compiled for it.
struct WeightsPlan {
    int tile, splits;
};
WeightsPlan weights_plan(int64_t M, int64_t experts, int64_t N, int64_t K) {
    const double even = double(M) / double(experts) / 64.0 + 0.5, stages = even < 1.0 ? 1.0 : even;
    const double slice = double(experts) * double(N) * double(K) * 4.0;
    WeightsPlan best{0, 1};
    float least = 0.0f;
    for (int p = 1; p <= 32; p *= 2) {
        if (p > 1 && (stages < 4.0 * p || slice * p > double(1 << 28))) break;
        auto count = [&](int bm, int bn) {
            return double(p) * double(experts) * double((N + bm - 1) / bm) * double((K + bn - 1) / bn);
        };
        const int t = cheapest(kDwTiles, stages / p, count, p > 1 ? 5 : 6);
        float us = kDwTiles[t].us(count(kDwTiles[t].bm, kDwTiles[t].bn), stages / p);
        if (p > 1) us += 4.0f + float(slice * (2 * p + 0.5) / 5.0e6);
        if (p == 1 || us < least) best = {t, p}, least = us;
    }
    return best;
}

// The tile of a launch of both, or -1: two launches.  A tile of the joint launch costs what it does in
// either; together they take nine tenths of the longest tile or of the CUs' share, whichever is more.
constexpr struct {
    TileCost dx, dw;
} kBothTiles[] = {{kDxTiles[0], kDwTiles[0]}, {kDxTiles[2], kDwTiles[1]}, {kDxTiles[3], kDwTiles[3]}};
int both_tile(const WeightsPlan &pl, int64_t M, int64_t experts, int64_t N, int64_t K) {
    if (pl.splits > 1) return -1;
    const double sx = double((N + 63) / 64), even = double(M) / double(experts) / 64.0 + 0.5, sw = even < 1.0 ? 1.0 : even;
    const GroupRowsGuess guess(M, experts);
    auto count_x = [&](int bm, int bn) { return guess.tiles(bm) * double((K + bn - 1) / bn); };
    auto count_w = [&](int bm, int bn) {
        return double(experts) * double((N + bm - 1) / bm) * double((K + bn - 1) / bn);
    };
    auto us = [&](const TileCost &t, double stages, auto count) { return t.us(count(t.bm, t.bn), stages); };
    float least = us(kDxTiles[rows_tile<true>(M, experts, K, N)], sx, count_x) + us(kDwTiles[pl.tile], sw, count_w);
    int best = -1;
    for (int i = 0; i < 3; ++i) {
        const TileCost &x = kBothTiles[i].dx, &w = kBothTiles[i].dw;
        const double total = (count_x(x.bm, x.bn) * (x.tile / x.per_cu + sx * x.stage) +
                              count_w(w.bm, w.bn) * (w.tile / w.per_cu + sw * w.stage)) / 256.0;
        double longest = x.tile + sx * x.stage;
        if (w.tile + sw * w.stage > longest) longest = w.tile + sw * w.stage;
        const float t = 5.0f + 0.9f * float(total > longest ? total : longest);
        if (t < least) best = i, least = t;
    }
    return best;
}

template <int KIND, bool TW>
hipError_t rows(const Grouped &a, const void *A, int64_t lda, void *C, int64_t ldc, int N, int K, hipStream_t st) {
#define SSG_TILE(i, CF) \
    case i: return rows_cfg<KIND, CF, TW>(a, A, lda, C, ldc, N, K, st)
    if constexpr (TW) {
        switch (rows_tile<true>(a.M, a.experts, N, K)) {
            SSG_TILE(0, Cfg32x64);
            SSG_TILE(1, Cfg64x64P);
            SSG_TILE(2, Cfg64x128P);
            SSG_TILE(3, Cfg128x128P);
            SSG_TILE(4, Cfg128x128);
            SSG_TILE(5, Cfg192x128P);
            default: return rows_cfg<KIND, CfgBigDense<true>, TW>(a, A, lda, C, ldc, N, K, st);
        }
    } else {
        switch (rows_tile<false>(a.M, a.experts, N, K)) {
            SSG_TILE(0, Cfg32x64);
            SSG_TILE(1, Cfg64x64);
            SSG_TILE(2, Cfg64x128);
            SSG_TILE(3, Cfg128x128);
            SSG_TILE(4, Cfg192x128P);
            SSG_TILE(5, Cfg192x256);
            default: return rows_cfg<KIND, Cfg256x256, TW>(a, A, lda, C, ldc, N, K, st);
        }
    }
#undef SSG_TILE
}

// Whether dw's longest groups go first, so that no long sum is the last to start (16384 rows of 64 experts,
// 1024 x 1024, dw 79.9 us in their own order, 74.6 sorted; 8192 of 8, 2048 x 2048, 95.2 and 90.1); with short
// sums finding the order costs more than it gives (64 rows of 32, 1024 x 2048, 29.1 and 36.4).
bool long_sums(const Grouped &a) { return a.M >= 128 * int64_t(a.experts); }

template <int KIND, class CF, bool SPLIT>
hipError_t weights_cfg(const Grouped &a, int splits, hipStream_t st) {
    using LY = Layout<KIND, CF>;
    GroupWeights<SPLIT ? 4 : 2> ex{};
    ex.offsets = a.offsets, ex.groups = a.experts, ex.rows = int(a.M), ex.splits = splits, ex.ldc = a.K;
    ex.sorted = long_sums(a);
    ex.lda = int(a.lddy), ex.ldw = int(a.ldx);
    const int64_t blocks = splits * a.experts * ((a.N + LY::BM - 1) / LY::BM) * ((a.K + LY::BN - 1) / LY::BN);
    if constexpr (SPLIT)
        return launch_cfg<KIND, CF, GroupWeights<4>, EPI_F32>(a.dy, a.x, a.ws, ex, blocks, int(a.N), int(a.K), 0, st);
    else return launch_cfg<KIND, CF>(a.dy, a.x, a.dw, ex, blocks, int(a.N), int(a.K), 0, st);
}

template <int KIND, bool SPLIT>
hipError_t weights_any(const Grouped &a, const WeightsPlan &pl, hipStream_t st) {
    switch (pl.tile) {
        case 0: return weights_cfg<KIND, Cfg32x64, SPLIT>(a, pl.splits, st);
        case 1: return weights_cfg<KIND, Cfg64x128P, SPLIT>(a, pl.splits, st);
        case 2: return weights_cfg<KIND, Cfg<2, 2, 2, 2, 2, 8, true, false>, SPLIT>(a, pl.splits, st);
        case 3: return weights_cfg<KIND, Cfg128x128P, SPLIT>(a, pl.splits, st);
        case 4: return weights_cfg<KIND, Cfg256x128P, SPLIT>(a, pl.splits, st);
        default: break;
    }
    if constexpr (SPLIT) return hipErrorInvalidValue;
    else return weights_cfg<KIND, CfgBigDense<true>, false>(a, 1, st);
}

template <int KIND>
hipError_t weights(const Grouped &a, const WeightsPlan &pl, hipStream_t st) {
    if (pl.splits == 1) return weights_any<KIND, false>(a, pl, st);
    hipError_t e = weights_any<KIND, true>(a, pl, st);
    if (e != hipSuccess) return e;
    using T = typename std::conditional<KIND == DENSE_F16, _Float16, __bf16>::type;
    const int64_t size = a.experts * a.N * a.K;  // (a multiple of 8)
    hipLaunchKernelGGL(group_sum_kernel<T>, dim3(unsigned((size / 8 + 255) / 256)), dim3(256), 0, st,
                       static_cast<const float *>(a.ws), pl.splits, size, static_cast<T *>(a.dw));
    return hipGetLastError();
}

// dx and dw in one launch: the first `first` workgroups are dx's tiles, the others dw's.  Small calls
// are two chains of latencies, which then run side by side, and one launch (1531 rows of 6 experts,
// 776 x 1000: 22.0 us in two launches, 17.9 in one; 307 rows of one, 176 x 2736: 12.5 and 7.1); the large
// ones are faster apart, each on its own tile (16384 rows of 16, 4096 x 1024: 343 and 353).  Over 100 calls
// of random sizes two launches take 1.37 times the better of both, and both_tile()'s choice 1.014.
template <int KIND, class CF>
__global__ void __launch_bounds__(CF::WM *CF::WN * 64 * (CF::PROD ? 2 : 1))
group_both_kernel(const uint8_t *__restrict__ dy, const uint8_t *__restrict__ x, const uint8_t *__restrict__ w, void *dx,
                  void *dw, int M, int N, int K, int first, GroupRows<true> of_rows, GroupWeights<2> of_weights) {
    constexpr int EPI = KIND == DENSE_F16 ? EPI_F16 : EPI_BF16;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Slabs<KIND, EPI, CF>::SMEM];
    if (int(blockIdx.x) < first)
        gemm_tile<KIND, EPI, CF>(dy, w, dx, M, K, N, (N + 63) / 64, of_rows, smem, blockIdx.x);
    else gemm_tile<KIND, EPI, CF>(dy, x, dw, N, K, 0, 0, of_weights, smem, blockIdx.x - first);
}

template <int KIND, class CF>
hipError_t both_cfg(const Grouped &a, hipStream_t st) {
    using LY = Layout<KIND, CF>;
    const int N = int(a.N), K = int(a.K);
    const GroupRows<true> r{a.offsets, a.experts, a.lddy * 2, a.lddx, a.N * a.K * 2, K, N, streams(a.M * K * 2)};
    GroupWeights<2> ex{};
    ex.offsets = a.offsets, ex.groups = a.experts, ex.rows = int(a.M), ex.splits = 1, ex.ldc = a.K;
    ex.sorted = long_sums(a);
    ex.lda = int(a.lddy), ex.ldw = int(a.ldx);
    const int64_t first = (group_tiles(a.M, a.experts, LY::BM, (K + LY::BN - 1) / LY::BN) + 7) / 8 * 8;
    const int64_t more = a.experts * int64_t((N + LY::BM - 1) / LY::BM) * ((K + LY::BN - 1) / LY::BN);
    hipLaunchKernelGGL((group_both_kernel<KIND, CF>), dim3(unsigned(first + more)), dim3(LY::NT), 0, st,
                       static_cast<const uint8_t *>(a.dy), static_cast<const uint8_t *>(a.x),
                       static_cast<const uint8_t *>(a.w), a.dx, a.dw, int(a.M), N, K, int(first), r, ex);
    return hipGetLastError();
}

template <int KIND>
hipError_t backward(const Grouped &a, hipStream_t st) {
    const WeightsPlan pl = weights_plan(a.M, a.experts, a.N, a.K);
    if (a.dx && a.dw && a.M > 0) {
        switch (both_tile(pl, a.M, a.experts, a.N, a.K)) {
            case 0: return both_cfg<KIND, Cfg32x64>(a, st);
            case 1: return both_cfg<KIND, Cfg64x128P>(a, st);
            case 2: return both_cfg<KIND, Cfg128x128P>(a, st);
            default: break;
        }
    }
    if (a.dx && a.M > 0) {
        const hipError_t e = rows<KIND, true>(a, a.dy, a.lddy, a.dx, a.lddx, int(a.K), int(a.N), st);
        if (e != hipSuccess) return e;
    }
    return a.dw ? weights<KIND>(a, pl, st) : hipSuccess;
}

}  // namespace

int64_t grouped_blocks(int64_t M, int64_t experts, int64_t N, int64_t K, bool backward) {
    auto of_rows = [&](const TileCost &t, int64_t n) { return group_tiles(M, experts, t.bm, (n + t.bn - 1) / t.bn); };
    auto of_weights = [&](const TileCost &t) {
        return experts * ((N + t.bm - 1) / t.bm) * ((K + t.bn - 1) / t.bn);
    };
    if (!backward) return of_rows(kFwdTiles[rows_tile<false>(M, experts, N, K)], N);
    const WeightsPlan pl = weights_plan(M, experts, N, K);
    const int both = both_tile(pl, M, experts, N, K);
    const int64_t dx = of_rows(kDxTiles[rows_tile<true>(M, experts, K, N)], K);
    int64_t most = pl.splits * of_weights(kDwTiles[pl.tile]);
    if (dx > most) most = dx;
    if (both >= 0) {
        const TileCost &t = kBothTiles[both].dx;
        const int64_t all = of_rows(t, K) + 8 + of_weights(t);
        if (all > most) most = all;
    }
    return most;
}

int grouped_tile(int product, int64_t M, int64_t experts, int64_t N, int64_t K) {
    if (product == 0) return rows_tile<false>(M, experts, N, K);
    if (product == 1) return rows_tile<true>(M, experts, K, N);
    const WeightsPlan pl = weights_plan(M, experts, N, K);
    return product == 2 ? pl.tile + 256 * pl.splits : both_tile(pl, M, experts, N, K);
}

int64_t grouped_slices_bytes(int64_t M, int64_t experts, int64_t N, int64_t K) {
    const int splits = weights_plan(M, experts, N, K).splits;
    return splits > 1 ? splits * experts * N * K * 4 : 0;
}

hipError_t launch_grouped_fwd(const Grouped &a, hipStream_t st) {
    if (a.dtype == DT_F16) return rows<DENSE_F16, false>(a, a.x, a.ldx, a.out, a.ldo, int(a.N), int(a.K), st);
    return rows<DENSE_BF16, false>(a, a.x, a.ldx, a.out, a.ldo, int(a.N), int(a.K), st);
}
hipError_t launch_grouped_bwd(const Grouped &a, hipStream_t st) {
    return a.dtype == DT_F16 ? backward<DENSE_F16>(a, st) : backward<DENSE_BF16>(a, st);
}

}  // namespace ssg

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
// groups have K loops of different lengths in one launch.
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

    template <class CF, int BM, int BN>
    __device__ __forceinline__ bool place(const uint8_t *&A, const uint8_t *&W, void *&C, int &M, int N, int, int &,
                                          int &n0) const {
        const group::Tile t = group::find_tile<BM>(offsets, groups, M, (N + BN - 1) / BN, CF::GM);
        if (t.group < 0) return false;
        A += t.row * a_row;
        W += t.group * w_bytes;
        C = static_cast<uint16_t *>(C) + t.row * ldc;
        M = t.rows;
        n0 = t.tile_n * BN;
        return true;
    }
};

// dw: every tile of every expert; M and N are the weight's sides.
struct GroupWeights {
    static constexpr bool kAfter = false, kEpilogue = false, kTransA = true, kTransW = true, kPlace = true;
    const int32_t *offsets;
    int groups, rows;
    int64_t a_row, ldc;  // (a_row: unused)
    int lda, ldw;
    int rows_a, rows_w;        // (unused: the stages' buffers take bytes_a and bytes_w)
    int64_t bytes_a, bytes_w;  // of the group's rows, from the tile's first column on

    template <class CF, int BM, int BN>
    __device__ __forceinline__ bool place(const uint8_t *&A, const uint8_t *&W, void *&C, int &M, int N, int,
                                          int &stages, int &n0) {
        const int tiles_n = (N + BN - 1) / BN, each = (M + BM - 1) / BM * tiles_n;
        // (every expert's tiles are spread over the XCDs: a popular expert is no XCD's alone)
        const int g = blockIdx.x / each, j = xcd_remap(blockIdx.x % each, each);
        int lo, hi;
        group::rows_of(offsets, groups, rows, g, lo, hi);
        const int m0 = j / tiles_n * BM;
        n0 = j % tiles_n * BN;
        A += (int64_t(lo) * lda + m0) * 2;
        W += int64_t(lo) * ldw * 2;
        C = static_cast<uint16_t *>(C) + (int64_t(g) * M + m0) * ldc;
        bytes_a = (int64_t(hi - lo - 1) * lda + M - m0) * 2;
        bytes_w = (int64_t(hi - lo - 1) * ldw + N) * 2;
        M -= m0;
        stages = (hi - lo + 63) / 64;
        return true;
    }
};

template <int KIND, class CF, class Extra>
hipError_t launch_cfg(const void *A, const void *W, void *C, const Extra &ex, int64_t blocks, int M, int N, int K,
                      hipStream_t st) {
    using LY = Layout<KIND, CF>;
    constexpr int EPI = KIND == DENSE_F16 ? EPI_F16 : EPI_BF16;
    hipLaunchKernelGGL((gemm_kernel<KIND, EPI, CF, Extra>), dim3(unsigned(blocks)), dim3(LY::NT), 0, st,
                       static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(W), nullptr, nullptr, nullptr, C,
                       M, N, K, (K + 63) / 64, ex);
    return hipGetLastError();
}

using Cfg32x128 = Cfg<1, 4, 1, 1, 4, 8, true, false>;
using Cfg64x128 = Cfg<2, 2, 1, 2, 3, 8, true, false>;
using Cfg128x128 = Cfg<2, 2, 2, 2, 4, 8, true, false, 0, true>;
using Cfg256x128 = Cfg<2, 2, 4, 2, 3, 8, true, false, 0, true>;

template <int KIND, class CF, bool TW>
hipError_t rows_cfg(const Grouped &a, const void *A, int64_t lda, void *C, int64_t ldc, int N, int K, hipStream_t st) {
    using LY = Layout<KIND, CF>;
    GroupRows<TW> ex{a.offsets, a.experts, lda * 2, ldc, int64_t(N) * K * 2, N, K};
    const int64_t blocks = group_tiles(a.M, a.experts, LY::BM, (N + LY::BN - 1) / LY::BN);
    return launch_cfg<KIND, CF>(A, a.w, C, ex, blocks, int(a.M), N, K, st);
}

template <int KIND, bool TW>
hipError_t rows(const Grouped &a, const void *A, int64_t lda, void *C, int64_t ldc, int N, int K, hipStream_t st) {
    const int64_t each = a.M / a.experts;
    if (each <= 32) return rows_cfg<KIND, Cfg32x128, TW>(a, A, lda, C, ldc, N, K, st);
    if (each <= 64) return rows_cfg<KIND, Cfg64x128, TW>(a, A, lda, C, ldc, N, K, st);
    if (each <= 256) return rows_cfg<KIND, Cfg128x128, TW>(a, A, lda, C, ldc, N, K, st);
    return rows_cfg<KIND, CfgBigDense<true>, TW>(a, A, lda, C, ldc, N, K, st);
}

template <int KIND, class CF>
hipError_t weights_cfg(const Grouped &a, hipStream_t st) {
    using LY = Layout<KIND, CF>;
    GroupWeights ex{};
    ex.offsets = a.offsets, ex.groups = a.experts, ex.rows = int(a.M), ex.ldc = a.K;
    ex.lda = int(a.lddy), ex.ldw = int(a.ldx);
    const int64_t blocks = a.experts * ((a.N + LY::BM - 1) / LY::BM) * ((a.K + LY::BN - 1) / LY::BN);
    return launch_cfg<KIND, CF>(a.dy, a.x, a.dw, ex, blocks, int(a.N), int(a.K), 0, st);
}

template <int KIND>
hipError_t weights(const Grouped &a, hipStream_t st) {
    if (a.experts * tiles(int(a.N), int(a.K), 128, 128) < 96) return weights_cfg<KIND, CfgT64<true, false>>(a, st);
    return weights_cfg<KIND, Cfg256x128>(a, st);
}

template <int KIND>
hipError_t backward(const Grouped &a, hipStream_t st) {
    if (a.dx && a.M > 0) {
        const hipError_t e = rows<KIND, true>(a, a.dy, a.lddy, a.dx, a.lddx, int(a.K), int(a.N), st);
        if (e != hipSuccess) return e;
    }
    return a.dw ? weights<KIND>(a, st) : hipSuccess;
}

}  // namespace

int64_t grouped_blocks(int64_t M, int64_t experts, int64_t N, int64_t K) {
    const int64_t side = N > K ? N : K;
    const int64_t fwd = group_tiles(M, experts, 32, (side + 127) / 128);
    const int64_t dw = experts * ((N + 63) / 64) * ((K + 63) / 64);
    return fwd > dw ? fwd : dw;
}

hipError_t launch_grouped_fwd(const Grouped &a, hipStream_t st) {
    if (a.dtype == DT_F16) return rows<DENSE_F16, false>(a, a.x, a.ldx, a.out, a.ldo, int(a.N), int(a.K), st);
    return rows<DENSE_BF16, false>(a, a.x, a.ldx, a.out, a.ldo, int(a.N), int(a.K), st);
}
hipError_t launch_grouped_bwd(const Grouped &a, hipStream_t st) {
    return a.dtype == DT_F16 ? backward<DENSE_F16>(a, st) : backward<DENSE_BF16>(a, st);
}

}  // namespace ssg

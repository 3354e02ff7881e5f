// 2:4 fp16 GEMM with low-rank adapters beside it: C = A . W + scale A down^T
// up^T, in one pass over C.  The skeleton of gemm_core.h runs as for
// w24_gemm_f16; between the main loop and the epilogue each wave adds its
// tokens' adapters to the accumulators (low_rank.h), so the sum is rounded
// once and the adapters cost no second read and write of C.
#include "gemm_core.h"
#include "gemm_tiles.h"
#include "launch.h"
#include "low_rank.h"

namespace ssg {

struct LowRankAfter {
    static constexpr bool kAfter = true, kEpilogue = false, kTransA = false, kTransW = false;
    const _Float16 *up, *low;
    const int32_t *index, *ranks;
    int adapters, R;

    template <class CF>
    __device__ __forceinline__ void after(floatx16 (&acc)[CF::TN][CF::TM], const int32_t *at, int mw, int nw, int M,
                                          int N) const {
        low_rank_expand<_Float16, CF::TN, CF::TM>(acc, up, low, at, ranks, adapters, R, mw, nw, M, N);
    }
};

template <class CF>
static hipError_t launch_lr(const void *A, const void *vals, const uint32_t *meta, const LowRankAfter &ex, void *C,
                            int M, int N, int K, hipStream_t st) {
    using LY = Layout<W24_F16, CF>;
    const int nb = ((M + LY::BM - 1) / LY::BM) * ((N + LY::BN - 1) / LY::BN);
    hipLaunchKernelGGL((gemm_kernel<W24_F16, EPI_F16, CF, LowRankAfter>), dim3(nb), dim3(LY::NT), 0, st,
                       static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(vals), meta, nullptr, nullptr, C,
                       M, N, K, K / (64 * CF::DK), ex);
    return hipGetLastError();
}

int low_rank_splits(int M, int N, int K) { return suggest_splits(W24_F16, M, N, K); }

// Tile choice as for the plain 2:4 fp16 GEMM (gemm_tiles.h).
hipError_t launch_w24_low_rank_f16(const void *A, const void *vals, const uint32_t *meta, const LowRank &lr,
                                   const void *low, void *C, int M, int N, int K, hipStream_t st) {
    const LowRankAfter ex{static_cast<const _Float16 *>(lr.up), static_cast<const _Float16 *>(low), lr.index, lr.ranks,
                          lr.adapters, lr.R};
    switch (pick_f16(M, N, K)) {
        case SHAPE_BIG: return launch_lr<CfgBig<true, 4>>(A, vals, meta, ex, C, M, N, K, st);
        case SHAPE_T64: return launch_lr<CfgT64<true, false>>(A, vals, meta, ex, C, M, N, K, st);
        case SHAPE_T32: return launch_lr<CfgT32<true>>(A, vals, meta, ex, C, M, N, K, st);
        case SHAPE_T64N: return launch_lr<CfgT64NP<true, true>>(A, vals, meta, ex, C, M, N, K, st);
        default: return launch_lr<CfgSmallP<true, true, 4>>(A, vals, meta, ex, C, M, N, K, st);
    }
}

}  // namespace ssg

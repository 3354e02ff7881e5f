// 2:4 fp16 GEMM with low-rank adapters beside it: C = A . W + scale A down^T
// up^T, in one pass over C.  The skeleton of gemm_core.h runs as for
// w24_gemm_f16; between the main loop and the epilogue each wave adds its
// tokens' adapters to the accumulators (low_rank.h), so the sum is rounded
// once and the adapters cost no second read and write of C.  4096 x 1024 x 4096,
// rank 64, 12 adapters: 39.3 us, least 37.6 (w24_gemm_f16 alone 30; a separate add
// would read and write 67 MB more, 13 us), after a shrink of 8.7.  The adapters' 8 us
// are the tile's end: every workgroup fetches its low values and pool rows at the same
// time, with no main loop left to hide them.
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

    // The tile's low values go to LDS once for all waves, 64 slots at a time, and
    // of its distinct adapters, two at a time, the channels' rows of the pool.  These
    // copies leave and arrive together at the end of a tile, so their bytes set
    // their time: read by every wave for itself they were 256 KiB a 256 x 256 tile
    // and 64 slots, instead of 96.
    // An adapter whose weights are not finite must not reach the tokens of other
    // requests through 0 * inf: such pieces are zeroed in LDS before use, and the
    // adapter's own tokens get NaN in those channels at the end (noted in `hit`, so
    // that the accumulators meet nothing but matrix instructions inside the loops:
    // a check there cost 6 to 17 of 45 us at 4096 x 1024 x 4096).
    template <class CF, int SMEM>
    __device__ __forceinline__ void after(floatx16 (&acc)[CF::TN][CF::TM], const int32_t *at, uint8_t *smem,
                                          bool loader, int m0, int n0, int M, int N) const {
        constexpr int TN = CF::TN, TM = CF::TM, NW = CF::WM * CF::WN, WAVES = CF::PROD ? 2 * NW : NW;
        constexpr int BM = CF::WM * TM * 32, BN = CF::WN * TN * 32, SEEN = (BM + 63) / 64;
        constexpr int LOW = BM * 256, UP = BN * 128;  // 64 slots: both planes; one adapter's rows
        static_assert(LOW + 2 * UP + BN / 4 <= SMEM, "scratch must fit in the stage ring");
        uint32_t *broken = reinterpret_cast<uint32_t *>(smem + LOW + 2 * UP);  // [2][BN / 32] channel bits
        // (opaque, so that nothing derived from it is kept in registers across the main loop)
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, h = lane >> 5, r = lane & 31;
        const int all = __builtin_amdgcn_readfirstlane(tid >> 6);  // wave of the workgroup
        const int wave = all % NW, wm = wave % CF::WM, wn = wave / CF::WM;
        const int ks = (R + 15) / 16, blocks = (M + 31) / 32;
        const int ws = R <= 16 ? 1 : R <= 32 ? 2 : 3;  // 16-byte pieces of a pool row, as a shift
        int mine[TM];
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            const int i = (wm * TM + tm) * 32 + r;
            mine[tm] = m0 + i < M ? at[i] : -1;
            if (mine[tm] != -1 && (mine[tm] < 0 || mine[tm] >= adapters)) {
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[tn][tm][i] = __builtin_nanf("");
            }
        }
        // Powers of two of the tokens' low values: the product so far is divided by them
        // before the first adapter, and everything multiplied at the end.
        int power[TM] = {};
        bool scaled = false;
        auto scale = [&](int sign) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int tm = 0; tm < TM; ++tm)
#pragma unroll
                    for (int i = 0; i < 16; ++i) acc[tn][tm][i] = __builtin_amdgcn_ldexpf(acc[tn][tm][i], sign * power[tm]);
        };
        uint32_t hit[TN][TM];  // channels whose weights of this token's adapter are broken
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) hit[tn][tm] = 0;
#pragma unroll 1
        for (int k0 = 0; k0 < R; k0 += 64) {
            const int steps = min(4, ks - k0 / 16);
            int seen[SEEN];
#pragma unroll
            for (int j = 0; j < SEEN; ++j) {
                const int i = j * 64 + lane;
                seen[j] = i < BM && m0 + i < M ? at[i] : -1;
                if (seen[j] >= adapters) seen[j] = -1;
            }
            // the next distinct adapter of the tile (every wave finds the same ones), -1: none
            auto next = [&]() {
                int a = -1;
#pragma unroll
                for (int j = SEEN - 1; j >= 0; --j) {
                    const uint64_t left = __ballot(seen[j] >= 0);
                    if (left) a = __builtin_amdgcn_readlane(seen[j], __builtin_ctzll(left));
                }
#pragma unroll
                for (int j = 0; j < SEEN; ++j)
                    if (seen[j] == a) seen[j] = -1;
                return a;
            };
            bool first = true;
#pragma unroll 1
            for (int a0 = next(); a0 >= 0; a0 = next()) {
                const int a1 = next();
                const bool opening = first && k0 == 0;
                const int rank0 = low_rank_of(ranks, a0, R), rank1 = a1 >= 0 ? low_rank_of(ranks, a1, R) : 0;
                if (!first || k0 > 0) __syncthreads();  // the last pair has been used
                if (first)
                    for (int j = all; j < BM / 32 * steps * 2; j += WAVES) {
                        const int plane = j / (BM / 32 * steps), tb = j / steps % (BM / 32), s = j % steps;
                        const void *src = g_low_zero;
                        if (m0 / 32 + tb < blocks)
                            src = low + plane * low_plane(M, R) +
                                  ((int64_t(m0 / 32 + tb) * ks + k0 / 16 + s) * 64 + lane) * 8;
                        tw_detail::tw_dma16(src, smem + ((plane * (BM / 32) + tb) * 4 + s) * 1024);
                    }
                first = false;
                const int pieces = BN >> (6 - ws);
                for (int j = all; j < (a1 >= 0 ? 2 * pieces : pieces); j += WAVES) {
                    const int u = j >= pieces, i = j - (u ? pieces : 0);
                    const int row = (i << (6 - ws)) + (lane >> ws);
                    const int k = k0 + ((lane & ((1 << ws) - 1)) ^ (row & ((1 << ws) - 1))) * 8;
                    const void *src = g_low_zero;
                    if (k < R) src = up + (int64_t(u ? a1 : a0) * N + min(n0 + row, N - 1)) * R + k;
                    tw_detail::tw_dma16(src, smem + LOW + u * UP + i * 1024);
                }
                if (tid < BN / 16) broken[tid] = 0;
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                __syncthreads();
                const int staged = a1 >= 0 ? 2 * pieces : pieces;
                for (int j0 = all; j0 < staged; j0 += 4 * WAVES) {
                    u32x4 v[4];
                    bool bad[4], any = false;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int j = j0 + q * WAVES, u = j >= pieces;
                        const int at_byte = LOW + (u ? UP - pieces * 1024 : 0) + j * 1024 + lane * 16;
                        v[q] = u32x4{0, 0, 0, 0};
                        if (j < staged) v[q] = *reinterpret_cast<const u32x4 *>(smem + at_byte);
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // (x * 0 has exponent bits only where x is not finite; slots past the rank do not count)
                        const int j = j0 + q * WAVES, u = j >= pieces, i = j - (u ? pieces : 0);
                        const int row = (i << (6 - ws)) + (lane >> ws);
                        const int k = k0 + ((lane & ((1 << ws) - 1)) ^ (row & ((1 << ws) - 1))) * 8;
                        const u32x4 z = __builtin_bit_cast(u32x4, __builtin_bit_cast(half8, v[q]) * half8{});
                        bad[q] = ((z.x | z.y | z.z | z.w) & 0x7c007c00u) != 0 &&
                                 not_finite<_Float16>(keep16(v[q], (u ? rank1 : rank0) - k));
                        any = any || bad[q];
                    }
                    if (__ballot(any) == 0) continue;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int j = j0 + q * WAVES, u = j >= pieces, i = j - (u ? pieces : 0);
                        const int row = (i << (6 - ws)) + (lane >> ws);
                        if (!bad[q]) continue;
                        *reinterpret_cast<u32x4 *>(smem + LOW + u * UP + i * 1024 + lane * 16) = u32x4{0, 0, 0, 0};
                        atomicOr(broken + u * (BN / 32) + row / 32, 1u << (row % 32));
                    }
                }
                __syncthreads();
                if (loader) continue;
                if (opening) {
#pragma unroll
                    for (int tm = 0; tm < TM; ++tm) {  // (slots 0..7, for both halves of the wave)
                        const uint8_t *p = smem + BM / 32 * 4096 + (wm * TM + tm) * 4096 + r * 16;
                        const int e = low_exponent_of(*reinterpret_cast<const u32x4 *>(p));
                        power[tm] = mine[tm] >= 0 && mine[tm] < adapters ? e : 0;
                        scaled = scaled || __ballot(power[tm] != 0) != 0;
                    }
                    if (scaled) scale(-1);
                }
#pragma unroll 1
                for (int u = 0; u < 2; ++u) {
                    const int a = u ? a1 : a0;
                    bool any = false;
#pragma unroll
                    for (int tm = 0; tm < TM; ++tm) any = any || __ballot(a >= 0 && mine[tm] == a) != 0;
                    if (!any) continue;
                    const int rank = u ? rank1 : rank0;
#pragma unroll 1
                    for (int s = 0; s < 4 && k0 + 16 * s < rank; ++s) {
                        const int k = k0 + 16 * s;
                        u32x4 w[TN];
#pragma unroll
                        for (int tn = 0; tn < TN; ++tn) {
                            const int row = (wn * TN + tn) * 32 + r;
                            const int piece = (2 * s + h) ^ (row & ((1 << ws) - 1));
                            w[tn] = keep16(
                                *reinterpret_cast<const u32x4 *>(smem + LOW + u * UP + (row << (ws + 4)) + piece * 16),
                                rank - k - 8 * h);
                        }
#pragma unroll
                        for (int tm = 0; tm < TM; ++tm) {
                            if (__ballot(mine[tm] == a) == 0) continue;
                            const uint8_t *p = smem + ((wm * TM + tm) * 4 + s) * 1024 + lane * 16;
                            u32x4 hi = *reinterpret_cast<const u32x4 *>(p);
                            u32x4 lo = *reinterpret_cast<const u32x4 *>(p + BM / 32 * 4096);
                            const bool use = mine[tm] == a && k + 8 * h < R;
                            hi = use ? hi : u32x4{0, 0, 0, 0};
                            lo = use ? lo_value<_Float16>(lo) : u32x4{0, 0, 0, 0};
#pragma unroll
                            for (int tn = 0; tn < TN; ++tn) {
                                acc[tn][tm] = mfma32<_Float16>(w[tn], hi, acc[tn][tm]);
                                acc[tn][tm] = mfma32<_Float16>(w[tn], lo, acc[tn][tm]);
                            }
                        }
                    }
#pragma unroll
                    for (int tn = 0; tn < TN; ++tn) {
                        const uint32_t rows = broken[u * (BN / 32) + wn * TN + tn];
#pragma unroll
                        for (int tm = 0; tm < TM; ++tm) hit[tn][tm] |= mine[tm] == a ? rows : 0u;
                    }
                }
            }
        }
        if (scaled) scale(1);
        uint32_t any = 0;
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) any |= hit[tn][tm];
        if (__ballot(any != 0) != 0) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int tm = 0; tm < TM; ++tm)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (hit[tn][tm] >> (8 * (i / 4) + 4 * h + i % 4) & 1) acc[tn][tm][i] = __builtin_nanf("");
        }
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

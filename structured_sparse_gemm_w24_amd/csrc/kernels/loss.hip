// Softmax cross entropy of a linear head over a large vocabulary, and its
// gradient, without keeping the logits, for gfx950.
//
//   z[m][v]  = x[m] . w[v]
//   lse[m]   = log sum_v exp z[m][v],   loss[m] = lse[m] - z[m][target[m]]
//   G[m][v]  = dloss[m] (exp(z[m][v] - lse[m]) - [v = target[m]])
//   dx = G w,   dw = G^T x                    (G = 0 in ignored rows)
//
// Bound by the matrix units: 2 M V D operations forward, 6 M V D backward (the
// logits once more, and the two products).  All products run on the GEMM
// skeleton (gemm_core.h) with epilogues of their own:
//   * forward, each tile reduces its logits to a maximum and a sum of
//     exponentials per row in registers and writes those 8 bytes a row; a second
//     launch merges a row's tiles in order;
//   * backward works through the vocabulary in pieces.  For a piece, the first
//     product's epilogue turns the logits into G [M][piece]; then dx += G w and
//     dw[piece] = G^T x.  What these sum over runs along the rows of w, of G and
//     of x, so they read those operands through transposing LDS reads as they
//     lie (with 256 x 128 tiles that is as fast as reading along the rows:
//     6144 x 1024 x 10240 bf16 126 us either way, both operands so 130;
//     transposed copies, and G written both ways round, cost 250 of 1365 us at
//     6144 x 30001 x 1024).  dx is summed over the pieces in fp32.
// G is rounded to the operands' 16 bits, as the products need it; its rows are
// divided by the largest finite |dloss| first (and, fp16, multiplied by 2^12, so that a
// probability of 2^-26 is still a normal number), which the products' outputs
// are multiplied by again in fp32.  In fp16 its steps are then 2^-36 of that factor, so
// rows that weigh less than about 2^-18 of the heaviest lose digits of their dx; a factor
// for each row would have to come out of the sum over rows in dw again.
// The rounding shows: 6144 x 1024 x 30001 bf16 is 0.0019 of its norm off the 64-bit
// result, where 32-bit probabilities and one rounding of the outputs give 0.0017; a
// second 16-bit part of G would run both gradient products again, 640 of 1090 us more.
// Measured on MI355X, several runs: forward 8192 x 1024 x 32000 fp16 501-522 us = 1029-1072
// TFLOP/s (the library's product alone 431-448 us); backward 6144 x 1024 x 30001 bf16
// 1069-1109 us = 1021-1059 TFLOP/s, in two pieces, each G 211-221 us, dx 164-168, dw 158-165.
// The matrix units are
// busy 0.57 of the forward and 0.41 / 0.62 / 0.54 of the three: what bounds them is
// LDS, whose reads and direct writes fill its port, and for G the epilogue (an
// exponential a logit and 184 MB of G written; a library product of that size, at
// the 1084 TFLOP/s it reaches at twice the width, takes 175).
#include "elem.h"
#include "gemm_core.h"
#include "gemm_tiles.h"
#include "launch.h"

namespace ssg {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

template <class T>
constexpr float kGradScale = __is_same(T, _Float16) ? 4096.0f : 1.0f;

// (max, sum of exp(z - max)) of two sets of logits; an empty or all -inf set
// has max -inf and sum 0.
__device__ __forceinline__ void merge(float &m, float &s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float at = top == -INFINITY ? 0.0f : top;
    s = s * exp_of(m - at) + s2 * exp_of(m2 - at);
    m = top;
}

// ---- forward epilogue: a tile's statistics and the targets' logits.
struct LossStats {
    static constexpr bool kAfter = false, kEpilogue = true, kTransA = false, kTransW = false;
    const int64_t *target;
    float *part;   // [tiles][M][2]
    float *logit;  // [M]
    int64_t v0;    // first vocabulary entry of this launch
    int tile0;     // its first tile

    template <class CF, int SMEM>
    __device__ __forceinline__ void epilogue(floatx16 (&acc)[CF::TN][CF::TM], uint8_t *smem, bool loader, int m0,
                                             int n0, int wave, int M, int N, int, int tile_n) const {
        constexpr int TN = CF::TN, TM = CF::TM, BM = CF::WM * TM * 32;
        static_assert(CF::WN * BM * 8 <= SMEM, "statistics must fit in the stage ring");
        const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
        const int wm = wave % CF::WM, wn = wave / CF::WM;
        const int nw = n0 + wn * TN * 32;
        float *s_max = reinterpret_cast<float *>(smem), *s_sum = s_max + CF::WN * BM;
        __syncthreads();  // every wave is done reading the stage buffers
        if (!loader) {
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) {
                const int room = N - nw - 4 * h;  // channels c < room exist
                const int row = wm * TM * 32 + tm * 32 + r, m = m0 + row;
                const int64_t t = m < M ? target[m] - v0 : -1;
                // the target's place among this lane's channels (those with bit 2 clear, from 4 h)
                const int at = t >= nw && t < nw + TN * 32 && t < N ? int(t) - nw - 4 * h : -1;
                float zt = 0.0f, top = -INFINITY;
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = tn * 32 + 8 * (i / 4) + i % 4;
                        const float z = c < room ? acc[tn][tm][i] : -INFINITY;
                        zt = c == at ? z : zt;
                        top = fmaxf(top, z);
                    }
                if (at >= 0 && (at & 4) == 0) logit[m] = zt;
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float ref = top == -INFINITY ? 0.0f : top;
                float sum = 0.0f;
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                    sum += tn * 32 + 8 * (i / 4) + i % 4 < room ? exp_of(acc[tn][tm][i] - ref) : 0.0f;
                sum += __shfl_xor(sum, 32, 64);
                if (h == 0) s_max[wn * BM + row] = top, s_sum[wn * BM + row] = sum;
            }
        }
        __syncthreads();
        if (int(threadIdx.x) < BM && m0 + int(threadIdx.x) < M) {
            float m = s_max[threadIdx.x], s = s_sum[threadIdx.x];
#pragma unroll
            for (int q = 1; q < CF::WN; ++q) merge(m, s, s_max[q * BM + threadIdx.x], s_sum[q * BM + threadIdx.x]);
            float *o = part + (int64_t(tile0 + tile_n) * M + m0 + threadIdx.x) * 2;
            o[0] = m;
            o[1] = s;
        }
    }
};

// Merges a row's tiles: 64 rows a workgroup, 16 threads a row.
__global__ void __launch_bounds__(1024)
loss_rows_kernel(const float *__restrict__ part, const float *__restrict__ logit, const int64_t *__restrict__ target,
                 int64_t ignore, int tiles, int64_t V, int M, float *__restrict__ loss, float *__restrict__ lse) {
    __shared__ float sm[16][64], ss[16][64];
    const int row = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int m = blockIdx.x * 64 + row;
    float top = -INFINITY, sum = 0.0f;
    if (m < M) {
        // the maximum first, so that the sums are independent of one another
#pragma unroll 4
        for (int t = q; t < tiles; t += 16) top = fmaxf(top, part[(int64_t(t) * M + m) * 2]);
        const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll 4
        for (int t = q; t < tiles; t += 16) {
            const float *p = part + (int64_t(t) * M + m) * 2;
            sum += p[1] * exp_of(p[0] - ref);
        }
    }
    sm[q][row] = top;
    ss[q][row] = sum;
    __syncthreads();
    if (q == 0 && m < M) {
        for (int i = 1; i < 16; ++i) merge(top, sum, sm[i][row], ss[i][row]);
        const float l = top + logf(sum);
        const int64_t t = target[m];
        lse[m] = l;
        loss[m] = t == ignore ? 0.0f : t < 0 || t >= V ? __builtin_nanf("") : l - logit[m];
    }
}

// ---- backward epilogue: logits to G [M][ldg], zeros past the last channel.
template <class T>
struct LossGrad {
    static constexpr bool kAfter = false, kEpilogue = true, kTransA = false, kTransW = false;
    const int64_t *target;
    int64_t ignore, V, v0;
    const float *dloss, *lse, *scale;  // scale[0] = largest finite |dloss|
    T *g;
    int ldg;

    template <class CF, int SMEM>
    __device__ __forceinline__ void epilogue(floatx16 (&acc)[CF::TN][CF::TM], uint8_t *smem, bool loader, int m0,
                                             int n0, int wave, int M, int N, int, int) const {
        constexpr int TN = CF::TN, TM = CF::TM, NWV = CF::WM * CF::WN;
        constexpr int GROW = TN * 64 + 16;  // slab row: TN * 32 channels
        constexpr int SLAB = 32 * GROW;
        static_assert(SLAB * NWV <= SMEM, "slabs must fit in the stage ring");
        const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
        const int wm = wave % CF::WM, wn = wave / CF::WM;
        const int mw = m0 + wm * TM * 32, nw = n0 + wn * TN * 32;
        uint8_t *slab = smem + wave * SLAB;
        const float most = scale[0];
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            __syncthreads();  // the stage buffers, or the slab of the block before, have been read
            if (!loader) {
                const int m = mw + tm * 32 + r;
                int at = -1;  // the target's place among this lane's channels
                float s = 0.0f, ref = 0.0f;
                if (m < M) {
                    const int64_t t = target[m];
                    if (t != ignore) {
                        s = most > 0.0f ? dloss[m] / most * kGradScale<T> : dloss[m] * 0.0f;
                        if (t < 0 || t >= V) s = __builtin_nanf("");
                        ref = lse[m];
                        const int64_t u = t - v0 - nw;
                        if (u >= 0 && u < TN * 32) at = int(u) - 4 * h;
                    }
                }
                const bool live = m < M && (s != 0.0f);
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        T e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int c = tn * 32 + 8 * q + i;
                            const float p = exp_of(acc[tn][tm][4 * q + i] - ref) - (c == at ? 1.0f : 0.0f);
                            e[i] = T(live && nw + c + 4 * h < N ? p * s : 0.0f);
                        }
                        __builtin_memcpy(slab + r * GROW + (tn * 32 + q * 8 + h * 4) * 2, e, 8);
                    }
            }
            __syncthreads();
            if (loader) continue;
            constexpr int CPR = TN * 4, RPI = 64 / CPR;  // 16-byte pieces a row, rows an instruction
#pragma unroll
            for (int i = 0; i < 32 / RPI; ++i) {
                const int row = i * RPI + lane / CPR, ch = lane % CPR;
                const int m = mw + tm * 32 + row, n = nw + ch * 8;
                const u32x4 o = *reinterpret_cast<const u32x4 *>(slab + row * GROW + ch * 16);
                if (m < M && n < ldg) st16(g + int64_t(m) * ldg + n, o);
            }
        }
        // the last tile of a row fills the padding that lies past it
        const int done = n0 + CF::WN * TN * 32, pad = (ldg - done) / 8;
        if (done >= N && pad > 0)
            for (int i = threadIdx.x; i < CF::WM * TM * 32 * pad; i += blockDim.x) {
                const int m = m0 + i / pad;
                if (m < M) st16(g + int64_t(m) * ldg + done + i % pad * 8, u32x4{0, 0, 0, 0});
            }
    }
};

// ---- epilogue of the two gradient products: out = T((acc + sum so far) * scale),
// or, between the pieces, the fp32 sum alone.
// w (and, TA, the first operand too) has k along its rows.
template <class T, bool TA>
struct LossOut {
    static constexpr bool kAfter = false, kEpilogue = true, kTransA = TA, kTransW = true;
    int lda, rows_a;  // (TA)
    int ldw, rows_w;
    const float *scale;  // [1]: largest finite |dloss| / kGradScale
    const float *prev;   // fp32 [M][ldp] or null
    float *next;         // fp32 [M][ldp] (may be prev; K split: a slice each), or null: out is written
    T *out;
    int64_t ldo;
    int ldp;
    bool wide;  // out's rows take 16-byte stores

    template <class CF, int SMEM>
    __device__ __forceinline__ void epilogue(floatx16 (&acc)[CF::TN][CF::TM], uint8_t *smem, bool loader, int m0,
                                             int n0, int wave, int M, int N, int, int) const {
        constexpr int TN = CF::TN, TM = CF::TM, NWV = CF::WM * CF::WN;
        constexpr int TP = TN > 2 ? 2 : TN;  // channel blocks a pass
        constexpr int ROW = TP * 32 + 4;
        static_assert(32 * ROW * 4 * NWV <= SMEM && TN % TP == 0, "slabs must fit in the stage ring");
        const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
        const int wm = wave % CF::WM, wn = wave / CF::WM;
        const int mw = m0 + wm * TM * 32, nw = n0 + wn * TN * 32;
        float *slab = reinterpret_cast<float *>(smem) + wave * 32 * ROW;
        const float f = scale[1];
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
            for (int tp = 0; tp < TN; tp += TP) {
                __syncthreads();
                if (!loader) {
#pragma unroll
                    for (int tn = 0; tn < TP; ++tn)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const floatx16 &a = acc[tp + tn][tm];
                            *reinterpret_cast<floatx4 *>(slab + r * ROW + tn * 32 + q * 8 + h * 4) =
                                floatx4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                        }
                }
                __syncthreads();
                if (loader) continue;
                constexpr int CPR = TP * 4, RPI = 64 / CPR;  // pieces of 8 values a row
#pragma unroll
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int row = i * RPI + lane / CPR, ch = lane % CPR * 8;
                    const int m = mw + tm * 32 + row, n = nw + tp * 32 + ch;
                    if (m >= M || n >= N) continue;
                    float v[8];
                    __builtin_memcpy(v, slab + row * ROW + ch, 32);
                    if (prev) {  // (padded to a multiple of 64 columns)
                        float p[8];
                        __builtin_memcpy(p, prev + int64_t(m) * ldp + n, 32);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += p[j];
                    }
                    if (next) {
                        __builtin_memcpy(next + (int64_t(blockIdx.y) * M + m) * ldp + n, v, 32);
                        continue;
                    }
                    T *o = out + int64_t(m) * ldo + n;
                    if (wide && n + 8 <= N) {
                        typename Elem<T>::Vec t;
#pragma unroll
                        for (int j = 0; j < 8; ++j) t[j] = T(v[j] * f);
                        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, t), reinterpret_cast<u32x4 *>(o));
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (n + j < N) o[j] = T(v[j] * f);
                    }
                }
            }
    }
};

// ---- copies.  Rows to a contiguous copy of dp columns, zeros past D.
__global__ void __launch_bounds__(256)
loss_pack_kernel(const uint16_t *__restrict__ src, int64_t ld, uint16_t *__restrict__ dst, int64_t rows, int D,
                 int dp) {
    const int64_t pieces = rows * (dp / 8);
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < pieces; i += int64_t(gridDim.x) * 256) {
        const int64_t m = i / (dp / 8);
        const int c = int(i % (dp / 8)) * 8;
        typename Elem<_Float16>::Vec v = {};
        if (c < D) v = load_raw(reinterpret_cast<const _Float16 *>(src) + m * ld, c, D);
        st16(dst + m * dp + c, __builtin_bit_cast(u32x4, v));
    }
}

__global__ void __launch_bounds__(256)
loss_zero_kernel(uint16_t *__restrict__ dst, int64_t ld, int64_t rows, int D) {
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * D; i += int64_t(gridDim.x) * 256)
        dst[i / D * ld + i % D] = 0;
}

// What the backward pass needs first.  Workgroup 0: out[0] = largest finite
// |dloss| of the rows that count, out[1] = out[0] / div.  (An infinite one as the
// common factor would make every other row 0 * inf; so such a row, and one that is
// NaN, is not finite in its own G alone.)  The others: x to contiguous rows of dp
// columns, zeros past D and in ignored rows, whose G is zero: read as they lie, an
// infinity or NaN there (padding that nothing has written) would reach all of
// dw = G^T x as 0 * inf.  Beside workgroup 0, which takes 8 us alone, the copy costs
// little: 6144 x 1024 10.6 us in all.
__global__ void __launch_bounds__(1024)
loss_prepare_kernel(const float *__restrict__ dloss, const int64_t *__restrict__ target, int64_t ignore, int M,
                    float div, float *__restrict__ out, const uint16_t *__restrict__ x, int64_t ldx,
                    uint16_t *__restrict__ rows, int D, int dp) {
    if (blockIdx.x > 0) {
        const int64_t pieces = int64_t(M) * (dp / 8);
        for (int64_t i = int64_t(blockIdx.x - 1) * 1024 + threadIdx.x; i < pieces; i += int64_t(gridDim.x - 1) * 1024) {
            const int64_t m = i / (dp / 8);
            const int c = int(i % (dp / 8)) * 8;
            typename Elem<_Float16>::Vec v = {};
            if (c < D && target[m] != ignore) v = load_raw(reinterpret_cast<const _Float16 *>(x) + m * ldx, c, D);
            st16(rows + m * dp + c, __builtin_bit_cast(u32x4, v));
        }
        return;
    }
    __shared__ float red[16];
    float top = 0.0f;
#pragma unroll 4
    for (int m = threadIdx.x; m < M; m += 1024)
        if (target[m] != ignore && fabsf(dloss[m]) <= __FLT_MAX__) top = fmaxf(top, fabsf(dloss[m]));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < 16; ++i) top = fmaxf(top, red[i]);
        out[0] = top;
        out[1] = top / div;
    }
}

// Sums the K splits' slices in order onto the pieces' sum so far (acc, null: none
// yet); last: out is written, else acc2.  4 columns a thread.
template <class T>
__global__ void __launch_bounds__(256)
loss_splits_kernel(const float *__restrict__ part, int splits, const float *acc, float *acc2, bool last,
                   const float *__restrict__ scale, T *__restrict__ out, int64_t ldo, int64_t M, int N, int ldp) {
    const int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
    const int64_t m = i / ldp;
    const int n = int(i % ldp);
    if (m >= M || n >= N) return;
    floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (acc) v = *reinterpret_cast<const floatx4 *>(acc + i);
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const floatx4 u = *reinterpret_cast<const floatx4 *>(part + s * M * ldp + i);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    if (!last) {
        *reinterpret_cast<floatx4 *>(acc2 + i) = v;
        return;
    }
    const float f = scale[1];
    for (int j = 0; j < 4; ++j)
        if (n + j < N) out[m * ldo + n + j] = T(v[j] * f);
}

template <int KIND, class CF, class Extra>
hipError_t product_cfg(const void *A, const void *W, const Extra &ex, int64_t M, int64_t N, int64_t K,
                       hipStream_t st, int splits = 1) {
    using LY = Layout<KIND, CF>;
    const int nb = int((M + LY::BM - 1) / LY::BM * ((N + LY::BN - 1) / LY::BN));
    hipLaunchKernelGGL((gemm_kernel<KIND, EPI_F16, CF, Extra>), dim3(nb, splits), dim3(LY::NT), 0, st,
                       static_cast<const uint8_t *>(A), static_cast<const uint8_t *>(W), nullptr, nullptr, nullptr,
                       nullptr, int(M), int(N), int(K), int((K + 63) / 64 / splits), ex);
    return hipGetLastError();
}

// Tiles of the products.  One workgroup of any but the smallest fills a CU, so a
// product takes ceil(tiles / 256) rounds, and the tile is the one with the least
// rounds * cost of a round.  Costs relative to 256 x 256, from bf16 products of
// M x N x K on MI355X (us; rounds in brackets):
//                        256 x 256   256 x 128   192 x 128   128 x 128
//   8192 x 32000 x 1024  492 (16)    635 (32)                693 (63)
//   read by transposing reads:
//   6144 x 1024 x 15104  322 (1)     187 (1)     163 (1)     205 (2)
//   15104 x 1024 x 6144  161 (1)     181 (2)     194 (3)     191 (4)
//   12608 x 768 x 8192   189 (1)     200 (2)     161 (2)     178 (3)
// The narrower tiles have four compute waves of half the tile's rows and columns
// (which read less from LDS per product than more, smaller ones: eight waves of
// 64 x 64 ran 127 where four of 128 x 64 ran 120) and four loader waves, which the
// transposing reads need: without them they cost 256 x 256 a tenth to a fifth.
enum LossTile { LT_256, LT_256X128, LT_192X128, LT_128, LT_64, LT_TILES };
struct LossTileShape {
    int bm, bn, cost, cost_trans;
};
constexpr LossTileShape kLossTiles[LT_TILES] = {
    {256, 256, 100, 115}, {256, 128, 68, 68}, {192, 128, 56, 56}, {128, 128, 40, 40}, {64, 64, 0, 0}};
using Cfg256x128 = Cfg<2, 2, 4, 2, 3, 8, true, false, 0, true>;
using Cfg192x128 = Cfg<2, 2, 3, 2, 4, 8, true, false, 0, true>;
using Cfg128x128 = Cfg<2, 2, 2, 2, 4, 8, true, false, 0, true>;

// Rounds times cost of the best tile, and the tile.
long loss_cost(int64_t M, int64_t N, bool trans, LossTile *tile) {
    constexpr long kCUs = 256;
    long best = 0;
    for (int t = LT_256; t < LT_64; ++t) {
        const LossTileShape &s = kLossTiles[t];
        const long rounds = (tiles(int(M), int(N), s.bm, s.bn) + kCUs - 1) / kCUs;
        const long c = rounds * (trans ? s.cost_trans : s.cost);
        if (t == LT_256 || c < best) best = c, *tile = LossTile(t);
    }
    // Fewer than 96 tiles of 128 x 128 leave most CUs idle: 64 x 64 (by graph, with the cut
    // at 48 / 96 / 192: 64 such tiles, 512 x 2048 x 1024, forward 19.1 / 16.7 / 16.8 us,
    // gradient 45 / 40 / 39; 96 tiles, 1024 x 1500 x 1024, 19.4 / 19.5 / 17.8 and 50 / 51 / 48;
    // the gradient of 2048 x 2048 x 1024, whose products have 128 and 256, 62.6 / 62.7 / 75.9).
    if (tiles(int(M), int(N), 128, 128) < 96) *tile = LT_64;
    return best;
}
LossTile loss_tile(int64_t M, int64_t N, bool trans) {
    LossTile t;
    loss_cost(M, N, trans, &t);
    return t;
}

int64_t loss_tile_n(int64_t M, int64_t N) { return kLossTiles[loss_tile(M, N, false)].bn; }

// K splits for dx [M][D]: with few tiles of a long sum (a small batch against the
// vocabulary) each tile's sum is a chain of K / 64 dependent stages that leaves
// most CUs idle; split, about two workgroups a CU share it, eight stages at
// least each (the whole backward call: bf16 187 x 264 x 5382 75 -> 35 us, fp16
// 38 x 1210 x 4306 83 -> 50 us).
int loss_splits(int64_t M, int64_t D, int64_t piece) {
    if (loss_tile(M, D, true) != LT_64) return 1;
    const long t = tiles(int(M), int(D), 64, 64), stages = long((piece + 63) / 64);
    long p = 512 / t;
    if (p > stages / 8) p = stages / 8;
    return int(p < 1 ? 1 : p > 64 ? 64 : p);
}

// A [M][K] . W [N][K]^T with an epilogue; K a multiple of 64 unless both are transposed.
template <class T, class Extra>
hipError_t product(const void *A, const void *W, const Extra &ex, int64_t M, int64_t N, int64_t K, hipStream_t st,
                   int splits = 1) {
    constexpr int KIND = __is_same(T, _Float16) ? DENSE_F16 : DENSE_BF16;
    switch (loss_tile(M, N, Extra::kTransW)) {
        case LT_256: return product_cfg<KIND, CfgBigDense<true>>(A, W, ex, M, N, K, st);
        case LT_256X128: return product_cfg<KIND, Cfg256x128>(A, W, ex, M, N, K, st);
        case LT_192X128: return product_cfg<KIND, Cfg192x128>(A, W, ex, M, N, K, st);
        case LT_128: return product_cfg<KIND, Cfg128x128>(A, W, ex, M, N, K, st);
        default: return product_cfg<KIND, CfgT64<true, false>>(A, W, ex, M, N, K, st, splits);
    }
}

// The operands as the products take them: contiguous rows of dp columns (the
// backward pass's x comes from loss_prepare_kernel).
hipError_t operands(const Loss &a, const LossPlan &pl, const void **x, const void **w, bool backward, hipStream_t st) {
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    *x = backward ? ws + pl.x : a.x;
    *w = a.w;
    auto pack = [&](const void *src, int64_t ld, int64_t at, int64_t rows) {
        const int64_t blocks = (rows * (pl.dp / 8) + 255) / 256;
        hipLaunchKernelGGL(loss_pack_kernel, dim3(int(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st,
                           static_cast<const uint16_t *>(src), ld, reinterpret_cast<uint16_t *>(ws + at), rows,
                           int(a.D), int(pl.dp));
        return hipGetLastError();
    };
    hipError_t e = hipSuccess;
    if (pl.pack_x && !backward) {
        if ((e = pack(a.x, a.ldx, pl.x, a.M)) != hipSuccess) return e;
        *x = ws + pl.x;
    }
    if (pl.pack_w) {
        if ((e = pack(a.w, a.ldw, pl.w, a.V)) != hipSuccess) return e;
        *w = ws + pl.w;
    }
    return e;
}

template <class T>
hipError_t fwd(const Loss &a, const LossPlan &pl, hipStream_t st) {
    const void *x, *w;
    hipError_t e = operands(a, pl, &x, &w, false, st);
    if (e != hipSuccess) return e;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    float *part = reinterpret_cast<float *>(ws + pl.part), *logit = reinterpret_cast<float *>(ws + pl.logit);
    int tile0 = 0;
    for (int64_t v0 = 0; v0 < a.V; v0 += pl.piece) {
        const int64_t n = a.V - v0 < pl.piece ? a.V - v0 : pl.piece;
        const LossStats ex{a.target, part, logit, v0, tile0};
        e = product<T>(x, static_cast<const T *>(w) + v0 * pl.dp, ex, a.M, n, pl.dp, st);
        if (e != hipSuccess) return e;
        const int64_t bn = loss_tile_n(a.M, n);
        tile0 += int((n + bn - 1) / bn);
    }
    hipLaunchKernelGGL(loss_rows_kernel, dim3(int((a.M + 63) / 64)), dim3(1024), 0, st, part, logit, a.target, a.ignore,
                       tile0, a.V, int(a.M), a.loss, a.lse);
    return hipGetLastError();
}

template <class T>
hipError_t bwd(const Loss &a, const LossPlan &pl, hipStream_t st) {
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    T *g = reinterpret_cast<T *>(ws + pl.g);
    float *acc = reinterpret_cast<float *>(ws + pl.acc), *scale = reinterpret_cast<float *>(ws + pl.scale);
    const int M = int(a.M), D = int(a.D), dp = int(pl.dp);
    if (M == 0) {  // no rows: no gradient
        hipLaunchKernelGGL(loss_zero_kernel, dim3(2048), dim3(256), 0, st, static_cast<uint16_t *>(a.dw), a.lddw, a.V, D);
        return hipGetLastError();
    }
    const void *x, *w;
    hipError_t e = operands(a, pl, &x, &w, true, st);
    if (e != hipSuccess) return e;
    const int64_t copies = (a.M * (dp / 8) + 1023) / 1024;
    hipLaunchKernelGGL(loss_prepare_kernel, dim3(1 + int(copies < 2048 ? copies : 2048)), dim3(1024), 0, st, a.dloss,
                       a.target, a.ignore, M, kGradScale<T>, scale, static_cast<const uint16_t *>(a.x), a.ldx,
                       reinterpret_cast<uint16_t *>(ws + pl.x), D, dp);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const bool wide_x = a.lddx % 8 == 0 && (reinterpret_cast<uintptr_t>(a.dx) & 15) == 0;
    const bool wide_w = a.lddw % 8 == 0 && (reinterpret_cast<uintptr_t>(a.dw) & 15) == 0;
    for (int64_t v0 = 0; v0 < a.V; v0 += pl.piece) {
        const int64_t n = a.V - v0 < pl.piece ? a.V - v0 : pl.piece;
        const int step = 64 * pl.splits, ldg = int((n + step - 1) / step * step);
        const bool first = v0 == 0, last = v0 + n == a.V;
        const T *wv = static_cast<const T *>(w) + v0 * dp;
        const LossGrad<T> grad{a.target, a.ignore, a.V, v0, a.dloss, a.lse, scale, g, ldg};
        if ((e = product<T>(x, wv, grad, M, n, dp, st)) != hipSuccess) return e;
        float *const so_far = first ? nullptr : acc;
        if (pl.splits > 1) {
            float *part = reinterpret_cast<float *>(ws + pl.part);
            const LossOut<T, false> to_part{0, 0, dp, int(n), scale, nullptr, part, nullptr, 0, dp, false};
            if ((e = product<T>(g, wv, to_part, M, D, ldg, st, pl.splits)) != hipSuccess) return e;
            const int64_t blocks = (a.M * dp / 4 + 255) / 256;
            hipLaunchKernelGGL((loss_splits_kernel<T>), dim3(int(blocks)), dim3(256), 0, st, part, pl.splits, so_far,
                               acc, last, scale, static_cast<T *>(a.dx), a.lddx, a.M, D, dp);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        } else {
            const LossOut<T, false> to_x{0,  0,       dp, int(n), scale, so_far, last ? nullptr : acc,
                                         static_cast<T *>(a.dx), a.lddx, dp, wide_x};
            if ((e = product<T>(g, wv, to_x, M, D, ldg, st)) != hipSuccess) return e;
        }
        const LossOut<T, true> to_w{ldg, M, dp, M, scale, nullptr, nullptr,
                                    static_cast<T *>(a.dw) + v0 * a.lddw, a.lddw, dp, wide_w};
        if ((e = product<T>(g, x, to_w, n, D, M, st)) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

LossPlan loss_plan(int64_t M, int64_t V, int64_t D, bool pack_x, bool pack_w, bool backward) {
    auto up = [](int64_t v, int64_t to) { return (v + to - 1) / to * to; };
    LossPlan p{};
    p.dp = up(D, 64);
    p.pack_x = pack_x;
    p.pack_w = pack_w;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += up(bytes, 256);
        return o;
    };
    if (pack_x || backward) p.x = take(M * p.dp * 2);
    if (pack_w) p.w = take(V * p.dp * 2);
    if (!backward) {
        // pieces only where w passes the products' 4 GiB, or the tiles (of 512 threads) the
        // 2^32 threads of a launch
        p.piece = (int64_t(4000) << 20) / (p.dp * 2) / 256 * 256;
        if (p.piece > V) p.piece = V;
        auto launch_tiles = [&](int64_t n) {
            const LossTileShape &t = kLossTiles[loss_tile(M, n, false)];
            return (M + t.bm - 1) / t.bm * ((n + t.bn - 1) / t.bn);
        };
        while (launch_tiles(p.piece) >= (int64_t(1) << 23)) p.piece = up(p.piece / 2, 256);
        p.tiles = 0;
        for (int64_t v0 = 0; v0 < V; v0 += p.piece) {
            const int64_t n = V - v0 < p.piece ? V - v0 : p.piece;
            const int64_t bn = loss_tile_n(M, n);
            p.tiles += (n + bn - 1) / bn;
        }
        p.part = take(p.tiles * M * 8);
        p.logit = take(M * 4);
    } else {
        // pieces of about equal size whose G takes, with the copy of x, at most 256 MiB
        // (but at least 2048 entries): of the counts from the least one on, the one
        // whose products fill their rounds best
        const int64_t copy = M * p.dp * 2, row = 2 * (M > 0 ? M : 1);
        int64_t most = ((int64_t(256) << 20) - copy) / row / 256 * 256;
        if (most < 2048) most = 2048;
        // (w's piece, and G with the copy, inside the products' 4 GiB; G alone of a batch
        // so tall that 256 entries are more)
        const int64_t reach_w = (int64_t(4000) << 20) / (p.dp * 2) / 256 * 256;
        int64_t reach = ((int64_t(4000) << 20) - copy) / row / 256 * 256;
        if (reach < 256) reach = 256;
        if (most > reach) most = reach;
        if (most > reach_w) most = reach_w;
        const int64_t least = (V + most - 1) / most;
        double best = 0.0;
        for (int64_t pieces = least; pieces < least + 6; ++pieces) {
            const int64_t n = up((V + pieces - 1) / pieces, 256);
            double cost = 0.0;
            LossTile t;
            for (int64_t v0 = 0; v0 < V; v0 += n) {
                const int64_t q = V - v0 < n ? V - v0 : n;
                cost += double(loss_cost(M, q, false, &t)) * p.dp + double(loss_cost(M, D, true, &t)) * q +
                        double(loss_cost(q, D, true, &t)) * M;
                cost += 32768.0;  // three launches, about 10 us
                if (q == n && v0 + 2 * n < V) {  // the other full pieces cost the same
                    const int64_t more = (V - v0) / n - 1;
                    cost *= double(more + 1);
                    v0 += more * n;
                }
            }
            if (pieces == least || cost < best) best = cost, p.piece = n;
        }
        if (p.piece > V) p.piece = V;
        p.splits = loss_splits(M > 0 ? M : 1, D, p.piece);
        p.g = take(M * up(p.piece, 64 * p.splits) * 2);
        p.part = p.splits > 1 ? take(p.splits * M * p.dp * 4) : at;
        p.acc = p.piece < V ? take(M * p.dp * 4) : at;
        p.scale = take(8);
    }
    p.total = at;
    return p;
}

hipError_t launch_loss_fwd(const Loss &a, const LossPlan &pl, hipStream_t st) {
    return a.dtype == DT_F16 ? fwd<_Float16>(a, pl, st) : fwd<__bf16>(a, pl, st);
}
hipError_t launch_loss_bwd(const Loss &a, const LossPlan &pl, hipStream_t st) {
    return a.dtype == DT_F16 ? bwd<_Float16>(a, pl, st) : bwd<__bf16>(a, pl, st);
}

}  // namespace ssg

// Internal launch entry points of the gfx950 kernels (not exported).
// Arguments are validated by the C-ABI layer before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssg {

// int8 GEMM output kinds (the values of the C-ABI's SSG_OUT_* constants)
enum OutKind { OUT_I32 = 0, OUT_F32 = 1, OUT_F16 = 2, OUT_I8 = 3 };

hipError_t launch_dense_f16(const void *A, const void *Wt, void *C, int M, int N, int K, hipStream_t st);
hipError_t launch_dense_i8(const void *A, const void *Wt, const float *scale, const float *bias, void *C,
                           int out, int M, int N, int K, hipStream_t st);
hipError_t launch_w24_f16(const void *A, const void *vals, const uint32_t *meta, void *C, int M, int N,
                          int K, hipStream_t st);
hipError_t launch_w24_i8(const void *A, const void *vals, const uint32_t *meta, const float *scale,
                         const float *bias, void *C, int out, int M, int N, int K, hipStream_t st);
// Tiles tile_order[t_first .. t_first + t_count); out_t: C is written
// transposed, Ct [N][M]; a_rowmajor: the A operand is row-major [M][K]
// instead of K-major At [K][M]; narrow: every tile keeps at most 64 columns
// (the narrow-tile configurations; a wider tile's window comes out NaN).
hipError_t launch_tw_f16(const void *At, const void *vals, const int32_t *offset_k,
                         const int32_t *offset_n, const int32_t *v_ptr, const int32_t *k_ptr,
                         const int32_t *n_ptr, const int32_t *tile_order, int t_first, int t_count,
                         int G, bool out_t, bool a_rowmajor, bool narrow, void *C, int M, int N, int K,
                         hipStream_t st);
// int8 tile-wise GEMM (K-major int8 At, condensed int8 tiles), epilogue as
// the int8 GEMMs' OUT_* kinds.
hipError_t launch_tw_i8(const void *At, const void *vals, const int32_t *offset_k, const int32_t *offset_n,
                        const int32_t *v_ptr, const int32_t *k_ptr, const int32_t *n_ptr,
                        const int32_t *tile_order, int T, int G, const float *scale, const float *bias,
                        void *C, int out, int M, int N, hipStream_t st);
hipError_t launch_transpose_f16(const void *A, void *At, int M, int K, hipStream_t st);

// Split K: kind is a GEMM kind (0 dense fp16, 1 2:4 fp16, 2 dense int8, 3 2:4
// int8).  The split launch writes split s's raw accumulators (fp32 / int32)
// to slice s of ws ([splits][M][N], 4 bytes each); the reduce launch sums the
// slices in split order and applies the kind's epilogue (out: OUT_* for int8).
hipError_t launch_gemm_partials(int kind, const void *A, const void *W, const uint32_t *meta, void *ws, int M,
                                int N, int K, int splits, hipStream_t st);
hipError_t launch_splitk_reduce(const void *ws, int splits, bool i8, const float *scale, const float *bias,
                                void *C, int out, int M, int N, hipStream_t st);
// K splits worth taking for a kind and shape (1 = do not split); a host-only
// rule from the tile choice, the resident workgroups per CU and the K stages.
int suggest_splits(int kind, int M, int N, int K);
// tile rows x columns the GEMM launchers pick for a kind (0-3) and shape
void tile_choice(int kind, int M, int N, int K, int *bm, int *bn);
// ---- layer norm, low-rank adapters, linear cross entropy.
// element types (the values of the C-ABI's SSG_DT_* constants)
enum DType { DT_F16 = 0, DT_BF16 = 1, DT_F32 = 2 };

// Rows of x and y (and of the residual and the kept sum) are ld* elements
// apart; w and b are of type wtype (the rows' type or fp32) or null.
struct LnFwd {
    int dtype, wtype;
    const void *x, *res, *w, *b;
    int64_t ldx, ldr, ldy, lds;
    float eps;
    void *y, *sum;
    float *mean, *rstd;
    int64_t M, N;
};
// dw, db: fp32 [N] or both null; part: layer_norm_slices() slices of [2][N]
// fp32 when they are not.
struct LnBwd {
    int dtype, wtype;
    const void *dy, *x;
    const float *mean, *rstd;
    const void *w, *dres;
    int64_t lddy, ldx, ldres, lddx;
    void *dx;
    float *dw, *db, *part;
    int64_t M, N;
};
hipError_t launch_layer_norm_fwd(const LnFwd &a, hipStream_t st);
hipError_t launch_layer_norm_bwd(const LnBwd &a, hipStream_t st);
int64_t layer_norm_slices(int dtype, int64_t M, int64_t N);

// Low-rank adapters (formulas in low_rank.h).  dtype: DT_F16 or DT_BF16.
struct LowRank {
    int dtype;
    const void *down, *up;  // [adapters][R][K], [adapters][N][R]
    const float *scale;     // [adapters] or null (ones)
    const int32_t *ranks;   // [adapters] or null (all R)
    const int32_t *index;   // [M]
    int adapters, R;
};
template <class T>
struct ShrinkTask {
    const T *x;
    int64_t ldx;
    const T *down;  // [adapters][R][K] (or [adapters][K][R])
    T *low;         // two planes
    int K;
    int32_t *key;  // [M], or null: wgrad's list (fp16, low_key in low_rank.h)
};
template <class T>
struct WgradTask {
    const T *z;
    int64_t ldz;
    const T *low;
    float *part;  // fp32 slices, or null: out is written
    T *out;
    int C, tiles;
    bool rows_c;  // the result's rows are z's columns ([C][R]), else [R][C]
    const int32_t *key;
};
struct LowRankBwd {
    LowRank lr;
    const void *dy, *x, *base;
    int64_t lddy, ldx, ldb, lddx;
    void *dx, *ddown, *dup, *ws;
    int M, N, K;
};
// Byte offsets in the backward pass's workspace, and its split of the tokens.
struct LowRankPlan {
    int64_t low, dlow, keys, counts, part, total;
    int range, slices, deals;
};
bool low_rank_few(int M);
int64_t low_rank_bytes(int64_t M, int R);  // both planes of the low-rank values
// K splits of the 2:4 product under low_rank_few()
int low_rank_splits(int M, int N, int K);
LowRankPlan low_rank_plan(int adapters, int R, int64_t M, int64_t N, int64_t K);
// base: rows of T (or null: zeros); splits > 0: `splits` fp32 slices [M][N].
hipError_t launch_low_rank_tokens(const LowRank &lr, const void *x, int64_t ldx, const void *base, int64_t ldb,
                                  int splits, void *out, int64_t ldo, int M, int N, int K, hipStream_t st);
hipError_t launch_low_rank_shrink(const LowRank &lr, const void *x, int64_t ldx, void *low, int M, int K,
                                  hipStream_t st);
// ws: low_rank_bytes() (unused with few tokens).
hipError_t launch_low_rank_add(const LowRank &lr, const void *x, int64_t ldx, const void *base, int64_t ldb, void *out,
                               int64_t ldo, int M, int N, int K, void *ws, hipStream_t st);
hipError_t launch_low_rank_bwd(const LowRankBwd &b, hipStream_t st);
hipError_t launch_w24_low_rank_f16(const void *A, const void *vals, const uint32_t *meta, const LowRank &lr,
                                   const void *low, void *C, int M, int N, int K, hipStream_t st);

// Linear cross entropy (formulas in loss.hip).
struct Loss {
    int dtype;  // DT_F16 or DT_BF16
    const void *x, *w;
    int64_t ldx, ldw;
    const int64_t *target;
    int64_t ignore;
    float *loss, *lse;  // forward: written; backward: lse read
    const float *dloss;
    void *dx, *dw;
    int64_t lddx, lddw;
    int64_t M, V, D;
    void *ws;
};
// Pieces of the vocabulary and byte offsets in the workspace.
struct LossPlan {
    int64_t dp;      // D rounded up to the products' step of 64
    bool pack_x, pack_w;
    int64_t piece;   // vocabulary entries of a piece
    int64_t tiles;   // forward: tiles of the vocabulary
    int splits;      // backward: K splits of dx's product
    int64_t x, w, part, logit, g, acc, scale, total;
};
LossPlan loss_plan(int64_t M, int64_t V, int64_t D, bool pack_x, bool pack_w, bool backward);
hipError_t launch_loss_fwd(const Loss &a, const LossPlan &pl, hipStream_t st);
hipError_t launch_loss_bwd(const Loss &a, const LossPlan &pl, hipStream_t st);

// K stages (one per 128 bytes of an A row) for a kind and K.
inline int gemm_k_stages(int kind, int K) { return (kind == 2 || kind == 3) ? K / 128 : K / 64; }

}  // namespace ssg

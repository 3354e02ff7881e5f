// Exported entry points beside the GEMMs: layer norm, low-rank adapters and
// the cross entropy of a linear head.  As in api.hip: arguments are checked on
// the host before any HIP call, nothing is allocated, nothing synchronises.
#include <hip/hip_runtime.h>

#include "device.h"
#include "kernels/launch.h"
#include "status.h"

namespace {

using ssg::check_device;
using ssg::fits_int;
using ssg::launched;

int ok() {
    ssg::clear_error();
    return SSG_OK;
}

int elem_bytes(int dtype) { return dtype == SSG_DT_F32 ? 4 : 2; }
bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) == 0; }

// Row strides of [M][N] matrices: at least a row, and every offset inside 2^62.
bool bad_ld(int64_t ld, int64_t M, int64_t N) { return ld < N || (M > 0 && ld > (int64_t(1) << 62) / M); }

int check_norm(const char *fn, int dtype, int wtype, const void *w, int64_t M, int64_t N) {
    if (dtype < SSG_DT_F16 || dtype > SSG_DT_F32) return ssg::fail(SSG_EINVAL, "%s: unknown dtype %d", fn, dtype);
    if (w && wtype != dtype && wtype != SSG_DT_F32)
        return ssg::fail(SSG_EINVAL, "%s: weight type %d must be the rows' type or fp32", fn, wtype);
    if (M < 0 || N <= 0 || !fits_int(M) || !fits_int(N))
        return ssg::fail(SSG_EINVAL, "%s: M=%lld N=%lld (need 0 <= M, 1 <= N, both below 2^31)", fn, (long long)M,
                         (long long)N);
    if (w && !aligned_to(w, elem_bytes(wtype))) return ssg::fail(SSG_EINVAL, "%s: weight misaligned", fn);
    return SSG_OK;
}

}  // namespace

SSG_API int layer_norm_forward(int32_t dtype, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                               const void *weight, const void *bias, int32_t wtype, float eps, void *y, int64_t ldy,
                               void *sum, int64_t lds, float *mean, float *rstd, int64_t M, int64_t N, void *stream) {
    const char *fn = "layer_norm_forward";
    int rc = check_norm(fn, dtype, wtype, weight ? weight : bias, M, N);
    if (rc) return rc;
    if (!(eps >= 0.0f)) return ssg::fail(SSG_EINVAL, "%s: eps must not be negative", fn);
    if ((residual == nullptr) != (sum == nullptr))
        return ssg::fail(SSG_EINVAL, "%s: residual and sum go together", fn);
    if ((mean == nullptr) != (rstd == nullptr)) return ssg::fail(SSG_EINVAL, "%s: mean and rstd go together", fn);
    if (bad_ld(ldx, M, N) || bad_ld(ldy, M, N) || (residual && (bad_ld(ldr, M, N) || bad_ld(lds, M, N))))
        return ssg::fail(SSG_EINVAL, "%s: a row stride is shorter than N=%lld", fn, (long long)N);
    if (M == 0) return ok();
    if (!x || !y) return ssg::fail(SSG_EINVAL, "%s: null pointer", fn);
    const int e = elem_bytes(dtype);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(residual, e) || !aligned_to(sum, e) ||
        !aligned_to(bias, elem_bytes(wtype)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return ssg::fail(SSG_EINVAL, "%s: a pointer is not aligned to its element", fn);
    if ((rc = check_device())) return rc;
    const ssg::LnFwd a{dtype, wtype, x, residual, weight, bias, ldx, ldr, ldy, lds, eps, y, sum, mean, rstd, M, N};
    return launched(ssg::launch_layer_norm_fwd(a, hipStream_t(stream)), fn);
}

SSG_API int64_t layer_norm_workspace_bytes(int32_t dtype, int64_t M, int64_t N) {
    if (dtype < SSG_DT_F16 || dtype > SSG_DT_F32 || M <= 0 || N <= 0 || !fits_int(M) || !fits_int(N)) return 0;
    return ssg::layer_norm_slices(dtype, M, N) * 2 * N * 4;
}

SSG_API int layer_norm_backward(int32_t dtype, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                const float *mean, const float *rstd, const void *weight, int32_t wtype,
                                const void *dres, int64_t ldres, void *dx, int64_t lddx, float *dweight, float *dbias,
                                int64_t M, int64_t N, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "layer_norm_backward";
    int rc = check_norm(fn, dtype, wtype, weight, M, N);
    if (rc) return rc;
    if ((dweight == nullptr) != (dbias == nullptr))
        return ssg::fail(SSG_EINVAL, "%s: dweight and dbias go together", fn);
    if (bad_ld(lddy, M, N) || bad_ld(ldx, M, N) || bad_ld(lddx, M, N) || (dres && bad_ld(ldres, M, N)))
        return ssg::fail(SSG_EINVAL, "%s: a row stride is shorter than N=%lld", fn, (long long)N);
    if (M == 0 && !dweight) return ok();
    const int e = elem_bytes(dtype);
    if (M > 0) {
        if (!dy || !x || !mean || !rstd || !dx) return ssg::fail(SSG_EINVAL, "%s: null pointer", fn);
        if (!aligned_to(dy, e) || !aligned_to(x, e) || !aligned_to(dx, e) || !aligned_to(dres, e) ||
            !aligned_to(mean, 4) || !aligned_to(rstd, 4))
            return ssg::fail(SSG_EINVAL, "%s: a pointer is not aligned to its element", fn);
    }
    if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4))
        return ssg::fail(SSG_EINVAL, "%s: a pointer is not aligned to its element", fn);
    const int64_t need = dweight ? layer_norm_workspace_bytes(dtype, M, N) : 0;
    if (need > 0) {
        if (!ws || !ssg::aligned16(ws)) return ssg::fail(SSG_EINVAL, "%s: workspace null or not 16-byte aligned", fn);
        if (ws_bytes < need)
            return ssg::fail(SSG_EINVAL, "%s: workspace of %lld bytes, %lld needed", fn, (long long)ws_bytes,
                             (long long)need);
    }
    if ((rc = check_device())) return rc;
    const ssg::LnBwd a{dtype, wtype, dy,   x,     mean, rstd, weight, dres, lddy,
                       ldx,   ldres, lddx, dx,    dweight, dbias, static_cast<float *>(ws), M, N};
    return launched(ssg::launch_layer_norm_bwd(a, hipStream_t(stream)), fn);
}

// ---------------------------------------------------------------- adapters
namespace {

constexpr int64_t kMaxTokens = int64_t(65535) * 2048;  // token ranges of the gradient launch

int check_low_rank(const char *fn, const ssg_low_rank *lr, int64_t M, int64_t N, int64_t K) {
    if (!lr) return ssg::fail(SSG_EINVAL, "%s: null adapter description", fn);
    if (lr->dtype != SSG_DT_F16 && lr->dtype != SSG_DT_BF16)
        return ssg::fail(SSG_EINVAL, "%s: adapter dtype %d must be fp16 or bf16", fn, lr->dtype);
    if (lr->R < 8 || lr->R > 128 || lr->R % 8)
        return ssg::fail(SSG_EINVAL, "%s: R=%d must be a multiple of 8, at most 128", fn, lr->R);
    if (lr->adapters < 1 || lr->adapters > 65535)
        return ssg::fail(SSG_EINVAL, "%s: adapters=%d must be in 1..65535", fn, lr->adapters);
    if (M < 0 || M > kMaxTokens || N < 8 || K < 8 || N % 8 || K % 8 || !fits_int(N) || !fits_int(K))
        return ssg::fail(SSG_EINVAL, "%s: M=%lld N=%lld K=%lld (need 0 <= M < 2^27, N and K positive multiples of 8)",
                         fn, (long long)M, (long long)N, (long long)K);
    // launch grids: tiles of 64 x 128 outputs
    if (!fits_int((M + 63) / 64 * ((N + 127) / 128)) || !fits_int((M + 63) / 64 * ((K + 127) / 128)))
        return ssg::fail(SSG_EINVAL, "%s: dimensions too large", fn);
    return SSG_OK;
}

int check_pool(const char *fn, const ssg_low_rank *lr) {
    if (!lr->down || !lr->up || !lr->index) return ssg::fail(SSG_EINVAL, "%s: null pointer", fn);
    if (!ssg::aligned16(lr->down) || !ssg::aligned16(lr->up))
        return ssg::fail(SSG_EINVAL, "%s: down and up must be 16-byte aligned", fn);
    if (!aligned_to(lr->index, 4) || !aligned_to(lr->ranks, 4) || !aligned_to(lr->scale, 4))
        return ssg::fail(SSG_EINVAL, "%s: index, ranks or scale misaligned", fn);
    return SSG_OK;
}

// A matrix of 16-bit rows read and written 16 bytes at a time.
int check_rows(const char *fn, const char *name, const void *p, int64_t ld, int64_t M, int64_t N) {
    if (bad_ld(ld, M, N) || ld % 8)
        return ssg::fail(SSG_EINVAL, "%s: row stride %lld of %s must be a multiple of 8, at least %lld", fn,
                         (long long)ld, name, (long long)N);
    if (!p) return ssg::fail(SSG_EINVAL, "%s: %s is null", fn, name);
    if (!ssg::aligned16(p)) return ssg::fail(SSG_EINVAL, "%s: %s must be 16-byte aligned", fn, name);
    return SSG_OK;
}

int check_ws(const char *fn, const void *ws, int64_t ws_bytes, int64_t need) {
    if (need <= 0) return SSG_OK;
    if (!ws || !ssg::aligned16(ws)) return ssg::fail(SSG_EINVAL, "%s: workspace null or not 16-byte aligned", fn);
    if (ws_bytes < need)
        return ssg::fail(SSG_EINVAL, "%s: workspace of %lld bytes, %lld needed", fn, (long long)ws_bytes,
                         (long long)need);
    return SSG_OK;
}

ssg::LowRank internal(const ssg_low_rank *lr) {
    return {lr->dtype, lr->down, lr->up, lr->scale, lr->ranks, lr->index, lr->adapters, lr->R};
}

bool plain_rank(int32_t R) { return R >= 8 && R <= 128 && R % 8 == 0; }

}  // namespace

SSG_API int64_t low_rank_workspace_bytes(int64_t M, int32_t R) {
    if (M <= 0 || M > kMaxTokens || !plain_rank(R) || ssg::low_rank_few(int(M))) return 0;
    return ssg::low_rank_bytes(M, R);
}

SSG_API int low_rank_add(const ssg_low_rank *lr, const void *x, int64_t ldx, const void *base, int64_t ldb, void *out,
                         int64_t ldo, int64_t M, int64_t N, int64_t K, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "low_rank_add";
    int rc = check_low_rank(fn, lr, M, N, K);
    if (rc) return rc;
    if (M == 0) return ok();
    if ((rc = check_pool(fn, lr))) return rc;
    if ((rc = check_rows(fn, "x", x, ldx, M, K)) || (base && (rc = check_rows(fn, "base", base, ldb, M, N))) ||
        (rc = check_rows(fn, "out", out, ldo, M, N)))
        return rc;
    if ((rc = check_ws(fn, ws, ws_bytes, low_rank_workspace_bytes(M, lr->R)))) return rc;
    if ((rc = check_device())) return rc;
    return launched(ssg::launch_low_rank_add(internal(lr), x, ldx, base, ldb, out, ldo, int(M), int(N), int(K), ws,
                                             hipStream_t(stream)),
                    fn);
}

SSG_API int64_t w24_low_rank_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t R) {
    if (M <= 0 || N <= 0 || K <= 0 || !fits_int(M) || !fits_int(N) || !fits_int(K) || !plain_rank(R)) return 0;
    if (!ssg::low_rank_few(int(M))) return ssg::low_rank_bytes(M, R);
    return int64_t(ssg::low_rank_splits(int(M), int(N), int(K))) * M * N * 4;
}

SSG_API int w24_low_rank_gemm_f16(const void *A, const void *vals, const uint32_t *meta, const ssg_low_rank *lr,
                                  void *C, int64_t M, int64_t N, int64_t K, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "w24_low_rank_gemm_f16";
    int rc = check_low_rank(fn, lr, M, N, K);
    if (rc) return rc;
    if (lr->dtype != SSG_DT_F16) return ssg::fail(SSG_EINVAL, "%s: the adapters must be fp16", fn);
    if ((rc = ssg::check_gemm(fn, A, vals, C, M, N, K, 64, 64))) return rc;
    if (M == 0) return ok();
    if (!meta || !ssg::aligned16(meta)) return ssg::fail(SSG_EINVAL, "%s: meta null or misaligned", fn);
    if ((rc = check_pool(fn, lr))) return rc;
    if ((rc = check_ws(fn, ws, ws_bytes, w24_low_rank_workspace_bytes(M, N, K, lr->R)))) return rc;
    if ((rc = check_device())) return rc;
    const hipStream_t st = hipStream_t(stream);
    const ssg::LowRank in = internal(lr);
    const int m = int(M), n = int(N), k = int(K);
    if (ssg::low_rank_few(m)) {
        // the 2:4 product's fp32 sums first, then adapters and rounding in one launch
        const int splits = ssg::low_rank_splits(m, n, k);
        if ((rc = launched(ssg::launch_gemm_partials(1, A, vals, meta, ws, m, n, k, splits, st), fn))) return rc;
        return launched(ssg::launch_low_rank_tokens(in, A, K, ws, N, splits, C, N, m, n, k, st), fn);
    }
    if ((rc = launched(ssg::launch_low_rank_shrink(in, A, K, ws, m, k, st), fn))) return rc;
    return launched(ssg::launch_w24_low_rank_f16(A, vals, meta, in, ws, C, m, n, k, st), fn);
}

SSG_API int64_t low_rank_backward_workspace_bytes(int32_t adapters, int32_t R, int64_t M, int64_t N, int64_t K) {
    if (adapters < 1 || adapters > 65535 || !plain_rank(R) || M < 0 || M > kMaxTokens || N < 8 || K < 8 || N % 8 ||
        K % 8 || !fits_int(N) || !fits_int(K))
        return 0;
    return ssg::low_rank_plan(adapters, R, M, N, K).total;
}

SSG_API int low_rank_backward(const ssg_low_rank *lr, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                              const void *base, int64_t ldb, void *dx, int64_t lddx, void *ddown, void *dup, int64_t M,
                              int64_t N, int64_t K, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "low_rank_backward";
    int rc = check_low_rank(fn, lr, M, N, K);
    if (rc) return rc;
    if (!ddown || !dup || !ssg::aligned16(ddown) || !ssg::aligned16(dup))
        return ssg::fail(SSG_EINVAL, "%s: ddown or dup null or not 16-byte aligned", fn);
    if (M > 0) {
        if ((rc = check_pool(fn, lr))) return rc;
        if ((rc = check_rows(fn, "dy", dy, lddy, M, N)) || (rc = check_rows(fn, "x", x, ldx, M, K)) ||
            (base && (rc = check_rows(fn, "base", base, ldb, M, K))) || (rc = check_rows(fn, "dx", dx, lddx, M, K)))
            return rc;
    }
    if ((rc = check_ws(fn, ws, ws_bytes, low_rank_backward_workspace_bytes(lr->adapters, lr->R, M, N, K)))) return rc;
    if ((rc = check_device())) return rc;
    const ssg::LowRankBwd b{internal(lr), dy, x, base, lddy, ldx, ldb, lddx, dx, ddown, dup, ws, int(M), int(N), int(K)};
    return launched(ssg::launch_low_rank_bwd(b, hipStream_t(stream)), fn);
}

// -------------------------------------------------------------------- loss
namespace {

// Operands the products cannot read where they lie get a packed copy.
bool packs(int64_t ld, int64_t D) { return ld != D || D % 64 != 0; }

bool plain_loss(int32_t dtype, int64_t M, int64_t V, int64_t D) {
    return (dtype == SSG_DT_F16 || dtype == SSG_DT_BF16) && M >= 0 && V >= 1 && D >= 1 && fits_int(M) && fits_int(V) &&
           fits_int(D) && M * ((D + 63) / 64 * 128) < (int64_t(1) << 32) && D < (1 << 20) && M < 8000000 &&
           (M + 63) / 64 * ((V + 63) / 64) < (int64_t(1) << 31);
}

int check_loss(const char *fn, int32_t dtype, const void *x, int64_t ldx, const void *w, int64_t ldw,
               const int64_t *target, int64_t M, int64_t V, int64_t D) {
    if (dtype != SSG_DT_F16 && dtype != SSG_DT_BF16)
        return ssg::fail(SSG_EINVAL, "%s: dtype %d must be fp16 or bf16", fn, dtype);
    if (!plain_loss(dtype, M, V, D))
        return ssg::fail(SSG_EINVAL, "%s: M=%lld V=%lld D=%lld (need 0 <= M < 8000000, 1 <= V, 1 <= D < 2^20, x below 4 GiB)", fn,
                         (long long)M, (long long)V, (long long)D);
    if (bad_ld(ldx, M, D) || bad_ld(ldw, V, D))
        return ssg::fail(SSG_EINVAL, "%s: a row stride is shorter than D=%lld", fn, (long long)D);
    if (M == 0) return SSG_OK;
    if (!x || !w || !target) return ssg::fail(SSG_EINVAL, "%s: null pointer", fn);
    if (!aligned_to(x, packs(ldx, D) ? 2 : 16) || !aligned_to(w, packs(ldw, D) ? 2 : 16) || !aligned_to(target, 8))
        return ssg::fail(SSG_EINVAL, "%s: x and w must be 16-byte aligned, target 8-byte", fn);
    return SSG_OK;
}

}  // namespace

SSG_API int64_t linear_cross_entropy_workspace_bytes(int32_t dtype, int64_t M, int64_t V, int64_t D, int64_t ldx,
                                                     int64_t ldw, int32_t backward) {
    if (!plain_loss(dtype, M, V, D) || M == 0) return 0;
    return ssg::loss_plan(M, V, D, packs(ldx, D), packs(ldw, D), backward != 0).total;
}

SSG_API int linear_cross_entropy_forward(int32_t dtype, const void *x, int64_t ldx, const void *w, int64_t ldw,
                                         const int64_t *target, int64_t ignore_index, float *loss, float *lse,
                                         int64_t M, int64_t V, int64_t D, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "linear_cross_entropy_forward";
    int rc = check_loss(fn, dtype, x, ldx, w, ldw, target, M, V, D);
    if (rc) return rc;
    if (M == 0) return ok();
    if (!loss || !lse || !aligned_to(loss, 4) || !aligned_to(lse, 4))
        return ssg::fail(SSG_EINVAL, "%s: loss or lse null or misaligned", fn);
    const ssg::LossPlan pl = ssg::loss_plan(M, V, D, packs(ldx, D), packs(ldw, D), false);
    if ((rc = check_ws(fn, ws, ws_bytes, pl.total))) return rc;
    if ((rc = check_device())) return rc;
    ssg::Loss a{};
    a.dtype = dtype, a.x = x, a.w = w, a.ldx = ldx, a.ldw = ldw, a.target = target, a.ignore = ignore_index;
    a.loss = loss, a.lse = lse, a.M = M, a.V = V, a.D = D, a.ws = ws;
    return launched(ssg::launch_loss_fwd(a, pl, hipStream_t(stream)), fn);
}

SSG_API int linear_cross_entropy_backward(int32_t dtype, const float *dloss, const void *x, int64_t ldx, const void *w,
                                          int64_t ldw, const int64_t *target, int64_t ignore_index, const float *lse,
                                          void *dx, int64_t lddx, void *dw, int64_t lddw, int64_t M, int64_t V,
                                          int64_t D, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "linear_cross_entropy_backward";
    int rc = check_loss(fn, dtype, x, ldx, w, ldw, target, M, V, D);
    if (rc) return rc;
    if (bad_ld(lddx, M, D) || bad_ld(lddw, V, D))
        return ssg::fail(SSG_EINVAL, "%s: a row stride is shorter than D=%lld", fn, (long long)D);
    if (!dw || !aligned_to(dw, 2) || (M > 0 && (!dx || !aligned_to(dx, 2))))
        return ssg::fail(SSG_EINVAL, "%s: dx or dw null or misaligned", fn);
    if (M > 0 && (!dloss || !lse || !aligned_to(dloss, 4) || !aligned_to(lse, 4)))
        return ssg::fail(SSG_EINVAL, "%s: dloss or lse null or misaligned", fn);
    const ssg::LossPlan pl = ssg::loss_plan(M, V, D, packs(ldx, D), packs(ldw, D), true);
    if (M > 0 && (rc = check_ws(fn, ws, ws_bytes, pl.total))) return rc;
    if ((rc = check_device())) return rc;
    ssg::Loss a{};
    a.dtype = dtype, a.x = x, a.w = w, a.ldx = ldx, a.ldw = ldw, a.target = target, a.ignore = ignore_index;
    a.dloss = dloss, a.lse = const_cast<float *>(lse), a.dx = dx, a.dw = dw, a.lddx = lddx, a.lddw = lddw;
    a.M = M, a.V = V, a.D = D, a.ws = ws;
    return launched(ssg::launch_loss_bwd(a, pl, hipStream_t(stream)), fn);
}

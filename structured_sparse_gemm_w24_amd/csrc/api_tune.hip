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

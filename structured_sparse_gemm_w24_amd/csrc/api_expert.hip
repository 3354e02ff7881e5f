// Exported entry points of expert layers: products grouped by expert, microscaled
// 4-bit products, the gradient norm.  As in api.hip: arguments are checked on the
// host before any HIP call, nothing is allocated, nothing synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <numeric>
#include <vector>

#include "device.h"
#include "kernels/launch.h"
#include "status.h"

namespace {

using ssg::check_device;
using ssg::fits_int;
using ssg::launched;

// A tile's 256 rows stay below 2 GiB (the kernels' offsets are of 32 bits), and the products' rows below
// 2^29 (so are their tile counts, and stages of 64 rows below 2^24).
constexpr int64_t kSide = int64_t(1) << 22, kGiB2 = int64_t(1) << 31, kRows = int64_t(1) << 29;

int ok() {
    ssg::clear_error();
    return SSG_OK;
}

int elem_bytes(int dtype) { return dtype == SSG_DT_F32 ? 4 : 2; }
bool known(int dtype) { return dtype >= SSG_DT_F16 && dtype <= SSG_DT_F32; }
bool half_type(int dtype) { return dtype == SSG_DT_F16 || dtype == SSG_DT_BF16; }
bool aligned_to(const void *p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) == 0; }
bool bad_ld(int64_t ld, int64_t M, int64_t N) { return ld < N || (M > 0 && ld > (int64_t(1) << 61) / M); }

int check_ws(const char *fn, const void *ws, int64_t have, int64_t need) {
    if (need > 0 && (!ws || !ssg::aligned16(ws)))
        return ssg::fail(SSG_EINVAL, "%s: workspace null or not 16-byte aligned", fn);
    if (have < need)
        return ssg::fail(SSG_EINVAL, "%s: workspace of %lld bytes, %lld needed", fn, (long long)have, (long long)need);
    return SSG_OK;
}

// Rows that the kernels read and write 16 bytes at a time.
int check_rows(const char *fn, const char *name, const void *p, int64_t ld, int64_t N) {
    if (ld < N || ld >= kSide || ld % 8)
        return ssg::fail(SSG_EINVAL, "%s: row stride %lld of %s must be a multiple of 8, at least %lld, below 2^22", fn,
                         (long long)ld, name, (long long)N);
    if (!p || !ssg::aligned16(p)) return ssg::fail(SSG_EINVAL, "%s: %s null or not 16-byte aligned", fn, name);
    return SSG_OK;
}

// Rows of any element alignment.
int check_any(const char *fn, const char *name, const void *p, int64_t ld, int64_t M, int64_t N, int dtype) {
    if (bad_ld(ld, M, N))
        return ssg::fail(SSG_EINVAL, "%s: row stride %lld of %s is shorter than %lld, or too long", fn, (long long)ld,
                         name, (long long)N);
    if (!p || !aligned_to(p, elem_bytes(dtype)))
        return ssg::fail(SSG_EINVAL, "%s: %s null or not aligned to its elements", fn, name);
    return SSG_OK;
}

int check_groups(const char *fn, const int32_t *offsets, int32_t experts) {
    if (experts < 1 || experts > 65535)
        return ssg::fail(SSG_EINVAL, "%s: experts=%d must be in 1..65535", fn, experts);
    if (!offsets || !aligned_to(offsets, 4)) return ssg::fail(SSG_EINVAL, "%s: offsets null or misaligned", fn);
    return SSG_OK;
}

bool grouped_dims(int64_t M, int64_t N, int64_t K) {
    return M >= 0 && M < kRows && N >= 8 && K >= 8 && N % 8 == 0 && K % 8 == 0 && N < kSide && K < kSide &&
           N * K * 2 < kGiB2;
}

int check_grouped(const char *fn, int32_t dtype, const int32_t *offsets, int32_t experts, int64_t M, int64_t N,
                  int64_t K, bool backward) {
    if (!half_type(dtype)) return ssg::fail(SSG_EINVAL, "%s: dtype %d must be fp16 or bf16", fn, dtype);
    if (!grouped_dims(M, N, K))
        return ssg::fail(SSG_EINVAL,
                         "%s: M=%lld N=%lld K=%lld (need 0 <= M < 2^29, N and K positive multiples of 8 below 2^22, a "
                         "weight below 2 GiB)",
                         fn, (long long)M, (long long)N, (long long)K);
    if (int rc = check_groups(fn, offsets, experts)) return rc;
    // (a launch takes fewer than 2^32 threads, in workgroups of up to 512)
    if (ssg::grouped_blocks(M, experts, N, K, backward) >= (int64_t(1) << 23))
        return ssg::fail(SSG_EINVAL, "%s: dimensions too large for one launch", fn);
    return SSG_OK;
}

// (the element kernels: two pieces of eight values a thread, 2^32 threads a launch; padded rows have 16
// pieces or more, so M stays below 2^29 as well)
bool mx_dims(int64_t M, int64_t K) {
    return M >= 0 && fits_int(M) && K >= 1 && K < kSide && M * (ssg::mxfp4_padded(K) / 8) < (int64_t(1) << 33) - 512;
}

int check_mx(const char *fn, int64_t M, int64_t K) {
    if (!mx_dims(M, K))
        return ssg::fail(SSG_EINVAL, "%s: M=%lld K=%lld (need 0 <= M < 2^29, 1 <= K < 2^22, below 2^36 padded values)", fn,
                         (long long)M, (long long)K);
    return SSG_OK;
}

int check_packed(const char *fn, const char *name, const uint8_t *codes, const uint8_t *scales) {
    if (!codes || !scales || !ssg::aligned16(codes) || !aligned_to(scales, 4))
        return ssg::fail(SSG_EINVAL, "%s: codes of %s null or not 16-byte aligned, or scales null or not 4-byte aligned",
                         fn, name);
    return SSG_OK;
}

int check_mx_gemm(const char *fn, const uint8_t *w, const uint8_t *w_scales, const int32_t *offsets, int32_t experts,
                  int dtype, const void *out, int64_t ldo, int64_t M, int64_t N, int64_t K) {
    int rc = check_mx(fn, M, K);
    if (rc) return rc;
    if (N < 1 || N >= kSide || N * ssg::mxfp4_padded(K) / 2 >= kGiB2)
        return ssg::fail(SSG_EINVAL, "%s: N=%lld K=%lld (need 1 <= N < 2^22, a weight's codes below 2 GiB)", fn,
                         (long long)N, (long long)K);
    if (offsets ? (rc = check_groups(fn, offsets, experts)) : experts != 1)
        return rc ? rc : ssg::fail(SSG_EINVAL, "%s: experts=%d without offsets", fn, experts);
    if (ssg::mxfp4_blocks(M, offsets ? experts : 0, N, K) >= (int64_t(1) << 23))
        return ssg::fail(SSG_EINVAL, "%s: dimensions too large for one launch", fn);
    if (M == 0) return SSG_OK;
    if ((rc = check_any(fn, "out", out, ldo, M, N, dtype))) return rc;
    return check_packed(fn, "w", w, w_scales);
}

// Memory that a call reads or writes: rows of `width` bytes, `step` apart (a run of memory: one row).
struct Area {
    const char *name;
    const void *p;
    int64_t rows, step, width;
};
Area run(const char *name, const void *p, int64_t bytes) { return {name, p, 1, bytes, bytes}; }
Area matrix(const char *name, const void *p, int64_t rows, int64_t ld, int64_t n, int bytes) {
    return {name, p, rows, rows > 1 ? ld * bytes : n * bytes, n * bytes};  // (one row: of any stride)
}

// Rows of one buffer beside each other (column slices, every other row) share no byte: they lie apart by
// their place in the common divisor of both steps.
bool meet(const Area &a, const Area &b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    if (pa + uintptr_t((a.rows - 1) * a.step + a.width) <= pb || pb + uintptr_t((b.rows - 1) * b.step + b.width) <= pa)
        return false;
    if (a.rows == 1 && b.rows == 1) return true;
    const int64_t g = a.rows == 1 ? b.step : b.rows == 1 ? a.step : std::gcd(a.step, b.step);
    const int64_t off = pb >= pa ? int64_t((pb - pa) % uintptr_t(g)) : g - 1 - int64_t((pa - pb - 1) % uintptr_t(g));
    return off < a.width || off + b.width > g;
}

// Nothing that is written may share a byte with anything else of the call.
int check_apart(const char *fn, std::initializer_list<Area> written, std::initializer_list<Area> read) {
    for (const Area *w = written.begin(); w != written.end(); ++w) {
        for (const Area *o = w + 1; o != written.end(); ++o)
            if (meet(*w, *o)) return ssg::fail(SSG_EINVAL, "%s: %s overlaps %s", fn, w->name, o->name);
        for (const Area &r : read)
            if (meet(*w, r)) return ssg::fail(SSG_EINVAL, "%s: %s overlaps %s", fn, w->name, r.name);
    }
    return SSG_OK;
}
Area offsets_area(const int32_t *offsets, int32_t experts) {
    return run("offsets", offsets, 4 * (int64_t(experts) + 1));
}
Area codes_area(const char *name, const uint8_t *p, int64_t rows, int64_t K) {
    return run(name, p, rows * (ssg::mxfp4_padded(K) / 2));
}
Area scales_area(const char *name, const uint8_t *p, int64_t rows, int64_t K) {
    return run(name, p, rows * (ssg::mxfp4_padded(K) / 32));
}

}  // namespace

// ------------------------------------------------------------ grouped products
SSG_API int grouped_gemm(int32_t dtype, const void *x, int64_t ldx, const void *w, const int32_t *offsets,
                         int32_t experts, void *out, int64_t ldo, int64_t M, int64_t N, int64_t K, void *stream) {
    const char *fn = "grouped_gemm";
    int rc = check_grouped(fn, dtype, offsets, experts, M, N, K, false);
    if (rc) return rc;
    if (M == 0) return ok();
    if ((rc = check_rows(fn, "x", x, ldx, K)) || (rc = check_rows(fn, "w", w, K, K)) ||
        (rc = check_rows(fn, "out", out, ldo, N)) ||
        (rc = check_apart(fn, {matrix("out", out, M, ldo, N, 2)},
                          {matrix("x", x, M, ldx, K, 2), run("w", w, experts * N * K * 2),
                           offsets_area(offsets, experts)})) ||
        (rc = check_device()))
        return rc;
    ssg::Grouped a{};
    a.dtype = dtype, a.x = x, a.w = w, a.offsets = offsets, a.experts = experts, a.ldx = ldx, a.out = out, a.ldo = ldo;
    a.M = M, a.N = N, a.K = K;
    return launched(ssg::launch_grouped_fwd(a, hipStream_t(stream)), fn);
}

SSG_API int64_t grouped_gemm_backward_workspace_bytes(int32_t experts, int64_t M, int64_t N, int64_t K) {
    if (experts < 1 || experts > 65535 || !grouped_dims(M, N, K)) return 0;
    return ssg::grouped_slices_bytes(M, experts, N, K);
}

SSG_API int grouped_gemm_backward(int32_t dtype, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                  const void *w, const int32_t *offsets, int32_t experts, void *dx, int64_t lddx,
                                  void *dw, int64_t M, int64_t N, int64_t K, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "grouped_gemm_backward";
    int rc = check_grouped(fn, dtype, offsets, experts, M, N, K, true);
    if (rc) return rc;
    if (M > 0) {
        if ((rc = check_rows(fn, "dy", dy, lddy, N))) return rc;
        if (dx && ((rc = check_rows(fn, "dx", dx, lddx, K)) || (rc = check_rows(fn, "w", w, K, K)))) return rc;
        if (dw && (rc = check_rows(fn, "x", x, ldx, K))) return rc;
    }
    if (dw && ((rc = check_rows(fn, "dw", dw, K, K)) ||
               (rc = check_ws(fn, ws, ws_bytes, grouped_gemm_backward_workspace_bytes(experts, M, N, K)))))
        return rc;
    if (!dw && (!dx || M == 0)) return ok();
    const int64_t pool = experts * N * K * 2, slices = dw ? grouped_gemm_backward_workspace_bytes(experts, M, N, K) : 0;
    if ((rc = check_apart(fn, {matrix("dx", dx, M, lddx, K, 2), run("dw", dw, pool), run("the workspace", ws, slices)},
                          {matrix("dy", dy, M, lddy, N, 2), matrix("x", dw ? x : nullptr, M, ldx, K, 2),
                           run("w", dx ? w : nullptr, pool), offsets_area(offsets, experts)})) ||
        (rc = check_device()))
        return rc;
    ssg::Grouped a{};
    a.dtype = dtype, a.x = x, a.w = w, a.dy = dy, a.offsets = offsets, a.experts = experts;
    a.ldx = ldx, a.lddy = lddy, a.dx = dx, a.lddx = lddx, a.dw = dw, a.ws = ws, a.M = M, a.N = N, a.K = K;
    return launched(ssg::launch_grouped_bwd(a, hipStream_t(stream)), fn);
}

SSG_API int32_t ssg_expert_tile(int32_t product, int32_t experts, int64_t M, int64_t N, int64_t K) {
    if (product < 0 || product > 4 || M < 1 || experts < (product == 4 ? 0 : 1) || experts > 65535) return -2;
    if (product < 4) return grouped_dims(M, N, K) ? ssg::grouped_tile(product, M, experts, N, K) : -2;
    if (!mx_dims(M, K) || N < 1 || N >= kSide) return -2;
    const int few = ssg::mxfp4_few_kind(M, experts, N, K);
    return few >= 0 ? 16 + few : ssg::mxfp4_tile(M, experts, N, K);
}

// ------------------------------------------------------------ microscaled 4 bit
SSG_API int mxfp4_quantize(int32_t dtype, const void *x, int64_t ldx, uint8_t *codes, uint8_t *scales, int64_t M,
                           int64_t K, void *stream) {
    const char *fn = "mxfp4_quantize";
    if (!known(dtype)) return ssg::fail(SSG_EINVAL, "%s: unknown dtype %d", fn, dtype);
    int rc = check_mx(fn, M, K);
    if (rc) return rc;
    if (M == 0) return ok();
    if ((rc = check_any(fn, "x", x, ldx, M, K, dtype)) || (rc = check_packed(fn, "the output", codes, scales)) ||
        (rc = check_apart(fn, {codes_area("codes", codes, M, K), scales_area("scales", scales, M, K)},
                          {matrix("x", x, M, ldx, K, elem_bytes(dtype))})) ||
        (rc = check_device()))
        return rc;
    return launched(ssg::launch_mxfp4_quantize(dtype, x, ldx, codes, scales, M, K, hipStream_t(stream)), fn);
}

SSG_API int mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int32_t dtype, void *out, int64_t ldo,
                             int64_t M, int64_t K, void *stream) {
    const char *fn = "mxfp4_dequantize";
    if (!known(dtype)) return ssg::fail(SSG_EINVAL, "%s: unknown dtype %d", fn, dtype);
    int rc = check_mx(fn, M, K);
    if (rc) return rc;
    if (M == 0) return ok();
    if ((rc = check_any(fn, "out", out, ldo, M, K, dtype)) || (rc = check_packed(fn, "the input", codes, scales)) ||
        (rc = check_apart(fn, {matrix("out", out, M, ldo, K, elem_bytes(dtype))},
                          {codes_area("codes", codes, M, K), scales_area("scales", scales, M, K)})) ||
        (rc = check_device()))
        return rc;
    return launched(ssg::launch_mxfp4_dequantize(dtype, codes, scales, out, ldo, M, K, hipStream_t(stream)), fn);
}

SSG_API int mxfp4_gemm(const uint8_t *a, const uint8_t *a_scales, const uint8_t *w, const uint8_t *w_scales,
                       const int32_t *offsets, int32_t experts, int32_t dtype, void *out, int64_t ldo, int64_t M,
                       int64_t N, int64_t K, void *stream) {
    const char *fn = "mxfp4_gemm";
    if (!known(dtype)) return ssg::fail(SSG_EINVAL, "%s: unknown dtype %d", fn, dtype);
    int rc = check_mx_gemm(fn, w, w_scales, offsets, experts, dtype, out, ldo, M, N, K);
    if (rc) return rc;
    if (M == 0) return ok();
    if ((rc = check_packed(fn, "a", a, a_scales)) ||
        (rc = check_apart(fn, {matrix("out", out, M, ldo, N, elem_bytes(dtype))},
                          {codes_area("a", a, M, K), scales_area("a's scales", a_scales, M, K),
                           codes_area("w", w, experts * N, K), scales_area("w's scales", w_scales, experts * N, K),
                           offsets_area(offsets, experts)})) ||
        (rc = check_device()))
        return rc;
    const ssg::Mxfp4Gemm g{a, a_scales, w, w_scales, offsets, experts, dtype, out, ldo, M, N, K};
    return launched(ssg::launch_mxfp4_gemm(g, hipStream_t(stream)), fn);
}

SSG_API int64_t mxfp4_linear_workspace_bytes(int64_t M, int64_t K) {
    if (!mx_dims(M, K)) return 0;
    const int64_t kp = ssg::mxfp4_padded(K);
    return M * (kp / 2) + M * (kp / 32);
}

SSG_API int mxfp4_linear(int32_t dtype, const void *x, int64_t ldx, const uint8_t *w, const uint8_t *w_scales,
                         const int32_t *offsets, int32_t experts, void *out, int64_t ldo, int64_t M, int64_t N,
                         int64_t K, void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "mxfp4_linear";
    if (!half_type(dtype)) return ssg::fail(SSG_EINVAL, "%s: dtype %d must be fp16 or bf16", fn, dtype);
    int rc = check_mx_gemm(fn, w, w_scales, offsets, experts, dtype, out, ldo, M, N, K);
    if (rc) return rc;
    if (M == 0) return ok();
    if ((rc = check_any(fn, "x", x, ldx, M, K, dtype)) ||
        (rc = check_ws(fn, ws, ws_bytes, mxfp4_linear_workspace_bytes(M, K))) ||
        (rc = check_apart(fn, {matrix("out", out, M, ldo, N, 2), run("the workspace", ws, mxfp4_linear_workspace_bytes(M, K))},
                          {matrix("x", x, M, ldx, K, 2), codes_area("w", w, experts * N, K),
                           scales_area("w's scales", w_scales, experts * N, K), offsets_area(offsets, experts)})) ||
        (rc = check_device()))
        return rc;
    if (ssg::mxfp4_few_kind(M, offsets ? experts : 0, N, K) >= 0) {
        const ssg::Mxfp4Gemm g{static_cast<const uint8_t *>(x), nullptr, w, w_scales, offsets, experts, dtype, out, ldo, M,
                               N, K};
        return launched(ssg::launch_mxfp4_few(g, dtype, ldx, hipStream_t(stream)), fn);
    }
    uint8_t *codes = static_cast<uint8_t *>(ws), *scales = codes + M * (ssg::mxfp4_padded(K) / 2);
    const hipError_t e = ssg::launch_mxfp4_quantize(dtype, x, ldx, codes, scales, M, K, hipStream_t(stream));
    if (e != hipSuccess) return launched(e, fn);
    const ssg::Mxfp4Gemm g{codes, scales, w, w_scales, offsets, experts, dtype, out, ldo, M, N, K};
    return launched(ssg::launch_mxfp4_gemm(g, hipStream_t(stream)), fn);
}

// ---------------------------------------------------------------- gradient norm
namespace {

// (up to 2^20 tensors and 2^44 bytes: piece and slot numbers stay below 2^31)
int check_list(const char *fn, int32_t n, const void *const *grads, const int64_t *sizes, const int32_t *dtypes) {
    if (n < 0 || n > (1 << 20)) return ssg::fail(SSG_EINVAL, "%s: n=%d tensors (need 0 <= n <= 2^20)", fn, n);
    int64_t bytes = 0;
    if (n > 0 && (!grads || !sizes || !dtypes)) return ssg::fail(SSG_EINVAL, "%s: null list", fn);
    for (int i = 0; i < n; ++i) {
        if (!known(dtypes[i])) return ssg::fail(SSG_EINVAL, "%s: unknown dtype %d of tensor %d", fn, dtypes[i], i);
        if (sizes[i] < 0 || sizes[i] >= (int64_t(1) << 40))
            return ssg::fail(SSG_EINVAL, "%s: tensor %d has %lld elements (need 0 <= size < 2^40)", fn, i,
                             (long long)sizes[i]);
        if (sizes[i] > 0 && (!grads[i] || !aligned_to(grads[i], elem_bytes(dtypes[i]))))
            return ssg::fail(SSG_EINVAL, "%s: tensor %d null or not aligned to its elements", fn, i);
        if ((bytes += sizes[i] * elem_bytes(dtypes[i])) > int64_t(1) << 44)
            return ssg::fail(SSG_EINVAL, "%s: tensors of more than 16 TiB", fn);
    }
    return SSG_OK;
}

struct Span {
    uintptr_t from, to;
    int tensor;
    bool written;
};

// What is written must be no one else's: spans in address order, a written one overlaps no other
// (an in-place tensor is one span) and not the norm that every workgroup reads.
int check_overlap(const char *fn, int32_t n, const void *const *grads, void *const *outs, const int64_t *sizes,
                  const int32_t *dtypes, const float *norm_in) {
    std::vector<Span> spans;
    try {
        spans.reserve(size_t(n) * 2 + 1);
    } catch (const std::bad_alloc &) {
        return ssg::fail(SSG_ENOSPC, "%s: no host memory for %d tensors", fn, n);
    }
    for (int i = 0; i < n; ++i) {
        if (sizes[i] == 0) continue;
        if (!outs[i] || !aligned_to(outs[i], elem_bytes(dtypes[i])))
            return ssg::fail(SSG_EINVAL, "%s: output %d null or not aligned to its elements", fn, i);
        const uintptr_t bytes = uintptr_t(sizes[i]) * uintptr_t(elem_bytes(dtypes[i]));
        const uintptr_t in = reinterpret_cast<uintptr_t>(grads[i]), to = reinterpret_cast<uintptr_t>(outs[i]);
        spans.push_back({to, to + bytes, i, true});
        if (in != to) spans.push_back({in, in + bytes, i, false});
    }
    if (norm_in) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(norm_in);
        spans.push_back({at, at + sizeof(float), -1, false});
    }
    std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
    uintptr_t any = 0, written = 0;  // furthest end so far, of all spans and of the written ones
    for (const Span &s : spans) {
        if (s.from < written || (s.written && s.from < any))
            return s.tensor < 0 ? ssg::fail(SSG_EINVAL, "%s: norm_in overlaps an output", fn)
                                : ssg::fail(SSG_EINVAL, "%s: tensor %d overlaps another input or output", fn, s.tensor);
        any = std::max(any, s.to);
        if (s.written) written = std::max(written, s.to);
    }
    return SSG_OK;
}

// The norm that is written and the workspace lie apart from each other and from every tensor.
int check_norm_apart(const char *fn, int32_t n, const void *const *grads, const void *const *outs, const int64_t *sizes,
                     const int32_t *dtypes, const float *norm, const void *ws) {
    const Area of_norm = run("norm", norm, sizeof(float)), of_ws = run("the workspace", ws, ssg::grad_norm_slots(n) * 8);
    if (int rc = check_apart(fn, {of_norm, of_ws}, {})) return rc;
    for (int i = 0; i < n; ++i) {
        const int64_t bytes = sizes[i] * elem_bytes(dtypes[i]);
        for (const Area &a : {run("a tensor", grads[i], bytes), run("an output", outs ? outs[i] : nullptr, bytes)})
            for (const Area &w : {of_norm, of_ws})
                if (meet(w, a)) return ssg::fail(SSG_EINVAL, "%s: %s overlaps %s (entry %d)", fn, w.name, a.name, i);
    }
    return SSG_OK;
}

}  // namespace

SSG_API int64_t grad_norm_workspace_bytes(int32_t n) { return n > 0 ? ssg::grad_norm_slots(n) * 8 : 0; }

SSG_API int grad_norm(int32_t n, const void *const *grads, const int64_t *sizes, const int32_t *dtypes, float *norm,
                      void *ws, int64_t ws_bytes, void *stream) {
    const char *fn = "grad_norm";
    int rc = check_list(fn, n, grads, sizes, dtypes);
    if (rc) return rc;
    if (!norm || !aligned_to(norm, 4)) return ssg::fail(SSG_EINVAL, "%s: norm null or misaligned", fn);
    if ((rc = check_ws(fn, ws, ws_bytes, grad_norm_workspace_bytes(n))) ||
        (rc = check_norm_apart(fn, n, grads, nullptr, sizes, dtypes, norm, n > 0 ? ws : nullptr)) || (rc = check_device()))
        return rc;
    const ssg::GradList l{n, grads, nullptr, sizes, dtypes};
    return launched(ssg::launch_grad_norm(l, static_cast<double *>(ws), norm, hipStream_t(stream)), fn);
}

SSG_API int clip_grad_norm(int32_t n, const void *const *grads, void *const *outs, const int64_t *sizes,
                           const int32_t *dtypes, double max_norm, const float *norm_in, float *norm, void *ws,
                           int64_t ws_bytes, void *stream) {
    const char *fn = "clip_grad_norm";
    int rc = check_list(fn, n, grads, sizes, dtypes);
    if (rc) return rc;
    if (!(max_norm >= 0.0)) return ssg::fail(SSG_EINVAL, "%s: max_norm=%g must be 0 or more", fn, max_norm);
    if (n > 0 && !outs) return ssg::fail(SSG_EINVAL, "%s: null list", fn);
    if ((rc = check_overlap(fn, n, grads, outs, sizes, dtypes, norm_in))) return rc;
    if (!norm_in) {
        if (!norm || !aligned_to(norm, 4)) return ssg::fail(SSG_EINVAL, "%s: norm null or misaligned", fn);
        if ((rc = check_ws(fn, ws, ws_bytes, grad_norm_workspace_bytes(n))) ||
            (rc = check_norm_apart(fn, n, grads, outs, sizes, dtypes, norm, n > 0 ? ws : nullptr)))
            return rc;
    } else if (!aligned_to(norm_in, 4)) {
        return ssg::fail(SSG_EINVAL, "%s: norm_in misaligned", fn);
    }
    if ((rc = check_device())) return rc;
    const ssg::GradList l{n, grads, outs, sizes, dtypes};
    return launched(ssg::launch_clip_grad_norm(l, max_norm, norm_in, static_cast<double *>(ws), norm,
                                               hipStream_t(stream)),
                    fn);
}

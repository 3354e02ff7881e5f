// Global norm of many tensors and their scaling to a largest norm.
//
//   norm = sqrt(sum over all tensors of x^2),   out = x min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: every element is read for the norm, read again and written for the
// scaling.  The tensors' addresses travel in the kernel arguments (a launch takes as
// many as fit in 4 KiB), so a call copies nothing to the device and captures into a
// graph.  A launch's tensors are cut into pieces of 16 KiB, which the workgroups of a grid of
// fixed size take in turn; each writes one partial sum and the sums are added in a fixed
// order.  So a launch walks through memory once from its first tensor to its last, and the
// scaling walks back the same way: what the norm read last (256 MB) may still be cached.  Squares and
// sums are fp64: an fp32 gradient of 1e30 does not overflow, and the order of summation shows in no
// digit of an fp32 norm.  290 tensors of 120 M values (360 MB to read, read again and write): 207 us in six
// launches, 5.2 TB/s; a copy that moves as much takes 209.
#include <cfloat>
#include <cmath>

#include "elem.h"
#include "launch.h"

namespace ssg {

namespace {

constexpr int kGrid = 1024;    // workgroups of a launch, at most
constexpr int kPiece = 16384;  // bytes
constexpr int kThreads = 256;
constexpr int kNormTensors = 190, kClipTensors = 136;
constexpr double kEps = 1e-6;

// size: elements, with the type in the bits above 2^56.
struct NormTable {
    const void *grad[kNormTensors];
    int64_t size[kNormTensors];
    uint32_t first[kNormTensors + 1];  // first piece of each tensor; at n: all pieces
    int n;
};
struct ClipTable {
    const void *grad[kClipTensors];
    void *out[kClipTensors];
    int64_t size[kClipTensors];
    uint32_t first[kClipTensors + 1];
    int n;
};
static_assert(sizeof(NormTable) <= 4000 && sizeof(ClipTable) <= 4000, "tables must fit in the kernel arguments");

// The tensor that piece p belongs to: how many start at or before it, 64 looked at a time (a search by
// halves is a chain of eight scalar loads, 2 us of a small call's 5).
template <class Table>
__device__ __forceinline__ int tensor_of(const Table &t, uint32_t p) {
    int before = 0;
    for (int i = 0; i < t.n; i += 64) {
        const int at = i + int(threadIdx.x & 63);
        before += __popcll(__ballot(at < t.n && t.first[at] <= p));
    }
    return before - 1;
}

template <class T>
__device__ __forceinline__ void add_squares(double &sum, typename Elem<T>::Vec v) {
#pragma unroll
    for (int i = 0; i < Elem<T>::V; ++i) {
        const double d = double(float(v[i]));
        sum = __builtin_fma(d, d, sum);
    }
}

// A piece: four 16-byte accesses a thread, kThreads apart.
template <class T>
__device__ __forceinline__ void piece_squares(double &sum, const void *p, int64_t at, int64_t n) {
    constexpr int V = Elem<T>::V, STEP = kThreads * V;
    const T *x = static_cast<const T *>(p) + at;
    const int64_t room = n - at;
    const int c = int(threadIdx.x) * V;
    typename Elem<T>::Vec v[4];
    if (room >= 4 * STEP) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fetch_raw<T, false>(x, c + i * STEP, 4 * STEP);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_raw(x, c + i * STEP, room);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) add_squares<T>(sum, v[i]);
}

// F: the factor's type.  The product is rounded to fp32 and then to T.
template <class T, class F>
__device__ __forceinline__ void piece_scale(F by, const void *p, void *q, int64_t at, int64_t n) {
    constexpr int V = Elem<T>::V, STEP = kThreads * V;
    const T *x = static_cast<const T *>(p) + at;
    T *y = static_cast<T *>(q) + at;
    const int64_t room = n - at;
    const int c = int(threadIdx.x) * V;
    typename Elem<T>::Vec v[4];
    if (room >= 4 * STEP) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fetch_raw<T, false>(x, c + i * STEP, 4 * STEP);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[V];
            to_float<T>(v[i], f);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = float(F(f[j]) * by);
            store_stream<T, false>(y, c + i * STEP, 4 * STEP, f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_raw(x, c + i * STEP, room);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[V];
            to_float<T>(v[i], f);
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = float(F(f[j]) * by);
            store_stream<T, true>(y, c + i * STEP, room, f);
        }
    }
}

// Sum over the workgroup; every thread gets it.
template <int T>
__device__ __forceinline__ double group_sum(double v, double *red) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += red[i];
    return v;
}

__global__ void __launch_bounds__(kThreads)
norm_squares_kernel(NormTable t, double *__restrict__ part) {
    __shared__ double red[kThreads / 64];
    const uint32_t pieces = t.first[t.n];
    double sum = 0.0;
    int at = tensor_of(t, blockIdx.x);
    for (uint32_t p = blockIdx.x; p < pieces; p += gridDim.x) {
        while (t.first[at + 1] <= p) ++at;
        const int64_t n = t.size[at] & ((int64_t(1) << 56) - 1);
        const int type = int(t.size[at] >> 56);
        const int64_t q = p - t.first[at];
        if (type == DT_F16) piece_squares<_Float16>(sum, t.grad[at], q * (kPiece / 2), n);
        else if (type == DT_BF16) piece_squares<__bf16>(sum, t.grad[at], q * (kPiece / 2), n);
        else piece_squares<float>(sum, t.grad[at], q * (kPiece / 4), n);
    }
    sum = group_sum<kThreads>(sum, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <int T>
__device__ __forceinline__ double sum_of(const double *part, int slots, double *red) {
    double sum = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < slots; i += T) sum += part[i];
    return group_sum<T>(sum, red);
}

// norm and total: either may be null.
__global__ void __launch_bounds__(1024)
norm_finish_kernel(const double *__restrict__ part, int slots, float *__restrict__ norm, double *__restrict__ total) {
    __shared__ double red[16];
    const double sum = sum_of<1024>(part, slots, red);
    if (threadIdx.x != 0) return;
    if (norm) norm[0] = float(sqrt(sum));
    if (total) total[0] = sum;
}

// Every workgroup adds the partial sums for itself: up to one a thread (kOwnSlots), or the one total that
// norm_finish_kernel left.  Of one a thread the sum is the same to the last bit in both kernels, so grad_norm
// and clipping tell one norm; and a launch that adds them once costs less than more of them in every workgroup
// of every launch, which is quadratic in the tensors (12000 of 100 KB, in a graph, 1.55 ms so and 3.86; 950 of them
// 119 us and 127; 290 of 800 KB 136 and 137).
constexpr int kOwnSlots = kThreads;

// Pieces from the last to the first.
template <class F>
__device__ __forceinline__ void scale_all(const ClipTable &t, F by) {
    const uint32_t pieces = t.first[t.n];
    int at = tensor_of(t, pieces - 1 - blockIdx.x);
    for (uint32_t back = blockIdx.x; back < pieces; back += gridDim.x) {
        const uint32_t p = pieces - 1 - back;
        while (t.first[at] > p) --at;
        if (by == F(1) && t.grad[at] == t.out[at]) continue;
        const int64_t size = t.size[at] & ((int64_t(1) << 56) - 1);
        const int type = int(t.size[at] >> 56);
        const int64_t q = p - t.first[at];
        if (type == DT_F16) piece_scale<_Float16>(by, t.grad[at], t.out[at], q * (kPiece / 2), size);
        else if (type == DT_BF16) piece_scale<__bf16>(by, t.grad[at], t.out[at], q * (kPiece / 2), size);
        else piece_scale<float>(by, t.grad[at], t.out[at], q * (kPiece / 4), size);
    }
}

// The factor is rounded to fp32 once, but below the normal fp32 values (norms near and past fp32's largest),
// where that would cost its digits, stays fp64.
__global__ void __launch_bounds__(kThreads)
clip_kernel(ClipTable t, double max_norm, const float *__restrict__ norm_in, const double *__restrict__ part, int slots,
            float *__restrict__ norm) {
    __shared__ double red[kThreads / 64];
    const double n = norm_in ? double(norm_in[0]) : sqrt(sum_of<kThreads>(part, slots, red));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = float(n);
    // (an infinite norm: 0, whatever max_norm is; a NaN stays one)
    const double c = n == double(INFINITY) ? 0.0 : max_norm / (n + kEps);
    if (c > 0.0 && c < double(FLT_MIN)) scale_all(t, c);
    else scale_all(t, c > 1.0 ? 1.0f : float(c));
}

int64_t pieces_of(const GradList &l, int i) {
    return (l.sizes[i] * (l.dtypes[i] == DT_F32 ? 4 : 2) + kPiece - 1) / kPiece;
}

// The end of the entries from i on that go into one table (those before i, backwards: their start).
template <int Most>
int table_end(const GradList &l, int i, bool back) {
    for (int n = 0; back ? i > 0 : i < l.n; i += back ? -1 : 1) {
        if (l.sizes[back ? i - 1 : i] == 0) continue;
        if (n == Most) break;
        ++n;
    }
    return i;
}

// Fills a table with the entries [i, end) that are not empty.
template <class Table, class F>
void fill(const GradList &l, int i, int end, Table &t, F more) {
    t.n = 0;
    uint32_t pieces = 0;
    for (; i < end; ++i) {
        if (l.sizes[i] == 0) continue;
        t.grad[t.n] = l.grads[i];
        t.size[t.n] = l.sizes[i] | int64_t(l.dtypes[i]) << 56;
        t.first[t.n] = pieces;
        more(t, i);
        pieces += uint32_t(pieces_of(l, i));
        ++t.n;
    }
    t.first[t.n] = pieces;
}

hipError_t squares(const GradList &l, double *ws, int &slots, hipStream_t st) {
    slots = 0;
    for (int i = 0; i < l.n;) {
        NormTable t;
        const int end = table_end<kNormTensors>(l, i, false);
        fill(l, i, end, t, [](NormTable &, int) {});
        i = end;
        if (t.n == 0) continue;
        const uint32_t pieces = t.first[t.n];
        const int grid = pieces < uint32_t(kGrid) ? int(pieces) : kGrid;
        hipLaunchKernelGGL(norm_squares_kernel, dim3(grid), dim3(kThreads), 0, st, t, ws + slots);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        slots += grid;
    }
    return hipSuccess;
}

hipError_t finish(const double *ws, int slots, float *norm, double *total, hipStream_t st) {
    hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(1024), 0, st, ws, slots, norm, total);
    return hipGetLastError();
}

}  // namespace

// Partial sums (every launch but the last takes kNormTensors tensors that are not empty), and their total.
int64_t grad_norm_slots(int n) { return (int64_t(n) + kNormTensors - 1) / kNormTensors * kGrid + 1; }

hipError_t launch_grad_norm(const GradList &l, double *ws, float *norm, hipStream_t st) {
    int slots;
    const hipError_t e = squares(l, ws, slots, st);
    return e != hipSuccess ? e : finish(ws, slots, norm, nullptr, st);
}

hipError_t launch_clip_grad_norm(const GradList &l, double max_norm, const float *norm_in, double *ws, float *norm,
                                 hipStream_t st) {
    int slots = 0;
    hipError_t e = norm_in ? hipSuccess : squares(l, ws, slots, st);
    if (e != hipSuccess) return e;
    const double *part = ws;
    if (slots > kOwnSlots) {
        if ((e = finish(ws, slots, nullptr, ws + slots, st)) != hipSuccess) return e;
        part = ws + slots, slots = 1;
    }
    bool told = norm_in != nullptr;  // the first scaling launch writes the norm
    for (int end = l.n; end > 0;) {
        ClipTable t;
        const int i = table_end<kClipTensors>(l, end, true);
        fill(l, i, end, t, [&](ClipTable &u, int at) { u.out[u.n] = l.outs[at]; });
        end = i;
        if (t.n == 0) continue;
        const uint32_t pieces = t.first[t.n];
        const int grid = pieces < uint32_t(2 * kGrid) ? int(pieces) : 2 * kGrid;
        hipLaunchKernelGGL(clip_kernel, dim3(grid), dim3(kThreads), 0, st, t, max_norm, norm_in, part, slots,
                           told ? nullptr : norm);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        told = true;
    }
    return told ? hipSuccess : finish(part, slots, norm, nullptr, st);
}

}  // namespace ssg

// Layer norm over the last axis, forward and backward, for gfx950.
//
//   forward   s = x (+ residual, rounded to the rows' type: the value that is
//             kept and that the backward pass reads)
//             mean = sum(s) / N,  rstd = 1 / sqrt(sum((s - mean)^2) / N + eps)
//             y = (s - mean) * rstd * w + b
//   backward  xh = (x - mean) * rstd,  g = dy * w
//             dx = rstd * (g - sum(g)/N - xh * sum(g * xh)/N)  (+ dres)
//             dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// Bound by memory: forward reads and writes every row once, backward reads dy
// and x (and dres) once and writes dx once.  A row therefore stays in registers
// as fp32 between the statistics and the output, held by TPR threads with C
// 16-byte chunks each; only rows past 16384 16-bit or 8192 fp32 elements (backward
// 8192 and 4096) are read again.  The variance is the sum of squared distances from the finished
// mean, so an offset that is large against the spread costs no digits.
// Workgroups are persistent over rows: w and b are loaded once, the next turn's
// rows are fetched while this turn's are reduced, and outputs are streaming
// stores (without the last two, forward ran 18.7 instead of 16.8 us at
// 12608 x 768 fp16 with a residual).  At most 768 of them, three a CU: by graph
// with 256 / 512 / 768 / 1536 / 4096, 12608 x 768 24.4 / 20.2 / 20.7 / 20.4 / 21.9
// us, without residual 23.2 / 17.7 / 16.1 / 16.1 / 17.5, 3000 x 8192 41.9 / 40.6 /
// 41.0 / 42.8 / 47.2, 1500 x 3001 fp32 20.0 / 16.6 / 15.2 / 18.1 / 18.2, 2865 x 4183
// bf16 43 / 31 / 36 / 36 / 45.  The backward pass keeps its column sums
// for dw and db in registers, adds those of a workgroup's rows through LDS and
// writes one slice a workgroup; a second launch sums the slices in order.  No
// atomics: results repeat bit for bit.  Its registers (w, dw, db, x, dy and the
// fetched row) set the split: one chunk a thread and 1024 threads keep 16 waves
// a CU and one slice a CU, where two to four chunks a thread ran at 1-3 waves a
// SIMD (12608 x 768 fp16: 21.4 us, 25.3 with two chunks and 768 slices;
// 4099 x 1537 bf16: 19.1 us, 37 with four chunks).
// Measured on MI355X in rotating buffers (233 MB): forward 12608 x 768 fp16 with
// residual 15.7-16.4 us = 4.7-4.9 TB/s, 4096 x 4096 23.9 us = 5.6 TB/s (a 1 GiB copy
// reaches 5.1); backward 21.4-22.3 us = 3.5 TB/s and 31.6 us = 4.2 TB/s, both
// launches.  Rows that end in part of a 16-byte piece have kernels of their own
// (TAIL): 3000 x 8191 fp16 forward 49.8 us = 4.0 TB/s, backward 62 us = 3.2 TB/s (8192
// wide 36.2 and 50.7), 2865 x 4183 bf16 31.5 us = 3.0 TB/s and 32.6 us, 4099 x
// 1537 bf16 without residual 12.4 us = 2.0 TB/s and 19.5 us.  Pieces cut at 16-byte boundaries
// instead of the row's start were slower (60 us at 2865 x 4183: two part pieces a row), and a
// row's sums would then depend on its place in the batch.  fp32: forward 1500 x 3001 with
// residual 15.0 us = 4.9 TB/s, backward 2000 x 4096 19.7 us = 5.4 TB/s and 3.9.  Rows past the
// register forms: forward 2000 x 20000 fp16 61 us (three reads of a row), backward 2000 x 12001
// fp16 52 + 32 + 5 us and 2000 x 8192 fp32 55 + 22 + 5 (dx, the column sums' slices, their sum).
#include "elem.h"
#include "launch.h"

namespace ssg {

namespace {

// Rows held in registers: TPR threads a row, C chunks of V elements a thread.
// TAIL: rows end in part of a chunk.
template <class T, class W, int TPR, int C, bool TAIL>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
ln_fwd_kernel(const T *x, int64_t ldx, const T *res, int64_t ldr, const W *__restrict__ w,
              const W *__restrict__ b, float eps, T *y, int64_t ldy, T *sum, int64_t lds, float *mean_out,
              float *rstd_out, int64_t M, int N) {
    constexpr int V = Elem<T>::V, NT = TPR < 256 ? 256 : TPR, RPB = NT / TPR;
    __shared__ float red[NT / 64];
    const int t = threadIdx.x % TPR;
    // The rows of the next turn are fetched while this turn's are reduced; the
    // first turn's, before the parameters are waited for.
    typename Elem<T>::Vec xr[C], rr[C];
    auto fetch = [&](int64_t m) {
        if (m >= M) return;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
            if (at < N) xr[c] = fetch_raw<T, TAIL>(x + m * ldx, at, N);
            if (res && at < N) rr[c] = fetch_raw<T, TAIL>(res + m * ldr, at, N);
        }
    };
    const int64_t step = int64_t(gridDim.x) * RPB;
    int64_t m = int64_t(blockIdx.x) * RPB + threadIdx.x / TPR;
#pragma unroll
    for (int c = 0; c < C; ++c) xr[c] = rr[c] = typename Elem<T>::Vec{};
    fetch(m);
    float wv[C][V], bv[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) wv[c][i] = 1.0f, bv[c][i] = 0.0f;
        if (w && at < N) load_param<V>(w, at, N, wv[c]);
        if (b && at < N) load_param<V>(b, at, N, bv[c]);
    }
    const float inv_n = 1.0f / float(N);
    for (; m < M; m += step) {
        float f[C][V];
        float acc = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
            to_float<T>(settle<T, TAIL>(xr[c], at, N), f[c]);
            if (res) {
                float g[V];
                to_float<T>(settle<T, TAIL>(rr[c], at, N), g);
#pragma unroll
                for (int i = 0; i < V; ++i) f[c][i] = rounded_sum<T>(f[c][i], g[i]);
                if (at < N) store_stream<T, TAIL>(sum + m * lds, at, N, f[c]);
            }
        }
        fetch(m + step);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) acc += f[c][i];
        const float mean = row_sum<TPR>(acc, red) * inv_n;
        acc = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                f[c][i] = at + i < N ? f[c][i] - mean : 0.0f;
                acc = fmaf(f[c][i], f[c][i], acc);
            }
        }
        const float var = row_sum<TPR>(acc, red) * inv_n;
        const float rstd = 1.0f / sqrtf(var + eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
            if (at >= N) continue;
#pragma unroll
            for (int i = 0; i < V; ++i) f[c][i] = fmaf(f[c][i] * rstd, wv[c][i], bv[c][i]);
            store_stream<T, TAIL>(y + m * ldy, at, N, f[c]);
        }
        if (mean_out && t == 0) mean_out[m] = mean, rstd_out[m] = rstd;
    }
}

// Rows longer than the register form holds: one workgroup a row, three sweeps.
template <class T, class W>
__global__ void __launch_bounds__(256)
ln_fwd_long_kernel(const T *x, int64_t ldx, const T *res, int64_t ldr, const W *__restrict__ w,
                   const W *__restrict__ b, float eps, T *y, int64_t ldy, T *sum, int64_t lds, float *mean_out,
                   float *rstd_out, int64_t M, int64_t N) {
    constexpr int V = Elem<T>::V;
    __shared__ float red[4];
    const float inv_n = 1.0f / float(N);
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        auto at_row = [&](int64_t c, float (&f)[V]) {
            load_vec(x + m * ldx, c, N, f);
            if (res) {
                float g[V];
                load_vec(res + m * ldr, c, N, g);
#pragma unroll
                for (int i = 0; i < V; ++i) f[i] = rounded_sum<T>(f[i], g[i]);
            }
        };
        float acc = 0.0f;
        for (int64_t c = int64_t(threadIdx.x) * V; c < N; c += 256 * V) {
            float f[V];
            at_row(c, f);
#pragma unroll
            for (int i = 0; i < V; ++i) acc += f[i];
        }
        const float mean = row_sum<256>(acc, red) * inv_n;
        acc = 0.0f;
        for (int64_t c = int64_t(threadIdx.x) * V; c < N; c += 256 * V) {
            float f[V];
            at_row(c, f);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = c + i < N ? f[i] - mean : 0.0f;
                acc = fmaf(d, d, acc);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<256>(acc, red) * inv_n + eps);
        // (each element is read by the thread that then writes it, so y or sum may be x or residual)
        for (int64_t c = int64_t(threadIdx.x) * V; c < N; c += 256 * V) {
            float f[V], wv[V], bv[V];
            at_row(c, f);
#pragma unroll
            for (int i = 0; i < V; ++i) wv[i] = 1.0f, bv[i] = 0.0f;
            if (w) load_param<V>(w, c, N, wv);
            if (b) load_param<V>(b, c, N, bv);
            if (res) store_vec(sum + m * lds, c, N, f);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = fmaf((f[i] - mean) * rstd, wv[i], bv[i]);
            store_vec(y + m * ldy, c, N, f);
        }
        if (mean_out && threadIdx.x == 0) mean_out[m] = mean, rstd_out[m] = rstd;
    }
}

// PARAM: also sum dw and db over this workgroup's rows into part[block][2][N].
// NT threads a workgroup, NT / TPR rows at a time.
template <class T, class W, int TPR, int C, int NT, bool PARAM, bool TAIL>
__global__ void __launch_bounds__(NT)
ln_bwd_kernel(const T *dy, int64_t lddy, const T *x, int64_t ldx, const float *__restrict__ mean,
              const float *__restrict__ rstd, const W *__restrict__ w, const T *dres, int64_t ldres, T *dx,
              int64_t lddx, float *__restrict__ part, int64_t M, int N) {
    constexpr int V = Elem<T>::V, RPB = NT / TPR, WPR = TPR / 64;
    __shared__ float red[2][RPB][WPR][2];
    __shared__ float cols[PARAM && RPB > 1 ? RPB * 2 * C * TPR * V : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    typename Elem<T>::Vec xr[C], gr[C], rr[C];
    float mu = 0.0f, rs = 0.0f;
    auto fetch = [&](int64_t m) {
        if (m >= M) return;
        mu = mean[m], rs = rstd[m];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
            if (at < N) xr[c] = fetch_raw<T, TAIL>(x + m * ldx, at, N), gr[c] = fetch_raw<T, TAIL>(dy + m * lddy, at, N);
            if (dres && at < N) rr[c] = fetch_raw<T, TAIL>(dres + m * ldres, at, N);
        }
    };
    const int64_t step = int64_t(gridDim.x) * RPB;
#pragma unroll
    for (int c = 0; c < C; ++c) xr[c] = gr[c] = rr[c] = typename Elem<T>::Vec{};
    fetch(int64_t(blockIdx.x) * RPB + sub);
    float wv[C][V], dw[C][V], db[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = (c * TPR + t) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) wv[c][i] = 1.0f, dw[c][i] = 0.0f, db[c][i] = 0.0f;
        if (w && at < N) load_param<V>(w, at, N, wv[c]);
    }
    const float inv_n = 1.0f / float(N);
    int turn = 0;
    // (the turns of a workgroup are the same for all its threads: past the last
    // row they only meet the barriers)
    for (int64_t base = int64_t(blockIdx.x) * RPB; base < M; base += step, turn ^= 1) {
        const int64_t m = base + sub;
        const bool live = m < M;
        float xh[C][V], g[C][V];
        typename Elem<T>::Vec rc[C];
        float a1 = 0.0f, a2 = 0.0f;
        const float rs_m = rs;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
            to_float<T>(settle<T, TAIL>(xr[c], at, N), xh[c]);
            to_float<T>(settle<T, TAIL>(gr[c], at, N), g[c]);
            rc[c] = rr[c];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[c][i] = live && at + i < N ? (xh[c][i] - mu) * rs : 0.0f;
                g[c][i] = live ? g[c][i] : 0.0f;
            }
        }
        fetch(m + step);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if constexpr (PARAM) {
                    dw[c][i] = fmaf(g[c][i], xh[c][i], dw[c][i]);
                    db[c][i] += g[c][i];
                }
                g[c][i] *= wv[c][i];
                a1 += g[c][i];
                a2 = fmaf(g[c][i], xh[c][i], a2);
            }
        a1 = wave_sum(a1);
        a2 = wave_sum(a2);
        if constexpr (WPR > 1) {
            // one exchange a row; the buffers alternate, so that the next row's
            // sums meet only readers that have passed its barrier
            if ((threadIdx.x & 63) == 0) red[turn][sub][t >> 6][0] = a1, red[turn][sub][t >> 6][1] = a2;
            __syncthreads();
            a1 = a2 = 0.0f;
#pragma unroll
            for (int i = 0; i < WPR; ++i) a1 += red[turn][sub][i][0], a2 += red[turn][sub][i][1];
        }
        const float c1 = a1 * inv_n, c2 = a2 * inv_n;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = (c * TPR + t) * V;
            if (at >= N || !live) continue;
            float r[V];
            to_float<T>(settle<T, TAIL>(rc[c], at, N), r);
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = fmaf(rs_m, fmaf(-xh[c][i], c2, g[c][i] - c1), r[i]);
            store_stream<T, TAIL>(dx + m * lddx, at, N, r);
        }
    }
    if constexpr (PARAM) {
        float *pw = part + int64_t(blockIdx.x) * 2 * N, *pb = pw + N;
        if constexpr (RPB > 1) {
            // the rows' partial sums of the workgroup, added in order
            constexpr int NC = C * TPR * V;
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    cols[(sub * 2 + 0) * NC + (c * V + i) * TPR + t] = dw[c][i];
                    cols[(sub * 2 + 1) * NC + (c * V + i) * TPR + t] = db[c][i];
                }
            __syncthreads();
            for (int j = threadIdx.x; j < N; j += NT) {
                const int chunk = j / V, i = j % V;
                const float *s = cols + ((chunk / TPR) * V + i) * TPR + chunk % TPR;
                float sw = 0.0f, sb = 0.0f;
                for (int q = 0; q < RPB; ++q) sw += s[(q * 2) * NC], sb += s[(q * 2 + 1) * NC];
                pw[j] = sw;
                pb[j] = sb;
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int at = (c * TPR + t) * V;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (at + i < N) pw[at + i] = dw[c][i], pb[at + i] = db[c][i];
            }
        }
    }
}

// Long rows: dx with one workgroup a row, two sweeps.
template <class T, class W>
__global__ void __launch_bounds__(256)
ln_bwd_long_kernel(const T *dy, int64_t lddy, const T *x, int64_t ldx, const float *__restrict__ mean,
                   const float *__restrict__ rstd, const W *__restrict__ w, const T *dres, int64_t ldres, T *dx,
                   int64_t lddx, int64_t M, int64_t N) {
    constexpr int V = Elem<T>::V;
    __shared__ float red[8];
    const float inv_n = 1.0f / float(N);
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        const float mu = mean[m], rs = rstd[m];
        auto at_row = [&](int64_t c, float (&xh)[V], float (&g)[V]) {
            float wv[V];
            load_vec(x + m * ldx, c, N, xh);
            load_vec(dy + m * lddy, c, N, g);
#pragma unroll
            for (int i = 0; i < V; ++i) wv[i] = 1.0f;
            if (w) load_param<V>(w, c, N, wv);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[i] = c + i < N ? (xh[i] - mu) * rs : 0.0f;
                g[i] = c + i < N ? g[i] * wv[i] : 0.0f;
            }
        };
        float a1 = 0.0f, a2 = 0.0f;
        for (int64_t c = int64_t(threadIdx.x) * V; c < N; c += 256 * V) {
            float xh[V], g[V];
            at_row(c, xh, g);
#pragma unroll
            for (int i = 0; i < V; ++i) a1 += g[i], a2 = fmaf(g[i], xh[i], a2);
        }
        const float c1 = row_sum<256>(a1, red) * inv_n;
        const float c2 = row_sum<256>(a2, red + 4) * inv_n;
        for (int64_t c = int64_t(threadIdx.x) * V; c < N; c += 256 * V) {
            float xh[V], g[V], r[V];
            at_row(c, xh, g);
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = 0.0f;
            if (dres) load_vec(dres + m * ldres, c, N, r);
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = fmaf(rs, fmaf(-xh[i], c2, g[i] - c1), r[i]);
            store_vec(dx + m * lddx, c, N, r);
        }
    }
}

// Long rows: column sums of a slice of rows, 256 columns x V a workgroup.
template <class T>
__global__ void __launch_bounds__(256)
ln_cols_kernel(const T *dy, int64_t lddy, const T *x, int64_t ldx, const float *__restrict__ mean,
               const float *__restrict__ rstd, float *__restrict__ part, int64_t M, int64_t N, int64_t rows) {
    constexpr int V = Elem<T>::V;
    const int64_t c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * V;
    if (c >= N) return;
    const int64_t first = int64_t(blockIdx.y) * rows, last = first + rows < M ? first + rows : M;
    float dw[V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dw[i] = 0.0f, db[i] = 0.0f;
    for (int64_t m = first; m < last; ++m) {
        float xv[V], g[V];
        load_vec(x + m * ldx, c, N, xv);
        load_vec(dy + m * lddy, c, N, g);
        const float mu = mean[m], rs = rstd[m];
#pragma unroll
        for (int i = 0; i < V; ++i) dw[i] = fmaf(g[i], (xv[i] - mu) * rs, dw[i]), db[i] += g[i];
    }
    float *pw = part + int64_t(blockIdx.y) * 2 * N, *pb = pw + N;
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (c + i < N) pw[c + i] = dw[i], pb[c + i] = db[i];
}

// Sums the workgroups' slices part[G][2N] in order: 32 columns a workgroup (a
// workgroup in turns: a launch ends before 2^32 threads), 32 threads a column, each
// over every 32nd slice, then their sums in order.
constexpr int kParamBlocks = 1 << 20;
__global__ void __launch_bounds__(1024)
ln_param_kernel(const float *__restrict__ part, int G, int64_t N, float *__restrict__ dw, float *__restrict__ db) {
    __shared__ float s[32][33];
    const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
    for (int64_t j0 = int64_t(blockIdx.x) * 32; j0 < 2 * N; j0 += int64_t(gridDim.x) * 32) {
        const int64_t j = j0 + col;
        float a = 0.0f;
        if (j < 2 * N)
            for (int g = lane; g < G; g += 32) a += part[int64_t(g) * 2 * N + j];
        s[lane][col] = a;
        __syncthreads();
        if (lane == 0 && j < 2 * N) {
            a = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) a += s[i][col];
            (j < N ? dw[j] : db[j - N]) = a;
        }
        __syncthreads();
    }
}

// Threads a row and chunks a thread of the register forms; tpr = 0: long rows.
struct LnShape {
    int tpr, c;
};
LnShape ln_fwd_shape(int64_t N, int v) {
    const int64_t chunks = (N + v - 1) / v;
    if (chunks <= 64) return {64, 1};
    if (chunks <= 128) return {64, 2};
    if (chunks <= 256) return {256, 1};
    if (chunks <= 512) return {256, 2};
    if (chunks <= 1024) return {256, 4};
    if (chunks <= 2048) return {1024, 2};
    return {0, 0};
}
LnShape ln_bwd_shape(int64_t N, int v) {
    const int64_t chunks = (N + v - 1) / v;
    if (chunks <= 64) return {64, 1};
    if (chunks <= 128) return {128, 1};
    if (chunks <= 256) return {256, 1};
    if (chunks <= 512) return {512, 1};
    if (chunks <= 1024) return {1024, 1};
    return {0, 0};
}

// Workgroups of a persistent grid over `groups` turns, at most `most`, the
// turns dealt evenly.
int even_blocks(int64_t groups, int most) {
    const int64_t turns = (groups + most - 1) / most;
    return int((groups + turns - 1) / turns);
}

constexpr int kBwdThreads = 1024, kBwdBlocks = 256;

int ln_bwd_blocks(int64_t M, int64_t N, int v) {
    const LnShape sh = ln_bwd_shape(N, v);
    if (M == 0) return 0;
    if (sh.tpr == 0) return int(M < 64 ? M : 64);
    const int nt = sh.tpr > kBwdThreads ? sh.tpr : kBwdThreads, rpb = nt / sh.tpr;
    return even_blocks((M + rpb - 1) / rpb, kBwdBlocks);
}

template <class T, class W>
hipError_t fwd(const LnFwd &a, hipStream_t st) {
    const LnShape sh = ln_fwd_shape(a.N, Elem<T>::V);
    const bool tail = a.N % Elem<T>::V != 0;
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    const W *w = static_cast<const W *>(a.w), *b = static_cast<const W *>(a.b);
    T *y = static_cast<T *>(a.y), *sum = static_cast<T *>(a.sum);
#define SSG_LN(TPR, C, TAIL)                                                                                       \
    if (sh.tpr == TPR && sh.c == C && tail == TAIL) {                                                              \
        constexpr int RPB = TPR < 256 ? 256 / TPR : 1;                                                             \
        hipLaunchKernelGGL((ln_fwd_kernel<T, W, TPR, C, TAIL>), dim3(even_blocks((a.M + RPB - 1) / RPB, 768)),           \
                           dim3(TPR < 256 ? 256 : TPR), 0, st, x, a.ldx, res, a.ldr, w, b, a.eps, y, a.ldy, sum,   \
                           a.lds, a.mean, a.rstd, a.M, int(a.N));                                                  \
        return hipGetLastError();                                                                                  \
    }
    SSG_LN(64, 1, false) SSG_LN(64, 2, false) SSG_LN(256, 1, false) SSG_LN(256, 2, false) SSG_LN(256, 4, false)
    SSG_LN(1024, 2, false)
    SSG_LN(64, 1, true) SSG_LN(64, 2, true) SSG_LN(256, 1, true) SSG_LN(256, 2, true) SSG_LN(256, 4, true)
    SSG_LN(1024, 2, true)
#undef SSG_LN
    hipLaunchKernelGGL((ln_fwd_long_kernel<T, W>), dim3(int(a.M < 2048 ? a.M : 2048)), dim3(256), 0, st, x, a.ldx, res,
                       a.ldr, w, b, a.eps, y, a.ldy, sum, a.lds, a.mean, a.rstd, a.M, a.N);
    return hipGetLastError();
}

template <class T, class W, bool PARAM>
hipError_t bwd(const LnBwd &a, hipStream_t st) {
    const LnShape sh = ln_bwd_shape(a.N, Elem<T>::V);
    const bool tail = a.N % Elem<T>::V != 0;
    const T *dy = static_cast<const T *>(a.dy), *x = static_cast<const T *>(a.x);
    const T *dres = static_cast<const T *>(a.dres);
    const W *w = static_cast<const W *>(a.w);
    T *dx = static_cast<T *>(a.dx);
    const int G = ln_bwd_blocks(a.M, a.N, Elem<T>::V);
    hipError_t e = hipSuccess;
    bool done = G == 0;
#define SSG_LN(TPR, C, TAIL)                                                                                         \
    if (!done && sh.tpr == TPR && sh.c == C && tail == TAIL) {                                                       \
        constexpr int NT = TPR > kBwdThreads ? TPR : kBwdThreads;                                                    \
        hipLaunchKernelGGL((ln_bwd_kernel<T, W, TPR, C, NT, PARAM, TAIL>), dim3(G), dim3(NT), 0, st, dy, a.lddy, x, a.ldx,     \
                           a.mean, a.rstd, w, dres, a.ldres, dx, a.lddx, a.part, a.M, int(a.N));                     \
        e = hipGetLastError();                                                                                       \
        done = true;                                                                                                 \
    }
    SSG_LN(64, 1, false) SSG_LN(128, 1, false) SSG_LN(256, 1, false) SSG_LN(512, 1, false) SSG_LN(1024, 1, false)
    SSG_LN(64, 1, true) SSG_LN(128, 1, true) SSG_LN(256, 1, true) SSG_LN(512, 1, true) SSG_LN(1024, 1, true)
#undef SSG_LN
    int slices = G;
    if (!done) {
        hipLaunchKernelGGL((ln_bwd_long_kernel<T, W>), dim3(int(a.M < 2048 ? a.M : 2048)), dim3(256), 0, st, dy, a.lddy,
                           x, a.ldx, a.mean, a.rstd, w, dres, a.ldres, dx, a.lddx, a.M, a.N);
        e = hipGetLastError();
        if constexpr (PARAM) {
            if (e != hipSuccess) return e;
            const int64_t rows = (a.M + G - 1) / G;
            slices = int((a.M + rows - 1) / rows);
            const int64_t cols = 256 * Elem<T>::V;
            hipLaunchKernelGGL((ln_cols_kernel<T>), dim3(int((a.N + cols - 1) / cols), slices), dim3(256), 0, st, dy,
                               a.lddy, x, a.ldx, a.mean, a.rstd, a.part, a.M, a.N, rows);
            e = hipGetLastError();
        }
    }
    if constexpr (PARAM) {
        if (e != hipSuccess) return e;
        const int64_t groups = (2 * a.N + 31) / 32;
        hipLaunchKernelGGL(ln_param_kernel, dim3(int(groups < kParamBlocks ? groups : kParamBlocks)), dim3(1024), 0, st,
                           a.part, slices, a.N, a.dw, a.db);
        e = hipGetLastError();
    }
    return e;
}

template <class T>
hipError_t fwd_t(const LnFwd &a, hipStream_t st) {
    if (a.wtype == DT_F32) return fwd<T, float>(a, st);
    return fwd<T, T>(a, st);
}
template <class T, class W>
hipError_t bwd_p(const LnBwd &a, hipStream_t st) {
    return a.dw ? bwd<T, W, true>(a, st) : bwd<T, W, false>(a, st);
}
template <class T>
hipError_t bwd_t(const LnBwd &a, hipStream_t st) {
    if (a.wtype == DT_F32) return bwd_p<T, float>(a, st);
    return bwd_p<T, T>(a, st);
}

}  // namespace

int64_t layer_norm_slices(int dtype, int64_t M, int64_t N) { return ln_bwd_blocks(M, N, dtype == DT_F32 ? 4 : 8); }

hipError_t launch_layer_norm_fwd(const LnFwd &a, hipStream_t st) {
    switch (a.dtype) {
        case DT_F16: return fwd_t<_Float16>(a, st);
        case DT_BF16: return fwd_t<__bf16>(a, st);
        default: return fwd<float, float>(a, st);
    }
}

hipError_t launch_layer_norm_bwd(const LnBwd &a, hipStream_t st) {
    switch (a.dtype) {
        case DT_F16: return bwd_t<_Float16>(a, st);
        case DT_BF16: return bwd_t<__bf16>(a, st);
        default: return bwd_p<float, float>(a, st);
    }
}

}  // namespace ssg

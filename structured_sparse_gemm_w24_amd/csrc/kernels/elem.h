// Element types of the kernels that take fp16, bf16 or fp32 rows: 16-byte
// vector access at any element alignment, conversion to fp32 and back (one
// rounding to nearest even), and wave / workgroup sums in a fixed order.
#pragma once

#include "common.h"

namespace ssg {

// V elements of T make one 16-byte access.
template <class T>
struct Elem {
    static constexpr int V = 16 / int(sizeof(T));
    typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T))));
};

// Loads elements [c, c + V) of a row of n elements, zeros past the row's end.
// Rows of an odd width start at any element, so the access is not assumed to
// be 16-byte aligned (gfx950 takes unaligned global vectors).  A row's last
// piece is read as the V elements that end with the row, and moved into place by
// settle(), which a caller that fetches ahead does when it uses them: read one by
// one, 16-bit elements wait for each other, two to a register, and that latency
// was most of an odd row's time (layer norm 2865 x 4183 bf16 51.8 us, so 31.8).
// TAIL false: rows are whole pieces (settling that has nothing to do cost the
// gradient of 12608 x 768 fp16 3 of 22 us).
template <class T, bool TAIL = true>
__device__ __forceinline__ typename Elem<T>::Vec fetch_raw(const T *row, int64_t c, int64_t n) {
    constexpr int V = Elem<T>::V;
    typename Elem<T>::Vec v = {};
    if constexpr (!TAIL) {
        if (c < n) __builtin_memcpy(&v, row + c, 16);
    } else if (n >= V) {
        if (c < n) __builtin_memcpy(&v, row + (c + V <= n ? c : n - V), 16);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < n) v[i] = row[c + i];
    }
    return v;
}
template <class T, bool TAIL = true>
__device__ __forceinline__ typename Elem<T>::Vec settle(typename Elem<T>::Vec v, int64_t c, int64_t n) {
    constexpr int V = Elem<T>::V;
    if (!TAIL || c + V <= n || c >= n || n < V) return v;
    const int k = int(c + V - n);  // elements to drop, 1 .. V - 1
    u32x4 d = __builtin_bit_cast(u32x4, v);
    if constexpr (V == 8) {
        if (k & 4) d = u32x4{d.z, d.w, 0u, 0u};
        if (k & 2) d = u32x4{d.y, d.z, d.w, 0u};
        if (k & 1) d = u32x4{d.x >> 16 | d.y << 16, d.y >> 16 | d.z << 16, d.z >> 16 | d.w << 16, d.w >> 16};
    } else {
        if (k & 2) d = u32x4{d.z, d.w, 0u, 0u};
        if (k & 1) d = u32x4{d.y, d.z, d.w, 0u};
    }
    return __builtin_bit_cast(typename Elem<T>::Vec, d);
}
template <class T>
__device__ __forceinline__ typename Elem<T>::Vec load_raw(const T *row, int64_t c, int64_t n) {
    return settle<T>(fetch_raw(row, c, n), c, n);
}

template <class T>
__device__ __forceinline__ void to_float(typename Elem<T>::Vec v, float (&f)[Elem<T>::V]) {
#pragma unroll
    for (int i = 0; i < Elem<T>::V; ++i) f[i] = float(v[i]);
}

template <class T>
__device__ __forceinline__ void load_vec(const T *row, int64_t c, int64_t n, float (&f)[Elem<T>::V]) {
    to_float<T>(load_raw(row, c, n), f);
}

// Stores elements [c, c + V) of a row, rounded to T; NTS: past the L2.
template <class T, bool NTS = false, bool TAIL = true>
__device__ __forceinline__ void store_vec(T *row, int64_t c, int64_t n, const float (&f)[Elem<T>::V]) {
    constexpr int V = Elem<T>::V;
    if (!TAIL || c + V <= n) {
        typename Elem<T>::Vec v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = T(f[i]);
        if constexpr (NTS) {
            typedef u32x4 Any __attribute__((aligned(2)));
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<Any *>(row + c));
        } else {
            __builtin_memcpy(row + c, &v, 16);
        }
    } else if (c < n) {
        // a row's last piece: 8, 4 and 2 bytes as its length has them (fp32: 8 and 4)
        typename Elem<T>::Vec v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = T(f[i]);
        u32x4 d = __builtin_bit_cast(u32x4, v);
        const int bytes = int(n - c) * int(sizeof(T));
        uint8_t *p = reinterpret_cast<uint8_t *>(row + c);
        if (bytes & 8) {
            __builtin_memcpy(p, &d, 8);
            d.x = d.z, d.y = d.w, p += 8;
        }
        if (bytes & 4) {
            __builtin_memcpy(p, &d, 4);
            d.x = d.y, p += 4;
        }
        if (sizeof(T) == 2 && bytes & 2) __builtin_memcpy(p, &d, 2);
    }
}
template <class T, bool TAIL>
__device__ __forceinline__ void store_stream(T *row, int64_t c, int64_t n, const float (&f)[Elem<T>::V]) {
    store_vec<T, true, TAIL>(row, c, n, f);
}

// a + b rounded to T by way of fp32.  The fp32 sum is made opaque, so that every
// use sees this one rounding (the compiler may otherwise round some uses to
// fp16 directly, which differs next to a tie).
template <class T>
__device__ __forceinline__ float rounded_sum(float a, float b) {
    float s = a + b;
    asm("" : "+v"(s));
    return float(T(s));
}

// V elements of an fp32 or T parameter vector.
template <int V, class T>
__device__ __forceinline__ void load_param(const T *p, int64_t c, int64_t n, float (&f)[V]) {
    constexpr int E = Elem<T>::V;
#pragma unroll
    for (int i = 0; i < V; i += E) {
        const typename Elem<T>::Vec v = load_raw(p, c + i, n);
#pragma unroll
        for (int j = 0; j < E; ++j) f[i + j] = float(v[j]);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// Sum over the T threads (a multiple of 64) that share a row; every thread
// gets it.  One wave needs no LDS; more exchange through red[T / 64], which
// the caller does not touch between calls (a barrier precedes its reuse).
template <int T>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (T > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < T / 64; ++i) v += red[i];
    }
    return v;
}

}  // namespace ssg

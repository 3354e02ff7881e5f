// The 4-bit format's scale bytes and codes, shared by the kernels that quantise (mxfp4.hip says the format).
#pragma once

#include <type_traits>

#include "elem.h"

namespace ssg {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), CTRL, 0xf, 0xf, false));
}

// Scale byte of the block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255 ? 255u : e > 2 ? e - 2 : 0u;
}
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);  // (255: not finite)
}

// Largest magnitude of the values added so far; bits(): as fp32 bits.
template <class T>
struct Top {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top = {0, 0};  // 16-bit types: two at a time
    __device__ __forceinline__ void add(typename Elem<T>::Vec v) {
        const u32x4 d = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, d[i] & 0x7fff7fffu));
    }
    __device__ __forceinline__ uint32_t bits() const {
        const uint16_t t = top.x > top.y ? top.x : top.y;
        if constexpr (std::is_same<T, __bf16>::value) return uint32_t(t) << 16;
        else return __builtin_bit_cast(uint32_t, float(__builtin_bit_cast(_Float16, t)));
    }
};
template <>
struct Top<float> {
    uint32_t top = 0;
    __device__ __forceinline__ void add(Elem<float>::Vec v) {
        const u32x4 d = __builtin_bit_cast(u32x4, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, d[i] & 0x7fffffffu);
    }
    __device__ __forceinline__ uint32_t bits() const { return top; }
};

// Eight values to eight codes: the instruction divides by the scale, a power of two, and rounds to the
// nearest code, ties to the even one, past 6 to 6.  A block that is not finite keeps codes 0.
template <class T>
__device__ __forceinline__ uint32_t codes_of(const typename Elem<T>::Vec (&v)[8 / Elem<T>::V], uint32_t byte) {
    if (byte == 255) return 0;
    const float by = scale_of(byte);
    uint32_t c = 0;
    if constexpr (std::is_same<T, _Float16>::value) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_shufflevector(v[0], v[0], 0, 1), by, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_shufflevector(v[0], v[0], 2, 3), by, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_shufflevector(v[0], v[0], 4, 5), by, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_shufflevector(v[0], v[0], 6, 7), by, 3);
    } else if constexpr (std::is_same<T, __bf16>::value) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_shufflevector(v[0], v[0], 0, 1), by, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_shufflevector(v[0], v[0], 2, 3), by, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_shufflevector(v[0], v[0], 4, 5), by, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_shufflevector(v[0], v[0], 6, 7), by, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0][0], v[0][1], by, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0][2], v[0][3], by, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[1][0], v[1][1], by, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[1][2], v[1][3], by, 3);
    }
    return c;
}

}  // namespace ssg

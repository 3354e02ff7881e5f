// Low-rank adapters: what the kernels share.
//
// Token m with adapter a = index[m] gets, beside its shared projection,
//   delta[m] = scale[a] * up[a] . (down[a] . x[m])
// down [n][R][K] and up [n][N][R] are pools of n adapters, R slots of rank
// each; adapter a uses the first ranks[a] slots (all R without ranks), and
// what lies in the others is not used.  index -1: no adapter.  Any other index
// outside [0, n) makes the token's output NaN: no pool row is read for it.
//
// The low-rank activations low[m][r] = scale[a] * (down[a] . x[m])[r] are
// handed from one kernel to the next as two values of the rows' type, hi =
// round(low) and lo = round(low - hi), two planes.  Both feed the
// matrix instructions, so that the split costs one more small product instead of
// the digits that a single 16-bit value would lose (16 bits of mantissa for
// bf16, 15 to 21 for fp16, against the 8 and 11 of the outputs).  A plane is laid out
// as the 32x32x16 instruction's operand: blocks of 32 tokens x 16 slots, in each
// the 16 bytes of lane (slot / 8 % 2) * 32 + token % 32 hold slots 8 (slot / 8)
// .. + 7, so that a wave reads a block as one contiguous KiB (read row by row,
// 32 rows an instruction, the loads took 4 times as many cache lines).
//
// fp16 has neither the range nor the small steps for values that are products of
// two of its numbers, so there a token's pair holds low * 2^-e, which puts the token's
// largest value into [2^-8, 2^15), where the pair's steps of 2^-23 are 15 bits of it or more
// (21 from 2^-2 on).  e is a multiple of 23, and 0 for values of ordinary size: narrower
// steps would hold more bits, but every e of an adapter costs wgrad another pass over its
// list (with steps of 20, 32 tokens of 26 adapters with values about 2^-5 took 23.4 us instead
// of 21.7, 6144 tokens about 2^-2, steps of 17, 56 instead of 52.5).  It travels in the last bits
// of lo, eight bits in every eight slots, which the readers take out; sums over one
// token's slots are multiplied by 2^e at their end.  Sums over tokens (wgrad) go
// through an adapter's tokens one e after another, from the least, and are brought to the
// next one's size between them.  (Multiplying each token's values by its 2^(e - largest)
// in the product's loop instead took 2 to 6 of 32 us there, with nothing to scale too.)
#pragma once

#include "elem.h"
#include "tw_common.h"

namespace ssg {

// Whether a token's pair carries a power of two (fp16).
template <class T>
constexpr bool kLowScaled = __is_same(T, _Float16);

// The power of two for a token whose largest value is `top`: in steps of 23, the
// width of [2^-8, 2^15), so that tokens of similar size have the same one.  The limits:
// values below 2^-54 are held to 2^-70, far below what a pool and an output in fp16
// can show, and 2^92 leaves the product in front of them room for 2^-92.
__device__ __forceinline__ int low_exponent(float top) {
    const int e = int(__builtin_bit_cast(uint32_t, top) >> 23) - 127 + 54;  // top = 1.. * 2^(e - 54)
    if (top == 0.0f) return 0;
    return min(max(e, 0) / 23 - 2, 4) * 23;
}
// Largest value of lanes i, i + 16, i + 32 and i + 48, for each of them (values >= 0).
__device__ __forceinline__ float max_of_groups(float v) {
    uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = max(uint32_t(a[0]), uint32_t(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __builtin_bit_cast(float, max(uint32_t(b[0]), uint32_t(b[1])));
}
// A token of wgrad's list: its adapter, and e as the low eight bits.
__device__ __forceinline__ int low_key(int adapter, int e) { return adapter << 8 | (e + 128); }
__device__ __forceinline__ int low_key_power(int key) { return (key & 255) - 128; }
// Eight slots of lo: their last bits to e (the even slots hold bits 0-3, the odd ones
// 4-7), and the values without them.
__device__ __forceinline__ int low_exponent_of(u32x4 lo) {
    constexpr uint32_t kBits = 0x00010001u;
    const uint32_t t = (lo.x & kBits) | (lo.y & kBits) << 1 | (lo.z & kBits) << 2 | (lo.w & kBits) << 3;
    return int8_t((t & 15) | t >> 12);
}
__device__ __forceinline__ uint32_t low_exponent_bit(int e, int slot) {
    return uint32_t(e) >> ((slot & 1) * 4 + (slot & 7) / 2) & 1;
}
template <class T>
__device__ __forceinline__ u32x4 lo_value(u32x4 lo) {
    if constexpr (!kLowScaled<T>) return lo;
    constexpr uint32_t kValue = 0xfffefffeu;
    return u32x4{lo.x & kValue, lo.y & kValue, lo.z & kValue, lo.w & kValue};
}

template <class T>
__device__ __forceinline__ floatx16 mfma32(u32x4 a, u32x4 b, floatx16 c) {
    if constexpr (sizeof(T) == 2 && __is_same(T, _Float16))
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}
template <class T>
__device__ __forceinline__ floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c) {
    if constexpr (sizeof(T) == 2 && __is_same(T, _Float16))
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0,
                                                      0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
}

// The first `n` of eight 16-bit elements, zeros after them.
__device__ __forceinline__ u32x4 keep16(u32x4 v, int n) {
    if (n >= 8) return v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 2 * i + 1 < n ? v[i] : 2 * i < n ? v[i] & 0xffffu : 0u;
    return v;
}

__device__ __forceinline__ int low_rank_of(const int32_t *ranks, int a, int R) {
    if (!ranks) return R;
    const int r = ranks[a];
    return r < 0 ? 0 : r > R ? R : r;
}

// Whether one of eight 16-bit elements is an infinity or NaN.
template <class T>
__device__ __forceinline__ bool not_finite(u32x4 v) {
    constexpr uint32_t kExp = __is_same(T, _Float16) ? 0x7c00u : 0x7f80u;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad = bad || (v[i] & kExp) == kExp || ((v[i] >> 16) & kExp) == kExp;
    return bad;
}

// An adapter whose weights are not finite must not reach the tokens of other
// requests through 0 * inf: its broken channels (rows of w) are taken out of the
// product, and its own tokens get NaN in them afterwards.  take_out() says whether
// the wave has such channels; the products between the two calls stay one block
// of independent matrix instructions.
template <class T, int TN>
__device__ __forceinline__ bool take_out(u32x4 (&w)[TN], bool (&bad)[TN]) {
    bool any = false;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) bad[tn] = not_finite<T>(w[tn]), any = any || bad[tn];
    if (__ballot(any) == 0) return false;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) w[tn] = bad[tn] ? u32x4{0, 0, 0, 0} : w[tn];
    return true;
}
template <int TN, int TM>
__device__ __forceinline__ void poison(floatx16 (&acc)[TN][TM], const bool (&bad)[TN], const bool (&use)[TM]) {
    const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
        const uint64_t b = __ballot(bad[tn]);
        const uint32_t rows = uint32_t(b) | uint32_t(b >> 32);
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (use[tm] && (rows >> (8 * (i / 4) + 4 * h + i % 4) & 1)) acc[tn][tm][i] = __builtin_nanf("");
    }
}

// Elements of one plane, and the place of 8 slots from r (a multiple of 8) of token m.
__host__ __device__ inline int64_t low_plane(int64_t M, int R) { return (M + 31) / 32 * 32 * ((R + 15) / 16 * 16); }
__device__ __forceinline__ int64_t low_at(int64_t m, int r, int R) {
    return ((m / 32 * ((R + 15) / 16) + r / 16) * 64 + (r / 8 % 2) * 32 + m % 32) * 8;
}

// Two operands of 8 consecutive rows a lane: transposing reads of the four rows
// at p (q) and of the four below them, at p4 (q4).  Waited for in the same
// statement: the compiler would place a wait for every load in flight before
// the builtin form, which it cannot tell apart from the direct-to-LDS loads'
// stores.
__device__ __forceinline__ void read_tr(uint32_t p, uint32_t p4, uint32_t q, uint32_t q4, u32x4 &u, u32x4 &v) {
    u32x2 u0, u1, v0, v1;
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4\n\t"
        "ds_read_b64_tr_b16 %1, %5\n\t"
        "ds_read_b64_tr_b16 %2, %6\n\t"
        "ds_read_b64_tr_b16 %3, %7\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(u0), "=&v"(u1), "=&v"(v0), "=&v"(v1)
        : "v"(p), "v"(p4), "v"(q), "v"(q4)
        : "memory");
    u = u32x4{u0.x, u0.y, u1.x, u1.y};
    v = u32x4{v0.x, v0.y, v1.x, v1.y};
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}

// Source of padding in direct-to-LDS loads.
static __device__ __attribute__((aligned(256))) uint16_t g_low_zero[128];

// Adds up[a] . low to accumulators of 32x32 blocks, zeros before: acc[tn][tm] holds, for the
// 32 tokens from mw + 32 tm (mw a multiple of 32), the channels nw + 32 tn +
// 8 (i/4) + 4 h + i%4 of token lane%32.  at[i]: index of token mw + i (anything
// past M).  Channels past the last repeat it (their results are not stored).
// The wave visits the distinct adapters of its tokens one after another, each
// with the other tokens' low values zeroed, up to 64 rank slots at a time: it
// copies its channels' rows of the pool to `lds` (TN * 4 KiB of its own) with
// whole-line direct-to-LDS loads and reads its operand from there.
// TRANS (TN even): the pool is [adapters][R][N], slots along the rows, and the
// operand comes through transposing LDS reads.
template <class T, int TN, int TM, bool TRANS>
__device__ __forceinline__ void low_rank_expand(floatx16 (&acc)[TN][TM], const T *__restrict__ up,
                                                const T *__restrict__ low, const int32_t *at,
                                                const int32_t *__restrict__ ranks, int adapters, int R, int mw, int nw,
                                                int M, int N, uint8_t *lds) {
    const int lane = threadIdx.x & 63, h = lane >> 5, r = lane & 31;
    const int64_t plane = low_plane(M, R);
    // 16-byte pieces of a pool row held at a time, as a shift
    const int ws = R <= 16 ? 1 : R <= 32 ? 2 : 3;
    int mine[TM], power[TM];  // (of its token)
    bool todo[TM];
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
        power[tm] = 0;
        mine[tm] = at[tm * 32 + r];
        if (mw + tm * 32 + r >= M) mine[tm] = -1;
        todo[tm] = mine[tm] >= 0 && mine[tm] < adapters;
        if (mine[tm] != -1 && !todo[tm]) {
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[tn][tm][i] = __builtin_nanf("");
        }
    }
    for (;;) {
        int a = -1;
#pragma unroll
        for (int tm = TM - 1; tm >= 0; --tm) {
            const uint64_t left = __ballot(todo[tm]);
            if (left) a = __builtin_amdgcn_readlane(mine[tm], __builtin_ctzll(left));
        }
        if (a < 0) break;
        {
            bool sel[TM];
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) {
                sel[tm] = todo[tm] && mine[tm] == a;
                todo[tm] = todo[tm] && !sel[tm];
            }
            const int rank = low_rank_of(ranks, a, R);
            const T *pool = up + int64_t(a) * N * R;
            for (int k0 = 0; k0 < R; k0 += 64) {
                // (the previous turn's reads are done before its bytes are replaced)
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                constexpr int PIECES = TN * 4;  // of a row of TN * 32 channels
                for (int j = 0; TRANS && j < TN * 4; ++j) {
                    const int row = (j * 64 + lane) / PIECES;
                    const int n = nw + (lane % PIECES ^ (4 * (row & 3) & (PIECES - 1))) * 8;
                    const void *src = g_low_zero;
                    if (k0 + row < rank && n < N) src = pool + int64_t(k0 + row) * N + n;
                    tw_detail::tw_dma16(src, lds + j * 1024);
                }
                for (int j = 0; !TRANS && j < TN << (ws - 1); ++j) {
                    const int row = (j << (6 - ws)) + (lane >> ws);
                    const int k = k0 + ((lane & ((1 << ws) - 1)) ^ (row & ((1 << ws) - 1))) * 8;
                    const void *src = g_low_zero;
                    if (k < R) src = pool + int64_t(min(nw + row, N - 1)) * R + k;
                    tw_detail::tw_dma16(src, lds + j * 1024);
                }
                u32x4 hi[4][TM], lo[4][TM];
#pragma unroll
                for (int s = 0; s < 4; ++s)
#pragma unroll
                    for (int tm = 0; tm < TM; ++tm) {
                        const int k = k0 + 16 * s + 8 * h;
                        hi[s][tm] = lo[s][tm] = u32x4{0, 0, 0, 0};
                        if (sel[tm] && k < R) {
                            const T *p = low + low_at(mw + tm * 32 + r, k, R);
                            hi[s][tm] = ld16(p);
                            lo[s][tm] = ld16(p + plane);
                        }
                    }
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                if (k0 >= rank) break;
                if constexpr (kLowScaled<T>) {
                    if (k0 == 0) {
#pragma unroll
                        for (int tm = 0; tm < TM; ++tm) {
                            // (the lower half's piece: the upper one's lies past R = 8)
                            const int e = low_exponent_of(lo[0][tm]);
                            if (__ballot(e != 0) != 0) {
                                const int own = __shfl(e, r, 64);
                                power[tm] = sel[tm] ? own : power[tm];
                            }
                        }
                    }
                }
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int k = k0 + 16 * s;
                    if (k >= rank) break;
                    u32x4 w[TN];
                    if constexpr (TRANS) {
                        static_assert(TN % 2 == 0, "channel blocks in pairs");
                        const int row = 16 * s + 8 * h + ((lane & 15) >> 2), c = (lane & 16) + 4 * (lane & 3);
                        auto at_block = [&](int tn) {
                            const int col = tn * 32 + c;
                            return lds_address(lds) + row * (PIECES * 16) +
                                   ((col >> 3) ^ (4 * (row & 3) & (PIECES - 1))) * 16 + (col & 7) * 2;
                        };
#pragma unroll
                        for (int tn = 0; tn < TN; tn += 2)
                            read_tr(at_block(tn), at_block(tn) + PIECES * 64, at_block(tn + 1),
                                    at_block(tn + 1) + PIECES * 64, w[tn], w[tn + 1]);
                    } else {
#pragma unroll
                        for (int tn = 0; tn < TN; ++tn) {
                            const int row = tn * 32 + r;
                            const int piece = (2 * s + h) ^ (row & ((1 << ws) - 1));
                            w[tn] = keep16(*reinterpret_cast<const u32x4 *>(lds + (row << (ws + 4)) + piece * 16),
                                           rank - k - 8 * h);
                        }
                    }
                    bool bad[TN];
                    const bool some = take_out<T>(w, bad);
#pragma unroll
                    for (int tm = 0; tm < TM; ++tm) {
                        const u32x4 l = lo_value<T>(lo[s][tm]);
#pragma unroll
                        for (int tn = 0; tn < TN; ++tn) {
                            acc[tn][tm] = mfma32<T>(w[tn], hi[s][tm], acc[tn][tm]);
                            acc[tn][tm] = mfma32<T>(w[tn], l, acc[tn][tm]);
                        }
                    }
                    if (some) poison(acc, bad, sel);
                }
            }
        }
    }
    if constexpr (kLowScaled<T>) {
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            if (__ballot(power[tm] != 0) == 0) continue;
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[tn][tm][i] = __builtin_amdgcn_ldexpf(acc[tn][tm][i], power[tm]);
        }
    }
}

}  // namespace ssg

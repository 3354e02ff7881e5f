// 4-bit products of few rows, quantising x on the way: C[m][n] = sum_k q(x[m][k]) w[n][k].
//
// A decode step's product is a few microseconds of waiting: for the launch, for memory, for the next
// launch.  Here one launch does both.  A workgroup is 32 rows x BN columns and its waves share K by
// units of 256 values (a 128-byte line of a packed row): each wave has its unit's weights under way,
// quantises the rows that there are into an LDS region of its own, without a barrier, and feeds the
// matrix instruction; the waves' sums meet in LDS in wave order.
//
// Measured (bf16, launches in a graph): 4 x 4096 x 1024 4.7 us, quantisation and product apart 7.0; 1 x 4096
// x 4096 6.8 and 10.4; 18 x 560 x 1508 6.9 and 8.1; a call from the host 9.8 and 12.5.  Bound by the
// launch and by one or two waits for memory.  Up to eight rows are quantised a row after another, four
// lanes a block; more of them by a lane for each block, whose loads touch a line for every row (of 16 rows,
// K = 3000, 8.5 us; row after row 9.5; of two rows, K = 2600, 6.8 and 4.6).
//
// The instruction's lane (h, r) holds one block of 32 values of row r.  Its sum may take the blocks in any
// order as long as both operands do: instruction i takes blocks 2i + h of a unit, neighbours in memory.
#include "gemm_core.h"
#include "group_place.h"
#include "launch.h"
#include "mx_codes.h"

namespace ssg {

namespace {

struct Few {
    const void *a;  // x, or packed codes
    const uint8_t *sa, *w, *sw;
    const int32_t *offsets;
    void *out;
    int64_t lda, ldo;
    int groups, M, N, K, kp;
};

// A unit's blocks 2i + h of one row, i = 0..3: codes, and the scales in a word's bytes.
struct Blocks {
    u32x4 code[4];
    uint32_t scale;
};
__device__ __forceinline__ uint32_t scales_of(u32x2 all, int h) {
    return __builtin_amdgcn_perm(all.y, all.x, h ? 0x07050301u : 0x06040200u);
}
__device__ __forceinline__ Blocks packed_blocks(const uint8_t *codes, const uint8_t *scales, int kp, int64_t row, int u,
                                                int h) {
    Blocks b{{}, 0};
    const uint8_t *const p = codes + row * (kp / 2) + u * 128 + h * 16;
    const uint32_t *const s = reinterpret_cast<const uint32_t *>(scales + row * (kp / 32) + u * 8);
    u32x2 all{s[0], 0};  // (rows are a multiple of 128 values: a unit is whole or half)
    b.code[0] = ld16(p), b.code[1] = ld16(p + 32);
    if (u * 256 + 128 < kp) all.y = s[1], b.code[2] = ld16(p + 64), b.code[3] = ld16(p + 96);
    b.scale = scales_of(all, h);
    return b;
}

// A wave's LDS: 8 rows of a unit's codes, 16 bytes apart from whole lines (reads of a column of rows at
// 128 bytes meet in one bank), and their scales.
constexpr int kRow = 144, kUnit = 8 * kRow + 8 * 8;

// Quantises a unit of the first `rows` <= 2 ITS rows (others stay as they are): two rows a step, a lane
// eight values, four lanes a block.
template <class T, bool TAIL, int ITS>
__device__ __forceinline__ void quantize_unit(uint8_t *lds, const T *x, int64_t ldx, int rows, int at, int K) {
    const int lane = threadIdx.x & 63, c = at + (lane & 31) * 8;
    typename Elem<T>::Vec v[ITS][1];
#pragma unroll
    for (int i = 0; i < ITS; ++i) v[i][0] = fetch_raw<T, TAIL>(x + min(2 * i + (lane >> 5), rows - 1) * ldx, c, K);
#pragma unroll
    for (int i = 0; i < ITS; ++i) {
        const int row = 2 * i + (lane >> 5);
        v[i][0] = settle<T, TAIL>(v[i][0], c, K);
        Top<T> most;
        most.add(v[i][0]);
        uint32_t top = most.bits();
        top = max(top, dpp<0xb1>(top));
        top = max(top, dpp<0x4e>(top));
        const uint32_t byte = scale_byte(top);
        *reinterpret_cast<uint32_t *>(lds + row * kRow + (lane & 31) * 4) = codes_of<T>(v[i], byte);
        if ((lane & 3) == 0) lds[8 * kRow + row * 8 + (lane & 31) / 4] = uint8_t(byte);
    }
}

// A unit of any row, as the instruction takes it: a lane quantises its own blocks.
template <class T, bool TAIL>
__device__ __forceinline__ Blocks quantized(const T *row, int u, int h, int K) {
    Blocks b{{}, 0};
    typename Elem<T>::Vec v[4][4][1];
    const int at = u * 256 + h * 32;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i / 4][i % 4][0] = fetch_raw<T, TAIL>(row, at + i / 4 * 64 + i % 4 * 8, K);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Top<T> top;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[i][j][0] = settle<T, TAIL>(v[i][j][0], at + i * 64 + j * 8, K);
            top.add(v[i][j][0]);
        }
        const uint32_t byte = scale_byte(top.bits());
        b.scale |= byte << (8 * i);
        b.code[i] = u32x4{codes_of<T>(v[i][0], byte), codes_of<T>(v[i][1], byte), codes_of<T>(v[i][2], byte),
                          codes_of<T>(v[i][3], byte)};
    }
    return b;
}

// T: x's type, or uint8_t: packed.  NB: blocks of 32 columns; NW: waves.
template <class T, class O, bool GROUPED, int NB, int NW, bool TAIL>
__global__ void __launch_bounds__(NW * 64)
few_rows_kernel(Few p) {
    constexpr int BN = 32 * NB, PITCH = BN + 4, V = 4;
    constexpr int REGION = 32 * PITCH * 4;  // a wave's sums, and before them the codes
    static_assert(REGION >= kUnit);
    __shared__ __attribute__((aligned(16))) uint8_t lds[NW][REGION];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int h = lane >> 5, r = lane & 31;
    const int tiles_n = (p.N + BN - 1) / BN;
    int row, rows, n0;
    const uint8_t *w = p.w, *sw = p.sw;
    if constexpr (GROUPED) {
        const group::Tile t = group::find_tile<32>(blockIdx.x, p.offsets, p.groups, p.M, tiles_n, 8);
        if (t.group < 0) return;
        row = t.row, rows = t.rows, n0 = t.tile_n * BN;
        w += int64_t(t.group) * p.N * (p.kp / 2);
        sw += int64_t(t.group) * p.N * (p.kp / 32);
    } else {
        const int b = xcd_remap(blockIdx.x, gridDim.x), tiles_m = (p.M + 31) / 32;
        row = b % tiles_m * 32, rows = p.M - row, n0 = b / tiles_m * BN;
    }
    rows = uniform(min(rows, 32));
    floatx16 acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = floatx16{};
    for (int u = wave; u * 256 < p.kp; u += NW) {
        Blocks a, b[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) b[i] = packed_blocks(w, sw, p.kp, min(n0 + 32 * i + r, p.N - 1), u, h);
        if constexpr (sizeof(T) == 1) {
            a = packed_blocks(static_cast<const uint8_t *>(p.a), p.sa, p.kp, row + min(r, rows - 1), u, h);
        } else {
            const T *const x = static_cast<const T *>(p.a) + row * p.lda;
            if (rows > 8) {
                a = quantized<T, TAIL>(x + min(r, rows - 1) * p.lda, u, h, p.K);
            } else {
                if (rows <= 2) quantize_unit<T, TAIL, 1>(lds[wave], x, p.lda, rows, u * 256, p.K);
                else quantize_unit<T, TAIL, 4>(lds[wave], x, p.lda, rows, u * 256, p.K);
                // (a wave's LDS accesses are done in order: only the compiler has to keep it)
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int i = 0; i < 4; ++i) a.code[i] = lds16(lds[wave] + (r & 7) * kRow + 32 * i + 16 * h);
                a.scale = scales_of(*reinterpret_cast<const u32x2 *>(lds[wave] + 8 * kRow + (r & 7) * 8), h);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            mma_f4<0>(acc[i], b[i].code[0], a.code[0], b[i].scale, a.scale);
            mma_f4<1>(acc[i], b[i].code[1], a.code[1], b[i].scale, a.scale);
            mma_f4<2>(acc[i], b[i].code[2], a.code[2], b[i].scale, a.scale);
            mma_f4<3>(acc[i], b[i].code[3], a.code[3], b[i].scale, a.scale);
        }
    }
    float *const sums = reinterpret_cast<float *>(lds[wave]);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<floatx4 *>(&sums[r * PITCH + 32 * i + 8 * q + 4 * h]) =
                floatx4{acc[i][4 * q], acc[i][4 * q + 1], acc[i][4 * q + 2], acc[i][4 * q + 3]};
    __syncthreads();
#pragma unroll
    for (int at = threadIdx.x; at < 32 * BN / V; at += NW * 64) {
        const int token = at / (BN / V), c = at % (BN / V) * V, n = n0 + c;
        if (token >= rows || n >= p.N) continue;
        auto part = [&](int i) {
            return *reinterpret_cast<const floatx4 *>(reinterpret_cast<const float *>(lds[i]) + token * PITCH + c);
        };
        floatx4 s = part(0);
#pragma unroll
        for (int i = 1; i < NW; ++i) s += part(i);
        O *const to = static_cast<O *>(p.out) + (int64_t(row) + token) * p.ldo + n;
        const O v[V] = {O(s.x), O(s.y), O(s.z), O(s.w)};
        if (n + V <= p.N) {
            __builtin_memcpy(to, v, sizeof(v));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (n + i < p.N) to[i] = v[i];
        }
    }
}

template <class T, class O, bool GROUPED, int NB, int NW>
hipError_t few_cfg(const Few &p, hipStream_t st) {
    const int64_t tiles_n = (p.N + 32 * NB - 1) / (32 * NB);
    const int64_t blocks = GROUPED ? group_tiles(p.M, p.groups, 32, tiles_n) : (p.M + 31) / 32 * tiles_n;
    auto k = few_rows_kernel<T, O, GROUPED, NB, NW, false>;
    if constexpr (sizeof(T) > 1)
        if (p.K % 8) k = few_rows_kernel<T, O, GROUPED, NB, NW, true>;
    hipLaunchKernelGGL(k, dim3(unsigned(blocks)), dim3(NW * 64), 0, st, p);
    return hipGetLastError();
}

template <class T, class O, bool GROUPED>
hipError_t few_any(const Few &p, hipStream_t st) {
    switch (mxfp4_few_kind(p.M, GROUPED ? p.groups : 0, p.N, p.K)) {
        case 0: return few_cfg<T, O, GROUPED, 1, 4>(p, st);
        case 1: return few_cfg<T, O, GROUPED, 1, 8>(p, st);
        default: return few_cfg<T, O, GROUPED, 2, 4>(p, st);
    }
}

template <class T, class O>
hipError_t few(const Few &p, hipStream_t st) {
    return p.offsets ? few_any<T, O, true>(p, st) : few_any<T, O, false>(p, st);
}

}  // namespace

hipError_t launch_mxfp4_few(const Mxfp4Gemm &g, int x_dtype, int64_t ldx, hipStream_t st) {
    const Few p{g.a, g.a_scales, g.w, g.w_scales, g.offsets, g.out, ldx, g.ldo, g.experts, int(g.M), int(g.N), int(g.K),
                int(mxfp4_padded(g.K))};
    if (x_dtype == DT_F16) return few<_Float16, _Float16>(p, st);
    if (x_dtype == DT_BF16) return few<__bf16, __bf16>(p, st);
    if (g.dtype == DT_F16) return few<uint8_t, _Float16>(p, st);
    if (g.dtype == DT_BF16) return few<uint8_t, __bf16>(p, st);
    return few<uint8_t, float>(p, st);
}

}  // namespace ssg

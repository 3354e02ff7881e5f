// Low-rank adapters of many requests beside a shared projection, for gfx950
// (formulas and formats in low_rank.h).
//
//   shrink   low[m] = scale[a] * (down[a] . x[m])          a = index[m]
//   expand   out[m] = base[m] + up[a] . low[m]
//   tokens   both in one launch on the vector units, for few tokens (and the
//            input gradient's second half, tokens_dx)
//   wgrad    ddown[a][r][k] = sum over a's tokens of (scale up[a]^T dy)[r] x[k]
//            dup[a][n][r]   = sum over a's tokens of dy[n] low[r]
// The input gradient is the same pair of kernels with the roles exchanged:
// dlow = shrink(dy, up^T), dx = expand(base, dlow, down^T), which take the pools
// as they lie through transposing LDS reads.
//
// Memory bound: shrink reads x once, expand reads base and writes out once,
// wgrad reads x and dy once; the pools are small beside them, and the products
// (2 M R (K + N) operations) far below the matrix units' rate.  Measured on
// MI355X, inputs in rotating buffers (HBM traffic by counter where named):
//   6144 x 1024 -> 4096 fp16, rank 16, 4 adapters, backward 47-52 us; medians:
//     both shrinks 18.0 us (64.8 MB: 3.6 TB/s), expand 8.1 us (26 MB: 3.2 TB/s),
//     wgrad 18.1 us (72.4 MB: 4.0 TB/s), wgrad_sum 4.1 us (least 15.8, 7.3, 16.4)
//   4096 x 1024 -> 1024 fp16, rank 128, 4 adapters, backward: 25.2, 15.3, 33.8, 5.5 us;
//   1755 x 2400 -> 1024, rank 64: 13.9, 10.3, 22.4, 4.1 us.  Bytes would take 5 to 10:
//     a slice of the pool is fetched, waited for and read before the next one leaves
//   1531 x 768 -> 2312 bf16, rank 32, 8 adapters: shrink 6.3, expand 8.4 us
//   32 tokens, 1024 -> 4096, 24 adapters of rank 16 (tokens): 4.6 us
// The small ones are a chain of a few dependent loads each, not bytes.
#include "launch.h"
#include "low_rank.h"
#include "tw_common.h"

namespace ssg {

namespace {

using namespace tw_detail;

// ---- shrink.  A workgroup takes 16 tokens, its NW waves every NW-th
// 64-wide slice of K; v_mfma 16x16x32 with the rank slots as rows and the
// tokens as columns (lane: row / column lane%16, k = 8 (lane/16)..; results:
// rows 4 (lane/16) + i of column lane%16).  The waves' sums are added in order
// through LDS.  RB: blocks of 16 rank slots.
// Two of a tile's adapters are taken at a time, on the same x values, so that a
// tile where one request ends and the next begins costs no second pass; the
// first x values are fetched before the indices are known.
// The pool's part of a slice is copied to LDS, for each wave its own, with
// whole-line direct-to-LDS loads (read as operands straight from memory, 16 rows
// of 64 bytes an instruction, the same pass took 18.0 us instead of 14.2 at
// 6144 x 4096 and 1024, rank 16).  TRANS: the pool is [adapters][K][R] (the gradient's use
// of `up`) and is read by transposing reads.
template <int RB>
constexpr int kShrinkUnroll = RB <= 2 ? 2 : 1;  // 64-wide slices of K in flight
template <class T, int RB, int NW, bool TRANS>
__device__ __forceinline__ void shrink_tile(const T *__restrict__ x, int64_t ldx, const T *__restrict__ down,
                                            const float *__restrict__ scale, const int32_t *__restrict__ ranks,
                                            const int32_t *__restrict__ index, int adapters, int R,
                                            T *__restrict__ low, int M, int K, int tile, int deal, int deals,
                                            floatx4 *part, float *tops, int32_t *__restrict__ key) {
    constexpr int UNROLL = kShrinkUnroll<RB>;
    constexpr int SLICE = RB * 2048;  // bytes of a slice in LDS
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, c = lane & 15;
    const int m = tile * 16 + c;
    const int step = NW * 64 * UNROLL;
    const T *row = x + int64_t(m) * ldx;
    u32x4 xv[UNROLL][2];
    auto fetch_x = [&](int k0) {
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k = k0 + u * NW * 64 + 32 * s + 8 * g;
                xv[u][s] = u32x4{0, 0, 0, 0};
                if (k < K && m < M) xv[u][s] = ld16(row + k);
            }
    };
    fetch_x(wave * 64);
    // every wave finds the distinct adapters of the same tokens, in the same order
    const int mine = m < M ? index[m] : -1;  // (each token in four lanes)
    bool todo = mine >= 0 && mine < adapters;
    // (a key for every token: those of an adapter are written with their values)
    if (kLowScaled<T> && key && deal == 0 && wave == 0 && g == 0 && m < M && !todo) key[m] = -1;
    bool held = true;  // xv holds the first slices
    int pair = 0;
    for (uint64_t left = __ballot(todo); left; left = __ballot(todo), ++pair) {
        const int a0 = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
        todo = todo && mine != a0;
        left = __ballot(todo);
        const int a1 = left ? __builtin_amdgcn_readlane(mine, __builtin_ctzll(left)) : -1;
        todo = todo && mine != a1;
        if (pair % deals != deal) continue;
        const int rank0 = low_rank_of(ranks, a0, R), rank1 = a1 >= 0 ? low_rank_of(ranks, a1, R) : 0;
        const float s0 = scale ? scale[a0] : 1.0f, s1 = scale && a1 >= 0 ? scale[a1] : 1.0f;
        __syncthreads();  // (the previous adapters' sums, in the same LDS, have been read)
        const T *pool0 = down + int64_t(a0) * R * K, *pool1 = down + int64_t(a1 < 0 ? 0 : a1) * R * K;
        floatx4 acc[2][RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) acc[0][b] = acc[1][b] = floatx4{0.f, 0.f, 0.f, 0.f};
        // one adapter's operand of the slices from k0
        uint8_t *own = reinterpret_cast<uint8_t *>(part) + wave * UNROLL * SLICE;
        auto fetch_pool = [&](const T *pool, int rank, u32x4 (&dv)[UNROLL][2][RB], int k0) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int ku = k0 + u * NW * 64;
                for (int j = 0; j < (TRANS ? R / 8 : RB * 2); ++j) {
                    const void *src = g_low_zero;
                    if constexpr (TRANS) {
                        const int64_t e = int64_t(ku) * R + (j * 64 + lane) * 8;
                        if (e < int64_t(K) * R) src = pool + e;
                    } else {  // rows of 128 bytes, 16-byte pieces swizzled by row
                        const int row = j * 8 + (lane >> 3), k = ku + ((lane & 7) ^ (row & 7)) * 8;
                        if (row < rank && k < K) src = pool + int64_t(row) * K + k;
                    }
                    tw_dma16(src, own + u * SLICE + j * 1024);
                }
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    if constexpr (TRANS) {  // (slots past R read what follows: their sums are not used)
                        const uint32_t p = lds_address(own) + u * SLICE + (8 * g + (c >> 2)) * (R * 2) +
                                           (b * 16 + 4 * (c & 3)) * 2;
                        read_tr(p, p + 8 * R, p + 64 * R, p + 72 * R, dv[u][0][b], dv[u][1][b]);
                    } else {
                        const uint8_t *p = own + u * SLICE + (b * 16 + c) * 128;
                        dv[u][0][b] = *reinterpret_cast<const u32x4 *>(p + (g ^ (c & 7)) * 16);
                        dv[u][1][b] = *reinterpret_cast<const u32x4 *>(p + ((4 + g) ^ (c & 7)) * 16);
                    }
                }
            // (the bytes are replaced only after these reads)
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        };
        auto product = [&](const u32x4 (&dv)[UNROLL][2][RB], int a, floatx4 (&to)[RB]) {
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const u32x4 v = mine == a ? xv[u][s] : u32x4{0, 0, 0, 0};
#pragma unroll
                    for (int b = 0; b < RB; ++b) to[b] = mfma16<T>(dv[u][s][b], v, to[b]);
                }
        };
        for (int k0 = wave * 64; k0 < K; k0 += step) {
            if (!held) fetch_x(k0);
            held = K <= step;
            u32x4 d[UNROLL][2][RB];
            fetch_pool(pool0, rank0, d, k0);
            product(d, a0, acc[0]);
            if (a1 >= 0) {
                fetch_pool(pool1, rank1, d, k0);
                product(d, a1, acc[1]);
            }
        }
        __syncthreads();  // (every wave has read its slices, which the sums replace)
#pragma unroll
        for (int b = 0; b < RB; ++b) {
            part[(b * NW + wave) * 64 + lane] = acc[0][b];
            if (a1 >= 0) part[((RB + b) * NW + wave) * 64 + lane] = acc[1][b];
        }
        __syncthreads();
        // A wave finishes the blocks of 16 slots q = wave, wave + NW of the pair's 2 RB.
        constexpr int QS = (2 * RB + NW - 1) / NW;
        // (opaque, so that nothing formed from it here is kept in registers across the loop above)
        int id = threadIdx.x;
        asm volatile("" : "+v"(id));
        const int turn = __builtin_amdgcn_readfirstlane(id >> 6);
        const int at = id & 63, g = at >> 4, c = at & 15, m = tile * 16 + c;
        const int count = (a1 >= 0 ? 2 : 1) * RB;
        float f[QS][4];
        int power = 0;
#pragma unroll
        for (int j = 0; j < QS; ++j) {
            const int q = turn + j * NW, r = q % RB * 16 + 4 * g;
            if (q >= count) break;
            floatx4 v = part[(q * NW) * 64 + at];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                const floatx4 u = part[(q * NW + w) * 64 + at];
                v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
            }
            // Slots past the rank: zeros, also beside an x that is not finite.
            int keep = (q < RB ? rank0 : rank1) - r;
            asm volatile("" : "+v"(keep));  // (formed here: ahead, it took registers of the loop)
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // The product is made opaque: the compiler otherwise forms hi a
                // second time with a multiply that rounds to fp16 directly, and
                // next to a tie the stored hi is then not the one lo was taken from.
                f[j][i] = i < keep ? v[i] * (q < RB ? s0 : s1) : 0.0f;
                asm("" : "+v"(f[j][i]));
                if (fabsf(f[j][i]) <= __FLT_MAX__) top = fmaxf(top, fabsf(f[j][i]));
            }
            if constexpr (kLowScaled<T>) {
                top = max_of_groups(top);
                if (RB == 1) power = low_exponent(top);
                else if (g == 0) tops[q * 16 + c] = top;
            }
        }
        if constexpr (kLowScaled<T> && RB > 1) __syncthreads();
#pragma unroll
        for (int j = 0; j < QS; ++j) {
            const int q = turn + j * NW, r = q % RB * 16 + 4 * g;
            if (q >= count) break;
            if constexpr (kLowScaled<T> && RB > 1) {
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < RB; ++i) top = fmaxf(top, tops[(q < RB ? i : RB + i) * 16 + c]);
                power = low_exponent(top);
            }
            if (mine != (q < RB ? a0 : a1) || r >= R) continue;
            if (kLowScaled<T> && key && r == 0) key[m] = low_key(mine, power);
            T hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = kLowScaled<T> ? __builtin_amdgcn_ldexpf(f[j][i], -power) : f[j][i];
                asm("" : "+v"(v));
                hi[i] = T(v);
                // (an infinite value has no rest: inf - inf is NaN)
                const float rest = v - float(hi[i]);
                lo[i] = T(fabsf(rest) <= __FLT_MAX__ ? rest : 0.0f);
                if constexpr (kLowScaled<T>) {
                    const uint16_t u = __builtin_bit_cast(uint16_t, lo[i]);
                    // (rounded once more, to even, where the last bit goes)
                    const uint32_t t = ((u + (u >> 1 & 1u)) & 0xfffeu) | low_exponent_bit(power, r + i);
                    lo[i] = __builtin_bit_cast(T, uint16_t(t));
                }
            }
            T *to = low + low_at(m, r & ~7, R) + (r & 4);
            __builtin_memcpy(to, hi, 8);
            __builtin_memcpy(to + low_plane(M, R), lo, 8);
        }
    }
}

// TRANS: of the first task's pool.
template <class T, int RB, int NW, bool TRANS>
__global__ void __launch_bounds__(NW * 64)
shrink_kernel(ShrinkTask<T> p, ShrinkTask<T> q, const float *__restrict__ scale, const int32_t *__restrict__ ranks,
              const int32_t *__restrict__ index, int adapters, int R, int M) {
    constexpr int SUMS = 2 * RB * NW * 64, SLICES = NW * kShrinkUnroll<RB> * RB * 2048 / 16;
    __shared__ floatx4 part[SUMS > SLICES ? SUMS : SLICES];
    __shared__ float tops[kLowScaled<T> && RB > 1 ? 2 * RB * 16 : 1];  // a token's largest value in each block
    if (blockIdx.y)
        shrink_tile<T, RB, NW, false>(q.x, q.ldx, q.down, scale, ranks, index, adapters, R, q.low, M, q.K, blockIdx.x,
                                      blockIdx.z, gridDim.z, part, tops, q.key);
    else
        shrink_tile<T, RB, NW, TRANS>(p.x, p.ldx, p.down, scale, ranks, index, adapters, R, p.low, M, p.K, blockIdx.x,
                                      blockIdx.z, gridDim.z, part, tops, p.key);
}

// ---- expand: a workgroup takes 64 tokens x 128 channels, a wave 32 x 64.
// The sums go through LDS as fp32 rows, so that base is read and out written
// 16 bytes a lane; out may be base.
// TRANS: the pool is [adapters][R][N] (the gradient's use of `down`).
constexpr int kExpandTN = 2;
template <class T, bool TRANS>
__global__ void __launch_bounds__(256, 3)
expand_kernel(const T *__restrict__ up, const T *__restrict__ low, const int32_t *__restrict__ index,
              const int32_t *__restrict__ ranks, int adapters, int R, const T *base, int64_t ldb, T *out, int64_t ldo,
              int M, int N) {
    constexpr int TN = kExpandTN, ROW = TN * 32 + 4, CPR = TN * 4, RPI = 64 / CPR, TURNS = 32 / RPI;
    __shared__ __attribute__((aligned(16))) float slab[4][32 * ROW];
    static_assert(32 * ROW * 4 >= TN * 4096, "the slab is low_rank_expand's scratch first");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = lane >> 5, r = lane & 31;
    const int tiles_n = (N + TN * 64 - 1) / (TN * 64);
    const int b = xcd_remap(blockIdx.x, gridDim.x);
    const int mw = (b / tiles_n) * 64 + (wave & 1) * 32, nw = (b % tiles_n) * TN * 64 + (wave >> 1) * TN * 32;
    const int ch = lane % CPR * 8, row0 = lane / CPR;
    u32x4 old[TURNS];
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int m = mw + i * RPI + row0, n = nw + ch;
        old[i] = u32x4{0, 0, 0, 0};
        if (base && m < M && n < N) old[i] = ld16(base + int64_t(m) * ldb + n);
    }
    floatx16 acc[TN][1];
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) acc[tn][0] = floatx16{};
    __shared__ int32_t at[64];
    if (threadIdx.x < 64) at[threadIdx.x] = int(mw - (wave & 1) * 32 + threadIdx.x) < M ? index[mw - (wave & 1) * 32 + threadIdx.x] : -1;
    __syncthreads();
    if (nw < N) low_rank_expand<T, TN, 1, TRANS>(acc, up, low, at + (wave & 1) * 32, ranks, adapters, R, mw, nw, M, N,
                                            reinterpret_cast<uint8_t *>(slab[wave]));
#pragma unroll
    for (int tn = 0; tn < TN; ++tn)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const floatx4 v = {acc[tn][0][4 * q], acc[tn][0][4 * q + 1], acc[tn][0][4 * q + 2], acc[tn][0][4 * q + 3]};
            *reinterpret_cast<floatx4 *>(&slab[wave][r * ROW + tn * 32 + q * 8 + h * 4]) = v;
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TURNS; ++i) {
        const int m = mw + i * RPI + row0, n = nw + ch;
        if (m >= M || n >= N) continue;
        const float *s = &slab[wave][(i * RPI + row0) * ROW + ch];
        const typename Elem<T>::Vec o = __builtin_bit_cast(typename Elem<T>::Vec, old[i]);
        typename Elem<T>::Vec v;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = T(float(o[j]) + s[j]);
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v),
                                    reinterpret_cast<u32x4 *>(out + int64_t(m) * ldo + n));
    }
}

// ---- few tokens: one launch on the vector units.  A workgroup takes one token
// and 512 channels and computes the token's low values by itself (the pool row
// comes from L2 for every workgroup but the first), in fp32 throughout.
// base: T rows, or `splits` fp32 slices [M][N] of a split product, summed here.
template <class T, bool PARTS>
__global__ void __launch_bounds__(512)
tokens_kernel(const T *__restrict__ x, int64_t ldx, const T *__restrict__ down, const T *__restrict__ up,
              const float *__restrict__ scale, const int32_t *__restrict__ ranks, const int32_t *__restrict__ index,
              int adapters, int R, const void *base, int64_t ldb, int splits, T *out, int64_t ldo, int M, int N,
              int K) {
    __shared__ float low[128];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = blockIdx.y, n = blockIdx.x * 512 + threadIdx.x;
    const int a = index[m];
    const bool live = a >= 0 && a < adapters;
    const int rank = live ? low_rank_of(ranks, a, R) : 0;
    float sum = 0.0f;
    if (n < N) {
        if constexpr (PARTS) {
            for (int s = 0; s < splits; ++s)
                sum += static_cast<const float *>(base)[(int64_t(s) * M + m) * N + n];
        } else if (base) {
            sum = float(static_cast<const T *>(base)[int64_t(m) * ldb + n]);
        }
    }
    const T *xr = x + int64_t(m) * ldx;
    for (int r0 = wave * 2; r0 < rank; r0 += 16) {
        const T *d0 = down + (int64_t(a) * R + r0) * K, *d1 = d0 + (r0 + 1 < rank ? K : 0);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 2
        for (int k = lane * 8; k < K; k += 512) {
            float xv[8], v0[8], v1[8];
            to_float<T>(__builtin_bit_cast(typename Elem<T>::Vec, ld16(xr + k)), xv);
            to_float<T>(__builtin_bit_cast(typename Elem<T>::Vec, ld16(d0 + k)), v0);
            to_float<T>(__builtin_bit_cast(typename Elem<T>::Vec, ld16(d1 + k)), v1);
#pragma unroll
            for (int i = 0; i < 8; ++i) s0 = fmaf(xv[i], v0[i], s0), s1 = fmaf(xv[i], v1[i], s1);
        }
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        if (lane == 0) {
            const float c = scale ? scale[a] : 1.0f;
            low[r0] = s0 * c;
            if (r0 + 1 < rank) low[r0 + 1] = s1 * c;
        }
    }
    __syncthreads();
    if (n >= N) return;
    if (live) {
        const T *u = up + (int64_t(a) * N + n) * R;
#pragma unroll 2
        for (int r = 0; r < rank; r += 8) {
            float v[8];
            to_float<T>(__builtin_bit_cast(typename Elem<T>::Vec, ld16(u + r)), v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r + i < rank) sum = fmaf(v[i], low[r + i], sum);
        }
    } else if (a != -1) {
        sum = __builtin_nanf("");
    }
    out[int64_t(m) * ldo + n] = T(sum);
}

// ---- few tokens' input gradient, dx[m] = base[m] + down[a]^T . dlow[m]: expand
// takes a tile's adapters one after another, which for a tile of many requests is
// a chain of pool loads (32 tokens of 26 adapters, 512 wide: 29 us, here 4.1; 77 of
// 32 adapters, 2048 wide: 26 us, here 3.9).  Here a
// workgroup takes one token and 512 columns, its waves every fourth rank slot.
template <class T>
__global__ void __launch_bounds__(256)
tokens_dx_kernel(const T *__restrict__ down, const T *__restrict__ dlow, const int32_t *__restrict__ index,
                 const int32_t *__restrict__ ranks, int adapters, int R, const T *base, int64_t ldb, T *out,
                 int64_t ldo, int M, int K) {
    __shared__ __attribute__((aligned(16))) float part[3][512];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int m = blockIdx.y, k = blockIdx.x * 512 + lane * 8;
    const int a = index[m];
    const bool live = a >= 0 && a < adapters;
    const int rank = live ? low_rank_of(ranks, a, R) : 0;
    using Vec = typename Elem<T>::Vec;
    float sum[8] = {};
    int power = 0;
    if (k < K) {
        const int64_t plane = low_plane(M, R);
        if (kLowScaled<T> && rank > 0) power = low_exponent_of(ld16(dlow + low_at(m, 0, R) + plane));
#pragma unroll 4
        for (int r = wave; r < rank; r += 4) {
            const T *l = dlow + low_at(m, r & ~7, R) + (r & 7);
            uint16_t lo = __builtin_bit_cast(uint16_t, l[plane]);
            if (kLowScaled<T>) lo &= 0xfffeu;
            const float f = float(__builtin_bit_cast(T, lo)) + float(l[0]);
            float v[8];
            to_float<T>(__builtin_bit_cast(Vec, ld16(down + (int64_t(a) * R + r) * K + k)), v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(f, v[i], sum[i]);
        }
    }
    if (wave > 0) __builtin_memcpy(&part[wave - 1][lane * 8], sum, 32);
    __syncthreads();
    if (wave > 0 || k >= K) return;
    float b[8] = {};
    if (base) to_float<T>(__builtin_bit_cast(Vec, ld16(base + int64_t(m) * ldb + k)), b);
    Vec o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float s = ((sum[i] + part[0][lane * 8 + i]) + part[1][lane * 8 + i]) + part[2][lane * 8 + i];
        if (kLowScaled<T>) s = __builtin_amdgcn_ldexpf(s, power);
        o[i] = T(live || a == -1 ? b[i] + s : __builtin_nanf(""));
    }
    st16(out + int64_t(m) * ldo + k, __builtin_bit_cast(u32x4, o));
}

// ---- wgrad: out[r][c] = sum over adapter a's tokens of low[m][r] z[m][c], z
// [M][C] one of x (out = ddown [R][K]) and dy (out = dup [N][R]).
// A workgroup takes 128 columns of z and one range of tokens, and the range's
// distinct adapters one after another (so every workgroup has the same number of
// tokens, however they fall to adapters; where those are few workgroups, the
// adapters are dealt over several): it lists the adapter's tokens in LDS,
// then works through the list 32 tokens at a time, their z rows and low values
// copied to LDS as they lie in memory ([token][column]) and read by transposing
// LDS reads, which give each lane 8 consecutive tokens of one column (lane i of a
// 16-lane group receives element i%4 of the 8-byte run read by lane 4e + i/4, e =
// 0..3).  Three stages are in flight beside the one in use.  The high and the low
// part of `low` have accumulators of their own.  Ranges write fp32 slices
// [range][adapter][R][C] that a second launch sums in order, of the adapters
// only that the range has.
constexpr int kListCap = 2048;  // tokens listed at a time

// Zeros for a workgroup's tile of one adapter's gradient: 128 columns from c0.
template <class T>
__device__ __forceinline__ void zero_tile(T *o, bool rows_c, int c0, int C, int R) {
    const int n = min(128, C - c0);
    for (int i = threadIdx.x; i < n * R; i += 256) {
        if (rows_c) o[int64_t(c0) * R + i] = T(0.0f);
        else o[int64_t(i / n) * C + c0 + i % n] = T(0.0f);
    }
}

template <class T, int RB>
__global__ void __launch_bounds__(256)
wgrad_kernel(WgradTask<T> p, WgradTask<T> q, const int32_t *__restrict__ index, const int32_t *__restrict__ ranks,
             int adapters, int R, int M, int range, int32_t *__restrict__ present) {
    constexpr int RT = RB * 16;                  // rank slots of a stage row
    constexpr int Z_STAGE = 32 * 128 * 2;        // [32][128]
    constexpr int L_STAGE = 32 * RT * 2;         // [32][RT], one part
    constexpr int STAGE = Z_STAGE + 2 * L_STAGE;
    constexpr int NB = 4;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[NB * STAGE];
    __shared__ int32_t list[kListCap];
    __shared__ int counts[4][kListCap / 256];
    __shared__ int least[2][4];
    constexpr int TURNS = kListCap / 256;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool second = int(blockIdx.x) >= p.tiles;
    const WgradTask<T> &w = second ? q : p;
    const int c0 = (int(blockIdx.x) - (second ? p.tiles : 0)) * 128;
    const int C = w.C, slice = blockIdx.y;
    const int first = slice * range, last = min(first + range, M);
    // this workgroup's adapters: deal, deal + deals, ..
    const int deal = blockIdx.z, deals = gridDim.z;
    const bool marks = w.part && blockIdx.x == 0;
    if (marks)
        for (int a = deal + tid * deals; a < adapters; a += 256 * deals) present[int64_t(slice) * adapters + a] = 0;

    // this thread's tokens of the range's piece c (only a large pool's single range,
    // kept that long for its slices' size, has more than one)
    const int pieces = (last - first + kListCap - 1) / kListCap;
    // (fp16: low_key's adapters and powers of two, which the shrink has written; one after another
    // by power within an adapter)
    int mine[TURNS];
    auto adapter = [](int v) { return kLowScaled<T> ? v >> 8 : v; };
    auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int m = first + c * kListCap + i * 256 + tid;
            if constexpr (kLowScaled<T>) {
                mine[i] = m < last ? w.key[m] : -1;
            } else {
                mine[i] = m < last ? index[m] : -1;
                if (mine[i] >= adapters) mine[i] = -1;
            }
            if (deals > 1 && mine[i] >= 0 && adapter(mine[i]) % deals != deal) mine[i] = -1;
        }
    };
    fetch(0);
    const int g = lane >> 4, j16 = lane & 15;
    const int64_t plane = low_plane(M, R);
    const uint32_t smem_addr = lds_address(smem);
    const int per_stage = 2 + (2 * RB - wave + 3) / 4;  // loads of this wave
    constexpr int kNone = 0x7fffffff;
    floatx4 acc[2][RB][2];
    auto scale = [&](int e) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[s][b][0][i] = __builtin_amdgcn_ldexpf(acc[s][b][0][i], e);
                    acc[s][b][1][i] = __builtin_amdgcn_ldexpf(acc[s][b][1][i], e);
                }
    };
    // this workgroup's adapters below `next`, and entries of `mine` below `from`, are done;
    // acc: the sums of adapter `now`, times 2^-power
    int turn = 0, next = deal, from = 0, now = -1, power = 0;
    for (;; turn ^= 1) {
        // the least entry that is not done
        int a = kNone;
        for (int c = 0; c < max(pieces, 1); ++c) {
            if (pieces > 1) fetch(c);
#pragma unroll
            for (int i = 0; i < TURNS; ++i)
                if (mine[i] >= from) a = min(a, mine[i]);
        }
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) a = min(a, __shfl_xor(a, d, 64));
        if (lane == 0) least[turn][wave] = a;
        __syncthreads();
        a = min(min(least[turn][0], least[turn][1]), min(least[turn][2], least[turn][3]));
        a = __builtin_amdgcn_readfirstlane(a);
        const int id = a == kNone ? kNone : adapter(a);
        if constexpr (kLowScaled<T>) {
            // to their size at the adapter's end, else to the next tokens' (the sums so far are the smaller ones)
            const int shift = id != now ? power : power - low_key_power(a);
            if (now >= 0 && shift != 0) scale(shift);
        }
        if (now >= 0 && id != now) {
            const int rank = w.part ? R : low_rank_of(ranks, now, R);
            // lane: rank slots 16 b + 4 g + i of column c0 + 32 wave + 16 cb + j16.  (Its place is opaque,
            // so that the addresses are formed here and not kept through the products.)
            int place = lane;
            asm volatile("" : "+v"(place));
            const int g = place >> 4, j16 = place & 15;
#pragma unroll
            for (int b = 0; b < RB; ++b)
#pragma unroll
                for (int cb = 0; cb < 2; ++cb) {
                    const int c = c0 + wave * 32 + cb * 16 + j16, r = b * 16 + 4 * g;
                    if (c >= C || r >= R) continue;
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = acc[0][b][cb][i] + acc[1][b][cb][i];
                    const int64_t mat = int64_t(R) * C;
                    if (w.part) {
                        float *o = w.part + (int64_t(slice) * adapters + now) * mat;
                        if (w.rows_c) {
                            __builtin_memcpy(o + int64_t(c) * R + r, v, 16);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[int64_t(r + i) * C + c] = v[i];
                        }
                    } else {
                        // Slots past the rank hold sums of zeros (NaN where x is not finite) times a z that
                        // need not be finite.  (Ranges' slices are cleared where they are summed: masks
                        // among those stores took 1.5 to 4 of 32 us at 4096 x 1024, rank 128.)
                        int keep = rank - r;
                        asm volatile("" : "+v"(keep));  // (formed here: ahead, all blocks' masks took registers)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = i < keep ? v[i] : 0.0f;
                        T *o = w.out + int64_t(now) * mat;
                        if (w.rows_c) {
                            T t[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) t[i] = T(v[i]);
                            __builtin_memcpy(o + int64_t(c) * R + r, t, 8);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[int64_t(r + i) * C + c] = T(v[i]);
                        }
                    }
                }
        }
        if (id != now) {
            if (!w.part) {
                // the one range writes every adapter: zeros for those without tokens
                const int upto = id == kNone ? adapters : id;
                for (int z = next; z < upto; z += deals) zero_tile(w.out + int64_t(z) * R * C, w.rows_c, c0, C, R);
            }
            if (id == kNone) return;
            next = id + deals;
            if (marks && tid == 0) present[int64_t(slice) * adapters + id] = 1;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int b = 0; b < RB; ++b) acc[s][b][0] = acc[s][b][1] = floatx4{0.f, 0.f, 0.f, 0.f};
        }
        now = id;
        from = a + 1;
        if constexpr (kLowScaled<T>) power = low_key_power(a);

        for (int c = 0; c < pieces; ++c) {
            // its tokens of the piece, in order
            if (pieces > 1) fetch(c);
            int total = 0;
            {
                uint64_t votes[TURNS];
#pragma unroll
                for (int i = 0; i < TURNS; ++i) {
                    votes[i] = __ballot(mine[i] == a);
                    if (lane == 0) counts[wave][i] = __builtin_popcountll(votes[i]);
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < TURNS; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        if (v == wave && mine[i] == a)
                            list[total + __builtin_popcountll(votes[i] & ((uint64_t(1) << lane) - 1))] =
                                first + c * kListCap + i * 256 + tid;
                        total += counts[v][i];
                    }
                __syncthreads();
            }
            total = __builtin_amdgcn_readfirstlane(total);

            // Direct-to-LDS loads of a stage: 8 KiB of z (row = 4 q + lane/16, 16-byte
            // chunk lane%16, swizzled), then 2 * RB KiB of low.
            auto issue = [&](int s) {
                uint8_t *base = smem + (s % NB) * STAGE;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int qq = j * 4 + wave, row = 4 * qq + g;
                    const int at = s * 32 + row, col = c0 + (j16 ^ (2 * (row & 3))) * 8;
                    const void *src = g_low_zero;
                    if (at < total && col < C) src = w.z + int64_t(list[at]) * w.ldz + col;
                    tw_dma16(src, base + qq * 1024);
                }
                for (int qq = wave; qq < 2 * RB; qq += 4) {
                    const int part = qq / RB, byte = (qq % RB) * 1024 + lane * 16;
                    const int row = byte / (RT * 2), r = byte % (RT * 2) / 2;
                    const int at = s * 32 + row;
                    const void *src = g_low_zero;
                    if (at < total && r < R) src = w.low + part * plane + low_at(list[at], r, R);
                    tw_dma16(src, base + Z_STAGE + qq * 1024);
                }
            };
            const int S = (total + 31) / 32;
            for (int s = 0; s < NB - 1 && s < S; ++s) issue(s);
            for (int s = 0; s < S; ++s) {
                // stage s has landed (younger ones may be in flight), and everyone is done with stage s - 1
                tw_wait_barrier(min(NB - 2, S - 1 - s) * per_stage);
                if (s + NB - 1 < S) issue(s + NB - 1);
                const uint32_t base = smem_addr + (s % NB) * STAGE;
                const int row = 8 * g + (j16 >> 2);
                uint32_t z_at[2];
#pragma unroll
                for (int cb = 0; cb < 2; ++cb) {
                    const int col = wave * 32 + cb * 16 + 4 * (j16 & 3);
                    z_at[cb] = base + row * 256 + ((col >> 3) ^ (2 * (row & 3))) * 16 + (col & 7) * 2;
                }
                const uint32_t l_at = base + Z_STAGE + row * (RT * 2) + 4 * (j16 & 3) * 2;
                u32x4 zv[2], lv[2][RB];
                read_tr(z_at[0], z_at[0] + 1024, z_at[1], z_at[1] + 1024, zv[0], zv[1]);
#pragma unroll
                for (int b = 0; b < RB; ++b) {
                    const uint32_t hi = l_at + b * 32, lo = hi + L_STAGE;
                    read_tr(hi, hi + RT * 8, lo, lo + RT * 8, lv[0][b], lv[1][b]);
                    lv[1][b] = lo_value<T>(lv[1][b]);
                }
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int b = 0; b < RB; ++b)
#pragma unroll
                        for (int cb = 0; cb < 2; ++cb) acc[part][b][cb] = mfma16<T>(lv[part][b], zv[cb], acc[part][b][cb]);
            }
        }
    }
}

// Sums the ranges' slices of the adapters that the ranges have, in order, and
// rounds once: one adapter a grid row, 4 values a thread (ddown [R][K], then dup
// [N][R]).  Slots past the rank get zeros.
template <class T>
__global__ void __launch_bounds__(256)
wgrad_sum_kernel(const float *__restrict__ part0, T *__restrict__ out0, int64_t n0, const float *__restrict__ part1,
                 T *__restrict__ out1, int64_t n1, int slices, const int32_t *__restrict__ present, int adapters,
                 const int32_t *__restrict__ ranks, int R, int K) {
    const int a = blockIdx.y, lane = threadIdx.x & 63;
    int64_t i = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;  // in the adapter's n0, then n1 values
    const bool second = i >= n0;
    const int64_t n = second ? n1 : n0;
    const float *part = second ? part1 : part0;
    T *out = second ? out1 : out0;
    if (second) i -= n0;
    const bool live = i < n;
    floatx4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int q0 = 0; q0 < slices; q0 += 64) {
        uint64_t has = __ballot(q0 + lane < slices && present[int64_t(q0 + lane) * adapters + a] != 0);
        while (has) {
            // four slices' loads at a time
            floatx4 v[4];
            int got = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
                if (!has) continue;
                const int q = q0 + __builtin_ctzll(has);
                has &= has - 1;
                got = u + 1;
                if (live) v[u] = *reinterpret_cast<const floatx4 *>(part + (int64_t(q) * adapters + a) * n + i);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (u < got) s.x += v[u].x, s.y += v[u].y, s.z += v[u].z, s.w += v[u].w;
        }
    }
    if (!live) return;
    const int rank = low_rank_of(ranks, a, R);
    if (rank < R) {  // ddown's first rank * K values are in use; in dup, 4 values lie in one row of R
        const int keep = second ? rank - int(i % R) : i < int64_t(rank) * K ? 4 : 0;
        s.x = keep > 0 ? s.x : 0.0f, s.y = keep > 1 ? s.y : 0.0f;
        s.z = keep > 2 ? s.z : 0.0f, s.w = keep > 3 ? s.w : 0.0f;
    }
    T t[4] = {T(s.x), T(s.y), T(s.z), T(s.w)};
    __builtin_memcpy(out + int64_t(a) * n + i, t, 8);
}

// One task, or the gradient's two (the first on the pool's other side).
template <class T, bool BOTH>
hipError_t shrink(const ShrinkTask<T> &p, const ShrinkTask<T> &q, const LowRank &lr, int M, hipStream_t st) {
    constexpr int NW = 8;
    // With few tiles, a tile's pairs of adapters (eight at most) are dealt over
    // workgroups: 32 tokens of 26 adapters, 512 wide, 14.7 -> 5.7 us, 77 tokens of 32
    // adapters, 2048 wide, 24.5 -> 9.3 us.
    const int nb = (M + 15) / 16 * (BOTH ? 2 : 1);
    const dim3 grid((M + 15) / 16, BOTH ? 2 : 1, nb <= 32 ? 8 : nb <= 128 ? 256 / nb : 1);
#define SSG_SHRINK(RB)                                                                                              \
    hipLaunchKernelGGL((shrink_kernel<T, RB, NW, BOTH>), grid, dim3(NW * 64), 0, st, p, q, lr.scale, lr.ranks,      \
                       lr.index, lr.adapters, lr.R, M)
    if (lr.R <= 16) SSG_SHRINK(1);
    else if (lr.R <= 32) SSG_SHRINK(2);
    else if (lr.R <= 64) SSG_SHRINK(4);
    else SSG_SHRINK(8);
#undef SSG_SHRINK
    return hipGetLastError();
}

template <class T, bool TRANS>
hipError_t expand(const T *up, const T *low, const LowRank &lr, const void *base, int64_t ldb, void *out, int64_t ldo,
                  int M, int N, hipStream_t st) {
    const int nb = (M + 63) / 64 * ((N + kExpandTN * 64 - 1) / (kExpandTN * 64));
    hipLaunchKernelGGL((expand_kernel<T, TRANS>), dim3(nb), dim3(256), 0, st, up, low, lr.index, lr.ranks, lr.adapters, lr.R,
                       static_cast<const T *>(base), ldb, static_cast<T *>(out), ldo, M, N);
    return hipGetLastError();
}

template <class T>
hipError_t add(const LowRank &lr, const void *x, int64_t ldx, const void *base, int64_t ldb, void *out, int64_t ldo,
               int M, int N, int K, void *ws, hipStream_t st) {
    T *low = static_cast<T *>(ws);
    if (low_rank_few(M)) return launch_low_rank_tokens(lr, x, ldx, base, ldb, 0, out, ldo, M, N, K, st);
    const ShrinkTask<T> p{static_cast<const T *>(x), ldx, static_cast<const T *>(lr.down), low, K, nullptr};
    const hipError_t e = shrink<T, false>(p, p, lr, M, st);
    if (e != hipSuccess) return e;
    return expand<T, false>(static_cast<const T *>(lr.up), low, lr, base, ldb, out, ldo, M, N, st);
}

template <class T>
hipError_t bwd(const LowRankBwd &b, hipStream_t st) {
    const LowRank &lr = b.lr;
    const int M = b.M, N = b.N, K = b.K, R = lr.R;
    const LowRankPlan pl = low_rank_plan(lr.adapters, R, M, N, K);
    uint8_t *ws = static_cast<uint8_t *>(b.ws);
    T *low = reinterpret_cast<T *>(ws + pl.low), *dlow = reinterpret_cast<T *>(ws + pl.dlow);
    int32_t *keys = reinterpret_cast<int32_t *>(ws + pl.keys);  // dy's tokens, then x's
    hipError_t e;
    if (M > 0) {
        const ShrinkTask<T> p{static_cast<const T *>(b.dy), b.lddy, static_cast<const T *>(lr.up), dlow, N, keys};
        const ShrinkTask<T> q{static_cast<const T *>(b.x), b.ldx, static_cast<const T *>(lr.down), low, K, keys + M};
        if ((e = shrink<T, true>(p, q, lr, M, st)) != hipSuccess) return e;
        if (low_rank_few(M)) {
            hipLaunchKernelGGL((tokens_dx_kernel<T>), dim3((K + 511) / 512, M), dim3(256), 0, st,
                               static_cast<const T *>(lr.down), dlow, lr.index, lr.ranks, lr.adapters, R,
                               static_cast<const T *>(b.base), b.ldb, static_cast<T *>(b.dx), b.lddx, M, K);
            e = hipGetLastError();
        } else {
            e = expand<T, true>(static_cast<const T *>(lr.down), dlow, lr, b.base, b.ldb, b.dx, b.lddx, M, K, st);
        }
        if (e != hipSuccess) return e;
    }
    const int64_t n0 = int64_t(lr.adapters) * R * K, n1 = int64_t(lr.adapters) * R * N;
    float *part0 = pl.slices > 1 ? reinterpret_cast<float *>(ws + pl.part) : nullptr;
    float *part1 = part0 ? part0 + pl.slices * n0 : nullptr;
    int32_t *counts = reinterpret_cast<int32_t *>(ws + pl.counts);
    const WgradTask<T> p{static_cast<const T *>(b.x), b.ldx, dlow, part0, static_cast<T *>(b.ddown), K, (K + 127) / 128,
                         false, keys};
    const WgradTask<T> q{static_cast<const T *>(b.dy), b.lddy, low, part1, static_cast<T *>(b.dup), N, (N + 127) / 128,
                         true, keys + M};
    const dim3 grid(p.tiles + q.tiles, pl.slices, pl.deals);
#define SSG_WGRAD(RB) \
    hipLaunchKernelGGL((wgrad_kernel<T, RB>), grid, dim3(256), 0, st, p, q, lr.index, lr.ranks, lr.adapters, R, M, pl.range, \
                       counts)
    if (R <= 16) SSG_WGRAD(1);
    else if (R <= 32) SSG_WGRAD(2);
    else if (R <= 64) SSG_WGRAD(4);
    else SSG_WGRAD(8);
#undef SSG_WGRAD
    if ((e = hipGetLastError()) != hipSuccess || pl.slices == 1) return e;
    const int64_t m0 = int64_t(R) * K, m1 = int64_t(R) * N;  // values of one adapter
    hipLaunchKernelGGL((wgrad_sum_kernel<T>), dim3(int(((m0 + m1) / 4 + 255) / 256), lr.adapters), dim3(256), 0, st,
                       part0, static_cast<T *>(b.ddown), m0, part1, static_cast<T *>(b.dup), m1, pl.slices, counts,
                       lr.adapters, lr.ranks, R, K);
    return hipGetLastError();
}

}  // namespace

int64_t low_rank_bytes(int64_t M, int R) { return low_plane(M, R) * 4; }

// Few tokens: one launch on the vector units (in the gradient, dx by token).  The
// tiled form takes a tile's adapters one after another, each a chain of waits; the
// tokens' form computes a token's low values again for every 512 channels.  Both, us a
// call by graph, fp16, K = N, tokens / tiled:
//   width  adapters  rank    32 tokens    64           128          256          512
//   1024   32        16      18 / 35      16 / 35      16 / 28      17 / 24      17 / 22
//   1024   1         128     19 / 21      20 / 22      21 / 22      28 / 22      49 / 22
//   4096   32        16      16 / 39      16 / 39      18 / 34      25 / 31      39 / 30
//   4096   32        128     41 / 135     73 / 148     110 / 119    186 / 93     301 / 78
//   4096   1         16      16 / 19      17 / 19      17 / 18      24 / 18      39 / 19
//   4096   1         128     29 / 30      46 / 30      86 / 30      161 / 33     309 / 35
//   4096   32        16, 2:4       22 / 76      25 / 81      31 / 76      47 / 73      67 / 52
//   4096   1         128, 2:4      42 / 71      59 / 73      103 / 73     184 / 73     333 / 55
//   4096   32        128, gradient 126 / 204    132 / 219    133 / 194    140 / 174    221 / 231
//   4096   1         128, gradient  49 / 50      51 / 53      62 / 60      75 / 67      90 / 72
// 128 is where they meet for many adapters of a high rank and for one of a low rank.
// It loses from 64 tokens on for one adapter of rank 64 and more at 4096 wide, and
// above 128 for many of a low rank: how many adapters the tokens have is not known
// here, and the workspace's size, which follows the form, depends on M and R alone.
bool low_rank_few(int M) { return M <= 128; }

LowRankPlan low_rank_plan(int adapters, int R, int64_t M, int64_t N, int64_t K) {
    auto up256 = [](int64_t v) { return (v + 255) / 256 * 256; };
    LowRankPlan p;
    p.low = 0;
    p.dlow = p.low + up256(low_plane(M, R) * 4);
    p.keys = p.dlow + up256(low_plane(M, R) * 4);
    p.part = p.keys + up256(2 * M * 4);
    // Token ranges: the workgroups that the CUs hold at once (by LDS), of at least
    // 256 tokens and at most what the list holds, in at most 256 MiB of slices;
    // one range if a large pool's slices do not fit.
    const int64_t cols = (N + 127) / 128 + (K + 127) / 128;
    const int64_t slots = 256 * (R <= 16 ? 3 : R <= 64 ? 2 : 1);
    const int64_t slice = int64_t(adapters) * R * (N + K) * 4;
    int64_t want = slots / cols > 0 ? slots / cols : 1;
    const int64_t most = M > 256 ? M / 256 : 1;
    if (want > most) want = most;
    const int64_t fit = (int64_t(256) << 20) / slice, cap = (M + kListCap - 1) / kListCap;
    if (want < cap) want = cap;
    if (want > fit) want = fit < cap ? 1 : fit;  // (one range if those of the list's length do not fit)
    int64_t range = want > 0 ? (M + want - 1) / want : M;
    range = (range + 31) / 32 * 32;
    if (want > 1 && range > kListCap) range = kListCap;
    if (range < 32) range = 32;
    p.range = int(range);
    p.slices = int(M > 0 ? (M + range - 1) / range : 1);
    // few workgroups: the adapters are dealt over more of them (fp16 32 tokens,
    // 512 x 136, rank 24, 26 adapters: the call 101 -> 45 us)
    const int64_t deals = slots / (cols * p.slices);
    p.deals = int(deals < 1 ? 1 : deals > adapters ? adapters : deals);
    p.counts = p.part;
    p.part += up256(int64_t(p.slices) * adapters * 4);
    p.total = p.part + (p.slices > 1 ? p.slices * slice : 0);
    return p;
}

hipError_t launch_low_rank_tokens(const LowRank &lr, const void *x, int64_t ldx, const void *base, int64_t ldb,
                                  int splits, void *out, int64_t ldo, int M, int N, int K, hipStream_t st) {
    const dim3 grid((N + 511) / 512, M);
#define SSG_TOK(T, PARTS)                                                                                            \
    hipLaunchKernelGGL((tokens_kernel<T, PARTS>), grid, dim3(512), 0, st, static_cast<const T *>(x), ldx,            \
                       static_cast<const T *>(lr.down), static_cast<const T *>(lr.up), lr.scale, lr.ranks, lr.index, \
                       lr.adapters, lr.R, base, ldb, splits, static_cast<T *>(out), ldo, M, N, K)
    if (lr.dtype == DT_F16) {
        if (splits > 0) SSG_TOK(_Float16, true);
        else SSG_TOK(_Float16, false);
    } else {
        SSG_TOK(__bf16, false);
    }
#undef SSG_TOK
    return hipGetLastError();
}

hipError_t launch_low_rank_shrink(const LowRank &lr, const void *x, int64_t ldx, void *low, int M, int K,
                                  hipStream_t st) {
    if (lr.dtype == DT_F16) {
        using T = _Float16;
        const ShrinkTask<T> p{static_cast<const T *>(x), ldx, static_cast<const T *>(lr.down), static_cast<T *>(low), K, nullptr};
        return shrink<T, false>(p, p, lr, M, st);
    }
    using T = __bf16;
    const ShrinkTask<T> p{static_cast<const T *>(x), ldx, static_cast<const T *>(lr.down), static_cast<T *>(low), K, nullptr};
    return shrink<T, false>(p, p, lr, M, st);
}

hipError_t launch_low_rank_add(const LowRank &lr, const void *x, int64_t ldx, const void *base, int64_t ldb, void *out,
                               int64_t ldo, int M, int N, int K, void *ws, hipStream_t st) {
    return lr.dtype == DT_F16 ? add<_Float16>(lr, x, ldx, base, ldb, out, ldo, M, N, K, ws, st)
                              : add<__bf16>(lr, x, ldx, base, ldb, out, ldo, M, N, K, ws, st);
}

hipError_t launch_low_rank_bwd(const LowRankBwd &b, hipStream_t st) {
    return b.lr.dtype == DT_F16 ? bwd<_Float16>(b, st) : bwd<__bf16>(b, st);
}

}  // namespace ssg

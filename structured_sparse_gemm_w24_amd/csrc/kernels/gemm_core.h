// The skeleton of the dense and 2:4-sparse GEMM kernels for gfx950.
//
// C[M][N] = A[M][K] . W[K][N].  The 2:4 kinds read W from its compressed
// form (two kept values per group of four along K plus 2-bit positions,
// GPUSQ-ViT "Boost Vision Transformer with GPU-Friendly Sparsity and
// Quantization", abstract) and feed the gfx950 sparse matrix instructions,
// whose sparse operand is the instruction's row operand.  W's sparsity runs
// along K inside an output column, so the kernels compute the transposed
// product C^T = W^T . A^T: instruction rows are output channels n (sparse
// operand: kept values of W^T row n), instruction columns are tokens m
// (dense operand: a row of A, K contiguous).  The hardware selects, per kept
// value, the matching activation by the 2-bit position; no software gather
// of A is needed.  The dense kinds run the same skeleton with the dense
// instruction so that the sparse-vs-dense comparison isolates the matrix
// instruction.
//
// Work decomposition
//   * workgroup = WM x WN waves (8 for the large tiles: two per SIMD); tile =
//     BM tokens x BN channels; every wave owns TM x TN 32x32 blocks
//     (BM = 32*WM*TM, BN = 32*WN*TN);
//   * K advances in stages of 128 bytes of an A row (f16: 64 k, i8: 128 k);
//     every stage is copied global -> LDS with direct-to-LDS loads (no
//     register staging) into a ring of STAGES buffers: stage s+STAGES is
//     fetched while stage s+1 is read into registers and stage s feeds the
//     matrix cores.  One explicit wait on the vector-memory counter plus one
//     barrier per stage hand a stage over;
//   * the sparse kinds' metadata either travels with each stage or, on the
//     tiles that use it, is fetched in blocks of several stages into a ring
//     of its own (fewer, longer row segments per load);
//   * on some tiles (SmallP, the sparse T64N) a second group of waves does
//     all the loading and the compute waves only read LDS and issue matrix
//     instructions; both groups meet at the same per-stage barrier;
//   * fragments are double-buffered in registers: the LDS reads of the next
//     k-step are issued between the matrix instructions of the current one
//     (scheduling hints interleave them), so one wave per SIMD keeps its
//     matrix pipe busy without waiting on LDS latency;
//   * LDS rows are XOR-swizzled in 16-byte chunks so that the rows read by one
//     fragment load fall into distinct banks; the direct-to-LDS lane order is
//     fixed (lane i writes bytes 16i..16i+15 of the wave's 1 KiB), so each lane
//     fetches the global chunk that belongs at its swizzled position;
//   * block ids are remapped so each XCD works on a contiguous range of tiles
//     (grouped GM tile-rows at a time), which keeps shared A rows and W
//     columns in that XCD's L2;
//   * epilogue: the accumulators go through LDS as row-major [token][channel]
//     slabs, so C is written as whole contiguous row segments, 16 bytes per
//     lane (fp16 kinds: fp16 rounded to nearest even; int8 kinds: raw int32,
//     or y = float(acc) * scale[n] (+ bias[n]) written as fp32, as fp16
//     rounded to nearest even, or as int8 rounded to nearest even and
//     saturated to [-128, 127]);
//   * a tile starts its K loop at stage 0 or, for the sparse 128 x 128 and
//     64 x 128 tiles, at a stage rotated by its tile id (measured per tile
//     shape, see ROT);
//   * split K (gridDim.y > 1, EPI_PART): workgroup (tile, y) runs K-stage range
//     y and writes its raw accumulators to slice y of a workspace, which
//     splitk.hip sums and finishes with the kind's epilogue.
//
// Instruction operand layouts (64-lane wave, h = lane / 32, r = lane % 32):
//   dense f16 32x32x16 : row-op lane holds k = 8h .. 8h+7 of its row r
//   dense i8  32x32x32 : k = 16h .. 16h+15
//   sparse f16 32x32x32: sparse row-op lane holds the 8 kept values of row r
//                        for k in [16h, 16h+16) (4 groups, ascending), slot c's
//                        two-bit position at bits 2c of the index operand; the
//                        dense column-op lane holds, as elements 0..7 and
//                        8..15, k = 8h .. 8h+7 and k = 16+8h .. 16+8h+7 of
//                        column r (measured on gfx950 with one-wave probes)
//   sparse i8 32x32x64 : sparse lane: 16 kept values for k in [32h, 32h+32),
//                        16 positions = 32 index bits; dense lane: elements
//                        0..15 = k 16h .., elements 16..31 = k 32+16h ..
//   accumulator        : lane holds rows 8*(i/4) + 4h + i%4 (i = 0..15) of
//                        column r
// The compressed pack stores slot j's position at bits 2*(j%16) of word j/16,
// which is exactly the index operand for these ranges, so meta words are fed
// to the instruction as stored (shifted by 16 bits for the upper f16 half).
#pragma once

#include "common.h"

namespace ssg {

// (DENSE_BF16 is used by the linear cross entropy and the experts' products,
// MX_F4 by the products of microscaled 4-bit operands.)
enum Kind { DENSE_F16 = 0, W24_F16 = 1, DENSE_I8 = 2, W24_I8 = 3, DENSE_BF16 = 4, MX_F4 = 5 };
// EPI_F16: fp16 kinds.  int8 kinds: EPI_I32 raw accumulators; the others
// compute y = float(acc) * scale[n] (+ bias[n]), each step rounded to nearest
// even, then store y as fp32, fp16 or saturated int8.  EPI_PART (split K, any
// kind): the raw accumulators (fp32 or int32) of K-split blockIdx.y go to its
// [M][N] slice of the workspace passed as C; a second kernel sums the slices.
// EPI_BF16, EPI_F32: the accumulators rounded to bf16, or as they are.
enum Epi {
    EPI_F16 = 0,
    EPI_I32 = 1,
    EPI_F32_SCALE = 2,
    EPI_F16_SCALE = 3,
    EPI_I8_SCALE = 4,
    EPI_PART = 5,
    EPI_BF16 = 6,
    EPI_F32 = 7
};

template <int KIND>
struct KindTraits;

template <>
struct KindTraits<DENSE_F16> {
    static constexpr bool kSparse = false, kI8 = false;
    static constexpr int kWB = 128;  // W bytes per row per stage
    static constexpr int kMW = 0;    // meta words per row per stage
    static constexpr int kNI = 4;    // instructions per stage
};
template <>
struct KindTraits<DENSE_BF16> : KindTraits<DENSE_F16> {};
// 4-bit values: a stage is 256 k; both operands bring 8 scale bytes a row (two words), one byte per 32 k.
template <>
struct KindTraits<MX_F4> : KindTraits<DENSE_F16> {};
template <>
struct KindTraits<W24_F16> {
    static constexpr bool kSparse = true, kI8 = false;
    static constexpr int kWB = 64, kMW = 2, kNI = 2;
};
template <>
struct KindTraits<DENSE_I8> {
    static constexpr bool kSparse = false, kI8 = true;
    static constexpr int kWB = 128, kMW = 0, kNI = 4;
};
template <>
struct KindTraits<W24_I8> {
    static constexpr bool kSparse = true, kI8 = true;
    static constexpr int kWB = 64, kMW = 4, kNI = 2;
};

// 16-byte chunk swizzles (see header comment).
__device__ __forceinline__ int swz128(int row, int col) { return col ^ ((row ^ (row >> 3)) & 7); }
__device__ __forceinline__ int swz256(int row, int col) { return col ^ (row & 15); }
__device__ __forceinline__ int swz64(int row, int col) { return col ^ (((row >> 1) ^ (row >> 3)) & 3); }
// swizzle of a row of RB bytes (64, 128 or 256)
template <int RB>
__device__ __forceinline__ int swzw(int row, int col) {
    if constexpr (RB == 64) return swz64(row, col);
    else if constexpr (RB == 128) return swz128(row, col);
    else return swz256(row, col);
}

template <int KIND>
struct AccOf {
    using T = typename std::conditional<KindTraits<KIND>::kI8, intx16, floatx16>::type;
};

__device__ __forceinline__ u32x4 lds16(const uint8_t *p) { return *reinterpret_cast<const u32x4 *>(p); }

typedef __attribute__((address_space(3))) void *lds_ptr_t;

// Direct-to-LDS loads through a buffer resource: lane i of the wave reads
// 16 (4) bytes at byte offset `off` of the buffer and writes them to
// wave_base + 16*i (4*i); wave_base must be uniform across the wave.  The
// buffer form moves a few per cent more per wave than the flat-address form
// (L2 → LDS microbenchmark on MI355X), and reads past the buffer's size
// return zeros instead of faulting.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, int(bytes), 0x00020000);
}
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint8_t *wave_base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)wave_base, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t off, uint8_t *wave_base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)wave_base, 4, off, 0, 0, 0);
}

// Waits until at most N vector-memory operations of this wave are
// outstanding, then synchronises the workgroup (no memory fence: LDS data
// here is produced by direct-to-LDS loads, which the counter tracks).
template <int N>
__device__ __forceinline__ void wait_vm_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}
// Same, after this wave's LDS reads have completed as well.
template <int N>
__device__ __forceinline__ void wait_lgkm_vm_barrier() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));

// Stores the first `room` elements of OB bytes (all 16 / OB, or fewer at a row's end; none
// below 1) at any element alignment.
template <int OB>
__device__ __forceinline__ void store_piece(uint8_t *p, u32x4 v, int room, bool stream) {
    typedef u32x4 Any __attribute__((aligned(2)));
    if (room >= 16 / OB) {
        if (stream) __builtin_nontemporal_store(v, reinterpret_cast<Any *>(p));
        else *reinterpret_cast<Any *>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 16 / OB - 1; ++i) {
        if (i >= room) break;
        if constexpr (OB == 4) reinterpret_cast<uint32_t *>(p)[i] = v[i];
        else reinterpret_cast<uint16_t *>(p)[i] = uint16_t(v[i / 2] >> (16 * (i % 2)));
    }
}

// One matrix instruction.  w: the row operand (kept W^T values, or dense W^T
// for the dense kinds); a: the column operand (activations).  For the sparse
// kinds a holds 32 bytes; the dense kinds use its low 16 bytes.
template <int KIND>
__device__ __forceinline__ void mma(typename AccOf<KIND>::T &acc, u32x4 w, u32x8 a, uint32_t idx) {
    if constexpr (KIND == W24_F16) {
        acc = __builtin_amdgcn_smfmac_f32_32x32x32_f16(__builtin_bit_cast(half8, w), __builtin_bit_cast(half16, a),
                                                        acc, int(idx), 0, 0);
    } else if constexpr (KIND == W24_I8) {
        acc = __builtin_amdgcn_smfmac_i32_32x32x64_i8(__builtin_bit_cast(intx4, w), __builtin_bit_cast(intx8, a), acc,
                                                       int(idx), 0, 0);
    } else if constexpr (KIND == DENSE_F16) {
        const u32x4 lo = __builtin_shufflevector(a, a, 0, 1, 2, 3);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, w), __builtin_bit_cast(half8, lo), acc,
                                                      0, 0, 0);
    } else if constexpr (KIND == DENSE_BF16) {
        const u32x4 lo = __builtin_shufflevector(a, a, 0, 1, 2, 3);
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, lo),
                                                       acc, 0, 0, 0);
    } else {
        const u32x4 lo = __builtin_shufflevector(a, a, 0, 1, 2, 3);
        acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(intx4, w), __builtin_bit_cast(intx4, lo), acc,
                                                     0, 0, 0);
    }
}

// The microscaled 4-bit instruction: 32 x 32 x 64, lane (h, r) holds k = 32h .. 32h+31 of its
// row r, i.e. one block, whose scale is byte OP of its scale word.
template <int OP>
__device__ __forceinline__ void mma_f4(floatx16 &acc, u32x4 w, u32x4 a, uint32_t sw, uint32_t sa) {
    const intx4 wi = __builtin_bit_cast(intx4, w), ai = __builtin_bit_cast(intx4, a);
    constexpr int kF4 = 4;  // operand format: E2M1
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        __builtin_shufflevector(wi, wi, 0, 1, 2, 3, 0, 1, 2, 3), __builtin_shufflevector(ai, ai, 0, 1, 2, 3, 0, 1, 2, 3),
        acc, kF4, kF4, OP, int(sw), OP, int(sa));
}

// Epilogue store of one 16-byte piece; nontemporal stores stream past L2.
template <bool NTS>
__device__ __forceinline__ void store16(void *p, u32x4 v) {
    if constexpr (NTS) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
    else *reinterpret_cast<u32x4 *>(p) = v;
}

// Tile configuration: WM x WN waves, TM x TN 32x32 blocks per wave, STAGES
// LDS stage buffers (prefetch distance), GM tile-rows per L2 group,
// nontemporal C stores, ROT: each tile starts its K loop at its own stage.
// By default every wave issues an equal share of each stage's direct-to-LDS
// loads.
// MP: K stages per metadata block of the sparse kinds (0: each stage's
// metadata travels with the stage).  PROD: the workgroup has as many
// loader waves as compute waves; the loader waves issue every direct-to-LDS
// load and the compute waves only read LDS and run the matrix instructions.
// NLD (without PROD): only compute waves 0..NLD-1 issue the loads (0: all).
// DK: K depth of a stage in units of 128 bytes of an A row.
template <int WM_, int WN_, int TM_, int TN_, int STAGES_, int GM_, bool NTS_, bool ROT_, int MP_ = 0,
          bool PROD_ = false, int NLD_ = 0, int DK_ = 1>
struct Cfg {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, STAGES = STAGES_, GM = GM_;
    static constexpr bool NTS = NTS_, ROT = ROT_, PROD = PROD_;
    static constexpr int MP = MP_, NLD = NLD_, DK = DK_;
    static constexpr bool DEEP = false;
};
// Four waves of 128 x 128 on a 256 x 256 tile (or TM x TN blocks each), a whole stage's fragments in
// registers.
template <int TM_, int TN_, int GM_, bool NTS_>
struct CfgDeep : Cfg<2, 2, TM_, TN_, 2, GM_, NTS_, false> {
    static constexpr bool DEEP = true;
};

template <int KIND, class CF>
struct Layout {
    using KT = KindTraits<KIND>;
    static constexpr int NW = CF::WM * CF::WN;           // compute waves (and loader waves)
    static constexpr int NT = NW * kWave * (CF::PROD ? 2 : 1);  // threads
    static constexpr int BM = CF::WM * CF::TM * 32;
    static constexpr int BN = CF::WN * CF::TN * 32;
    static constexpr int DK = CF::DK;
    static constexpr int AB = 128 * DK;      // A bytes per row per stage
    static constexpr int NI = KT::kNI * DK;  // matrix instructions (k-steps) per stage
    static constexpr int WB = KT::kWB * DK;
    static constexpr int MW = KT::kMW * DK;
    static constexpr int A_STAGE = BM * AB;
    static constexpr int W_STAGE = BN * WB;
    static constexpr int M_BYTES = BN * MW * 4;  // metadata bytes of one stage
    // Metadata blocks (MP > 0): the metadata of MP consecutive stages sits
    // in one block of its own ring instead of in the stage buffers, stored
    // row-major [BN][MP * MW] words, so that every 256-byte load covers
    // MP * MW * 4 contiguous bytes of a row (8 rows) rather than 8 or 16
    // bytes of 32 or 16 rows: the loads touch MP times fewer cache lines.
    // A block is fetched in MP parts, one with each of the MP stage loads
    // before its first stage; MSLOTS blocks are kept so that a part never
    // overwrites a block that a stage still in the ring reads.
    static constexpr int MP = KT::kSparse ? CF::MP : 0;
    static constexpr int M_STAGE = MP ? 0 : M_BYTES;
    static constexpr int STAGE = A_STAGE + W_STAGE + M_STAGE;
    // MX_F4: scale blocks, the scales of two stages, 16 bytes a row, A's rows then W's, in a ring of
    // three behind the stages.  Block c is fetched in two parts with the loads of stages 2c - 1 and 2c.
    // (Fetched stage by stage they are 8 bytes a row, so as many cache lines as all the codes: 8192^3
    // on the 256 x 256 tile 310 us, without any scales 279.)  In chunks of 64 rows; waves past a part's
    // last chunk fetch it once more, so that all issue alike.
    static constexpr int S_AROWS = (BM + 63) / 64 * 64;
    static constexpr int S_CHUNKS = KIND == MX_F4 ? S_AROWS / 64 + (BN + 63) / 64 : 0;
    static constexpr int S_PART = (S_CHUNKS + 1) / 2;
    static constexpr int S_BLOCK = S_CHUNKS * 1024;
    static constexpr int S_RING = 3 * S_BLOCK;
    static_assert(S_CHUNKS == 0 || DK == 1, "scale blocks are of two stages of 256 k");
    static constexpr int RW = MP * MW;  // words per row in a block
    static constexpr int MBLK = MP * M_BYTES;
    static constexpr int MSLOTS = MP ? 2 + (CF::STAGES - 2 + MP - 1) / MP : 0;
    static constexpr int MRING = MSLOTS * MBLK;
    static_assert(MP == 0 || (64 % RW == 0 && BN % MP == 0), "metadata block shape");
    // direct-to-LDS instructions per wave per stage (each moves 1 KiB, or
    // 256 bytes for the 4-byte meta loads).  A 64-channel fp16 tile has 2
    // meta chunks of 256 bytes for 4 waves: then waves w and w + MCH load the
    // same chunk into the same LDS bytes (identical data), so that every wave
    // issues the same number of loads per stage and one counter value means
    // "stage complete" for all of them.
    static constexpr int MCH = M_BYTES / 256;
    // waves that issue the loads (the loader group, or the first NLD compute waves)
    static constexpr int NL = CF::PROD || CF::NLD == 0 ? NW : CF::NLD;
    static constexpr int LA = A_STAGE / 1024 / NL;
    static constexpr int LW = W_STAGE / 1024 / NL;
    static constexpr int LM = MCH >= NL ? MCH / NL : (MCH > 0 ? 1 : 0);
    static constexpr int LS = (S_PART + NL - 1) / NL;
    static constexpr int L = LA + LW + LM + LS;
    static_assert(LA * NL * 1024 == A_STAGE && LW * NL * 1024 == W_STAGE && MCH * 256 == M_BYTES &&
                      (MCH == 0 || MCH % NL == 0 || NL % MCH == 0),
                  "stage does not split evenly over the waves");
    // meta chunk of this wave's j-th meta load (no modulo unless chunks are
    // shared: on the 128 x 256 int8 tiles it cost the registers that keep
    // two workgroups per CU)
    static __device__ __forceinline__ int mchunk(int j, int wave) {
        if constexpr (MCH >= NL) return j * NL + wave;
        else return wave % (MCH > 0 ? MCH : 1);
    }
    // word position of (row, w) inside a metadata block: XOR-swizzled so that
    // the 32 rows of one fragment read fall into distinct banks
    static __device__ __forceinline__ int mword(int row, int w) {
        return row * RW + (w ^ ((row * RW / 32) & (RW - 1)));
    }
};

// What a kernel adds to the plain product: Extra::kAfter -- index[M] is fetched
// to LDS ahead of the first stage, and after() runs between the main loop and
// the epilogue, with the accumulators and the tile's indices;
// Extra::kEpilogue -- epilogue() takes the place of the store to C; kTransA /
// kTransW (dense 16-bit kinds) -- the operand lies the other way round, A as
// [rows_a][lda] and W as [rows_w][ldw] with k along the rows (zeros past the
// last one), and is read through transposing LDS reads.  Extra::kPlace --
// place() finds the workgroup's tile (one of many products of one launch): it
// moves the operands' pointers to the tile's rows and sets M, the tile's place
// in N and the number of K stages, or returns false where there is no such
// tile; A's rows are then lda elements apart, and K may end inside a stage
// (chunks past it are read as zeros).  Plain GEMMs have none of them.
struct NoExtra {
    static constexpr bool kAfter = false, kEpilogue = false, kTransA = false, kTransW = false, kPlace = false;
};

template <class Extra>
__device__ __forceinline__ int lda_of(const Extra &e) {
    if constexpr (Extra::kTransA) return e.lda;
    else return 0;
}
template <class Extra>
__device__ __forceinline__ int64_t a_row_of(const Extra &e, int64_t row) {
    if constexpr (Extra::kPlace) return e.a_row;
    else return row;
}
template <class Extra>
__device__ __forceinline__ int ldw_of(const Extra &e) {
    if constexpr (Extra::kTransW) return e.ldw;
    else return 0;
}
template <class Extra>
__device__ __forceinline__ uint32_t bytes_a_of(const Extra &e) {
    if constexpr (Extra::kTransA) return uint32_t(int64_t(e.rows_a) * e.lda * 2);
    else return 0;
}
template <class Extra>
__device__ __forceinline__ uint32_t bytes_w_of(const Extra &e) {
    if constexpr (Extra::kTransW) return uint32_t(int64_t(e.rows_w) * e.ldw * 2);
    else return 0;
}

// Transposed operand in LDS: 16-byte chunk of a row of `chunks` chunks.  One
// transposing fragment read takes 64 bytes of rows k..k+3 and k+8..k+11: the
// first four fall into distinct quarters of the banks.
__device__ __forceinline__ int swzk(int row, int col, int chunks) { return col ^ ((4 * (row & 3)) & (chunks - 1)); }

// Eight consecutive k of one column from a [k][column] image: lane j of a
// 16-lane group points at row j/4 and columns 4 (j%4).., and receives column j
// of rows 0..3; the second read takes the four rows after them.
__device__ __forceinline__ u32x4 lds_tr8(const uint8_t *p, int row_bytes) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 *lds_s4;
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p)));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4)(p + 4 * row_bytes)));
    return u32x4{lo.x, lo.y, hi.x, hi.y};
}

template <int KIND, int EPI, class CF, class Extra>
__global__ void __launch_bounds__(CF::WM *CF::WN * 64 * (CF::PROD ? 2 : 1))
gemm_kernel(const uint8_t *__restrict__ A, const uint8_t *__restrict__ Wv, const uint32_t *__restrict__ meta,
            const float *__restrict__ scale, const float *__restrict__ bias, void *__restrict__ C, int M, int N,
            int K, int stages, Extra extra) {
    using KT = KindTraits<KIND>;
    using LY = Layout<KIND, CF>;
    using Acc = typename AccOf<KIND>::T;
    constexpr int TM = CF::TM, TN = CF::TN, GM = CF::GM, NB = CF::STAGES;
    constexpr int WM = CF::WM;
    constexpr int BM = LY::BM, BN = LY::BN, WB = LY::WB, MW = LY::MW;
    constexpr int A_STAGE = LY::A_STAGE, W_STAGE = LY::W_STAGE, STAGE = LY::STAGE;
    constexpr int SA = KT::kI8 ? 1 : 2;  // bytes per element
    constexpr bool F4 = KIND == MX_F4;
    // LDS-staged epilogue: each wave owns 32 token rows x TN*32 channels per pass
    constexpr int OB = (EPI == EPI_F16 || EPI == EPI_F16_SCALE || EPI == EPI_BF16) ? 2
                                                                                   : (EPI == EPI_I8_SCALE ? 1 : 4);  // output bytes
    constexpr int EROW = TN * 32 * OB + 16;       // padded LDS row (odd multiple of 16 B)
    constexpr int EWAVE = 32 * EROW;
    constexpr int EPASS = (TM * EWAVE * LY::NW <= CF::STAGES * STAGE) ? TM : 1;
    constexpr int SMEM_EPI = EPASS * EWAVE * LY::NW;
    constexpr int SMEM_MAIN = CF::STAGES * STAGE + LY::MRING + LY::S_RING;
    constexpr int SMEM = (SMEM_MAIN > SMEM_EPI) ? SMEM_MAIN : SMEM_EPI;

    __shared__ __attribute__((aligned(1024))) uint8_t smem[SMEM];
    __shared__ int32_t s_index[Extra::kAfter ? BM < 64 ? 64 : BM : 1];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    // With loader waves (PROD), waves NW.. load and waves 0..NW-1 compute;
    // `wave` is a wave's index within its group.
    constexpr bool PROD = CF::PROD;
    const bool loader = PROD && (tid >> 6) >= LY::NW;
    const int wave = loader ? (tid >> 6) - LY::NW : tid >> 6;
    const int wm = wave % WM, wn = wave / WM;
    const int h = lane >> 5, r = lane & 31;

    // ---- tile assignment: XCD-contiguous ranges, GM tile-rows per group
    int b = 0, tile_m = 0, tile_n = 0, m0 = 0, n0 = 0;
    if constexpr (Extra::kPlace) {
        const uint8_t *a = A, *w = Wv;
        void *c = C;
        if (!extra.template place<CF, BM, BN>(a, w, c, M, N, K, stages, n0)) return;
        A = a, Wv = w, C = c;
    } else {
        const int tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
        b = xcd_remap(blockIdx.x, tiles_m * tiles_n);
        const int group = b / (GM * tiles_n);
        const int first_m = group * GM;
        const int gm = min(tiles_m - first_m, GM);
        const int in_group = b % (GM * tiles_n);
        tile_m = first_m + in_group % gm;
        tile_n = in_group / gm;
        m0 = tile_m * BM, n0 = tile_n * BN;
    }

    const int64_t k_row = F4 ? int64_t(K) / 2 : int64_t(K) * SA;  // bytes of K values
    const int64_t a_row = a_row_of(extra, k_row);                 // bytes between A rows
    const int64_t w_row = KT::kSparse ? k_row / 2 : k_row;        // bytes per W row
    const int64_t m_row = K / 32;                            // meta words per row
    // S = K stages of this workgroup (128 bytes of an A row each): all of them,
    // or, with K split over gridDim.y, split blockIdx.y's equal share.  The
    // mask is a value-range hint (the host's 4 GiB operand limit keeps S below
    // 2^19): with S known to be small the compiler keeps the stage address
    // arithmetic narrow, which holds the 128 x 256 tiles within the 256
    // registers that two workgroups per CU allow (260 without it).
    const int S = stages & 0xffffff;
    const int ks0 = int(blockIdx.y) * S;

    // ---- direct-to-LDS sources: instruction j of this wave fills the wave's
    // j-th KiB of the A (or W) stage; lane -> (row, position) -> global chunk.
    // (32-bit byte offsets from the uniform base pointers keep the per-lane
    // address state small.)
    uint32_t oa[LY::LA];
#pragma unroll
    for (int j = 0; j < LY::LA; ++j) {
        const int byte = (j * LY::NL + wave) * 1024 + lane * 16;
        if constexpr (Extra::kTransA) {  // (columns past M: finite or not, they stay in rows that are not stored)
            const int row = byte / (BM * 2), pos = (byte / 16) % (BM / 8);
            oa[j] = uint32_t(row) * uint32_t(extra.lda * 2) + uint32_t(m0 * 2) + swzk(row, pos, BM / 8) * 16;
        } else {
            const int row = byte / LY::AB, pos = (byte / 16) % (LY::AB / 16);
            oa[j] = uint32_t(min(m0 + row, M - 1)) * uint32_t(a_row) + swzw<LY::AB>(row, pos) * 16;
        }
    }
    uint32_t ow[LY::LW];
#pragma unroll
    for (int j = 0; j < LY::LW; ++j) {
        const int byte = (j * LY::NL + wave) * 1024 + lane * 16;
        if constexpr (Extra::kTransW) {
            const int row = byte / (BN * 2), pos = (byte / 16) % (BN / 8);
            ow[j] = uint32_t(row) * uint32_t(extra.ldw * 2) + uint32_t(n0 * 2) + swzk(row, pos, BN / 8) * 16;
        } else {
            const int row = byte / WB, pos = (byte / 16) % (WB / 16);
            ow[j] = uint32_t(min(n0 + row, N - 1)) * uint32_t(w_row) + swzw<WB>(row, pos) * 16;
        }
    }
    uint32_t om[LY::LM > 0 ? LY::LM : 1];
#pragma unroll
    for (int j = 0; j < LY::LM; ++j) {
        const int word = LY::mchunk(j, wave) * 64 + lane;  // row-major [BN][MW]
        const int row = word / (MW > 0 ? MW : 1), w = word % (MW > 0 ? MW : 1);
        om[j] = (uint32_t(min(n0 + row, N - 1)) * uint32_t(m_row) + w) * 4;
    }
    constexpr int RW = LY::MP ? LY::RW : 1;
    const uint8_t *meta_b = reinterpret_cast<const uint8_t *>(meta);

    // Where a tile starts its K loop.  From stage 0, the tiles in flight on an
    // XCD read the same K slice at about the same time, so one L2 fill serves
    // several of them; rotated (tile b starts at stage b mod S), they read
    // different slices, which spreads their requests over more memory
    // channels but gives up that sharing.  The K reduction may run in any
    // order, and the order is fixed per tile, so results stay deterministic
    // either way.  Which one is faster was measured per tile shape on MI355X
    // (ROT in the tile configurations below).
    const int rot = CF::ROT ? b % S : 0;
    // (the host caps A and W below 4 GiB, so every byte count fits 32 bits)
    // (transposed operands end with their last row: a partial last stage reads zeros past it)
    const __amdgpu_buffer_rsrc_t bufA =
        buffer_of(A, Extra::kTransA  ? bytes_a_of(extra)
                     : Extra::kPlace ? uint32_t(int64_t(min(M, BM) - 1) * a_row + k_row)
                                     : uint32_t(int64_t(M) * a_row));
    const __amdgpu_buffer_rsrc_t bufW =
        buffer_of(Wv, Extra::kTransW ? bytes_w_of(extra) : uint32_t(int64_t(N) * w_row));
    const __amdgpu_buffer_rsrc_t bufM = buffer_of(meta_b, KT::kSparse ? uint32_t(int64_t(N) * m_row * 4) : 0u);
    // Part t - (c - 1) * MP - 1 of metadata block c = ceil(t / MP), loaded
    // with the loads of stage t (t < 0: the prologue's parts of block 0).
    // Each part is MCH 256-byte chunks, BN / MP rows.  Lane's word is (row,
    // stored position p) of the block; it holds word w = p ^ swizzle of the
    // row's metadata for block stage q = w / MW, i.e. local stage c * MP + q
    // (past the last stage: any valid word, never read).
    auto issue_meta = [&](int t) {
        if constexpr (LY::MP > 0) {
            constexpr int MPr = LY::MP > 0 ? LY::MP : 1;
            const int c = (t + MPr - 1) / MPr;  // ceil(t / MP); t + MP - 1 >= 0
            const int part = t - (c * MPr - MPr + 1);
            uint8_t *blk = smem + NB * STAGE + (c % LY::MSLOTS) * LY::MBLK;
#pragma unroll
            for (int j = 0; j < LY::LM; ++j) {
                const int row = (part * LY::MCH + LY::mchunk(j, wave)) * (64 / RW) + lane / RW;
                const int w = (lane % RW) ^ ((row * RW / 32) & (RW - 1));
                const int sl = min(c * MPr + w / MW, S - 1);
                const int sg = ks0 + ((sl + rot < S) ? sl + rot : sl + rot - S);
                const uint32_t off =
                    (uint32_t(min(n0 + row, N - 1)) * uint32_t(m_row) + uint32_t(sg * MW + w % MW)) * 4;
                dma4(bufM, off, blk + (part * LY::MCH + LY::mchunk(j, wave)) * 256);
            }
        }
    };
    const bool issuer = LY::NL == LY::NW || wave < LY::NL;  // (with PROD: the loaders)
    // The last stage of a K that ends inside it (place() launches, whose buffers, a tile's rows of
    // A and one weight, end below 2 GiB):
    // chunks past the end are read past the buffer, i.e. as zeros.
    [[maybe_unused]] auto issue_end = [&](uint8_t *base, int sg) {
        constexpr uint32_t kNone = 0x80000000u;
        const int room = int(k_row) - sg * LY::AB;
#pragma unroll
        for (int j = 0; j < LY::LA; ++j) {
            const int byte = (j * LY::NL + wave) * 1024 + lane * 16;
            const int row = byte / LY::AB, pos = (byte / 16) % (LY::AB / 16);
            const bool in = swzw<LY::AB>(row, pos) * 16 < room;
            dma16(bufA, in ? oa[j] + uint32_t(sg * LY::AB) : kNone, base + (j * LY::NL + wave) * 1024);
        }
#pragma unroll
        for (int j = 0; j < LY::LW; ++j) {
            if constexpr (Extra::kTransW) {
                dma16(bufW, ow[j] + uint32_t(sg) * uint32_t(ldw_of(extra) * 128), base + A_STAGE + (j * LY::NL + wave) * 1024);
            } else {
                const int byte = (j * LY::NL + wave) * 1024 + lane * 16;
                const int row = byte / WB, pos = (byte / 16) % (WB / 16);
                const bool in = swzw<WB>(row, pos) * 16 < room;
                dma16(bufW, in ? ow[j] + uint32_t(sg * WB) : kNone, base + A_STAGE + (j * LY::NL + wave) * 1024);
            }
        }
    };
    // MX_F4: part t + 1 - 2c of scale block c = ceil(t / 2), with the loads of stage t.  (Past the end of
    // a row it may bring the next row's scales: load_scales() leaves them out.)
    [[maybe_unused]] auto issue_scales = [&](int t) {
        if constexpr (F4) {
            const int c = (t + 1) >> 1, part = (t + 1) & 1, s_row = K / 32;
            const __amdgpu_buffer_rsrc_t bufSA = buffer_of(extra.sa, uint32_t(min(M, BM) * s_row));
            const __amdgpu_buffer_rsrc_t bufSW = buffer_of(extra.sw, uint32_t(N * s_row));
            uint8_t *block = smem + NB * STAGE + c % 3 * LY::S_BLOCK;
#pragma unroll
            for (int j = 0; j < LY::LS; ++j) {
                const int chunk = min(part * LY::S_PART + min(j * LY::NL + wave, LY::S_PART - 1), LY::S_CHUNKS - 1);
                const int row = chunk * 64 + lane;
                if (chunk < LY::S_AROWS / 64)  // (uniform)
                    dma16(bufSA, uint32_t(min(m0 + row, M - 1)) * uint32_t(s_row) + uint32_t(c * 16), block + chunk * 1024);
                else
                    dma16(bufSW, uint32_t(min(n0 + row - LY::S_AROWS, N - 1)) * uint32_t(s_row) + uint32_t(c * 16),
                          block + chunk * 1024);
            }
        }
    };
    // whole: stage s is known to lie inside K (no branch parts what the scheduler may interleave).
    auto issue = [&](int s, auto whole) {
        if (!issuer) return;
        uint8_t *base = smem + (s % NB) * STAGE;
        const int sg = ks0 + ((s + rot < S) ? s + rot : s + rot - S);  // global K stage
        if constexpr (F4) issue_scales(s);
        if constexpr (Extra::kPlace && !Extra::kTransA && !decltype(whole)::value) {
            if ((sg + 1) * LY::AB > int(k_row)) {
                issue_end(base, sg);
                return;
            }
        }
        if constexpr (Extra::kPlace && Extra::kTransA) {
            // rows of a group may reach past 32-bit offsets: each stage has a buffer of its own
            const int64_t sa = int64_t(sg) * extra.lda * 128, sw = int64_t(sg) * extra.ldw * 128;
            const __amdgpu_buffer_rsrc_t a = buffer_of(A + sa, uint32_t(min(extra.bytes_a - sa, int64_t(0x7fffffff))));
            const __amdgpu_buffer_rsrc_t w = buffer_of(Wv + sw, uint32_t(min(extra.bytes_w - sw, int64_t(0x7fffffff))));
#pragma unroll
            for (int j = 0; j < LY::LA; ++j) dma16(a, oa[j], base + (j * LY::NL + wave) * 1024);
#pragma unroll
            for (int j = 0; j < LY::LW; ++j) dma16(w, ow[j], base + A_STAGE + (j * LY::NL + wave) * 1024);
            return;
        }
#pragma unroll
        for (int j = 0; j < LY::LA; ++j)
            dma16(bufA, oa[j] + (Extra::kTransA ? uint32_t(sg) * uint32_t(lda_of(extra) * 128) : uint32_t(sg * LY::AB)), base + (j * LY::NL + wave) * 1024);
#pragma unroll
        for (int j = 0; j < LY::LW; ++j)
            dma16(bufW, ow[j] + (Extra::kTransW ? uint32_t(sg) * uint32_t(ldw_of(extra) * 128) : uint32_t(sg * WB)), base + A_STAGE + (j * LY::NL + wave) * 1024);
        if constexpr (LY::MP == 0) {
#pragma unroll
            for (int j = 0; j < LY::LM; ++j)
                dma4(bufM, om[j] + uint32_t(sg * MW * 4), base + A_STAGE + W_STAGE + LY::mchunk(j, wave) * 256);
        } else {
            issue_meta(s);
        }
    };

    // Fragments of one k-step (one matrix instruction deep) for the wave's
    // TN channel blocks and TM token blocks.
    struct Frag {
        u32x4 w[TN];
        uint32_t idx[TN];
        u32x8 a[TM];
        uint32_t sw[F4 ? TN : 1], sa[F4 ? TM : 1];  // MX_F4: this lane's block's scale in byte 2 (k-step % 2)
    };
    // byte of a [k][column] stage that this lane points at for k-step kk, block column `row`
    [[maybe_unused]] auto tr_at = [&](int row, int kk, int columns) {
        const int k = 16 * kk + 8 * h + ((lane & 15) >> 2), col = row - (r & 15) + 4 * (lane & 3);
        return k * (columns * 2) + swzk(k, col >> 3, columns / 8) * 16 + (col & 7) * 2;
    };
    auto load_frag = [&](int s, int kk, Frag &F) {
        const uint8_t *bA = smem + (s % NB) * STAGE;
        const uint8_t *bW = bA + A_STAGE;
        const uint32_t *bM = reinterpret_cast<const uint32_t *>(bA + A_STAGE + W_STAGE);
        constexpr int MPr = LY::MP > 0 ? LY::MP : 1;
        const uint32_t *bB =
            reinterpret_cast<const uint32_t *>(smem + NB * STAGE + ((s / MPr) % (LY::MP ? LY::MSLOTS : 1)) * LY::MBLK);
        const int q = (s % MPr) * MW;  // first word of stage s in a block row
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
            const int row = wn * TN * 32 + tn * 32 + r;
            if constexpr (!Extra::kTransW) F.w[tn] = lds16(bW + row * WB + swzw<WB>(row, 2 * kk + h) * 16);
            else F.w[tn] = lds_tr8(bW + tr_at(row, kk, BN), BN * 2);
            if constexpr (LY::MP > 0 && KIND == W24_F16) F.idx[tn] = bB[LY::mword(row, q + kk)] >> (16 * h);
            else if constexpr (LY::MP > 0 && KIND == W24_I8) F.idx[tn] = bB[LY::mword(row, q + 2 * kk + h)];
            else if constexpr (KIND == W24_F16) F.idx[tn] = bM[row * MW + kk] >> (16 * h);
            else if constexpr (KIND == W24_I8) F.idx[tn] = bM[row * MW + 2 * kk + h];
            else F.idx[tn] = 0;
        }
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            const int row = wm * TM * 32 + tm * 32 + r;
            if constexpr (KT::kSparse) {
                // two 16-byte pieces of the 64-byte window: bytes 16h.. and 32+16h..
                const u32x4 lo = lds16(bA + row * LY::AB + swzw<LY::AB>(row, 4 * kk + h) * 16);
                const u32x4 hi = lds16(bA + row * LY::AB + swzw<LY::AB>(row, 4 * kk + 2 + h) * 16);
                F.a[tm] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            } else if constexpr (Extra::kTransA) {
                const u32x4 lo = lds_tr8(bA + tr_at(row, kk, BM), BM * 2);
                F.a[tm] = __builtin_shufflevector(lo, lo, 0, 1, 2, 3, 0, 1, 2, 3);
            } else {
                const u32x4 lo = lds16(bA + row * LY::AB + swzw<LY::AB>(row, 2 * kk + h) * 16);
                F.a[tm] = __builtin_shufflevector(lo, lo, 0, 1, 2, 3, 0, 1, 2, 3);
            }
        }
    };

    // MX_F4: one word of scales serves two k-steps (none past the end of K).
    [[maybe_unused]] auto load_scales = [&](int s, int kk, Frag &F, const Frag &before) {
        if constexpr (F4) {
            const uint8_t *b = smem + NB * STAGE + (s >> 1) % 3 * LY::S_BLOCK + (s & 1) * 8 + kk / 2 * 4;
            const uint32_t live = (s * 2 + kk / 2) * 4 < K / 32 ? 0xffffffffu : 0u;
            auto word = [&](int row) { return (*reinterpret_cast<const uint32_t *>(b + row * 16) & live) >> (8 * h); };
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
                F.sw[tn] = kk % 2 ? before.sw[tn] : word(LY::S_AROWS + wn * TN * 32 + tn * 32 + r);
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) F.sa[tm] = kk % 2 ? before.sa[tm] : word(wm * TM * 32 + tm * 32 + r);
        }
    };

    Acc acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = Acc{};

    auto mma_frag = [&](const Frag &F, [[maybe_unused]] int kk) {
#pragma unroll
        for (int tn = 0; tn < TN; ++tn)
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) {
                if constexpr (F4) {
                    const u32x4 a = __builtin_shufflevector(F.a[tm], F.a[tm], 0, 1, 2, 3);
                    if (kk % 2) mma_f4<2>(acc[tn][tm], F.w[tn], a, F.sw[tn], F.sa[tm]);
                    else mma_f4<0>(acc[tn][tm], F.w[tn], a, F.sw[tn], F.sa[tm]);
                } else {
                    mma<KIND>(acc[tn][tm], F.w[tn], F.a[tm], F.idx[tn]);
                }
            }
    };
    // Interleave hint: one matrix instruction, then its share of LDS reads.
    constexpr int NMMA = TN * TM;
    constexpr int NRD = TN * (KT::kSparse || Extra::kTransW ? 2 : 1) + TM * (KT::kSparse || Extra::kTransA ? 2 : 1);
    constexpr int RPM = (NRD + NMMA - 1) / NMMA;
    auto interleave = [&]() {
#pragma unroll
        for (int i = 0; i < NMMA; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);    // matrix
            __builtin_amdgcn_sched_group_barrier(0x100, RPM, 0);  // LDS reads
        }
    };

    // Pipeline: NB stage buffers, the stage s+NB is fetched while stage s+1 is
    // read into registers and stage s feeds the matrix cores.  Within a stage
    // the next k-step's fragments are read during the current k-step's
    // instructions; the stage hand-off (wait + barrier) sits before the last
    // k-step's instructions so that the next stage's first fragments overlap
    // them too.
    if constexpr (Extra::kAfter) {
        // (the oldest loads of their waves, so the first stage's wait covers them; zeros past M)
        const __amdgpu_buffer_rsrc_t bufI = buffer_of(extra.index, uint32_t(M) * 4u);
        if ((!PROD || loader) && wave < (BM + 63) / 64)
            for (int j = wave; j < (BM + 63) / 64; j += LY::NW)
                dma4(bufI, uint32_t(m0 + j * 64 + lane) * 4u, reinterpret_cast<uint8_t *>(s_index + j * 64));
    }
    if (!PROD || loader) {
        if constexpr (LY::MP > 1)
            for (int t = 1 - LY::MP; t < 0; ++t) issue_meta(t);
        if constexpr (F4) issue_scales(-1);
#pragma unroll
        for (int s = 0; s < NB; ++s)
            if (s < S) issue(s, std::false_type{});
    }
    if (NB < S) wait_vm_barrier<(NB - 1) * LY::L>();
    else wait_vm_barrier<0>();
    if (loader) {
        // the same barriers as the compute waves' stages: after the one that
        // ends stage s, stage s's buffer is free for stage s + NB
        int s = 0;
        for (; s + NB < S; ++s) {
            wait_vm_barrier<(NB - 2) * LY::L>();
            issue(s + NB, std::false_type{});
        }
        for (; s < S; ++s) wait_vm_barrier<0>();
    } else if constexpr (CF::DEEP) {
        // One wave a SIMD with registers for a whole stage's fragments: they are read a stage's last
        // k-step ahead of their use (and the last one in the first), so that a stage's buffer is free
        // again after its first k-step, and the loads into it have a stage and a half to arrive instead
        // of one.  Two barriers a stage: its reads are done, the next stage is there.
        static_assert(!PROD && NB == 2 && LY::NL == LY::NW);
        constexpr int NI = LY::NI;
        Frag F[NI];
        auto load = [&](int s, int kk) {
            load_frag(s, kk, F[kk]);
            if constexpr (F4) load_scales(s, kk, F[kk], F[kk & ~1]);
        };
#pragma unroll
        for (int kk = 0; kk + 1 < NI; ++kk) load(0, kk);
        // PHASE 0: stage s + NB is fetched, and whole; 1: fetched; 2: there is none
        auto stage = [&](int s, auto phase) {
            constexpr int PHASE = decltype(phase)::value;
#pragma unroll
            for (int kk = 0; kk < NI; ++kk) {
                if (kk == 0) load(s, NI - 1);
                if (kk == 1 && PHASE < 2) {
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    if constexpr (PHASE == 0) issue(s + NB, std::true_type{});
                    else issue(s + NB, std::false_type{});
                }
                if (kk == NI - 1) {
                    if constexpr (PHASE < 2) wait_vm_barrier<LY::L>();
                    else wait_vm_barrier<0>();
#pragma unroll
                    for (int k = 0; k + 1 < NI; ++k) load(s + 1, k);
                }
                mma_frag(F[kk], kk);
#pragma unroll
                for (int i = 0; i < TN * TM; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix
                    if (kk == NI - 1) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // LDS reads
                    else if (kk == 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                    else if (PHASE < 2 && i % 2 == 0) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // loads
                }
            }
        };
        const int whole = Extra::kPlace && !Extra::kTransA ? int(k_row / LY::AB) : S;
        int s = 0;
        for (; s + NB < whole; ++s) stage(s, std::integral_constant<int, 0>{});
        for (; s + NB < S; ++s) stage(s, std::integral_constant<int, 1>{});
        for (; s < S; ++s) stage(s, std::integral_constant<int, 2>{});
    } else {
        Frag F[2];
        load_frag(0, 0, F[0]);
        if constexpr (F4) load_scales(0, 0, F[0], F[0]);

        // One stage; STEADY: the ring still has a stage to fetch (s + NB < S).
        // The next stage's first fragments are read unconditionally: on the last
        // stage this reads a valid, stale buffer whose values are never used.
        auto stage = [&](int s, auto steady) {
#pragma unroll
            for (int kk = 0; kk < LY::NI; ++kk) {
                Frag &cur = F[kk & 1];
                Frag &nxt = F[(kk + 1) & 1];
                if (kk + 1 < LY::NI) {
                    load_frag(s, kk + 1, nxt);
                    if constexpr (F4) load_scales(s, kk + 1, nxt, cur);
                } else {
                    // stage s is fully in registers; stage s+1 must be complete
                    if constexpr (decltype(steady)::value) {
                        wait_lgkm_vm_barrier<(NB - 2) * LY::L>();
                        if constexpr (!PROD) issue(s + NB, std::false_type{});  // reuses stage s's buffer
                    } else {
                        wait_lgkm_vm_barrier<0>();
                    }
                    load_frag(s + 1, 0, nxt);
                    if constexpr (F4) load_scales(s + 1, 0, nxt, cur);
                }
                mma_frag(cur, kk);
                interleave();
            }
        };
        int s = 0;
        for (; s + NB < S; ++s) stage(s, std::true_type{});
        for (; s < S; ++s) stage(s, std::false_type{});
    }

    if constexpr (Extra::kAfter) {
        __syncthreads();  // (the stage ring is its scratch: every wave is done reading it)
        extra.template after<CF, SMEM>(acc, s_index, smem, loader, m0, n0, M, N);
    }
    if constexpr (Extra::kEpilogue) {
        extra.template epilogue<CF, SMEM>(acc, smem, loader, m0, n0, wave, M, N, tile_m, tile_n);
        return;
    }

    // ---- epilogue.  Lane (h, r) holds, for 32x32 block (tn, tm) and q = 0..3,
    // channels n = tn*32 + 8q + 4h .. +3 of token m = tm*32 + r.
    auto convert = [&](const Acc &v, int q, int n) -> u32x4 {
        u32x4 o = u32x4{0, 0, 0, 0};
        if constexpr (EPI == EPI_F16) {
            o.x = pack_half2_rne(v[4 * q + 0], v[4 * q + 1]);
            o.y = pack_half2_rne(v[4 * q + 2], v[4 * q + 3]);
        } else if constexpr (EPI == EPI_BF16) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            const bf16x4 t = {__bf16(v[4 * q + 0]), __bf16(v[4 * q + 1]), __bf16(v[4 * q + 2]), __bf16(v[4 * q + 3])};
            const u32x2 u = __builtin_bit_cast(u32x2, t);
            o.x = u.x, o.y = u.y;
        } else if constexpr (EPI == EPI_PART || EPI == EPI_F32) {
            // (whole 4-vectors are bit-cast: a bit-cast of a single element of
            // the 16-wide accumulator vector yielded element 0 for every lane)
            using E4 = typename std::conditional<KT::kI8, intx4, floatx4>::type;
            const E4 t = E4{v[4 * q + 0], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
            o = __builtin_bit_cast(u32x4, t);
        } else if constexpr (EPI == EPI_I32) {
            o.x = uint32_t(v[4 * q + 0]);
            o.y = uint32_t(v[4 * q + 1]);
            o.z = uint32_t(v[4 * q + 2]);
            o.w = uint32_t(v[4 * q + 3]);
        } else {
            const int nc = min(n, N - 4);
            const floatx4 sc = *reinterpret_cast<const floatx4 *>(scale + nc);
            floatx4 f;
            f.x = __fmul_rn(float(v[4 * q + 0]), sc.x);
            f.y = __fmul_rn(float(v[4 * q + 1]), sc.y);
            f.z = __fmul_rn(float(v[4 * q + 2]), sc.z);
            f.w = __fmul_rn(float(v[4 * q + 3]), sc.w);
            if (bias) {
                const floatx4 bi = *reinterpret_cast<const floatx4 *>(bias + nc);
                f.x = __fadd_rn(f.x, bi.x);
                f.y = __fadd_rn(f.y, bi.y);
                f.z = __fadd_rn(f.z, bi.z);
                f.w = __fadd_rn(f.w, bi.w);
            }
            if constexpr (EPI == EPI_F32_SCALE) {
                o = __builtin_bit_cast(u32x4, f);
            } else if constexpr (EPI == EPI_F16_SCALE) {
                o.x = pack_half2_rne(f.x, f.y);
                o.y = pack_half2_rne(f.z, f.w);
            } else {
                // round to nearest even, saturate, pack four int8 into one word
                auto q8 = [](float y) -> uint32_t {
                    const float r = fminf(fmaxf(__builtin_rintf(y), -128.0f), 127.0f);
                    return uint32_t(int32_t(r)) & 0xffu;
                };
                o.x = q8(f.x) | (q8(f.y) << 8) | (q8(f.z) << 16) | (q8(f.w) << 24);
            }
        }
        return o;
    };

    // Stage 32-token slabs of the wave's accumulators through LDS as
    // row-major [token][channel], then store whole row segments
    // (TN*32*OB contiguous bytes per token) with 16 bytes per lane.
    constexpr int CPR = TN * 32 * OB / 16;  // 16-byte chunks per token row
    constexpr int RPI = kWave / CPR;        // token rows per store instruction
    static_assert(RPI * CPR == kWave, "row segment must tile a wave");
    __syncthreads();  // every wave is done reading the stage buffers
    uint8_t *const Cb = reinterpret_cast<uint8_t *>(C) + (EPI == EPI_PART ? int64_t(blockIdx.y) * M * N * OB : 0);
    // (with after(), recomputed: the main loop has no registers to keep them in)
    [[maybe_unused]] auto late = [](int waves, int each) {
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));
        return (waves ? (t >> 6) % LY::NW % waves : (t >> 6) % LY::NW / WM) * each;
    };
    const int row_of_wave = Extra::kAfter ? late(WM, TM * 32) : wm * TM * 32;
    uint8_t *ew = smem + wave * EPASS * EWAVE;  // (compute waves)
    const int nw = n0 + (Extra::kAfter ? late(0, TN * 32) : wn * TN * 32);  // first channel of the wave
#pragma unroll
    for (int tp = 0; tp < TM; tp += EPASS) {
        if (!loader) {
#pragma unroll
            for (int e = 0; e < EPASS; ++e) {
                uint8_t *slab = ew + e * EWAVE + r * EROW;
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int c = tn * 32 + q * 8 + h * 4;
                        const u32x4 o = convert(acc[tn][tp + e], q, nw + c);
                        if constexpr (OB == 1) *reinterpret_cast<uint32_t *>(slab + c) = o.x;
                        else if constexpr (OB == 2) *reinterpret_cast<u32x2 *>(slab + c * 2) = u32x2{o.x, o.y};
                        else *reinterpret_cast<u32x4 *>(slab + c * 4) = o;
                    }
            }
        }
        __syncthreads();
        if (!loader) {
#pragma unroll
            for (int e = 0; e < EPASS; ++e) {
#pragma unroll
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int row = i * RPI + lane / CPR, ch = lane % CPR;
                    const int m = m0 + row_of_wave + (tp + e) * 32 + row;
                    const int n = nw + ch * (16 / OB);
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(ew + e * EWAVE + row * EROW + ch * 16);
                    if constexpr (Extra::kPlace) {
                        store_piece<OB>(Cb + (int64_t(m) * extra.ldc + n) * OB, v, m < M ? N - n : 0, CF::NTS && extra.stream);
                    } else {
                        if (m < M && n < N) store16<CF::NTS>(Cb + (int64_t(m) * N + n) * OB, v);
                    }
                }
            }
        }
        if (tp + EPASS < TM) __syncthreads();
    }
}

}  // namespace ssg

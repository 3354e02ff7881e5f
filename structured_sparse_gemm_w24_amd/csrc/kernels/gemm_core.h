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
// (the same at `off` + `more`, the latter uniform; only `off` is checked against the buffer's size)
__device__ __forceinline__ void dma16s(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t more, uint8_t *wave_base) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)wave_base, 16, off, more, 0, 0);
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
        if (stream) {
            asm volatile("" ::: "memory");  // (else the compiler makes one plain store of the two)
            __builtin_nontemporal_store(v, reinterpret_cast<Any *>(p));
            asm volatile("" ::: "memory");
        } else {
            *reinterpret_cast<Any *>(p) = v;
        }
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

// What place() found, as scalars: the same in every lane, but computed in vector registers it makes each
// load loop over the lanes' buffer descriptors.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint64_t lo = uint32_t(uniform(int(uint32_t(v)))), hi = uint32_t(uniform(int(uint32_t(v >> 32))));
    return reinterpret_cast<const uint8_t *>(hi << 32 | lo);
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
// registers, so that a stage's buffer is free after the first quarter of its matrix instructions.
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

// LDS-staged epilogue: each wave owns 32 token rows x TN*32 channels per pass; and the LDS of a kernel.
template <int KIND, int EPI, class CF>
struct Slabs {
    using LY = Layout<KIND, CF>;
    static constexpr int OB = (EPI == EPI_F16 || EPI == EPI_F16_SCALE || EPI == EPI_BF16) ? 2
                              : (EPI == EPI_I8_SCALE ? 1 : 4);  // output bytes
    static constexpr int EROW = CF::TN * 32 * OB + 16;  // padded LDS row (odd multiple of 16 B)
    static constexpr int EWAVE = 32 * EROW;
    static constexpr int EPASS = (CF::TM * EWAVE * LY::NW <= CF::STAGES * LY::STAGE) ? CF::TM : 1;
    static constexpr int SMEM_EPI = EPASS * EWAVE * LY::NW;
    static constexpr int SMEM_MAIN = CF::STAGES * LY::STAGE + LY::MRING + LY::S_RING;
    static constexpr int SMEM = (SMEM_MAIN > SMEM_EPI) ? SMEM_MAIN : SMEM_EPI;
};

template <int KIND, int EPI, class CF, class Extra>
__global__ void __launch_bounds__(CF::WM *CF::WN * 64 * (CF::PROD ? 2 : 1))
gemm_kernel(const uint8_t *__restrict__ A, const uint8_t *__restrict__ Wv, const uint32_t *__restrict__ meta,
            const float *__restrict__ scale, const float *__restrict__ bias, void *__restrict__ C, int M, int N,
            int K, int stages, Extra extra) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[Slabs<KIND, EPI, CF>::SMEM];
    __shared__ int32_t s_index[Extra::kAfter ? Layout<KIND, CF>::BM < 64 ? 64 : Layout<KIND, CF>::BM : 1];
    const int block = blockIdx.x;
#include "gemm_tile.h"
}

// The same for a kernel whose launch holds the tiles of two products.
template <int KIND, int EPI, class CF, class Extra>
__device__ __forceinline__ void
gemm_tile(const uint8_t *__restrict__ A, const uint8_t *__restrict__ Wv, void *__restrict__ C, int M, int N, int K,
          int stages, Extra extra, uint8_t *smem, int block) {
    const uint32_t *meta = nullptr;
    const float *scale = nullptr, *bias = nullptr;
    int32_t *s_index = nullptr;
#include "gemm_tile.h"
}

}  // namespace ssg

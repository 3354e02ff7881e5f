// One tile of a GEMM launch: the body of gemm_kernel() and of gemm_tile() (gemm_core.h), included by
// both.  As a function that the kernel calls, the same statements compile to other registers and
// another order, and the 2:4 kernels ran 4 to 5 % slower (fp16 6304 x 4096 x 1024 50.1 us, so 52.3).
//
// In scope: KIND, EPI, CF, Extra; A, Wv, meta, scale, bias, C, M, N, K, stages, extra; smem, s_index;
// block, the tile's number in the launch or in a part of it.

    using KT = KindTraits<KIND>;
    using LY = Layout<KIND, CF>;
    using SL = Slabs<KIND, EPI, CF>;
    using Acc = typename AccOf<KIND>::T;
    constexpr int TM = CF::TM, TN = CF::TN, GM = CF::GM, NB = CF::STAGES;
    constexpr int WM = CF::WM;
    constexpr int BM = LY::BM, BN = LY::BN, WB = LY::WB, MW = LY::MW;
    constexpr int A_STAGE = LY::A_STAGE, W_STAGE = LY::W_STAGE, STAGE = LY::STAGE;
    constexpr int SA = KT::kI8 ? 1 : 2;  // bytes per element
    constexpr bool F4 = KIND == MX_F4;
    constexpr int OB = SL::OB, EROW = SL::EROW, EWAVE = SL::EWAVE, EPASS = SL::EPASS;
    [[maybe_unused]] constexpr int SMEM = SL::SMEM;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    // With loader waves (PROD), waves NW.. load and waves 0..NW-1 compute;
    // `wave` is a wave's index within its group.
    constexpr bool PROD = CF::PROD;
    const bool loader = PROD && (tid >> 6) >= LY::NW;
    // (DEEP: known to be uniform, so that where a load goes in LDS is a scalar)
    const int wave = CF::DEEP ? __builtin_amdgcn_readfirstlane(tid >> 6) : loader ? (tid >> 6) - LY::NW : tid >> 6;
    const int wm = wave % WM, wn = wave / WM;
    const int h = lane >> 5, r = lane & 31;

    // ---- tile assignment: XCD-contiguous ranges, GM tile-rows per group
    int b = 0, tile_m = 0, tile_n = 0, m0 = 0, n0 = 0;
    if constexpr (Extra::kPlace) {
        const uint8_t *a = A, *w = Wv;
        void *c = C;
        if (!extra.template place<CF, BM, BN>(block, a, w, c, M, N, K, stages, n0)) return;
        A = uniform(a), Wv = uniform(w), C = c;
        M = uniform(M);
    } else {
        const int tiles_m = (M + BM - 1) / BM, tiles_n = (N + BN - 1) / BN;
        b = xcd_remap(block, tiles_m * tiles_n);
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
                     : Extra::kPlace ? uint32_t(uniform(int(int64_t(min(M, BM) - 1) * a_row + k_row)))
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
            auto room = [](int64_t bytes) { return uint32_t(uniform(int(min(bytes, int64_t(0x7fffffff))))); };
            const __amdgpu_buffer_rsrc_t a = buffer_of(uniform(A + sa), room(extra.bytes_a - sa));
            const __amdgpu_buffer_rsrc_t w = buffer_of(uniform(Wv + sw), room(extra.bytes_w - sw));
#pragma unroll
            for (int j = 0; j < LY::LA; ++j) dma16(a, oa[j], base + (j * LY::NL + wave) * 1024);
#pragma unroll
            for (int j = 0; j < LY::LW; ++j) dma16(w, ow[j], base + A_STAGE + (j * LY::NL + wave) * 1024);
            return;
        }
        if constexpr (CF::DEEP && decltype(whole)::value) {
            // The stage in the scalar offset, which the buffer's range check leaves out: only for operands
            // whose rows a whole stage never leaves.  (A transposed W is read past its last row's end where
            // the tile is wider, and the check has to see all of the offset.)
#pragma unroll
            for (int j = 0; j < LY::LA; ++j) dma16s(bufA, oa[j], uint32_t(sg * LY::AB), base + (j * LY::NL + wave) * 1024);
#pragma unroll
            for (int j = 0; j < LY::LW; ++j) {
                uint8_t *const to = base + A_STAGE + (j * LY::NL + wave) * 1024;
                if constexpr (Extra::kTransW) dma16(bufW, ow[j] + uint32_t(sg) * uint32_t(ldw_of(extra) * 128), to);
                else dma16s(bufW, ow[j], uint32_t(sg * WB), to);
            }
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
    [[maybe_unused]] auto load_scales = [&](int s, int kk, Frag &F, const Frag &before, auto whole) {
        if constexpr (F4) {
            const uint8_t *b = smem + NB * STAGE + (s >> 1) % 3 * LY::S_BLOCK + (s & 1) * 8 + kk / 2 * 4;
            const uint32_t live = decltype(whole)::value || (s * 2 + kk / 2) * 4 < K / 32 ? 0xffffffffu : 0u;
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
        // Where this lane's chunks lie in a stage.  Of the swizzle of a row r + 32 t only bit 2, t % 2,
        // depends on t, and in k-step kk it is that of k-step kk ^ 2 of t's neighbour: four places an
        // operand and constant distances from them serve all its rows (each place found by itself is
        // two of the three vector instructions beside every matrix instruction of a stage).  A transposed
        // operand has a place for each t, and its k-steps at constant distances.
        static_assert(NI == 4 && LY::AB == 128 && WB == 128);
        int at_a[Extra::kTransA ? TM : NI], at_w[Extra::kTransW ? TN : NI];
        auto place_t = [&](int row, int columns) {
            const int k = 8 * h + ((lane & 15) >> 2), col = row - (r & 15) + 4 * (lane & 3);
            return k * (columns * 2) + swzk(k, col >> 3, columns / 8) * 16 + (col & 7) * 2;
        };
#pragma unroll
        for (int t = 0; t < (Extra::kTransA ? TM : NI); ++t) {
            const int row = wm * TM * 32 + r;
            at_a[t] = Extra::kTransA ? place_t(row + t * 32, BM) : row * 128 + swz128(row, 2 * t + h) * 16;
        }
#pragma unroll
        for (int t = 0; t < (Extra::kTransW ? TN : NI); ++t) {
            const int row = wn * TN * 32 + r;
            at_w[t] = A_STAGE + (Extra::kTransW ? place_t(row + t * 32, BN) : row * 128 + swz128(row, 2 * t + h) * 16);
        }
        auto load = [&](int s, int kk, auto whole) {
            const uint8_t *b = smem + (s & 1) * STAGE;
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) {
                if constexpr (Extra::kTransW) F[kk].w[tn] = lds_tr8(b + at_w[tn] + kk * (32 * BN), BN * 2);
                else F[kk].w[tn] = lds16(b + at_w[kk ^ (tn & 1) * 2] + tn * 4096);
            }
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) {
                u32x4 lo;
                if constexpr (Extra::kTransA) lo = lds_tr8(b + at_a[tm] + kk * (32 * BM), BM * 2);
                else lo = lds16(b + at_a[kk ^ (tm & 1) * 2] + tm * 4096);
                F[kk].a[tm] = __builtin_shufflevector(lo, lo, 0, 1, 2, 3, 0, 1, 2, 3);
            }
            if constexpr (F4) load_scales(s, kk, F[kk], F[kk & ~1], whole);
        };
#pragma unroll
        for (int kk = 0; kk + 1 < NI; ++kk) load(0, kk, std::false_type{});
        // PHASE 0: stage s + NB is fetched, and whole; 1: fetched; 2: there is none
        auto stage = [&](int s, auto phase) {
            constexpr int PHASE = decltype(phase)::value;
#pragma unroll
            for (int kk = 0; kk < NI; ++kk) {
                if (kk == 0) load(s, NI - 1, std::integral_constant<bool, PHASE == 0>{});
                if (kk == 1 && PHASE < 2) {
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    if constexpr (PHASE == 0) issue(s + NB, std::true_type{});
                    else issue(s + NB, std::false_type{});
                }
                if (kk == NI - 1) {
                    if constexpr (PHASE < 2) wait_vm_barrier<LY::L>();
                    else wait_vm_barrier<0>();
#pragma unroll
                    for (int k = 0; k + 1 < NI; ++k) load(s + 1, k, std::integral_constant<bool, PHASE == 0>{});
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
        if constexpr (F4) load_scales(0, 0, F[0], F[0], std::false_type{});

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
                    if constexpr (F4) load_scales(s, kk + 1, nxt, cur, std::false_type{});
                } else {
                    // stage s is fully in registers; stage s+1 must be complete
                    if constexpr (decltype(steady)::value) {
                        wait_lgkm_vm_barrier<(NB - 2) * LY::L>();
                        if constexpr (!PROD) issue(s + NB, std::false_type{});  // reuses stage s's buffer
                    } else {
                        wait_lgkm_vm_barrier<0>();
                    }
                    load_frag(s + 1, 0, nxt);
                    if constexpr (F4) load_scales(s + 1, 0, nxt, cur, std::false_type{});
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

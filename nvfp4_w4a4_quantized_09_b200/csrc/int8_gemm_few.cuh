// int8_gemm_few.cuh -- the int8 GEMM for few tokens (M <= 128), where the
// weight streams from memory once.  Included by int8_gemm.cu.
//
// Tiles of all the tokens x BN channels, in one of three ways:
//   * The tokens are the MMA's rows (64 of them up to 64 tokens, then 128) and
//     the channels its N = BN, a multiple of 16 up to 256.  BN is free, so the
//     launcher picks it to fill whole rounds of the SMs.  Only the tokens' own
//     rows are loaded (NT = M rounded up to 8); the MMA reads all its rows from
//     the tile's start, those beyond NT are whatever shared memory holds there,
//     and the accumulator lanes they fill are never read.
//   * kSwap, for M <= 32 and 224 channels an SM or more: the channels are the
//     MMA's 128 rows and the tokens its N = 16 or 32.  The same weight bytes then
//     take an eighth to a quarter of the multiplications, and with them of the
//     power, which in a long stream holds the SM clock down (8 x 34816 x 5120
//     back to back: 28.0 us swapped, 29.0 not; 8 x 151936 x 5120: 117 and 124;
//     in short runs 27.4 and 26.9, 115 and 116).  In a decode step of 16 layers
//     (norm, projections of 24640 and 5120 channels, norm, MLP 34816 / 17408)
//     and a head of 151936 channels, where those two widths run swapped: 1502,
//     1510 and 1560 us for 1, 8 and 32 tokens, 1528, 1552 and 1602 with none
//     swapped.  With fewer channels the fixed tile height fills the rounds worse
//     (32 x 24640 x 5120: 22.4 us swapped, 21.4 not; 1 x 5120 x 5120: 8.5 and 7.3).
//   * kSplit, where the tiles are few or narrow and K is long: a cluster of 2, 4
//     or 8 CTAs shares a tile's K, and each of them then owns a slice of the
//     tile's columns, to which the others' sums come through distributed shared
//     memory.  A narrow tile spends its time bringing the tokens in again (they
//     weigh more than its channels) at a rate that one SM bounds; wider tiles
//     with a part of K each bring in less.  The exchange costs 2 us and more:
//     100 x 5120 x 17408 19.6 us, 27.2 by whole tiles; 128 x 2048 x 17408 12.2
//     and 25.4; 16 x 2048 x 17408 10.0 and 13.7; 1 x 256 x 17408 6.9 and 12.4
//     (weights from memory).  Near the border the rule may miss: 64 x 5120 x 5120
//     takes 8.9 shared, 8.3 whole.
// Common to all:
//   * A pipeline stage holds U = 1, 2, 4 or 8 steps of 128 values of K, the
//     most that 58 KB take: each stage costs the MMA warp a handshake during
//     which the tensor pipe idles, and each operand one copy.
//   * Persistent (but for kSplit, one tile a cluster): the ring runs across
//     tiles, two accumulators of 256 columns.
//   * Launched as a programmatic dependent: every role that touches global
//     memory first waits for the previous grid (griddepcontrol.wait); the
//     first ring of weights is prefetched into L2 before that (5 to 7 % of a
//     call, measured for 24640 and 34816 channels).
// Bound by memory: 8 x 34816 x 5120 27.4 us = 6.5 TB/s, 1 x 24640 x 5120 20.0 us
// = 6.3 TB/s, 100 x 24640 x 5120 22.4 us = 5.9 TB/s, 1 x 5120 x 17408 16.7 us =
// 5.3 TB/s, 8 x 151936 x 5120 115 us = 6.8 TB/s (CUDA-graph replay).  Small
// products are bound by what a launch costs around its stream: 16 x 2048 x 2048
// 3.6 us, 1 x 5120 x 5120 7.2 us for 26 MB.
//
// Roles (10 warps): 0 TMA producer; 1 TMEM owner and MMA issuer; 2..9 epilogue,
// two warps per TMEM lane quarter on alternate 16-column chunks.  Every wait is
// bounded; on a timeout all roles stop and drain what is in flight.

constexpr int kFewThreads = 320;
constexpr int kFewMaxTokens = 128;
constexpr int kSwapTokens = 32;                      // at most: channels as the MMA's rows
constexpr int kSwapSteps = 2;                        // k-steps per stage of its tiles
constexpr int kFewMaxStages = 16;
constexpr int kFewMaxBN = 256;
constexpr uint32_t kFewSmem = 227 * 1024;            // whole: one CTA per SM
constexpr uint32_t kFewBars = (2 * kFewMaxStages + 5) * 8;
constexpr uint32_t kFewScales = 2 * kFewMaxBN * 4;    // channel scales, one set per accumulator
constexpr uint32_t kFewRing = (kFewSmem - 1024 - kFewBars - kFewScales - 16) / 1024 * 1024;

struct FewArgs {
    const float* sa;
    const float* sw;
    uint16_t* y;
    int64_t ldy;
    int M, N, K;
    int n_tiles, k_steps;
    int nt;          // token rows loaded: M rounded up to 8 (16 when swapped)
    int bn;          // channels per tile
    int wide;        // one copy brings a stage's U steps of an operand
    int stages;
    int splits;      // CTAs of a cluster that share a tile's K
    uint64_t timeout_ns;
    int* status;
};

// k-steps per stage and ring depth of a tile shape.
__host__ __device__ constexpr void few_config(int nt, int bn, int* u, int* stages) {
    const int step = (nt + bn) * kStepBytes;
    int uu = 58 * 1024 / step;
    uu = uu >= 8 ? 8 : uu >= 4 ? 4 : uu >= 2 ? 2 : 1;
    int st = static_cast<int>(kFewRing) / (uu * step);
    *u = uu;
    *stages = st > kFewMaxStages ? kFewMaxStages : st;
}

constexpr bool swap_steps_match() {
    for (int nt = 16; nt <= kSwapTokens; nt += 16) {
        int u = 0, st = 0;
        few_config(nt, kRows, &u, &st);
        if (u != kSwapSteps) return false;
    }
    return true;
}
static_assert(swap_steps_match(), "the swapped form is built for one number of k-steps per stage");

// Every shape keeps at least three stages, and the MMA's 128 token rows from
// the last A tile's start end inside the ring (the B tiles follow the A tiles).
constexpr bool few_configs_fit() {
    for (int nt = 8; nt <= kFewMaxTokens; nt += 8)
        for (int bn = 16; bn <= kFewMaxBN; bn += 16) {
            int u = 0, st = 0;
            few_config(nt, bn, &u, &st);
            if (st < 3 || static_cast<uint32_t>(st * u * (nt + bn) * kStepBytes) > kFewRing) return false;
            if (st * u * bn < kRows - nt) return false;
        }
    return true;
}
static_assert(few_configs_fit(), "a few-token configuration does not fit");
static_assert(kFewRing >= kMaxExchange, "the ring takes in the other CTAs' sums");
static_assert(kFewSmem > 228 * 1024 / 2, "two CTAs could share an SM and its 512 TMEM columns");

template <int U, bool kSwap, bool kSplit>
__global__ void __launch_bounds__(kFewThreads, 1)
int8_gemm_few_kernel(const __grid_constant__ CUtensorMap tmap_a,
                     const __grid_constant__ CUtensorMap tmap_w, const FewArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int STAGES = args.stages, BN = args.bn;
    const uint32_t a_step = static_cast<uint32_t>(args.nt) * kStepBytes;
    const uint32_t b_step = static_cast<uint32_t>(BN) * kStepBytes;
    const uint32_t off_b = static_cast<uint32_t>(STAGES * U) * a_step;
    float* s_scales = reinterpret_cast<float*>(smem + kFewRing);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kFewRing + kFewScales);
    uint64_t* empty = full + kFewMaxStages;
    uint64_t* tmem_full = empty + kFewMaxStages;        // [2]
    uint64_t* tmem_empty = tmem_full + 2;               // [2]
    uint64_t* drain = tmem_empty + 2;
    uint32_t* s_tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem_base + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int k_stages = (args.k_steps + U - 1) / U;     // stages per tile
    // this CTA's tiles and its stages of each: all, or its part of one tile's
    const int rank = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
    const int first = kSplit ? static_cast<int>(blockIdx.x) / args.splits : static_cast<int>(blockIdx.x);
    const int stride = kSplit ? args.n_tiles : static_cast<int>(gridDim.x);
    const int ks0 = kSplit ? rank * k_stages / args.splits : 0;
    const int ks1 = kSplit ? (rank + 1) * k_stages / args.splits : k_stages;
    grid_launch_dependents();

    if (warp == 0) {
        if (lane < STAGES) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < 2) {
            mbar_init(&tmem_full[lane], 1);
            mbar_init(&tmem_empty[lane], kEpiWarps);
        }
        if (lane == 0) {
            mbar_init(drain, 1);
            *s_abort = 0;
            prefetch_tmap(&tmap_a);
            prefetch_tmap(&tmap_w);
        }
        fence_mbar_init();
        __syncwarp();
        named_barrier_arrive(2, kFewThreads);            // the stream starts without the others
    } else {
        if (warp == 1) {
            tmem_alloc(s_tmem_base, 512);
            tmem_relinquish();
        }
        tc_fence_before();
        named_barrier_sync(2, kFewThreads);
        tc_fence_after();
    }
    const uint32_t tmem_base = warp == 0 ? 0u : *s_tmem_base;

    // The two feeding roles run as whole warps with one lane issuing.  A
    // wait that gives up raises `failed`; from then on the role's waits return
    // at once and it issues nothing.
    const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
    const bool leader = elect_one();
    if (warp == 0) {
        // ---------------- TMA producer ----------------
        // While the previous grid finishes, the first ring of weights moves
        // into L2 (a hint: nothing of it is read before the wait).
        if (leader && args.wide) {
            const int ahead = min(ks0 + STAGES, ks1);
            for (int ks = ks0; ks < ahead; ++ks)
                tma_prefetch_3d(&tmap_w, 0, first * BN, ks * U);
        }
        grid_dependency_wait();
        const uint64_t pol_w = l2_policy_evict_first();   // each weight byte is read once
        const uint64_t pol_a = l2_policy_evict_last();    // tokens are read by every tile
        uint32_t issued = 0, issued_parity = 0;
        bool failed = false;
        int stage = 0;
        uint32_t phase = 0;
        bool ready = true;                                // the ring starts empty
        for (int nt = first; nt < args.n_tiles; nt += stride) {
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!ready) failed |= !mbar_spin(empty0 + 8 * stage, phase ^ 1u, failed ? 1 : kSpinTries);
                const int next = stage + 1 == STAGES ? 0 : stage + 1;
                const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
                ready = mbar_peek(empty0 + 8 * next, next_phase ^ 1u);
                const int k0 = ks * U;
                uint8_t* sb = smem + off_b + stage * U * b_step;
                uint8_t* sa = smem + stage * U * a_step;
                if (leader && !failed) {
                    if (args.wide) {
                        // steps beyond K read as zeros, and count as bytes
                        mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(U) * (a_step + b_step));
                        tma_load_3d(sb, &tmap_w, &full[stage], 0, nt * BN, k0, pol_w);
                        tma_load_3d(sa, &tmap_a, &full[stage], 0, 0, k0, pol_a);
                    } else {
                        const int steps = min(U, args.k_steps - k0);
                        mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(steps) * (a_step + b_step));
                        for (int i = 0; i < steps; ++i) {
                            tma_load_3d(sb + i * b_step, &tmap_w, &full[stage], (k0 + i) * kStepBytes,
                                        nt * BN, 0, pol_w);
                            tma_load_3d(sa + i * a_step, &tmap_a, &full[stage], (k0 + i) * kStepBytes, 0, 0,
                                        pol_a);
                        }
                    }
                }
                __syncwarp();
                if (!failed) {
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                }
                stage = next;
                phase = next_phase;
            }
        }
        if (__any_sync(0xFFFFFFFFu, failed) && lane == 0) {
            *s_abort = 1;
            atomicExch(args.status, kDevTimeout);
            // leave no copy in flight: wait (bounded) for every stage issued
            int local_abort = 0;
            for (int st = 0; st < STAGES; ++st)
                if (issued & (1u << st))
                    mbar_wait_bounded(&full[st], (issued_parity >> st) & 1u, args.timeout_ns,
                                      &local_abort, args.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        // nothing here reads memory; the bounded waits below begin when the
        // previous grid, however long it takes, has finished
        grid_dependency_wait();
        // D's rows are the tokens, or with kSwap the channels
        const uint32_t idesc = kSwap ? int8_idesc(kRows, args.nt) : int8_idesc(args.nt <= 64 ? 64 : kRows, BN);
        const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(kSwap ? smem + off_b : smem));
        const uint64_t db0 = sdesc_kmajor_sw128(smem_u32(kSwap ? smem : smem + off_b));
        const uint32_t da_step = (kSwap ? b_step : a_step) >> 4;
        const uint32_t db_step = (kSwap ? a_step : b_step) >> 4;
        const int last_n = (args.K - (k_stages - 1) * U * kStepBytes + 31) / 32;   // MMAs of the last stage
        const uint32_t acc_empty0 = smem_u32(tmem_empty);
        bool failed = false;
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ready = false;
        for (int nt = first; nt < args.n_tiles; nt += stride) {
            failed |= !mbar_spin(acc_empty0 + 8 * acc, acc_phase ^ 1u, failed ? 1 : kSpinTries);
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * 256;
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!ready) failed |= !mbar_spin(full0 + 8 * stage, phase, failed ? 1 : kSpinTries);
                tc_fence_after();
                const int next = stage + 1 == STAGES ? 0 : stage + 1;
                const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
                ready = mbar_peek(full0 + 8 * next, next_phase);
                // descriptor start addresses advance by 2 per 32 bytes of K
                const uint64_t da = da0 + static_cast<uint64_t>(stage * U) * da_step;
                const uint64_t db = db0 + static_cast<uint64_t>(stage * U) * db_step;
                if (leader && !failed) {
                    if (ks + 1 < k_stages) {
#pragma unroll
                        for (int i = 0; i < U; ++i)
#pragma unroll
                            for (int j = 0; j < kStepBytes / 32; ++j)
                                tc_mma_i8(d_tmem, da + i * da_step + 2 * j, db + i * db_step + 2 * j, idesc,
                                          static_cast<uint32_t>((ks - ks0) | i | j));
                    } else {
                        // the last stage ends with K
                        for (int i = 0; i < last_n; ++i) {
                            const uint32_t j = 2 * (i & 3);
                            tc_mma_i8(d_tmem, da + (i >> 2) * da_step + j, db + (i >> 2) * db_step + j, idesc,
                                      static_cast<uint32_t>((ks - ks0) | i));
                        }
                    }
                    tc_commit(&empty[stage]);
                    if (ks == ks1 - 1) tc_commit(&tmem_full[acc]);
                }
                __syncwarp();
                stage = next;
                phase = next_phase;
            }
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
        // every tcgen05 operation issued above has finished before TMEM is freed
        if (__any_sync(0xFFFFFFFFu, failed) && lane == 0) {
            *s_abort = 1;
            atomicExch(args.status, kDevTimeout);
        }
        __syncwarp();
        if (elect_one()) {
            tc_commit(drain);
            int local_abort = 0;
            mbar_wait_bounded(drain, 0, args.timeout_ns, &local_abort, args.status);
        }
        __syncwarp();
    } else if constexpr (kSwap) {
        // ---------------- epilogue (warps 2..9), rows of D are channels ----------------
        // lane -> channel, 16 tokens at a time; a warp's stores of one token are
        // consecutive in memory.
        const int q = warp & 3;
        const int half = (warp - 2) >> 2;
        const int tid = threadIdx.x - 64;
        const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        grid_dependency_wait();
        if (tid < args.M) s_scales[tid] = args.sa[tid];
        named_barrier_sync(1, 32 * kEpiWarps);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int nt = first; nt < args.n_tiles; nt += stride) {
            const int n = nt * kRows + q * 32 + lane;
            const bool mine = n < args.N;
            const float sw = mine ? args.sw[n] : 0.0f;      // on its way while the MMAs run
            if (!mbar_wait_warp(&tmem_full[acc], acc_phase, args.timeout_ns, s_abort, args.status)) break;
            tc_fence_after();
            for (int c = half * 16; c < args.M; c += 32) {
                uint32_t r[16];
                tmem_ld_16cols(tq + acc * 256 + c, r);
                tmem_ld_wait();
                if (mine) {
                    uint16_t* yp = args.y + static_cast<int64_t>(c) * args.ldy + n;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < args.M)
                            yp[j * args.ldy] = __bfloat16_as_ushort(__float2bfloat16_rn(
                                scale_f32(static_cast<int32_t>(r[j]), s_scales[c + j], sw)));
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tmem_empty[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    } else if constexpr (kSplit) {
        // ---------------- epilogue (warps 2..9): this CTA's sums are complete ----------------
        const int tid = threadIdx.x - 64, n = first * BN + tid;
        grid_dependency_wait();
        s_scales[tid] = tid < BN && n < args.N ? args.sw[n] : 0.0f;
        mbar_wait_warp(&tmem_full[0], 0, args.timeout_ns, s_abort, args.status);
        __syncwarp();
    } else {
        // ---------------- epilogue (warps 2..9) ----------------
        // lane -> token (the first 16 lanes of a quarter where D has 64 rows); 16
        // channels at a time, a 32-byte sector of the row, the next chunk's TMEM
        // load under way meanwhile.  The channels' scales pass through shared
        // memory while the MMAs run.
        constexpr int kChunks = kFewMaxBN / 32;       // per warp
        const int q = warp & 3;                       // TMEM lane quarter of this warp
        const int half = (warp - 2) >> 2;
        const int per_q = args.nt <= 64 ? 16 : 32;
        const int m0 = q * per_q;
        const bool mine = lane < per_q && m0 + lane < args.M;
        const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * 16;
        const int tid = threadIdx.x - 64;
        grid_dependency_wait();
        const float sa = mine ? args.sa[m0 + lane] : 0.0f;
        uint16_t* yrow = args.y + static_cast<int64_t>(m0 + lane) * args.ldy;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool failed = false;      // a warp that gave up still meets the others at the barrier
        for (int nt = first; nt < args.n_tiles; nt += stride) {
            float* s_sw = s_scales + acc * kFewMaxBN;  // last read two tiles ago, before the previous barrier
            s_sw[tid] = nt * BN + tid < args.N && tid < BN ? args.sw[nt * BN + tid] : 0.0f;
            named_barrier_sync(1, 32 * kEpiWarps);
            if (!failed)
                failed = !mbar_wait_warp(&tmem_full[acc], acc_phase, args.timeout_ns, s_abort, args.status);
            if (failed) continue;
            tc_fence_after();
            // columns of the tile inside the matrix, in chunks of this warp
            const int cols = min(BN, args.N - nt * BN) - half * 16;
            const int nch = m0 < args.M && cols > 0 ? (cols + 31) / 32 : 0;   // warp-uniform
            const uint32_t src = tq + acc * 256;
            uint32_t r[2][16];
            if (nch > 0) tmem_ld_16cols(src, r[0]);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                if (i >= nch) break;
                tmem_ld_wait();
                if (i + 1 < nch) tmem_ld_16cols(src + 32 * (i + 1), r[(i + 1) & 1]);
                const int c = half * 16 + 32 * i, n0 = nt * BN + c;
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 w4 = *reinterpret_cast<const float4*>(s_sw + c + 4 * j);
                    o[2 * j] = scale_bf16x2(r[i & 1][4 * j], r[i & 1][4 * j + 1], sa, w4.x, w4.y);
                    o[2 * j + 1] = scale_bf16x2(r[i & 1][4 * j + 2], r[i & 1][4 * j + 3], sa, w4.z, w4.w);
                }
                if (mine) {
                    uint16_t* yp = yrow + n0;
                    if (n0 + 16 <= args.N) {
                        *reinterpret_cast<uint4*>(yp) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(yp + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (n0 + j < args.N) yp[j] = static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1)));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tmem_empty[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }

    if constexpr (kSplit) {
        const int m = (warp & 3) * (args.nt <= 64 ? 16 : 32) + lane;
        const Slices sl = {args.splits, rank, 1, 0, slice_chunks(BN, args.splits),
                           min(BN, args.N - first * BN + 15) / 16};
        exchange_and_store(sl, tmem_base, smem_u32(smem), s_scales, args.sa, args.y, args.ldy, m, m, args.M,
                           args.nt <= 64 ? 16 : 32, first * BN, args.N);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, 512);
    }
}

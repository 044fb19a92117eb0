// int8_gemm_few.cuh -- the int8 GEMM for few tokens (M <= 256), where the
// weight streams from memory once.  Included by int8_gemm.cu.
//
//   * Operands swapped: 128 weight rows sit on the MMA's M side and the
//     tokens, padded to NT = 16..256, on its N side, so a tile is 128 outputs
//     wide in n whatever the token count.
//   * K is split over a cluster of S CTAs, each accumulating its slice of a
//     tile in TMEM.  The sums are integers, so S is free to follow N: the
//     launcher picks the S whose rounds of tiles leave the fewest idle steps.
//   * Persistent: cluster c takes weight tiles c, c + C, c + 2C, ...; the
//     shared-memory ring runs across tiles, so weight loads stay in flight
//     while earlier tiles drain.
//   * S > 1: the partial sums are reduced through distributed shared memory,
//     in units of up to kFewChunk tokens.  Every CTA pushes its partials of a
//     row to the CTA that owns the row (R = 128 / S rounded up to a multiple
//     of 4 rows each); the owner adds them, scales and stores.  Handshakes are
//     mbarriers arrived on across the cluster.
//   * S = 1: the accumulator is scaled and stored by the warps that read it.
//   * Launched as a programmatic dependent: every role that touches global
//     memory first waits for the previous grid (griddepcontrol.wait).
//
// Roles (10 warps): 0 TMA producer; 1 TMEM owner and MMA issuer; 2..5 readers
// of the accumulator (one per TMEM lane quarter: push partials, or store for
// S = 1); 6..9 reducers.  Every wait is bounded; on a timeout all roles stop,
// drain what is in flight and meet at the final cluster barrier.

constexpr int kFewThreads = 320;
constexpr int kFewMaxTokens = 256;
constexpr int kFewMaxSplit = 8;
constexpr int kFewMaxStages = 10;
constexpr int kFewMaxAcc = 4;
constexpr int kFewMaxParts = 4;
constexpr int kFewChunk = 64;                       // tokens per exchanged unit
constexpr uint32_t kFewBudget = 216 * 1024;         // ring + partial buffers
constexpr uint32_t kFewMinSmem = 116 * 1024;        // > half an SM: one CTA per SM

struct FewArgs {
    const float* sa;
    const float* sw;
    uint16_t* y;
    int64_t ldy;
    int M, N, K;
    int n_tiles, k_steps;
    int nt;          // MMA N: tokens padded to a multiple of 16
    int split;       // CTAs per cluster along K
    int stages;      // ring depth
    int nparts;      // partial-sum buffers (0 when split == 1)
    int nacc;        // TMEM accumulators, 512 / nacc columns apart
    uint64_t timeout_ns;
    int* status;
};

// Rows of a tile that each CTA of the cluster owns, and a unit's bytes.
__host__ __device__ constexpr int few_rows(int split) { return ((kRows + split - 1) / split + 3) / 4 * 4; }
__host__ __device__ constexpr uint32_t few_part_bytes(int nt, int split) {
    return static_cast<uint32_t>((nt < kFewChunk ? nt : kFewChunk) * few_rows(split) * split * 4);
}
__host__ __device__ constexpr uint32_t few_stage_bytes(int nt) {
    return static_cast<uint32_t>((kRows + nt) * kStepBytes);
}

struct FewLayout {
    uint32_t off_x, off_part, off_bar, off_scale, off_misc, bytes;
};

__host__ __device__ constexpr FewLayout few_layout(int nt, int split, int stages, int nparts) {
    FewLayout L{};
    L.off_x = static_cast<uint32_t>(stages) * kRows * kStepBytes;
    L.off_part = L.off_x + static_cast<uint32_t>(stages) * nt * kStepBytes;
    L.off_bar = L.off_part + static_cast<uint32_t>(nparts) * few_part_bytes(nt, split);
    L.off_scale = L.off_bar + (2 * kFewMaxStages + 2 * kFewMaxAcc + 2 * kFewMaxParts + 1) * 8;
    L.off_misc = L.off_scale + kFewMaxTokens * 4;
    const uint32_t bytes = L.off_misc + 16 + 1024;   // + slack for 1024-byte alignment
    L.bytes = bytes < kFewMinSmem ? kFewMinSmem : bytes;
    return L;
}

// Accumulators, partial buffers and ring depth.
__host__ __device__ constexpr void few_config(int nt, int split, int* stages, int* nparts, int* nacc) {
    const int np = split == 1 ? 0 : (nt <= 16 ? 4 : 2);
    int st = static_cast<int>((kFewBudget - np * few_part_bytes(nt, split)) / few_stage_bytes(nt));
    *stages = st > kFewMaxStages ? kFewMaxStages : st;
    *nparts = np;
    *nacc = nt <= 128 ? 4 : 2;
}

constexpr bool few_configs_fit() {
    for (int nt = 16; nt <= kFewMaxTokens; nt += 16)
        for (int s = 1; s <= kFewMaxSplit; ++s) {
            int st = 0, np = 0, na = 0;
            few_config(nt, s, &st, &np, &na);
            const FewLayout L = few_layout(nt, s, st, np);
            if (st < 2 || L.bytes > 227 * 1024 || np > kFewMaxParts || na > kFewMaxAcc || nt > 512 / na)
                return false;
            if (few_rows(s) * (s - 1) >= kRows || few_rows(s) * s < kRows) return false;
            if (L.off_x % 1024 != 0 || L.off_part % 16 != 0 || L.off_bar % 8 != 0) return false;
        }
    return true;
}
static_assert(few_configs_fit(), "a few-token configuration exceeds a hardware limit");
static_assert(2 * kFewMinSmem > 228 * 1024, "two CTAs could share an SM and its 512 TMEM columns");

__global__ void __launch_bounds__(kFewThreads, 1)
int8_gemm_few_kernel(const __grid_constant__ CUtensorMap tmap_w,
                     const __grid_constant__ CUtensorMap tmap_x,
                     const __grid_constant__ FewArgs args) {
    const int NT = args.nt, S = args.split, STAGES = args.stages, NPART = args.nparts, NACC = args.nacc;
    const uint32_t ACC_STRIDE = 512 / NACC;
    const FewLayout L = few_layout(NT, S, STAGES, NPART);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.off_bar);
    uint64_t* empty = full + kFewMaxStages;
    uint64_t* tmem_full = empty + kFewMaxStages;
    uint64_t* tmem_empty = tmem_full + kFewMaxAcc;
    uint64_t* part_full = tmem_empty + kFewMaxAcc;    // partials of my rows landed
    uint64_t* part_free = part_full + kFewMaxParts;   // every owner done with a buffer
    uint64_t* drain = part_free + kFewMaxParts;
    float* s_sa = reinterpret_cast<float*>(smem + L.off_scale);
    uint32_t* s_tmem_base = reinterpret_cast<uint32_t*>(smem + L.off_misc);
    volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L.off_misc + 4);
    int32_t* part = reinterpret_cast<int32_t*>(smem + L.off_part);   // [NPART][S][CH][R]

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    grid_launch_dependents();
    const int rank = static_cast<int>(cluster_ctarank());
    const int cluster_id = blockIdx.x / S;
    const int num_clusters = gridDim.x / S;
    const int k_begin = (rank * args.k_steps) / S;
    const int k_end = ((rank + 1) * args.k_steps) / S;
    const int R = few_rows(S);
    const int CH = NT < kFewChunk ? NT : kFewChunk;
    const int chunks = (args.M + CH - 1) / CH;          // units per tile
    const int owned = min(R, kRows - rank * R);         // rows of a tile this CTA owns

    if (warp == 0) {
        if (lane < STAGES) {
            mbar_init(&full[lane], 1);
            mbar_init(&empty[lane], 1);
        }
        if (lane < kFewMaxAcc) {
            mbar_init(&tmem_full[lane], 1);
            mbar_init(&tmem_empty[lane], 4);                              // the four reader warps
        }
        if (lane < NPART) {
            mbar_init(&part_full[lane], static_cast<uint32_t>(owned * S));  // each row from each CTA
            mbar_init(&part_free[lane], 4 * S);                           // 4 reducer warps of each CTA
        }
        if (lane == 0) {
            mbar_init(drain, 1);
            *s_abort = 0;
            prefetch_tmap(&tmap_w);
            prefetch_tmap(&tmap_x);
        }
        fence_mbar_init();
        __syncwarp();
        named_barrier_arrive(2, kFewThreads);
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
    // every thread arrives now; the roles that touch a peer wait before their
    // first remote access, the others at the end
    cluster_arrive();

    const int last_kb = args.k_steps - 1;
    const int last_n = (args.K - last_kb * kStepBytes + 31) / 32;   // MMAs of the last k-step
    const uint32_t s_w0 = smem_u32(smem);
    const uint32_t s_x0 = smem_u32(smem + L.off_x);
    const uint32_t x_stride = static_cast<uint32_t>(NT) * kStepBytes;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        grid_dependency_wait();
        const uint64_t pol_w = l2_policy_evict_first();   // each weight byte is read once
        const uint64_t pol_x = l2_policy_evict_last();    // tokens are read by every tile
        const uint32_t tx = few_stage_bytes(NT);
        uint32_t issued = 0, issued_parity = 0;
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        for (int nt = cluster_id; nt < args.n_tiles && ok; nt += num_clusters) {
            for (int kb = k_begin; kb < k_end; ++kb) {
                if (!mbar_spin_warp(&empty[stage], phase ^ 1u, args.timeout_ns, s_abort, args.status)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[stage], tx);
                    tma_load_2d(smem + stage * (kRows * kStepBytes), &tmap_w, &full[stage],
                                kb * kStepBytes, nt * kRows, pol_w);
                    tma_load_2d(smem + L.off_x + stage * x_stride, &tmap_x, &full[stage],
                                kb * kStepBytes, 0, pol_x);
                }
                __syncwarp();
                issued |= 1u << stage;
                issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && lane == 0) {
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
        const uint32_t idesc = int8_idesc(kRows, NT);
        const uint64_t dw0 = sdesc_kmajor_sw128(s_w0);
        const uint64_t dx0 = sdesc_kmajor_sw128(s_x0);
        bool ok = true;
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        for (int nt = cluster_id; nt < args.n_tiles && ok; nt += num_clusters) {
            if (!mbar_spin_warp(&tmem_empty[acc], acc_phase ^ 1u, args.timeout_ns, s_abort, args.status)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * ACC_STRIDE;
            for (int kb = k_begin; kb < k_end; ++kb) {
                if (!mbar_spin_warp(&full[stage], phase, args.timeout_ns, s_abort, args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // descriptor start addresses advance by 2 per 32 bytes of K
                const uint64_t dw = dw0 + static_cast<uint64_t>(stage * (kRows * kStepBytes / 16));
                const uint64_t dx = dx0 + static_cast<uint64_t>(stage * (x_stride / 16));
                const uint32_t first = kb != k_begin;
                const int nmma = kb == last_kb ? last_n : kStepBytes / 32;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kStepBytes / 32; ++j)
                        if (j < nmma)
                            tc_mma_i8(d_tmem, dw + 2 * j, dx + 2 * j, idesc, first | static_cast<uint32_t>(j));
                    tc_commit(&empty[stage]);
                }
                __syncwarp();
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok && elect_one()) tc_commit(&tmem_full[acc]);
            __syncwarp();
            if (++acc == NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
        // every tcgen05 operation issued above has finished before TMEM is freed
        if (elect_one()) {
            tc_commit(drain);
            int local_abort = 0;
            mbar_wait_bounded(drain, 0, args.timeout_ns, &local_abort, args.status);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ---------------- accumulator readers (warps 2..5) ----------------
        const int q = warp & 3;                       // TMEM lane quarter of this warp
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        const int row = q * 32 + lane;
        const int owner = row / R;
        const int rr = row - owner * R;
        if (S == 1) {
            // the token scales are these warps' own here
            grid_dependency_wait();
            for (int t = threadIdx.x - 64; t < args.M; t += 128) s_sa[t] = args.sa[t];
            named_barrier_sync(1, 128);
        }
        const uint32_t part_owner = mapa_shared(smem_u32(part), static_cast<uint32_t>(owner));
        const uint32_t full_owner = mapa_shared(smem_u32(part_full), static_cast<uint32_t>(owner));
        cluster_wait();                               // the owners' barriers are initialised
        int acc = 0, pb = 0;
        uint32_t acc_phase = 0, free_phase = 1;       // the first pass over the buffers waits for nothing
        bool ok = true;
        for (int nt = cluster_id; nt < args.n_tiles && ok; nt += num_clusters) {
            const int n = nt * kRows + row;
            const float sw = S == 1 && n < args.N ? args.sw[n] : 0.0f;
            if (!mbar_wait_warp(&tmem_full[acc], acc_phase, args.timeout_ns, s_abort, args.status)) break;
            tc_fence_after();
            const uint32_t src = tmem_base + lane_base + acc * ACC_STRIDE;
            if (S == 1) {
                uint16_t* yn = args.y + n;
                for (int c = 0; c < args.M; c += 16) {
                    uint32_t r[16];
                    tmem_ld_16cols(src + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < args.M && n < args.N)
                            yn[static_cast<int64_t>(c + j) * args.ldy] =
                                scale_bf16(static_cast<int32_t>(r[j]), s_sa[c + j], sw);
                }
            } else {
                for (int ch = 0; ch < chunks; ++ch) {
                    int got = 1;
                    if (lane == 0)
                        got = mbar_wait_cluster_bounded(&part_free[pb], free_phase, args.timeout_ns,
                                                        s_abort, args.status);
                    if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
                        ok = false;
                        break;
                    }
                    const int c0 = ch * CH, cn = min(CH, args.M - c0);
                    const uint32_t dst = part_owner + static_cast<uint32_t>(
                        (((pb * S + rank) * CH) * R + rr) * 4);
                    for (int c = 0; c < cn; c += 16) {
                        uint32_t r[16];
                        tmem_ld_16cols(src + c0 + c, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j < cn)
                                st_shared_cluster_f32(dst + static_cast<uint32_t>((c + j) * R * 4),
                                                      __uint_as_float(r[j]));
                    }
                    mbar_arrive_cluster(full_owner + pb * 8);   // my row's partials have landed
                    if (++pb == NPART) {
                        pb = 0;
                        free_phase ^= 1u;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tmem_empty[acc]);       // the MMA may reuse it
            if (++acc == NACC) {
                acc = 0;
                acc_phase ^= 1u;
            }
        }
    } else if (S > 1) {
        // ---------------- reducers (warps 6..9) ----------------
        // thread -> 4 consecutive owned rows and every tstep-th token
        const int tid = threadIdx.x - 6 * 32;
        grid_dependency_wait();
        for (int t = tid; t < args.M; t += 128) s_sa[t] = args.sa[t];
        named_barrier_sync(1, 128);
        cluster_wait();                               // the peers' barriers are initialised
        const int ngroups = owned / 4;
        const int tstep = 128 / ngroups;
        const int t_first = tid / ngroups;            // >= tstep: this thread has no token
        const int rg = 4 * (tid - t_first * ngroups);
        int pb = 0;
        uint32_t use = 0;
        bool ok = true;
        for (int nt = cluster_id; nt < args.n_tiles && ok; nt += num_clusters) {
            const int n0 = nt * kRows + rank * R + rg;
            float sw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) sw[u] = n0 + u < args.N ? args.sw[n0 + u] : 0.0f;
            for (int ch = 0; ch < chunks; ++ch) {
                int got = 1;
                if (lane == 0)
                    got = mbar_wait_cluster_bounded(&part_full[pb], use, args.timeout_ns, s_abort, args.status);
                if (!__shfl_sync(0xFFFFFFFFu, got, 0)) {
                    ok = false;
                    break;
                }
                // this lane's own acquire (lane 0 waited for the phase)
                mbar_try_wait_cluster(&part_full[pb], use);
                const int c0 = ch * CH, cn = min(CH, args.M - c0);
                const int32_t* pbuf = part + static_cast<size_t>(pb) * S * CH * R + rg;
                if (t_first < tstep) {
                    for (int t = t_first; t < cn; t += tstep) {
                        int4 sum = *reinterpret_cast<const int4*>(pbuf + t * R);
                        for (int s = 1; s < S; ++s) {
                            const int4 p = *reinterpret_cast<const int4*>(pbuf + (s * CH + t) * R);
                            sum.x += p.x, sum.y += p.y, sum.z += p.z, sum.w += p.w;
                        }
                        const float sa = s_sa[c0 + t];
                        uint16_t* yp = args.y + static_cast<int64_t>(c0 + t) * args.ldy + n0;
                        const uint32_t v0 = scale_bf16(sum.x, sa, sw[0]), v1 = scale_bf16(sum.y, sa, sw[1]);
                        const uint32_t v2 = scale_bf16(sum.z, sa, sw[2]), v3 = scale_bf16(sum.w, sa, sw[3]);
                        if (n0 + 3 < args.N) {
                            *reinterpret_cast<uint2*>(yp) = make_uint2(v0 | (v1 << 16), v2 | (v3 << 16));
                        } else {
                            if (n0 < args.N) yp[0] = static_cast<uint16_t>(v0);
                            if (n0 + 1 < args.N) yp[1] = static_cast<uint16_t>(v1);
                            if (n0 + 2 < args.N) yp[2] = static_cast<uint16_t>(v2);
                        }
                    }
                }
                __syncwarp();
                // this warp has consumed buffer pb: tell every CTA of the cluster
                if (lane < S)
                    mbar_arrive_cluster_relaxed(
                        mapa_shared(smem_u32(&part_free[pb]), static_cast<uint32_t>(lane)));
                if (++pb == NPART) {
                    pb = 0;
                    use ^= 1u;
                }
            }
        }
    }

    // no CTA leaves while a peer may still write into its shared memory or
    // arrive on its barriers
    tc_fence_before();
    __syncwarp();
    if (warp < 2 || (warp >= 6 && S == 1)) cluster_wait();   // the roles that did not wait above
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, 512);
}

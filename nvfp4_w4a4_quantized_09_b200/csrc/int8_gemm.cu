// int8_gemm.cu -- product of two int8 matrices with one FP32 scale per token
// (row of A) and per channel (row of W):
//
//   acc[m, n] = sum_k a[m, k] * w[n, k]             (exact in 32 bits)
//   y[m, n] = bf16( fl32( fl32( fl32(acc) * sa[m] ) * sw[n] ) )
//
// K is at most 131056, so |acc| <= 128 * 128 * K < 2^31: the sum cannot
// overflow, and integer addition gives the same bits in any order.  Tile sizes
// and splits of K are therefore free choices that no result depends on; both
// kernels and every configuration of them give the same bits.
//
//   M <= 128   int8_gemm_few_kernel (int8_gemm_few.cuh): one CTA per tile of all
//              tokens x BN channels, the weight streamed once.
//   M > 128    int8_gemm_pair_kernel: a CTA pair per 256 x BN tile.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "host_common.h"
#include "int8_mma.cuh"
#include "nvfp4.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int64_t kMaxK = 131056;
constexpr int kRows = 128;                      // rows of an operand tile per CTA
constexpr int kStepBytes = 128;                 // values of K per pipeline stage
constexpr uint64_t kTimeoutNs = 1000000000ull;  // 1 s per wait

// The product's value: the sum rounded to binary32, both scales, BF16 bits.
__device__ __forceinline__ float scale_f32(int32_t acc, float sa, float sw) {
    return __fmul_rn(__fmul_rn(__int2float_rn(acc), sa), sw);
}
// Two neighbouring values as packed BF16 (the low half first).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t acc0, uint32_t acc1, float sa, float sw0, float sw1) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(scale_f32(static_cast<int32_t>(acc0), sa, sw0),
                                                   scale_f32(static_cast<int32_t>(acc1), sa, sw1));
    return *reinterpret_cast<const uint32_t*>(&v);
}

constexpr int kEpiWarps = 8;                    // two per TMEM lane quarter
constexpr int kMaxSplits = 8;                   // CTAs of a cluster that share a tile's K

// A tile whose K the CTAs of a cluster share: `splits` of them (in the pair
// kernel pairs of them) hold sums of 128 rows x BN columns in TMEM, and number r
// owns the r-th slice (the last ones may be shorter, or empty).
struct Slices {
    int splits, rank;
    int step, offset;                           // owner r is CTA step * r + offset of the cluster
    int slice;                                  // chunks of 16 columns each owns
    int chunks;                                 // of the tile inside the matrix
};
__host__ __device__ constexpr int slice_chunks(int bn, int splits) { return (bn / 16 + splits - 1) / splits; }
// What an owner's shared memory takes in: 8 KB a chunk from each of the others.
constexpr uint32_t kMaxExchange = 7 * 2 * 8192;
constexpr bool exchanges_fit() {
    for (int splits = 2; splits <= kMaxSplits; splits *= 2)
        for (int bn = 16; bn <= 256; bn += 16)
            if (static_cast<uint32_t>(splits - 1) * slice_chunks(bn, splits) * 8192 > kMaxExchange) return false;
    return true;
}
static_assert(exchanges_fit(), "the sums of a tile do not fit where its ring was");

// By all threads of every CTA of the cluster, once its sums are complete.  Every
// CTA stores its sums of the other slices into their owners' shared memory,
// where the ring (at `ring`) has served; the owner adds them to its own and
// stores the product.  Integers: the order is free.  A lane is a row (`m` of the
// tile, `row` of the matrix; `per_q` of a warp's lanes are in use), 4 columns of
// consecutive rows are consecutive 16 bytes.
__device__ __forceinline__ void exchange_and_store(const Slices& sl, uint32_t tmem_base, uint32_t ring,
                                                   const float* s_sw, const float* gsa, uint16_t* y, int64_t ldy,
                                                   int m, int row, int M, int per_q, int n_base, int N) {
    constexpr uint32_t kUnit = kRows * 16;      // 4 columns of all rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = (warp - 2) >> 2;
    const bool warp_mine = warp >= 2 && row - lane < M;
    const bool mine = warp_mine && lane < per_q && row < M;
    const uint32_t tq = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    ring += static_cast<uint32_t>(m) * 16;
    cluster_sync();                             // every ring has been read
    tc_fence_after();
    if (warp_mine) {
        for (int c = half; c < sl.chunks; c += 2) {
            const int owner = c / sl.slice;
            if (owner == sl.rank) continue;
            uint32_t r[16];
            tmem_ld_16cols(tq + 16 * c, r);
            tmem_ld_wait();
            const int slot = (sl.rank - (sl.rank > owner)) * sl.slice + c - owner * sl.slice;
            const uint32_t to = mapa_shared(ring, sl.step * owner + sl.offset) + static_cast<uint32_t>(slot) * 4 * kUnit;
            if (mine)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    st_cluster_v4(to + g * kUnit, r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]);
            __syncwarp();
        }
    }
    __syncwarp();
    cluster_sync();                             // every sum has arrived
    if (warp_mine) {
        const float sa = mine ? gsa[row] : 0.0f;
        const int c0 = sl.rank * sl.slice, end = min(sl.chunks, c0 + sl.slice);
        for (int c = c0 + half; c < end; c += 2) {
            uint32_t r[16];
            tmem_ld_16cols(tq + 16 * c, r);
            tmem_ld_wait();
            if (mine) {
                uint32_t from = ring + static_cast<uint32_t>(c - c0) * 4 * kUnit;
                for (int i = 1; i < sl.splits; ++i, from += static_cast<uint32_t>(sl.slice) * 4 * kUnit)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint4 v = lds128(from + g * kUnit);
                        r[4 * g] += v.x, r[4 * g + 1] += v.y, r[4 * g + 2] += v.z, r[4 * g + 3] += v.w;
                    }
                uint32_t o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    o[j] = scale_bf16x2(r[2 * j], r[2 * j + 1], sa, s_sw[16 * c + 2 * j], s_sw[16 * c + 2 * j + 1]);
                const int n0 = n_base + 16 * c;
                uint16_t* yp = y + static_cast<int64_t>(row) * ldy + n0;
                if (n0 + 16 <= N) {
                    *reinterpret_cast<uint4*>(yp) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(yp + 8) = make_uint4(o[4], o[5], o[6], o[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (n0 + j < N) yp[j] = static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1)));
                }
            }
            __syncwarp();
        }
    }
    __syncwarp();
}

#include "int8_gemm_few.cuh"

// ---------------------------------------------------------------------------
// CTA-pair kernel (cta_group::2).  A cluster of two CTAs on two SMs computes a
// 256 x BN tile (BN a multiple of 32 up to 256, chosen by the launcher so that
// the tiles fill whole rounds of the pairs): each CTA loads its 128 rows of A
// and its BN / 2 rows of W per k-step of 128, the even CTA issues the MMAs
// (M = 256, N = BN, K = 32), accumulator rows 0..127 live in the even CTA's
// TMEM and 128..255 in the odd one's.  Two accumulators of 256 columns each:
// the epilogue drains one while the MMAs fill the other -- or, with wide tiles
// of 2 BN columns, both belong to one tile: A is loaded once for the two.
// With kSplit a cluster of two or four pairs shares a tile's K and each pair owns
// a slice of its columns, to which the others' sums come through distributed
// shared memory: for narrow products of long rows, whose k-steps cost the same
// however narrow the tile is (160 x 5120 x 17408 25 us, 36.3 by whole tiles; 256 x
// 2048 x 17408 17.3 and 36.8; 384 x 1024 x 28672 21.4 and 57; but 512 x 5120 x 5120
// 15.4 whole, 26 shared).
//   warp 0      TMA producer (both CTAs; bytes counted on the even CTA's barrier)
//   warp 1      MMA issuer (even CTA), TMEM owner
//   warps 2..9  epilogue: two warps per TMEM lane quarter take alternate
//               32-column chunks: scales, BF16, a 32 x 32 tile staged in the
//               64-byte swizzle and one TMA store of it (rows beyond M and
//               whole 16-byte pieces beyond N clipped by the tensor map)
// 8192 x 34816 x 5120 takes 780 us by itself (3.74 P op/s; the tensor pipe is
// busy 97 % of the SMs' active time), 885 us in short runs and 955 to 1015 us
// back to back, where the power limit holds the SMs at some 1.3 GHz.  Smaller
// products are bound by shared memory, which the copies' writes and the MMAs'
// reads share, and by how the tiles fill the rounds: 1000 x 5120 x 17408 61 to 63
// us, 1000 x 5120 x 5120 21.6 us, 512 x 24640 x 5120 48 us, 200 x 24640 x 5120 29
// us, 517 x 2051 x 1040 6.7 us.  With a short K the epilogue is as long as the
// k-steps of a tile and takes shared memory from them: 2178 x 11003 x 816 33 us
// (12 by bytes), 1088 x 12998 x 1232 24 us (11).  Six stages of 32 KB against
// five: 1000 and 1062 us for the
// largest; spinning feed waits against suspending ones: 70 and 78 us for 1000
// tokens; bands of 16 M tiles where A fits in L2: 2 to 3 % slower.
// ---------------------------------------------------------------------------
constexpr int kPairThreads = 320;
constexpr int kPairMaxStages = 8;
constexpr int kPairMaxBN = 256;
constexpr int kEpiBytes = 32 * 64;              // one staged 32 x 32 BF16 tile
constexpr int kEpiBufs = 2;
constexpr uint32_t kPairEpi = kEpiWarps * kEpiBufs * kEpiBytes;
constexpr uint32_t kPairBars = (2 * kPairMaxStages + 5) * 8;
constexpr uint32_t kPairSmem = 227 * 1024;      // whole: one CTA per SM
constexpr uint32_t kPairRing = (kPairSmem - 1024 - kPairEpi - kPairBars - 16) / 1024 * 1024;

struct PairArgs {
    const float* sa;
    const float* sw;
    uint16_t* y;
    int64_t ldy;
    int M, N, K;
    int m_tiles, n_tiles, k_steps;
    int group_m;                                // raster: m-tiles visited per n sweep
    int bn;                                     // columns of an accumulator
    int wide;                                   // 1: a tile fills both accumulators, 2 bn columns
    int stages;
    int splits;                                 // pairs of a cluster that share a tile's K
    uint64_t timeout_ns;
    int* status;
};

__host__ __device__ constexpr uint32_t pair_stage_bytes(int bn, int wide) {
    return static_cast<uint32_t>(kRows + ((bn / 2) << wide)) * kStepBytes;
}
__host__ __device__ constexpr int pair_stages(int bn, int wide) {
    return static_cast<int>(kPairRing / pair_stage_bytes(bn, wide)) < kPairMaxStages
               ? static_cast<int>(kPairRing / pair_stage_bytes(bn, wide)) : kPairMaxStages;
}
static_assert(kPairRing >= kMaxExchange, "the ring takes in the other pairs' sums");
static_assert(pair_stages(256, 0) >= 6 && pair_stages(256, 1) >= 4, "the widest tiles keep a deep ring");
static_assert(kPairSmem > 228 * 1024 / 2, "two CTAs could share an SM and its 512 TMEM columns");

__device__ __forceinline__ void pair_tile(int t, const PairArgs& a, int& mt, int& nt) {
    const int group_m = min(a.group_m, a.m_tiles);
    const int per_group = group_m * a.n_tiles;
    const int grp = t / per_group;
    const int first_m = grp * group_m;
    const int gsize = min(group_m, a.m_tiles - first_m);
    const int local = t - grp * per_group;
    mt = first_m + local % gsize;
    nt = local / gsize;
}

template <bool kSplit>
__global__ void __launch_bounds__(kPairThreads, 1)
int8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmap_a,
                      const __grid_constant__ CUtensorMap tmap_b,
                      const __grid_constant__ CUtensorMap tmap_y, const PairArgs args) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int STAGES = args.stages;
    const int BN = args.bn;
    constexpr uint32_t A_BYTES = kRows * kStepBytes;
    const int wide = args.wide;
    const int TN = BN << wide;                           // columns of a tile
    const uint32_t HALF_B = static_cast<uint32_t>(BN / 2) * kStepBytes;   // this CTA's rows of BN
    const uint32_t B_BYTES = HALF_B << wide;
    const uint32_t off_b = STAGES * A_BYTES;
    uint8_t* epi = smem + kPairRing;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + kPairEpi);
    uint64_t* empty = full + kPairMaxStages;
    uint64_t* tmem_full = empty + kPairMaxStages;       // [2]
    uint64_t* tmem_empty = tmem_full + 2;               // [2]
    uint64_t* drain = tmem_empty + 2;
    uint32_t* s_tmem_base = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem_base + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t ctarank = cluster_ctarank();
    const uint32_t rank = ctarank & 1u;                  // 0: issues the pair's MMAs
    const uint32_t even = kSplit ? ctarank & ~1u : 0u;   // the pair's even CTA in the cluster
    const int total_tiles = args.m_tiles * args.n_tiles;
    // this pair's tiles and its k-steps of each: all, or its part of one tile's
    const int split = static_cast<int>(even >> 1);
    const int pair = static_cast<int>(blockIdx.x) / (kSplit ? 2 * args.splits : 2);
    const int npairs = kSplit ? total_tiles : static_cast<int>(gridDim.x >> 1);
    const int kb0 = kSplit ? split * args.k_steps / args.splits : 0;
    const int kb1 = kSplit ? (split + 1) * args.k_steps / args.splits : args.k_steps;
    grid_launch_dependents();

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tmem_full[i], 1);
            mbar_init(&tmem_empty[i], 2 * kEpiWarps);    // both CTAs' epilogue warps
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        fence_mbar_init();
        prefetch_tmap(&tmap_a);
        prefetch_tmap(&tmap_b);
        prefetch_tmap(&tmap_y);
    }
    if (warp == 1) {
        tmem_alloc_pair(s_tmem_base, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                      // barriers of both CTAs initialised
    tc_fence_after();
    const uint32_t tmem_base = *s_tmem_base;
    const uint32_t full0_leader = mapa_shared(smem_u32(&full[0]), even);
    const uint32_t tmem_empty_leader = mapa_shared(smem_u32(tmem_empty), even);

    // The two feeding roles run as whole warps with one lane issuing.  A
    // wait that gives up raises `failed`; from then on the role's waits return
    // at once and it issues nothing.
    const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
    const bool leader = elect_one();
    if (warp == 0) {
        // ---------------- TMA producer (both CTAs) ----------------
        // With one M tile the weight streams from memory once, as for few
        // tokens: while the previous grid finishes, its first ring moves into
        // L2 (a hint: nothing of it is read before the wait).
        const bool once = args.m_tiles == 1;
        if (leader && once) {
            const int ahead = min(kb0 + STAGES, kb1);
            for (int kb = kb0; kb < ahead; ++kb)
                for (int h = 0; h <= wide; ++h)
                    tma_prefetch_2d(&tmap_b, kb * kStepBytes,
                                    pair * TN + h * BN + static_cast<int>(rank) * (BN / 2));
        }
        grid_dependency_wait();
        const uint64_t pol = l2_policy_evict_last();
        const uint64_t pol_w = once ? l2_policy_evict_first() : pol;
        int stage = 0;
        uint32_t phase = 0;
        uint32_t armed = 0, armed_parity = 0;   // stages the even CTA expects bytes on
        bool failed = false, ready = true;      // the ring starts empty
        for (int t = pair; t < total_tiles; t += npairs) {
            int mt, nt;
            pair_tile(t, args, mt, nt);
            const int ya = mt * 256 + static_cast<int>(rank) * kRows;
            const int yb = nt * TN + static_cast<int>(rank) * (BN / 2);
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!ready) failed |= !mbar_spin(empty0 + 8 * stage, phase ^ 1u, failed ? 1 : kSpinTries);
                const int next = stage + 1 == STAGES ? 0 : stage + 1;
                const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
                ready = mbar_peek(empty0 + 8 * next, next_phase ^ 1u);
                const uint32_t fb = full0_leader + stage * 8;
                if (leader && !failed) {
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (A_BYTES + B_BYTES));
                    tma_load_2d_pair(smem + stage * A_BYTES, &tmap_a, fb, kb * kStepBytes, ya, pol);
                    uint8_t* sb = smem + off_b + stage * B_BYTES;
                    tma_load_2d_pair(sb, &tmap_b, fb, kb * kStepBytes, yb, pol_w);
                    if (wide) tma_load_2d_pair(sb + HALF_B, &tmap_b, fb, kb * kStepBytes, yb + BN, pol_w);
                }
                __syncwarp();
                if (rank == 0 && !failed) {
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                }
                stage = next;
                phase = next_phase;
            }
        }
        if (__any_sync(0xFFFFFFFFu, failed) && lane == 0) {
            *s_abort = 1;
            atomicExch(args.status, kDevTimeout);
            // leave no copy of either CTA in flight on the stages armed here
            int local_abort = 0;
            for (int s = 0; s < STAGES; ++s)
                if (armed & (1u << s))
                    mbar_wait_bounded(&full[s], (armed_parity >> s) & 1u, args.timeout_ns,
                                      &local_abort, args.status);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer (even CTA) ----------------
            // nothing here reads memory; the bounded waits below begin when the
            // previous grid, however long it takes, has finished
            grid_dependency_wait();
            const uint32_t idesc = int8_idesc(256, BN);
            const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(smem));
            const uint64_t db0 = sdesc_kmajor_sw128(smem_u32(smem + off_b));
            const int last_kb = args.k_steps - 1;
            const int last_n = (args.K - last_kb * kStepBytes + 31) / 32;   // MMAs of the last k-step
            const uint32_t acc_empty0 = smem_u32(tmem_empty);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool failed = false, ready = false;
            for (int t = pair; t < total_tiles; t += npairs) {
                failed |= !mbar_spin(acc_empty0 + 8 * acc, acc_phase ^ 1u, failed ? 1 : kSpinTries);
                if (wide) failed |= !mbar_spin(acc_empty0 + 8, acc_phase ^ 1u, failed ? 1 : kSpinTries);
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!ready) failed |= !mbar_spin(full0 + 8 * stage, phase, failed ? 1 : kSpinTries);
                    tc_fence_after();
                    const int next = stage + 1 == STAGES ? 0 : stage + 1;
                    const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
                    ready = mbar_peek(full0 + 8 * next, next_phase);
                    // descriptor start addresses advance by 2 per 32 bytes of K
                    const uint64_t da = da0 + static_cast<uint64_t>(stage * (A_BYTES / 16));
                    const uint64_t db = db0 + static_cast<uint64_t>(stage * (B_BYTES / 16));
                    const int nmma = kb == last_kb ? last_n : kStepBytes / 32;
                    if (leader && !failed) {
#pragma unroll
                        for (int j = 0; j < kStepBytes / 32; ++j)
                            if (j < nmma)
                                tc_mma_i8_pair(d_tmem, da + 2 * j, db + 2 * j, idesc,
                                               static_cast<uint32_t>((kb - kb0) | j));
                        if (wide) {
                            const uint64_t db1 = db + (HALF_B >> 4);
#pragma unroll
                            for (int j = 0; j < kStepBytes / 32; ++j)
                                if (j < nmma)
                                    tc_mma_i8_pair(tmem_base + 256, da + 2 * j, db1 + 2 * j, idesc,
                                                   static_cast<uint32_t>((kb - kb0) | j));
                        }
                        tc_commit_pair(&empty[stage], 0x3 << even);
                        if (kb == kb1 - 1) {
                            tc_commit_pair(&tmem_full[acc], 0x3 << even);
                            if (wide) tc_commit_pair(&tmem_full[1], 0x3 << even);
                        }
                    }
                    __syncwarp();
                    stage = next;
                    phase = next_phase;
                }
                if (wide) {                   // both accumulators, every tile
                    acc_phase ^= 1u;
                } else {
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
            // every tcgen05 operation issued above has finished before TMEM is freed
            if (__any_sync(0xFFFFFFFFu, failed) && lane == 0) {
                *s_abort = 1;
                atomicExch(args.status, kDevTimeout);
            }
            __syncwarp();
            if (elect_one()) {
                tc_commit_pair(drain, 0x1 << even);
                int local_abort = 0;
                mbar_wait_bounded(drain, 0, args.timeout_ns, &local_abort, args.status);
            }
            __syncwarp();
        }
    } else if constexpr (kSplit) {
        // ---------------- epilogue (warps 2..9): this pair's sums are complete ----------------
        const int tid = threadIdx.x - 64;
        int mt, nt;
        pair_tile(pair, args, mt, nt);
        grid_dependency_wait();
        reinterpret_cast<float*>(epi)[tid] = tid < BN && nt * BN + tid < args.N ? args.sw[nt * BN + tid] : 0.0f;
        mbar_wait_warp(&tmem_full[0], 0, args.timeout_ns, s_abort, args.status);
        __syncwarp();
    } else {
        // ---------------- epilogue (warps 2..9, both CTAs) ----------------
        grid_dependency_wait();
        constexpr int kChunks = kPairMaxBN / 64;          // per warp
        const int q = warp & 3;
        const int half = (warp - 2) >> 2;
        const uint64_t pol_y = l2_policy_evict_first();
        uint8_t* stage_y = epi + (warp - 2) * (kEpiBufs * kEpiBytes);
        const uint32_t swz = static_cast<uint32_t>((lane >> 1) & 3);
        const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        int acc = 0, buf = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int t = pair; t < total_tiles && ok; t += npairs) {
            int mt, nt;
            pair_tile(t, args, mt, nt);
            const int m0 = mt * 256 + static_cast<int>(rank) * kRows + q * 32;   // row of lane 0
            const float sa = m0 + lane < args.M ? args.sa[m0 + lane] : 0.0f;
            // an accumulator at a time: one a tile, or both of a wide one
            for (int h = 0; h <= wide; ++h) {
                const int nb = nt * TN + h * BN;
                // its channels' scales are on their way while the MMAs run
                float sw[kChunks];
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    const int c = half * 32 + 64 * i + lane;
                    sw[i] = m0 < args.M && c < BN && nb + c < args.N ? args.sw[nb + c] : 0.0f;
                }
                if (!mbar_wait_warp(&tmem_full[acc], acc_phase, args.timeout_ns, s_abort, args.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (m0 < args.M) {                                         // warp-uniform
#pragma unroll
                    for (int i = 0; i < kChunks; ++i) {
                        const int c = half * 32 + 64 * i;
                        const int n0 = nb + c;
                        if (c >= BN || n0 >= args.N) break;                // warp-uniform
                        uint32_t r[32];
                        tmem_ld_32cols(tq + acc * 256 + c, r);
                        tmem_ld_wait();
                        uint32_t o[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            o[j] = scale_bf16x2(r[2 * j], r[2 * j + 1], sa, __shfl_sync(0xFFFFFFFFu, sw[i], 2 * j),
                                                __shfl_sync(0xFFFFFFFFu, sw[i], 2 * j + 1));
                        }
                        if (n0 + 32 > args.N && (args.N & 7) != 0) {       // warp-uniform
                            // TMA stores whole 16-byte pieces of a row: columns
                            // that end inside one are stored from here
                            if (m0 + lane < args.M) {
                                uint16_t* yp = args.y + static_cast<int64_t>(m0 + lane) * args.ldy + n0;
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (n0 + j < args.N)
                                        yp[j] = static_cast<uint16_t>(o[j >> 1] >> (16 * (j & 1)));
                            }
                            continue;
                        }
                        // the store that last used this buffer has finished reading it
                        uint8_t* sb = stage_y + buf * kEpiBytes;
                        const uint32_t sy = smem_u32(sb);
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        __syncwarp();
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            sts128(sy + lane * 64 + ((static_cast<uint32_t>(u) ^ swz) << 4), o[4 * u],
                                   o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&tmap_y, sb, n0, m0, pol_y);
                            bulk_commit_group();
                        }
                        buf ^= 1;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(tmem_empty_leader + acc * 8);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
        // every store of this warp has completed before the CTA exits
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    if constexpr (kSplit) {
        int mt, nt;
        pair_tile(pair, args, mt, nt);
        const int m = (warp & 3) * 32 + lane;
        const Slices sl = {args.splits, split, 2, static_cast<int>(rank), slice_chunks(BN, args.splits),
                           min(BN, args.N - nt * BN + 15) / 16};
        exchange_and_store(sl, tmem_base, smem_u32(smem), reinterpret_cast<const float*>(epi), args.sa, args.y,
                           args.ldy, m, mt * 256 + static_cast<int>(rank) * kRows + m, args.M, 32, nt * BN, args.N);
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                                      // no CTA leaves while its peer may signal it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);

// Looked up once (a thread-safe local static); nullptr when the driver has none.
EncodeFn tensor_map_encoder() {
    static const EncodeFn fn = []() -> EncodeFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        return nullptr;
    }();
    return fn;
}

// 2-D map of a [rows, cols] matrix, row stride in bytes; zero fill (loads) and
// clipping (stores) beyond it.
bool make_map(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols,
              int64_t stride_bytes, int box_cols, int box_rows, CUtensorMapSwizzle swizzle,
              CUtensorMapL2promotion promo) {
    const EncodeFn fn = tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride_bytes)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle, promo, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_codes_map(CUtensorMap* m, const int8_t* base, int64_t rows, int64_t K, int box_rows) {
    return make_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rows, K, K, kStepBytes, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// The same codes as [K / 128][rows][128 bytes], read in boxes of u k-steps: one
// copy lays u swizzled tiles of 128 bytes a row one behind the other.  Where K
// is no multiple of 128 the map is [1][rows][K], read a step at a time.
bool make_steps_map(CUtensorMap* m, const int8_t* base, int64_t rows, int64_t K, int box_rows, int u) {
    const EncodeFn fn = tensor_map_encoder();
    if (!fn) return false;
    const bool whole = K % kStepBytes == 0;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(whole ? kStepBytes : K), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(whole ? K / kStepBytes : 1)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(whole ? kStepBytes : K)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kStepBytes), static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(whole ? u : 1)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operands {
    const int8_t* a;
    const int8_t* w;
    const float* sa;
    const float* sw;
    uint16_t* y;
    int64_t ldy;
    int M, N, K;
};

// The launches are programmatic dependents: the kernels wait for the previous
// grid before they touch global memory, so only their set-up overlaps it.
void launch_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&attr)[2], int cluster, int threads,
                   uint32_t smem, cudaStream_t stream) {
    *cfg = {};
    cfg->blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg->dynamicSmemBytes = smem;
    cfg->stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 2;
}

nvfp4_status launch_few(const Operands& o, const DeviceInfo& info, int* status, cudaStream_t stream) {
    using Kernel = void (*)(CUtensorMap, CUtensorMap, FewArgs);
    static const Kernel whole[4] = {
        int8_gemm_few_kernel<1, false, false>, int8_gemm_few_kernel<2, false, false>,
        int8_gemm_few_kernel<4, false, false>, int8_gemm_few_kernel<8, false, false>};
    static const Kernel shared[4] = {
        int8_gemm_few_kernel<1, false, true>, int8_gemm_few_kernel<2, false, true>,
        int8_gemm_few_kernel<4, false, true>, int8_gemm_few_kernel<8, false, true>};
    static const Kernel swapped = int8_gemm_few_kernel<kSwapSteps, true, false>;
    static PerDeviceOnce once;
    static int resident[kMaxDevices][kMaxSplits + 1];     // clusters of 2, 4 and 8 CTAs that fit the device
    int dev = 0;
    nvfp4_status st = current_device(&dev);
    if (st != NVFP4_OK) return st;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    st = once.run(dev, [&] {
        for (const Kernel k : {whole[0], whole[1], whole[2], whole[3], shared[0], shared[1], shared[2], shared[3],
                               swapped})
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) != cudaSuccess)
                return NVFP4_ERR_CUDA;
        for (int s = 2; s <= kMaxSplits; s *= 2) {
            launch_config(&cfg, attr, s, kFewThreads, kFewSmem, nullptr);
            cfg.gridDim = dim3(static_cast<unsigned>(info.sms / s * s), 1, 1);
            if (cudaOccupancyMaxActiveClusters(&resident[dev][s], shared[0], &cfg) != cudaSuccess)
                return NVFP4_ERR_CUDA;
        }
        return NVFP4_OK;
    });
    if (st != NVFP4_OK) return st;
    FewArgs f = {};
    f.sa = o.sa, f.sw = o.sw, f.y = o.y, f.ldy = o.ldy, f.M = o.M, f.N = o.N, f.K = o.K;
    f.k_steps = (o.K + kStepBytes - 1) / kStepBytes;
    f.timeout_ns = kTimeoutNs;
    f.status = status;
    // Channels as the MMA's rows: a long stream of few tokens (see the top of
    // int8_gemm_few.cuh), long enough for the power limit to show and to fill
    // rounds of 128-channel tiles.
    const bool swap = o.M <= kSwapTokens && o.N >= 224 * info.sms;
    f.nt = swap ? (o.M + 15) / 16 * 16 : (o.M + 7) / 8 * 8;
    // Tile width and the split of K, by cycles.  Over all rounds of tiles an SM
    // spends on each k-step the larger of its MMAs (four of BN / 2, 56 at the
    // least or 44 with 64 rows, and 300 for a stage's handshake) and its feed
    // (48 bytes a cycle); memory as a whole delivers some 3400 bytes of weights
    // a cycle.  The slower of the two decides; a quarter of the SMs' share is
    // added, so that among widths that memory bounds the least loaded SMs win.
    // Sharing K among the CTAs of a cluster costs 3000 and 200 for each of them,
    // and the exchange of the sums, 10 bytes a cycle: of the mean slice, but of
    // eight CTAs' the longest, since slices of one and two chunks leave some of
    // them none (60 shapes where that decides: 6 % less time on average, 128 x 2048
    // x 17408 12.2 us instead of 15.0; 13 % more at the worst).  On the 77 shapes of
    // up to 128 tokens that the figures were fitted to, the choice takes 1 %
    // longer than the best of all widths and splits on average, 17 % at the worst
    // (of 3.6 us); on 70 others 2 %, 21 % at the worst (of 3.1 us).
    int u = 0;
    int64_t best = 0;
    const int64_t memory = o.N * static_cast<int64_t>(kStepBytes) / 3400;
    if (swap) {
        f.bn = kRows, f.splits = 1;
        few_config(f.nt, f.bn, &u, &f.stages);
    }
    for (int splits = 1; !swap && splits <= kMaxSplits; splits *= 2) {
        const int fit = splits == 1 ? info.sms : resident[dev][splits];
        if (fit <= 0) continue;
        for (int bn = 16 * splits; bn <= kFewMaxBN; bn += 16) {
            const int64_t tiles = (o.N + bn - 1) / bn;
            int bu = 0, bs = 0;
            few_config(f.nt, bn, &bu, &bs);
            if (splits > 1 && f.k_steps < bu * splits) continue;       // a stage for every CTA
            const int64_t step = std::max(4 * std::max(f.nt <= 64 ? 44 : 56, bn / 2) + 300 / bu,
                                          (f.nt + bn) * kStepBytes / 48);
            const int64_t sm = (tiles + fit - 1) / fit * step / splits;
            const int share = splits < kMaxSplits ? bn / splits : 16 * slice_chunks(bn, splits);
            const int64_t cost = f.k_steps * (std::max(sm, memory) + sm / 4) +
                                 (splits > 1 ? 3000 + 200 * splits + f.nt * share * 4 * (splits - 1) / 10 : 0);
            if (best == 0 || cost < best) best = cost, f.bn = bn, f.stages = bs, f.splits = splits, u = bu;
        }
    }
    f.n_tiles = (o.N + f.bn - 1) / f.bn;
    const Kernel kern = swap ? swapped : (f.splits > 1 ? shared : whole)[u == 8 ? 3 : u / 2];
    CUtensorMap ta, tw;
    f.wide = o.K % kStepBytes == 0;
    if (!make_steps_map(&ta, o.a, o.M, o.K, f.nt, u) || !make_steps_map(&tw, o.w, o.N, o.K, f.bn, u))
        return NVFP4_ERR_CUDA;
    launch_config(&cfg, attr, f.splits, kFewThreads, kFewSmem, stream);
    cfg.gridDim = dim3(static_cast<unsigned>(f.splits > 1 ? f.n_tiles * f.splits : std::min(f.n_tiles, info.sms)), 1,
                       1);
    if (cudaLaunchKernelEx(&cfg, kern, ta, tw, f) != cudaSuccess) return NVFP4_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

nvfp4_status launch_pair(const Operands& o, const DeviceInfo& info, int* status, cudaStream_t stream) {
    using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, PairArgs);
    static const Kernel kernels[2] = {int8_gemm_pair_kernel<false>, int8_gemm_pair_kernel<true>};
    static PerDeviceOnce once;
    static int resident[kMaxDevices][kMaxSplits / 2 + 1];  // clusters of 2 and 4 pairs that fit the device
    int dev = 0;
    nvfp4_status st = current_device(&dev);
    if (st != NVFP4_OK) return st;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    st = once.run(dev, [&] {
        for (const Kernel k : kernels)
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem) != cudaSuccess)
                return NVFP4_ERR_CUDA;
        for (int s = 2; s <= kMaxSplits / 2; s *= 2) {
            launch_config(&cfg, attr, 2 * s, kPairThreads, kPairSmem, nullptr);
            cfg.gridDim = dim3(static_cast<unsigned>(info.sms / (2 * s) * (2 * s)), 1, 1);
            if (cudaOccupancyMaxActiveClusters(&resident[dev][s], kernels[1], &cfg) != cudaSuccess)
                return NVFP4_ERR_CUDA;
        }
        return NVFP4_OK;
    });
    if (st != NVFP4_OK) return st;
    PairArgs p = {};
    p.sa = o.sa, p.sw = o.sw, p.y = o.y, p.ldy = o.ldy, p.M = o.M, p.N = o.N, p.K = o.K;
    p.m_tiles = (o.M + 255) / 256;
    p.k_steps = (o.K + kStepBytes - 1) / kStepBytes;
    p.timeout_ns = kTimeoutNs;
    p.status = status;
    const int max_pairs = info.sms / 2;
    // Tile width and the split of K, by cycles of shared memory, which the
    // copies' writes and the MMAs' reads share at 128 bytes a cycle: a k-step of BN
    // columns writes 128 + BN / 2 rows of 128 bytes and reads 128 + BN (450 cycles
    // at the least); a wide one, of 2 BN columns, writes 128 + BN rows and reads
    // twice 128 + BN, which is less than two narrow ones, but no MMAs overlap its
    // epilogue (28 BN cycles; of narrow tiles the last one's 16 BN count).  A round
    // of tiles costs 1500 besides; sharing K among pairs 2000 and the exchange of
    // the sums, 10 bytes a cycle.  Take what costs least, the widest among equals.
    // (Measured for 1000 x 5120 x 17408, cycles a k-step: 393, 483, 519, 532 and 583
    // for BN = 128 to 256; the product takes 61 us in wide tiles of 320 columns, one
    // round, and 70 in narrow ones of 160, two rounds.  Over 130 shapes of 129 to
    // 2500 tokens, 60 of them not fitted to, the choice takes 1 % longer than the
    // best on average, 10 % at the worst.  An epilogue longer than its tile's
    // k-steps has no term: at a few k-steps, 2178 x 11003 x 816 or 1142 x 27401 x
    // 272, the sum is 1.4 to 1.6 times too low.)
    int64_t best = 0;
    for (int splits = 1; splits <= kMaxSplits / 2; splits *= 2) {
        const int fit = splits == 1 ? max_pairs : resident[dev][splits];
        if (fit <= 0 || p.k_steps < splits) continue;
        for (int wide = splits == 1; wide >= 0; --wide)
            for (int bn = kPairMaxBN; bn >= (wide ? 160 : 64); bn -= 32) {
                const int64_t tiles = static_cast<int64_t>(p.m_tiles) * ((o.N + (bn << wide) - 1) / (bn << wide));
                const int64_t rounds = (tiles + fit - 1) / fit;
                const int64_t step = wide ? 384 + 3 * bn : std::max(256 + 3 * bn / 2, 450);
                int64_t cost = rounds * (p.k_steps * step / splits + 1500);
                if (splits > 1)
                    cost += rounds * (2000 + kRows * bn * 4 * (splits - 1) / splits / 10);
                else
                    cost += wide ? rounds * 28 * bn : 16 * bn;
                if (best == 0 || cost < best) best = cost, p.bn = bn, p.wide = wide, p.splits = splits;
            }
    }
    p.n_tiles = (o.N + (p.bn << p.wide) - 1) / (p.bn << p.wide);
    p.stages = pair_stages(p.bn, p.wide);
    // Raster: when A fits comfortably in L2, sweep every M tile for each N tile
    // (the weight then streams from HBM once); otherwise bands of 16 M tiles.
    p.group_m = static_cast<int64_t>(o.M) * o.K <= (int64_t(48) << 20) ? 1 << 30 : 16;
    const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    const int pairs = static_cast<int>(p.splits > 1 ? tiles * p.splits : std::min<int64_t>(tiles, max_pairs));
    CUtensorMap ta, tb, ty;
    if (!make_codes_map(&ta, o.a, o.M, o.K, kRows) || !make_codes_map(&tb, o.w, o.N, o.K, p.bn / 2) ||
        !make_map(&ty, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, o.y, o.M, o.N, o.ldy * 2, 32, 32,
                  CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE))
        return NVFP4_ERR_CUDA;
    launch_config(&cfg, attr, 2 * p.splits, kPairThreads, kPairSmem, stream);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
    if (cudaLaunchKernelEx(&cfg, kernels[p.splits > 1], ta, tb, ty, p) != cudaSuccess) return NVFP4_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_int8_gemm(const int8_t* a_codes, const float* a_scale,
                                        const int8_t* w_codes, const float* w_scale, void* y,
                                        int64_t ldy, int64_t M, int64_t N, int64_t K, void* stream) {
    if (M < 0 || N < 0 || K < 0) return NVFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || K < 16 || K > kMaxK) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    // tile indices and row numbers are 32-bit in the kernels; a tile's rows may
    // pass the last one by less than 512, a walk over the tiles by the grid
    constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
    if (M > kMaxDim || N > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return NVFP4_OK;
    if (ldy < N || ldy % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    if (extent_too_large(M, ldy, 2)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (((M + 127) / 128) * ((N + 63) / 64) >= (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!a_codes || !a_scale || !w_codes || !w_scale || !y) return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(a_codes) || !aligned16(w_codes) || !aligned16(y) ||
        (reinterpret_cast<uintptr_t>(a_scale) & 3u) != 0 || (reinterpret_cast<uintptr_t>(w_scale) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    // every CTA reads the operands and scales while others write y
    const size_t yb = extent_bytes(M, ldy, N, 2);
    if (overlaps(a_codes, static_cast<size_t>(M * K), y, yb) ||
        overlaps(w_codes, static_cast<size_t>(N * K), y, yb) ||
        overlaps(a_scale, static_cast<size_t>(M) * 4, y, yb) ||
        overlaps(w_scale, static_cast<size_t>(N) * 4, y, yb))
        return NVFP4_ERR_INVALID_ARG;
    DeviceInfo info;
    const nvfp4_status st = require_sm100(&info);
    if (st != NVFP4_OK) return st;
    int* status = device_status_ptr();
    if (!status) return NVFP4_ERR_CUDA;
    const Operands o = {a_codes, w_codes, a_scale, w_scale, static_cast<uint16_t*>(y), ldy,
                        static_cast<int>(M), static_cast<int>(N), static_cast<int>(K)};
    return M <= kFewMaxTokens ? launch_few(o, info, status, as_stream(stream))
                              : launch_pair(o, info, status, as_stream(stream));
}

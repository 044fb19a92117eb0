// int8_rows.cu -- rows of a BF16 matrix to int8 codes with one FP32 scale per
// row: plain (an activation's tokens, a weight's output channels) or fused
// with the residual addition and root-mean-square norm in front of a layer.
//
//   r = fl32(x + residual)           (x without a residual)
//   t = fl32(r * fl32(weight + weight_offset))      (t = x without a norm)
//   T = max |t| over the row, raised to 2^-100
//   code = RNE(fl32(t * fl32(127 / T))),  |code| <= 127
//   scale = fl32(T / 127)  [norm: fl32(that * rstd), rstd = 1 / sqrt(mean(r^2) + eps)]
//
// The norm's factor rstd is common to the row, so it cancels from the codes
// (v = t * rstd and its largest magnitude carry it alike) and appears in the
// scale alone.  Hence one reduction per row, of sum r^2 and max |t| together,
// and codes that no summation order can change.  The codes stay within +-127:
// with u = 2^-24, t * fl32(127 / T) <= 127 (1 + u)^2 < 127.5.  2^-100 keeps
// 127 / T below 2^107 (a row that small is quantized in steps of 2^-100 / 127);
// an all-zero row has scale 1.  A row with a NaN or an infinity (in x, in the
// sum or in t, or a sum of squares beyond binary32) gets scale NaN and codes 0,
// so the products that use it are NaN in that row and nowhere else.
// r and the sum of squares are binary32; r is rounded to BF16 only where it is
// stored, and the norm takes the unrounded value.
//
// Bound by memory: 7 bytes per element for the norm with a residual (2 + 2 read,
// 2 + 1 written), 3 without and for the plain quantizer.  On a B200 (copies run
// at 6.55 TB/s), CUDA-graph replay over rotating inputs:
//   norm  32768 x 5120 182 us = 6.4 TB/s, 8192 x 5120 47.7 us = 6.2,
//         16384 x 8192 148 us = 6.4, 8192 x 17408 160-164 us = 6.1-6.3, 4096 x
//         32768 190 us = 4.9 (staged in shared memory; 240 with a second pass
//         over the row), 1000 x 131072 262 us = 3.5 (two passes);
//         without a residual 8192 x 5120 26 us = 4.8 (by then the instructions:
//         fewer registers and more CTAs are slower), 4096 x 32768 81 us = 5.0
//   plain 8191 x 17408 67.6 us = 6.3, 8192 x 5120 21.6 us = 5.8, 4096 x 32768
//         62 us = 6.5, 3000 x 49152 81 us = 5.5 (staged)
//   one row of 5120 2.2 us, eight of 17408 2.1 us
// What brought it there: one pass with the next row's loads in flight during
// the reduction (norm 8192 x 5120: 70.6 us in two passes); the plain row held
// in 16 bits and compared as 16-bit integers, so that two CTAs share an SM
// (8191 x 17408: 77.3 us with binary32 held).  Packed f32x2 arithmetic was
// slower (its register pairs spill: 61 us for norm 8192 x 5120), and its
// multiplication is fused into the addition after it, which changes codes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "host_common.h"
#include "nvfp4.h"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr float kTiny = 0x1p-100f;

struct RowArgs {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* residual;      // null: none
    int64_t ldr;
    const uint16_t* weight;        // norm only
    float weight_offset;
    float eps;
    float inv_cols;                // fl32(1 / cols)
    uint16_t* residual_out;        // null: none
    int64_t ldo;
    int64_t rows;
    int32_t cols;
    uint8_t* codes;
    float* scale;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const uint32_t l = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(hi));
    return l | (h << 16);
}

// 16-byte load that does not allocate in L1.  An ordinary (coherent) load: the
// residual may be rewritten in place by the thread that reads it.
__device__ __forceinline__ uint4 ld_row16(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight weights, again for every row: volatile, or the compiler would keep them.
__device__ __forceinline__ uint4 ld_weight(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Eight values of r = x (+ residual), binary32.
template <bool kRes>
__device__ __forceinline__ void sum_r(const uint4& xv, const uint4& rv, float (&r)[8]) {
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
    const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = bf16_lo(xw[i]);
        r[2 * i + 1] = bf16_hi(xw[i]);
        if (kRes) {
            r[2 * i] = __fadd_rn(r[2 * i], bf16_lo(rw[i]));
            r[2 * i + 1] = __fadd_rn(r[2 * i + 1], bf16_hi(rw[i]));
        }
    }
}

template <bool kNorm>
__device__ __forceinline__ void weigh(const uint4& wv, float offset, const float (&r)[8], float (&t)[8]) {
    const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[2 * i] = kNorm ? __fmul_rn(r[2 * i], __fadd_rn(bf16_lo(ww[i]), offset)) : r[2 * i];
        t[2 * i + 1] = kNorm ? __fmul_rn(r[2 * i + 1], __fadd_rn(bf16_hi(ww[i]), offset)) : r[2 * i + 1];
    }
}

__device__ __forceinline__ uint4 pack8(const float (&r)[8]) {
    return make_uint4(pack_bf16(r[0], r[1]), pack_bf16(r[2], r[3]), pack_bf16(r[4], r[5]), pack_bf16(r[6], r[7]));
}

// 8 codes from t and the multiplier fl32(127 / T).  |t * mult| < 127.5, so
// adding 1.5 * 2^23 rounds the product to an integer (ties to even) and leaves
// its two's complement in the low byte: full-rate additions in place of
// conversions, which run at a quarter of the rate.
__device__ __forceinline__ uint2 encode8(const float (&t)[8], float mult) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(t[i], mult), 12582912.0f));
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

template <bool kNorm>
__device__ __forceinline__ void tally(const float (&r)[8], const float (&t)[8], float& sum, uint32_t& top) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (kNorm) sum = __fmaf_rn(r[i], r[i], sum);
        top = max(top, __float_as_uint(t[i]) & 0x7FFFFFFFu);    // NaN above infinity above all else
    }
}

// No norm: BF16 magnitudes compared as 16-bit integers, two at a time.
__device__ __forceinline__ uint32_t tally16(const uint4& xv, uint32_t top2) {
    top2 = __vmaxu2(top2, xv.x & 0x7FFF7FFFu);
    top2 = __vmaxu2(top2, xv.y & 0x7FFF7FFFu);
    top2 = __vmaxu2(top2, xv.z & 0x7FFF7FFFu);
    return __vmaxu2(top2, xv.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t top_bits(uint32_t top2) { return max(top2 & 0xFFFFu, top2 >> 16) << 16; }

// Sum and maximum over the CTA's `warps` warps, the same in every thread: one
// barrier, `red` alternating between two buffers from row to row.
template <bool kNorm>
__device__ __forceinline__ void reduce_row(float& sum, uint32_t& top, uint2* red, int warps) {
    if (kNorm) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (warps == 1) return;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = make_uint2(__float_as_uint(sum), top);
    __syncthreads();
    const uint2 v = lane < warps ? red[lane] : make_uint2(0, 0);
    if (kNorm) {
        sum = __uint_as_float(v.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    top = __reduce_max_sync(0xFFFFFFFFu, v.y);
}

// The row's multiplier (bad rows: false) and, from one thread, its scale.
template <bool kNorm>
__device__ __forceinline__ bool finish_row(const RowArgs& a, int64_t row, float sum, uint32_t top, float* mult) {
    const bool ok = top < 0x7F800000u && (!kNorm || sum < __uint_as_float(0x7F800000u));
    const float T = fmaxf(__uint_as_float(top), kTiny);
    *mult = __fdiv_rn(127.0f, T);
    if (threadIdx.x == 0) {
        float s = __fdiv_rn(T, 127.0f);
        if (kNorm) s = __fmul_rn(s, __frsqrt_rn(__fmaf_rn(sum, a.inv_cols, a.eps)));
        if (top == 0) s = 1.0f;
        a.scale[row] = ok ? s : __uint_as_float(0x7FC00000u);
    }
    return ok;
}

// Rows that fit a CTA's registers: V vectors of 8 per thread, the vectors of a
// thread blockDim.x apart.  Each CTA walks rows, and the next row's loads leave
// before the current row's reduction.  Between that and the encoding the norm
// holds t (and with V = 2 its weights, which longer rows read from L1 again);
// without a norm the row is held as loaded.  What counts is bytes in flight and
// warps: thread counts and register limits are set so that two CTAs or more
// share an SM where that is possible, or one has up to 32 warps (norm with a
// residual, 8192 x 17408: 191 us with V = 4 and the weights held, in 17 warps;
// 164 with V = 3 in 23.  Reading the weights again with V = 2: 8192 x 5120 without a
// residual 34 us against 26.  A row shared by a cluster of CTAs: a cluster
// barrier a row, 301 us for 8192 x 17408).
constexpr int row_max_threads(bool norm, int v) { return norm ? 1024 : v == 2 ? 768 : 640; }
constexpr int row_min_ctas(bool norm, int v) { return norm || v == 8 ? 1 : 2; }

template <bool kNorm, bool kRes, int V>
__global__ void __launch_bounds__(row_max_threads(kNorm, V), row_min_ctas(kNorm, V)) row_int8_kernel(const RowArgs a) {
    __shared__ uint2 s_red[2][32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int vecs = a.cols / 8;
    const int warps = blockDim.x >> 5;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    constexpr bool kHeld = V == 2;                  // the weights stay in registers
    uint4 w[kHeld ? V : 1], xv[V], rv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        const bool in = v < vecs;
        if (kHeld) w[j] = kNorm && in ? *reinterpret_cast<const uint4*>(a.weight + 8 * v) : zero;
        xv[j] = in ? ld_row16(a.x + blockIdx.x * a.ldx + 8 * v) : zero;
        rv[j] = kRes && in ? ld_row16(a.residual + blockIdx.x * a.ldr + 8 * v) : zero;
    }
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        float t[kNorm ? V : 1][8];
        uint4 held[kNorm ? 1 : V];
        float sum = 0.0f;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if constexpr (kNorm) {
                float r[8];
                sum_r<kRes>(xv[j], rv[j], r);
                const int v = threadIdx.x + j * blockDim.x;
                if constexpr (kHeld)
                    weigh<kNorm>(w[j], a.weight_offset, r, t[j]);
                else
                    weigh<kNorm>(v < vecs ? ld_weight(a.weight + 8 * v) : zero, a.weight_offset, r, t[j]);
                tally<kNorm>(r, t[j], sum, top);
                if (kRes && v < vecs && a.residual_out)
                    *reinterpret_cast<uint4*>(a.residual_out + row * a.ldo + 8 * v) = pack8(r);
            } else {
                held[j] = xv[j];
                top = tally16(xv[j], top);
            }
        }
        const int64_t next = row + gridDim.x;
        if (next < a.rows) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int v = threadIdx.x + j * blockDim.x;
                if (v < vecs) {
                    xv[j] = ld_row16(a.x + next * a.ldx + 8 * v);
                    if (kRes) rv[j] = ld_row16(a.residual + next * a.ldr + 8 * v);
                }
            }
        }
        if constexpr (!kNorm) top = top_bits(top);
        reduce_row<kNorm>(sum, top, s_red[buf], warps);
        float mult;
        const bool ok = finish_row<kNorm>(a, row, sum, top, &mult);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int v = threadIdx.x + j * blockDim.x;
            if (v < vecs) {
                uint2 c = make_uint2(0, 0);
                if constexpr (kNorm) {
                    if (ok) c = encode8(t[j], mult);
                } else {
                    float x8[8];
                    sum_r<false>(held[j], zero, x8);
                    if (ok) c = encode8(x8, mult);
                }
                *reinterpret_cast<uint2*>(a.codes + row * a.cols + 8 * v) = c;
            }
        }
    }
}

// Longer rows: t waits in shared memory (as x itself, in 16 bits, without a
// norm) between the reduction and the encoding.  Each thread reads back what it
// wrote.  Two CTAs of 512 threads share an SM where their rows fit, else one has
// 1024 (norm 4096 x 32768: 188 us, 214 with 512; plain 3000 x 49152: 81 us with two
// CTAs, 103 with one).  Beyond shared memory the row is read twice.
// A thread's sum of squares is one chain of binary32 additions: at most 56 of
// them in a row that fits on chip, so that the scale errs by 2^-18 at the most.
// Rows read twice may have any length (a chain of 32768, 2^25 columns, erred by
// 2.4e-4): their batches of 32 are added up in binary64.
constexpr int kLongThreads = 1024;              // half of them where two CTAs share an SM
constexpr int kHalfSmem = 112 * 1024;
constexpr int kLongBatch = 4;
constexpr int kLongSmem = 200 * 1024;

template <bool kNorm, bool kRes, bool kStaged>
__global__ void __launch_bounds__(kLongThreads, 1) row_int8_long_kernel(const RowArgs a) {
    __shared__ uint2 s_red[2][32];
    extern __shared__ uint4 s_row[];
    // rows of any length: the next grid is let in early only where this one is
    // short beside the bounded waits of the kernels that may follow
    if (kStaged) grid_launch_dependents();
    grid_dependency_wait();
    const int vecs = a.cols / 8, threads = blockDim.x;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        const uint16_t* x = a.x + row * a.ldx;
        const uint16_t* res = kRes ? a.residual + row * a.ldr : nullptr;
        uint16_t* out = kRes && a.residual_out ? a.residual_out + row * a.ldo : nullptr;
        float sum = 0.0f;
        double total = 0.0;
        uint32_t top = 0;
        for (int v0 = threadIdx.x; v0 < vecs; v0 += threads * kLongBatch) {
            uint4 xv[kLongBatch], rv[kLongBatch];
#pragma unroll
            for (int j = 0; j < kLongBatch; ++j) {
                const int64_t at = 8 * static_cast<int64_t>(v0 + j * threads);
                if (v0 + j * threads < vecs) {
                    xv[j] = ld_row16(x + at);
                    rv[j] = kRes ? ld_row16(res + at) : zero;
                }
            }
#pragma unroll
            for (int j = 0; j < kLongBatch; ++j) {
                const int v = v0 + j * threads;
                const int64_t at = 8 * static_cast<int64_t>(v);
                if (v >= vecs) break;
                if constexpr (kNorm) {
                    const uint4 wv = *reinterpret_cast<const uint4*>(a.weight + at);
                    float r[8], t[8];
                    sum_r<kRes>(xv[j], rv[j], r);
                    weigh<true>(wv, a.weight_offset, r, t);
                    tally<true>(r, t, sum, top);
                    if constexpr (kStaged) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            s_row[2 * v + i] = make_uint4(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]),
                                                          __float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]));
                        if (out) *reinterpret_cast<uint4*>(out + at) = pack8(r);
                    }
                } else {
                    top = tally16(xv[j], top);
                    if constexpr (kStaged) s_row[v] = xv[j];
                }
            }
            if constexpr (kNorm && !kStaged) total += static_cast<double>(sum), sum = 0.0f;
        }
        if constexpr (kNorm && !kStaged) sum = static_cast<float>(total);
        if constexpr (!kNorm) top = top_bits(top);
        reduce_row<kNorm>(sum, top, s_red[buf], threads / 32);
        float mult;
        const bool ok = finish_row<kNorm>(a, row, sum, top, &mult);
        for (int v = threadIdx.x; v < vecs; v += threads) {
            const int64_t at = 8 * static_cast<int64_t>(v);
            float t[8];
            if constexpr (kStaged && kNorm) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 q = s_row[2 * v + i];
                    t[4 * i] = __uint_as_float(q.x), t[4 * i + 1] = __uint_as_float(q.y);
                    t[4 * i + 2] = __uint_as_float(q.z), t[4 * i + 3] = __uint_as_float(q.w);
                }
            } else if constexpr (kStaged) {
                sum_r<false>(s_row[v], zero, t);
            } else {
                // beyond shared memory: the row once more, from cache
                float r[8];
                sum_r<kRes>(ld_row16(x + at), kRes ? ld_row16(res + at) : zero, r);
                if (out) *reinterpret_cast<uint4*>(out + at) = pack8(r);
                if constexpr (kNorm) {
                    weigh<true>(*reinterpret_cast<const uint4*>(a.weight + at), a.weight_offset, r, t);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = r[i];
                }
            }
            *reinterpret_cast<uint2*>(a.codes + row * a.cols + at) = ok ? encode8(t, mult) : make_uint2(0, 0);
        }
    }
}

// One kernel's launch state: CTAs per SM for each thread count in warps, 0
// until measured (racing threads measure the same value).
struct Resident {
    std::atomic<int> per_sm[kMaxDevices][33] = {};
};

nvfp4_status launch(void (*kern)(RowArgs), std::atomic<int>& cached, int threads, int smem, const RowArgs& a,
                    const DeviceInfo& dev, void* stream) {
    // resident CTAs only: each walks its share of the rows
    int per_sm = cached.load(std::memory_order_acquire);
    if (per_sm <= 0) {
        if (smem > 0 &&
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLongSmem) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess || per_sm <= 0)
            return NVFP4_ERR_CUDA;
        cached.store(per_sm, std::memory_order_release);
    }
    const int64_t cap = static_cast<int64_t>(dev.sms) * per_sm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows < cap ? a.rows : cap), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = as_stream(stream);
    // a programmatic dependent: the kernels wait for the previous grid before
    // they touch global memory, so only their set-up overlaps it
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return NVFP4_ERR_CUDA;
    return cuda_status(cudaGetLastError());
}

template <bool kNorm, bool kRes, int V>
bool try_rows(const RowArgs& a, const DeviceInfo& dev, int id, void* stream, nvfp4_status* st) {
    static Resident resident;
    const int threads = ((a.cols / 8 + V - 1) / V + 31) / 32 * 32;
    if (threads > row_max_threads(kNorm, V)) return false;
    *st = launch(row_int8_kernel<kNorm, kRes, V>, resident.per_sm[id][threads / 32], threads, 0, a, dev, stream);
    return true;
}

template <bool kNorm, bool kRes>
nvfp4_status launch_rows(const RowArgs& a, void* stream) {
    DeviceInfo dev;
    int id = 0;
    nvfp4_status st = require_sm100(&dev);
    if (st == NVFP4_OK) st = current_device(&id);
    if (st != NVFP4_OK) return st;
    // the fewest vectors per thread whose threads fit a CTA
    if (try_rows<kNorm, kRes, 2>(a, dev, id, stream, &st)) return st;
    if constexpr (kNorm)
        if (try_rows<kNorm, kRes, 3>(a, dev, id, stream, &st)) return st;
    if constexpr (!kRes)
        if (try_rows<kNorm, kRes, 4>(a, dev, id, stream, &st)) return st;
    if constexpr (!kNorm)
        if (try_rows<kNorm, kRes, 8>(a, dev, id, stream, &st)) return st;
    // CTAs per SM by the row's KB of shared memory
    static std::atomic<int> staged[kMaxDevices][kLongSmem / 1024 + 1], unstaged[kMaxDevices];
    const int64_t bytes = static_cast<int64_t>(a.cols) * (kNorm ? 4 : 2);
    if (bytes <= kLongSmem) {
        const int smem = static_cast<int>((bytes + 1023) / 1024 * 1024);
        return launch(row_int8_long_kernel<kNorm, kRes, true>, staged[id][smem / 1024],
                      smem > kHalfSmem ? kLongThreads : kLongThreads / 2, smem, a, dev,
                      stream);
    }
    return launch(row_int8_long_kernel<kNorm, kRes, false>, unstaged[id], kLongThreads, 0, a, dev, stream);
}

// Same address and stride: every element is read by the thread that rewrites
// it, before it does (in place).  Any other overlap is refused.
bool clashes(const void* in, int64_t ldi, const void* out, int64_t ldo, int64_t rows, int64_t cols) {
    if (in == out && ldi == ldo) return false;
    return overlaps(in, extent_bytes(rows, ldi, cols, 2), out, extent_bytes(rows, ldo, cols, 2));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_int8_quantize(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                            int8_t* codes, float* scale, void* stream) {
    if (rows < 0 || cols < 0) return NVFP4_ERR_INVALID_ARG;
    if (cols % 16 != 0 || ld % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    if (cols == 0 || cols >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!x || !codes || !scale || ld < cols) return NVFP4_ERR_INVALID_ARG;
    if (extent_too_large(rows, ld, 2)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(x) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scale) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    const size_t xb = extent_bytes(rows, ld, cols, 2), cb = static_cast<size_t>(rows * cols);
    const size_t sb = static_cast<size_t>(rows) * 4;
    if (overlaps(x, xb, codes, cb) || overlaps(x, xb, scale, sb) || overlaps(codes, cb, scale, sb))
        return NVFP4_ERR_INVALID_ARG;
    RowArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ld;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.codes = reinterpret_cast<uint8_t*>(codes);
    a.scale = scale;
    return launch_rows<false, false>(a, stream);
}

extern "C" nvfp4_status nvfp4_add_rms_norm_int8(const void* x, int64_t ldx, const void* residual,
                                                int64_t ldr, const void* weight, float weight_offset,
                                                float eps, int64_t rows, int64_t cols,
                                                void* residual_out, int64_t ldo, int8_t* codes,
                                                float* scale, void* stream) {
    if (rows < 0 || cols < 0) return NVFP4_ERR_INVALID_ARG;
    // a positive normal eps, so that an all-zero row has a finite factor
    if (!(eps >= 0x1p-126f) || !(eps < 0x1p127f) || !(weight_offset > -0x1p100f) ||
        !(weight_offset < 0x1p100f))
        return NVFP4_ERR_INVALID_ARG;
    if (!residual && residual_out) return NVFP4_ERR_INVALID_ARG;
    if (cols % 16 != 0 || ldx % 8 != 0 || (residual && ldr % 8 != 0) || (residual_out && ldo % 8 != 0))
        return NVFP4_ERR_ALIGNMENT;
    if (cols == 0 || cols >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return NVFP4_OK;
    if (!x || !weight || !codes || !scale || ldx < cols || (residual && ldr < cols) ||
        (residual_out && ldo < cols))
        return NVFP4_ERR_INVALID_ARG;
    if (extent_too_large(rows, ldx, 2) || (residual && extent_too_large(rows, ldr, 2)) ||
        (residual_out && extent_too_large(rows, ldo, 2)))
        return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
        !aligned16(codes) || (reinterpret_cast<uintptr_t>(scale) & 3u) != 0)
        return NVFP4_ERR_ALIGNMENT;
    const size_t xb = extent_bytes(rows, ldx, cols, 2), wb = static_cast<size_t>(cols) * 2;
    const size_t rb = residual ? extent_bytes(rows, ldr, cols, 2) : 0;
    const size_t ob = residual_out ? extent_bytes(rows, ldo, cols, 2) : 0;
    const size_t cb = static_cast<size_t>(rows * cols), sb = static_cast<size_t>(rows) * 4;
    const void* outs[3] = {residual_out, codes, scale};
    const size_t outb[3] = {ob, cb, sb};
    for (int i = 0; i < 3; ++i) {
        if (overlaps(outs[i], outb[i], weight, wb)) return NVFP4_ERR_INVALID_ARG;
        if (i > 0 && (overlaps(outs[i], outb[i], x, xb) || overlaps(outs[i], outb[i], residual, rb)))
            return NVFP4_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], outb[i], outs[j], outb[j])) return NVFP4_ERR_INVALID_ARG;
    }
    if (residual_out && (clashes(x, ldx, residual_out, ldo, rows, cols) ||
                         clashes(residual, ldr, residual_out, ldo, rows, cols)))
        return NVFP4_ERR_INVALID_ARG;
    RowArgs a = {};
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.residual = static_cast<const uint16_t*>(residual);
    a.ldr = ldr;
    a.weight = static_cast<const uint16_t*>(weight);
    a.weight_offset = weight_offset;
    a.eps = eps;
    a.inv_cols = 1.0f / static_cast<float>(cols);
    a.residual_out = static_cast<uint16_t*>(residual_out);
    a.ldo = ldo;
    a.rows = rows;
    a.cols = static_cast<int32_t>(cols);
    a.codes = reinterpret_cast<uint8_t*>(codes);
    a.scale = scale;
    return residual ? launch_rows<true, true>(a, stream) : launch_rows<true, false>(a, stream);
}

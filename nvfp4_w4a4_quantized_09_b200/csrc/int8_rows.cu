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
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

// Eight values of a row: r (the stored residual's value before rounding).
template <bool kNorm>
__device__ __forceinline__ void load_r(const RowArgs& a, int64_t row, int vec, float (&r)[8]) {
    const uint4 xv = *reinterpret_cast<const uint4*>(a.x + row * a.ldx + 8 * static_cast<int64_t>(vec));
    const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = bf16_lo(xw[i]);
        r[2 * i + 1] = bf16_hi(xw[i]);
    }
    if (kNorm && a.residual) {
        const uint4 rv =
            *reinterpret_cast<const uint4*>(a.residual + row * a.ldr + 8 * static_cast<int64_t>(vec));
        const uint32_t rw[4] = {rv.x, rv.y, rv.z, rv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = __fadd_rn(r[2 * i], bf16_lo(rw[i]));
            r[2 * i + 1] = __fadd_rn(r[2 * i + 1], bf16_hi(rw[i]));
        }
    }
}

template <bool kNorm>
__device__ __forceinline__ void weigh(const RowArgs& a, int vec, const float (&r)[8], float (&t)[8]) {
    if constexpr (kNorm) {
        const uint4 wv = *reinterpret_cast<const uint4*>(a.weight + 8 * static_cast<int64_t>(vec));
        const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[2 * i] = __fmul_rn(r[2 * i], __fadd_rn(bf16_lo(ww[i]), a.weight_offset));
            t[2 * i + 1] = __fmul_rn(r[2 * i + 1], __fadd_rn(bf16_hi(ww[i]), a.weight_offset));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = r[i];
    }
}

// 8 codes from t and the multiplier fl32(127 / T).
__device__ __forceinline__ uint2 encode8(const float (&t)[8], float mult) {
    uint32_t b[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        b[i >> 2] |= (static_cast<uint32_t>(__float2int_rn(__fmul_rn(t[i], mult))) & 0xFFu) << (8 * (i & 3));
    return make_uint2(b[0], b[1]);
}

// One CTA per row at a time, two passes over it (the second from cache).
constexpr int kRowThreads = 256;

template <bool kNorm>
__global__ void __launch_bounds__(kRowThreads) row_int8_kernel(const RowArgs a) {
    __shared__ float s_sum[2][kRowThreads / 32];
    __shared__ uint32_t s_max[2][kRowThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int vecs = a.cols / 8;
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
        float sum = 0.0f;
        uint32_t top = 0;
        for (int v = threadIdx.x; v < vecs; v += kRowThreads) {
            float r[8], t[8];
            load_r<kNorm>(a, row, v, r);
            weigh<kNorm>(a, v, r, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (kNorm) sum = __fmaf_rn(r[i], r[i], sum);
                top = max(top, __float_as_uint(t[i]) & 0x7FFFFFFFu);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        top = __reduce_max_sync(0xFFFFFFFFu, top);
        if (lane == 0) {
            s_sum[buf][warp] = sum;
            s_max[buf][warp] = top;
        }
        __syncthreads();
        sum = 0.0f;
        top = 0;
#pragma unroll
        for (int w = 0; w < kRowThreads / 32; ++w) {
            sum += s_sum[buf][w];
            top = max(top, s_max[buf][w]);
        }
        const bool bad = top >= 0x7F800000u || (kNorm && !(sum < __uint_as_float(0x7F800000u)));
        const float T = fmaxf(__uint_as_float(top), kTiny);
        const float mult = bad ? 0.0f : __fdiv_rn(127.0f, T);
        if (threadIdx.x == 0) {
            float s = __fdiv_rn(T, 127.0f);
            if (kNorm) s = __fmul_rn(s, __frsqrt_rn(__fmaf_rn(sum, a.inv_cols, a.eps)));
            if (top == 0) s = 1.0f;
            a.scale[row] = bad ? __uint_as_float(0x7FC00000u) : s;
        }
        for (int v = threadIdx.x; v < vecs; v += kRowThreads) {
            float r[8], t[8];
            load_r<kNorm>(a, row, v, r);
            weigh<kNorm>(a, v, r, t);
            if (kNorm && a.residual_out) {
                uint4 o;
                o.x = pack_bf16(r[0], r[1]);
                o.y = pack_bf16(r[2], r[3]);
                o.z = pack_bf16(r[4], r[5]);
                o.w = pack_bf16(r[6], r[7]);
                *reinterpret_cast<uint4*>(a.residual_out + row * a.ldo + 8 * static_cast<int64_t>(v)) = o;
            }
            const uint2 c = bad ? make_uint2(0, 0) : encode8(t, mult);
            *reinterpret_cast<uint2*>(a.codes + row * a.cols + 8 * static_cast<int64_t>(v)) = c;
        }
    }
}

template <bool kNorm>
nvfp4_status launch_rows(const RowArgs& a, void* stream) {
    DeviceInfo dev;
    const nvfp4_status st = require_sm100(&dev);
    if (st != NVFP4_OK) return st;
    const int64_t cap = static_cast<int64_t>(dev.sms) * 8;
    const int64_t grid = a.rows < cap ? a.rows : cap;
    row_int8_kernel<kNorm><<<static_cast<unsigned>(grid), kRowThreads, 0, as_stream(stream)>>>(a);
    return cuda_status(cudaGetLastError());
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
    return launch_rows<false>(a, stream);
}

extern "C" nvfp4_status nvfp4_add_rms_norm_int8(const void* x, int64_t ldx, const void* residual,
                                                int64_t ldr, const void* weight, float weight_offset,
                                                float eps, int64_t rows, int64_t cols,
                                                void* residual_out, int64_t ldo, int8_t* codes,
                                                float* scale, void* stream) {
    if (rows < 0 || cols < 0) return NVFP4_ERR_INVALID_ARG;
    // a positive normal eps, so that an all-zero row has a finite factor
    if (!(eps >= 0x1p-126f) || !(eps < 0x1p127f) || !(weight_offset > -0x1p127f) ||
        !(weight_offset < 0x1p127f))
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
    return launch_rows<true>(a, stream);
}

// int8_gemm.cu -- product of two int8 matrices with one FP32 scale per token
// (row of A) and per channel (row of W):
//
//   acc[m, n] = sum_k a[m, k] * w[n, k]             (exact in 32 bits)
//   y[m, n] = bf16( fl32( fl32( fl32(acc) * sa[m] ) * sw[n] ) )
//
// K is at most 131056, so |acc| <= 128 * 128 * K < 2^31: the sum cannot
// overflow, and integer addition gives the same bits in any order.  Tile sizes
// and splits of K are therefore free choices that no result depends on.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "host_common.h"
#include "nvfp4.h"

namespace nvfp4 {
namespace {

constexpr int64_t kMaxK = 131056;

struct Int8GemmArgs {
    const int8_t* a;
    const int8_t* w;
    const float* sa;
    const float* sw;
    uint16_t* y;
    int64_t ldy;
    int M, N, K;
};

// 64 x 64 outputs per CTA, 4 x 4 per thread, four products per dp4a.
constexpr int kTile = 64;
constexpr int kStep = 64;      // bytes of K per step

__global__ void __launch_bounds__(256) int8_gemm_kernel(const Int8GemmArgs g) {
    __shared__ int32_t as[kTile][kStep / 4 + 1], ws[kTile][kStep / 4 + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTile, n0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 16;
    for (int k0 = 0; k0 < g.K; k0 += kStep) {
        int4 av = make_int4(0, 0, 0, 0), wv = av;
        if (k0 + lc < g.K) {
            if (m0 + lr < g.M) av = *reinterpret_cast<const int4*>(g.a + (m0 + lr) * g.K + k0 + lc);
            if (n0 + lr < g.N) wv = *reinterpret_cast<const int4*>(g.w + (n0 + lr) * g.K + k0 + lc);
        }
        __syncthreads();
        as[lr][lc / 4] = av.x, as[lr][lc / 4 + 1] = av.y, as[lr][lc / 4 + 2] = av.z, as[lr][lc / 4 + 3] = av.w;
        ws[lr][lc / 4] = wv.x, ws[lr][lc / 4 + 1] = wv.y, ws[lr][lc / 4 + 2] = wv.z, ws[lr][lc / 4 + 3] = wv.w;
        __syncthreads();
        for (int k = 0; k < kStep / 4; ++k) {
            int a4[4], w4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a4[i] = as[ty + 16 * i][k];
                w4[i] = ws[tx + 16 * i][k];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a4[i], w4[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty + 16 * i;
        if (m >= g.M) continue;
        const float sa = g.sa[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx + 16 * j;
            if (n >= g.N) continue;
            const float v = __fmul_rn(__fmul_rn(__int2float_rn(acc[i][j]), sa), g.sw[n]);
            g.y[m * g.ldy + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
        }
    }
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_int8_gemm(const int8_t* a_codes, const float* a_scale,
                                        const int8_t* w_codes, const float* w_scale, void* y,
                                        int64_t ldy, int64_t M, int64_t N, int64_t K, void* stream) {
    if (M < 0 || N < 0 || K < 0) return NVFP4_ERR_INVALID_ARG;
    if (K % 16 != 0 || K < 16 || K > kMaxK) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return NVFP4_OK;
    if (ldy < N || ldy % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    if (extent_too_large(M, ldy, 2)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (((M + 127) / 128) * ((N + 127) / 128) >= (int64_t(1) << 30)) return NVFP4_ERR_UNSUPPORTED_SHAPE;
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
    DeviceInfo dev;
    const nvfp4_status st = require_sm100(&dev);
    if (st != NVFP4_OK) return st;
    Int8GemmArgs g = {a_codes, w_codes, a_scale, w_scale, static_cast<uint16_t*>(y), ldy,
                      static_cast<int>(M), static_cast<int>(N), static_cast<int>(K)};
    const dim3 grid(static_cast<unsigned>((N + kTile - 1) / kTile), static_cast<unsigned>((M + kTile - 1) / kTile));
    if (grid.y > 65535) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    int8_gemm_kernel<<<grid, 256, 0, as_stream(stream)>>>(g);
    return cuda_status(cudaGetLastError());
}

// int8_mma.cuh -- the 8-bit-integer matrix instruction of sm_100a:
// D[tmem, s32] (+)= A[smem, s8] * B[smem, s8]^T, 32 values of K (32 bytes of a
// K-major row) per instruction, both operands in the 128-byte swizzle.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace nvfp4 {

// kind::i8 instruction descriptor: S32 accumulator (format 2 at bit 4, no
// saturation), signed 8-bit A and B (format 1 at bits 7 and 10), both K-major,
// N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t int8_idesc(int m, int n) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// CTA pair: M = 256 (128 rows of A from each CTA), B split along N between the
// two CTAs, accumulator rows in each CTA's tensor memory.
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tries of mbar_spin before it gives up: at some 20 cycles a try at the least,
// a bound of a fraction of a second to a few seconds.
constexpr uint32_t kSpinTries = 1u << 25;

// The feed loops' waits, by every lane of the warp.  mbar_peek tests a phase
// without waiting; mbar_spin tests it until it has completed or `tries` tests
// have failed (false then).  A loop peeks at its next stage before it issues
// the work of the current one and spins only where that failed: a completed
// phase costs some 60 cycles to test, and the tensor pipe runs dry meanwhile
// when the test stands between two batches of MMAs (measured for batches of
// four MMAs of 50-64 cycles: 366 cycles a batch with a wait in front of each,
// 300 with the peek and the election hoisted, 206-256 with no wait at all).
__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity, uint32_t tries) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %3;\n\t"
        "SPIN:\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.gt.s32 q, n, 0;\n\t"
        "@q bra SPIN;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(tries)
        : "memory");
    return done != 0;
}

// Bring a box into L2, a hint that nothing waits for.  L2 is where this GPU's
// memory is coherent, so a box that an earlier kernel is still writing may be
// prefetched: the later load reads what that kernel wrote.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t x, int32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(map), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z)
                 : "memory");
}

// 16 bytes into the shared memory of a CTA of the cluster (an address from
// mapa_shared).
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// 3-D tiled TMA load (no multicast), bytes counted on this CTA's `bar`.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x,
                                            int32_t y, int32_t z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}

}  // namespace nvfp4

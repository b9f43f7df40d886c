// moe_w4.cuh -- what the two kernels of moe_expert_w4 (and the layer for a few
// tokens) share: sizes, the 4-bit codes as 16-bit numbers, the 16-row tensor-core
// product, and the gated SiLU.
#pragma once

#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

struct W4Args {
    int E, C, K, N, M, group;          // M rows of the matrix: N, or 2N with the gate
    int nkb;                           // blocks of 128 inputs
};

// A packed word's 8 codes as four pairs of 16-bit numbers (q - 8) / kW4Unit, the
// pair (2i, 2i+1) to r[i]. The low byte of a 16-bit half, taken as the bits of a
// bf16 or fp16 number, is that integer times the type's lowest subnormal (the
// step to the first normal numbers is linear), so a mask leaves code 2i's 4 bits
// as n or 16 n such units and one exact fused multiply-add makes (n - 8) / kW4Unit
// of it: no shift but one by 8 for the upper two codes of each half. The unit, a
// power of two, goes into the group's scale.
template <bool F16>
constexpr float kW4Unit = F16 ? 512.0f : 64.0f;

template <bool F16>
__device__ __forceinline__ uint32_t w4_fma(uint32_t n, uint32_t by, uint32_t less) {
    uint32_t r;
    if constexpr (F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(n), "r"(by), "r"(less));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(n), "r"(by), "r"(less));
    return r;
}
template <bool F16>
__device__ __forceinline__ void w4_pairs(uint32_t word, uint32_t (&r)[4]) {
    // fp16: units of 2^-24, times 2^15 or 2^11, less 8 / 512; bf16: of 2^-133, times 2^127 or 2^123, less 8 / 64
    constexpr uint32_t kBy = F16 ? 0x78007800u : 0x7F007F00u, kBy16 = F16 ? 0x68006800u : 0x7D007D00u;
    constexpr uint32_t kLess = F16 ? 0xA400A400u : 0xBE00BE00u;
    const uint32_t up = word >> 8;
    r[0] = w4_fma<F16>(word & 0x000F000Fu, kBy, kLess);
    r[1] = w4_fma<F16>(word & 0x00F000F0u, kBy16, kLess);
    r[2] = w4_fma<F16>(up & 0x000F000Fu, kBy, kLess);
    r[3] = w4_fma<F16>(up & 0x00F000F0u, kBy16, kLess);
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 codes -> two fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}

// v / (1 + exp(-v)) with the division of 2 ulp, which the rounding to bf16 hides (its 0 for denominators past 2^126
// is where the quotient is below 1e-36).
__device__ __forceinline__ float silu(float v) { return __fdividef(v, __fadd_rn(1.0f, expf(-v))); }

__device__ __forceinline__ void put_bf16(uint16_t *p, float v) {
    *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
}

// The kernel for many rows per expert (moe_w4_tiles.cu): tcgen05 tiles. The
// workspace holds w4_tiles_workspace_bytes.
size_t w4_tiles_workspace_bytes(const Dims &d, const W4Args &a);
int launch_w4_tiles(const Dims &d, const W4Args &a, cudaStream_t st, const void *x, const float *x_scale,
                    const int32_t *counts, const void *w_q, const void *w_scale, void *y, void *workspace);

}  // namespace moe

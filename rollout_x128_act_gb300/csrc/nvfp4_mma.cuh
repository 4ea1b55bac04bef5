// Products of NVFP4 weights and BF16 activations on the warp-level tensor
// instructions: decoding, and the MMA that takes the decoded pairs.
//
// The bits of an E2M1 code placed at a BF16's sign and at the low exponent and
// top mantissa bits are that code's value times 2^-126 (the subnormal codes
// included); times the block scale * 2^110 this is the exact product
// e2m1 * e4m3 (6 significant bits) * 2^-16, and 2^16 is multiplied into the
// final scale.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace jetq {

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes of a word -> four BF16 pairs (element j, element j + 4) of
// value * scale * 2^-16; `scale` holds the block scale * 2^110 twice.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t (&p)[4])
{
    const __nv_bfloat162 s = *reinterpret_cast<const __nv_bfloat162 *>(&scale);
    const uint32_t w8 = w >> 8;
    // a nibble at bits 3..0 (7..4): one product puts its sign at bit 15 and its magnitude at bits 8..6
    const uint32_t t[4] = {(w & 0x000F000Fu) * 0x1040u, (w & 0x00F000F0u) * 0x104u, (w8 & 0x000F000Fu) * 0x1040u,
                           (w8 & 0x00F000F0u) * 0x104u};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t b = t[j] & 0x81C081C0u;
        const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&b), s);
        p[j] = *reinterpret_cast<const uint32_t *>(&v);
    }
}

// Two E4M3 scales (a 16-bit word) -> their values * 2^110 as BF16 pairs.
__device__ __forceinline__ void decode_scales(uint32_t s2, uint32_t (&out)[2])
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)s2));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f;
        asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)(h >> (16 * i))));
        const __nv_bfloat162 b = __float2bfloat162_rn(f * 0x1p110f);
        out[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
}

} // namespace jetq

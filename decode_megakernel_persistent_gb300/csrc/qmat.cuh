// qmat.cuh -- device helpers of the 4-bit matrices' format (qmat.cu, qmat_mul.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "qmat.h"

namespace ll {

// Code i of a word of 8 is at bits (4 f + 3) % 32, f = i / 2 + 4 (i % 2): turned right by 4 p bits,
// the word has codes 2 p and 2 p + 1 in bits 3..6 of its halves. There they are the upper four
// of bf16's seven mantissa bits, so that (word & 0x00780078) | 0x41804180 is the bf16 pair 16 + c:
// one logical operation for two codes, beside the shift. In fp16, with ten mantissa bits, the same three bits
// further up. magic: 0x41804180, or (HALF) 0x4c004c00.
template <bool HALF>
__device__ __forceinline__ uint32_t qm_turn(uint32_t w, int p) {
    if (HALF) return p == 0 ? w << 3 : p == 3 ? __funnelshift_r(w, w, 9) : w >> (4 * p - 3);
    return p == 0 ? w : p == 3 ? __funnelshift_r(w, w, 12) : w >> (4 * p);
}

// Codes 2 p and 2 p + 1 as a pair, c - 8 (EXACT) or 16 + c.
template <bool HALF, bool EXACT>
__device__ __forceinline__ uint32_t qm_codes(uint32_t w, int p, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(qm_turn<HALF>(w, p)), "r"(HALF ? 0x03c003c0u : 0x00780078u), "r"(magic));  // (a & b) | c
    if (!EXACT) return r;
    if (HALF) {
        const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&r), __float2half2_rn(24.f));
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&r), __float2bfloat162_rn(24.f));
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace ll

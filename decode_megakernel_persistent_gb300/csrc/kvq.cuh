// kvq.cuh -- device helpers of the packed KV cache's format, shared by kvq.cu and
// kvq_attn.cu.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace ll {

__device__ __forceinline__ uint32_t kvq_prmt(uint32_t a, uint32_t b, uint32_t sel) {
    return __byte_perm(a, b, sel);
}

__device__ __forceinline__ __half2 kvq_h2(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }
__device__ __forceinline__ uint32_t kvq_u32(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }

// A group's parameters (lo, step) that stand for NaN.
__device__ __forceinline__ bool kvq_is_nan(uint32_t par) {
    return (par & 0x7fffu) > 0x7c00u || (par >> 16 & 0x7fffu) > 0x7c00u;
}

// Four pairs of codes as fp16 numbers from two cells of 4 codes each: out[i] =
// (code i of cell a, code i of cell b). fp16 holds 1024 + c exactly as the bits
// 0x6400 | c (c < 1024), and 1024 + 16 c as 0x6400 | c << 4, so a code becomes a
// number by one logical operation and one exact subtraction (or multiply-add).
// 4 bits: x holds cell a in its low half and cell b in its high half.
__device__ __forceinline__ void kvq_codes4(uint32_t x, __half2 (&out)[4]) {
    const __half2 m1024 = __float2half2_rn(-1024.f), r16 = __float2half2_rn(0.0625f), m64 = __float2half2_rn(-64.f);
    const uint32_t y = x >> 8;
    out[0] = __hadd2(kvq_h2((x & 0x000f000fu) | 0x64006400u), m1024);
    out[1] = __hfma2(kvq_h2((x & 0x00f000f0u) | 0x64006400u), r16, m64);
    out[2] = __hadd2(kvq_h2((y & 0x000f000fu) | 0x64006400u), m1024);
    out[3] = __hfma2(kvq_h2((y & 0x00f000f0u) | 0x64006400u), r16, m64);
}

// 8 bits: the cells are whole words a and b.
__device__ __forceinline__ void kvq_codes8(uint32_t a, uint32_t b, __half2 (&out)[4]) {
    const __half2 m1024 = __float2half2_rn(-1024.f);
    const uint32_t lo = kvq_prmt(a, b, 0x5140), hi = kvq_prmt(a, b, 0x7362);  // bytes a0 b0 a1 b1, a2 b2 a3 b3
    out[0] = __hadd2(kvq_h2(kvq_prmt(lo, 0x64646464u, 0x4140)), m1024);
    out[1] = __hadd2(kvq_h2(kvq_prmt(lo, 0x64646464u, 0x4342)), m1024);
    out[2] = __hadd2(kvq_h2(kvq_prmt(hi, 0x64646464u, 0x4140)), m1024);
    out[3] = __hadd2(kvq_h2(kvq_prmt(hi, 0x64646464u, 0x4342)), m1024);
}

}  // namespace ll

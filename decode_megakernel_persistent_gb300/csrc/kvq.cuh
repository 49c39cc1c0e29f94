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

// Two fp32 operations at once.
__device__ __forceinline__ uint64_t kvq_pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void kvq_split(uint64_t p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t kvq_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t kvq_mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t kvq_add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A group's parameters (lo, step) that stand for NaN.
__device__ __forceinline__ bool kvq_is_nan(uint32_t par) {
    return (par & 0x7fffu) > 0x7c00u || (par >> 16 & 0x7fffu) > 0x7c00u;
}

// Constants of the unpacking, held in registers: an instruction takes one immediate
// operand, and without them every mask-and-or became two instructions (the compiler
// puts constants that it knows back into the code).
struct KvqConsts {
    uint32_t c1024, r16, m64;  // fp16 pairs 1024, 1/16, -64
    __device__ __forceinline__ KvqConsts() {
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(c1024));
        asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(r16));
        asm volatile("mov.b32 %0, 0xd400d400;" : "=r"(m64));
    }
};

__device__ __forceinline__ uint32_t kvq_and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));  // (a & b) | c
    return r;
}

// Four pairs of codes as fp16 numbers from two cells of 4 codes each: out[i] =
// (code i of cell a, code i of cell b). fp16 holds 1024 + c exactly as the bits
// 0x6400 | c (c < 1024), and 1024 + 16 c as 0x6400 | c << 4, so a code becomes a
// number by one logical operation and one exact subtraction (or multiply-add).
// 4 bits: x holds cell a in its low half and cell b in its high half.
__device__ __forceinline__ void kvq_codes4(uint32_t x, const KvqConsts &k, __half2 (&out)[4]) {
    const __half2 m1024 = __float2half2_rn(-1024.f);
    const uint32_t y = x >> 8;
    out[0] = __hadd2(kvq_h2(kvq_and_or(x, 0x000f000fu, k.c1024)), m1024);
    out[1] = __hfma2(kvq_h2(kvq_and_or(x, 0x00f000f0u, k.c1024)), kvq_h2(k.r16), kvq_h2(k.m64));
    out[2] = __hadd2(kvq_h2(kvq_and_or(y, 0x000f000fu, k.c1024)), m1024);
    out[3] = __hfma2(kvq_h2(kvq_and_or(y, 0x00f000f0u, k.c1024)), kvq_h2(k.r16), kvq_h2(k.m64));
}

// 8 bits: the cells are whole words a and b.
__device__ __forceinline__ void kvq_codes8(uint32_t a, uint32_t b, const KvqConsts &k, __half2 (&out)[4]) {
    const __half2 m1024 = __float2half2_rn(-1024.f);
    const uint32_t lo = kvq_prmt(a, b, 0x5140), hi = kvq_prmt(a, b, 0x7362);  // bytes a0 b0 a1 b1, a2 b2 a3 b3
    out[0] = __hadd2(kvq_h2(kvq_prmt(lo, k.c1024, 0x7170)), m1024);
    out[1] = __hadd2(kvq_h2(kvq_prmt(lo, k.c1024, 0x7372)), m1024);
    out[2] = __hadd2(kvq_h2(kvq_prmt(hi, k.c1024, 0x7170)), m1024);
    out[3] = __hadd2(kvq_h2(kvq_prmt(hi, k.c1024, 0x7372)), m1024);
}

}  // namespace ll

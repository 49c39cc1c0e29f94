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

// Whether a group's parameters (lo, step) stand for a NaN or an infinity at some code: values
// grow or fall with the code and a lo that is not finite reaches every one, so the largest code tells.
template <int BITS>
__device__ __forceinline__ bool kvq_not_finite(uint32_t par) {
    const __half v = __hfma(__ushort_as_half(uint16_t(par >> 16)), __int2half_rn((1 << BITS) - 1), __ushort_as_half(uint16_t(par)));
    return (__half_as_ushort(v) & 0x7c00u) == 0x7c00u;
}
// The value of dim d (of 32) of a row's group gr.
template <int BITS, int HD>
__device__ __forceinline__ __half kvq_value(const uint8_t *codes, uint32_t par, int gr, int d) {
    const int el = ((d >> 2) * (HD / 32) + gr) * 4 + (d & 3);
    const int code = BITS == 8 ? codes[el] : codes[el >> 1] >> (4 * (el & 1)) & 15;
    return __hfma(__ushort_as_half(uint16_t(par >> 16)), __int2half_rn(code), __ushort_as_half(uint16_t(par)));
}
// A pair of values, those that are not finite as zeros.
__device__ __forceinline__ uint32_t kvq_finite2(uint32_t v) {
    if ((v & 0x7c00u) == 0x7c00u) v &= 0xffff0000u;
    if ((v & 0x7c000000u) == 0x7c000000u) v &= 0xffffu;
    return v;
}
// Bit d: dim d of a row's group gr is not finite. (Rows like that are rare: a loop, of few registers.)
template <int BITS, int HD>
__device__ __forceinline__ uint32_t kvq_not_finite_dims(const uint8_t *codes, uint32_t par, int gr) {
    uint32_t dims = 0;
#pragma unroll 1
    for (int d = 0; d < 32; d++) {
        const __half v = kvq_value<BITS, HD>(codes, par, gr, d);
        if ((__half_as_ushort(v) & 0x7c00u) == 0x7c00u) dims |= 1u << d;
    }
    return dims;
}
// The values of a row's group gr that are not finite become finite ones: by code 0 where lo and step are
// finite, otherwise (all of them are not) by the parameters that are returned.
template <int BITS, int HD>
__device__ __forceinline__ uint32_t kvq_make_finite(uint8_t *codes, uint32_t par, int gr) {
    if ((par & 0x7c00u) == 0x7c00u || (par & 0x7c000000u) == 0x7c000000u) return 0;
    const uint32_t dims = kvq_not_finite_dims<BITS, HD>(codes, par, gr);
#pragma unroll 1
    for (int d = 0; d < 32; d++) {
        const int el = ((d >> 2) * (HD / 32) + gr) * 4 + (d & 3);
        if (!(dims >> d & 1)) continue;
        if (BITS == 8)
            codes[el] = 0;
        else
            codes[el >> 1] &= el & 1 ? 0x0f : 0xf0;
    }
    return par;
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

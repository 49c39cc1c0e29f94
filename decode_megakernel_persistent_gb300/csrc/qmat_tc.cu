// qmat_tc.cu -- y = x W^T (+ add) with W in 4 bits on the fifth-generation tensor cores: many rows x, or large
// matrices (qmat_mul.cu has the other kernel, and the rule).
//
//   y[i][r] = sum over groups G of  step (sum_k c x) + lo (sum_k x),   k in G
//
// A code c needs no arithmetic to become an operand: the bits 0000cccc, read as an e4m3 number, are c / 512 (up to 7 a
// subnormal, from 8 on a normal one), so unpacking is a shift and a mask for four codes. x enters as e4m3 too: as it
// is; or bf16 as two terms (hi, and 32 times what is left of it), fp32 as four, of 4 bits and a sign each, scaled by a
// power of two for a row and 128 columns. Two terms hold bf16's 8 bits exactly down to 2^-14 of the largest of the
// 128 (what is lost below is 2^-22 of it at most), four hold 20 bits of fp32. Products are exact, sums fp32; lo, step and
// the scales meet them in fp32, once a group.
//
// That is for fp32 outputs, or fp32 x. bf16 outputs of bf16 or e4m3 x (HALF) take W's values themselves, rounded to fp16
// (2^-12 of a value at most), and x in fp16, scaled by a power of two a row (bf16's 8 bits exactly down to 2^-28 of the
// largest; e4m3 times its scale rounded to 11 bits): three times the instructions a code, but one sum over all columns, where
// taking the sums of 64 columns of x a group of 128 from tensor memory cost more. The roundings add 2e-4 of the
// outputs' norm to the 1.6e-3 of their own.
//
// A block takes 128 rows at a time and walks their columns in tiles of 128, a unit each. Sixteen warps, in four sets that
// take units in turn, unpack 32 rows each from a ring of their own (cp.async) into tensor memory, the products' A operand,
// a row to a lane; x stays in shared memory, unpacked once a block, as B. One warp issues the products; four warps, a row
// to a thread, take the sums from tensor memory (a group's, joined in registers with its parameters, or HALF a row
// block's). Blocks of a cluster share the columns: each row's shares then meet through shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "call.h"
#include "kvq_attn.cuh"
#include "qmat.h"

namespace ll {
namespace {

struct TcArgs {
    const uint4 *codes;
    const uint4 *params;    // (lo, step), 4 rows to 16 bytes
    int rows, cols, KT, RT;
    const void *x;
    int64_t x_stride;
    int x_type;
    const float *scale;     // e4m3: [n][scale_row], the tile's or (scale_step 0) the row's
    int scale_row, scale_step;
    bool vec;               // x's rows take 8-value loads
    const void *add;
    int64_t add_stride;
    void *y;
    int64_t y_stride;
    bool y_f32;
    int n;
    KvqWaits waits;
    // the plan
    int terms, tokens;      // columns of x's operand a token takes, tokens of a pass over the matrix
    int cluster, slice;     // blocks that share the columns, tiles of a block
    int depth;              // units of a warp in flight
};

constexpr int SETS = 4, UNPACK = 4 * SETS, FLUSH = 4, W_MMA = UNPACK + FLUSH, THREADS = 32 * (W_MMA + 1);
constexpr int MAX_SMEM = 232448 - 2048, MAX_CLUSTER = 8;

// What a block keeps of x, by bytes from `base` on (a 1,024-byte border):
//   operand  [slice][N][128]      K-major rows of a tile's columns in e4m3, in the 128-byte swizzle
//   scale    [slice][NC] floats   of a tile's column
//   sum      [slice][PG][NC]      of a group's x (in the column of its first term)
// or HALF
//   operand  [slice][2][N][128]   the same in fp16, 64 columns after 64
//   scale    [NC] floats          of a token; then the largest of each, as bits
template <int NC, int PG, bool HALF>
struct Shape {
    static constexpr int N = NC < 16 ? 16 : NC;                  // columns of a product: 16 at least
    static constexpr int TILE = N * (HALF ? 256 : 128);
    static constexpr int A_COLS = HALF ? 64 : 32;                // of tensor memory: a stage of A
    static constexpr int SD = HALF ? 2 : N <= 32 ? 8 : 4;        // sums
    static constexpr int TM_A = SD * N, SA = (512 - TM_A) / A_COLS < 8 ? (512 - TM_A) / A_COLS : 8;
    static constexpr int SLOT = 2048 + (HALF ? 128 * PG : 0);    // a warp's unit in its ring: codes, parameters
    static __host__ __device__ int x_bytes(int slice) { return slice * TILE + (HALF ? 2 * NC * 4 : slice * NC * 4 * (1 + PG)); }
};

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// Until all but the last n groups of copies have landed.
__device__ __forceinline__ void wait_copies(int n) {
    switch (n) {
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
        case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
        case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
        case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
    return u;
}
__device__ __forceinline__ ulonglong2 lds_two_pairs(uint32_t at) {
    ulonglong2 u;
    asm volatile("ld.shared.v2.u64 {%0,%1}, [%2];" : "=l"(u.x), "=l"(u.y) : "r"(at) : "memory");
    return u;
}
__device__ __forceinline__ uint32_t to_e4m3(float lo, float hi) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
    return h;
}
__device__ __forceinline__ float2 from_e4m3(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Shared-memory descriptor of a K-major tile in the 128-byte swizzle (rows of 128 bytes, 8-row groups 1,024 bytes apart).
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3fffu) | uint64_t(1u) << 16 | uint64_t(1024u >> 4) << 32 | uint64_t(1u) << 46 | uint64_t(2u) << 61;
}
// e4m3 (kind::f8f6f4) or fp16 (kind::f16) A and B, fp32 sums, M = 128.
template <int N>
constexpr uint32_t IDESC = (1u << 4) | (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
// (by a whole warp, of which one elected lane, the same at every call, carries it out)
template <bool HALF>
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    if (HALF)
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
            "r"(a), "l"(b), "r"(idesc), "r"(add)
            : "memory");
    else asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {  // arrives once all products issued so far are done
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Bounded wait: once the limit passes, with *err set, or once another's has, the block goes on without waits to its
// end, as if all had come: its loops and whole-warp instructions stay together, and its outputs become NaN.
__device__ __noinline__ void wait_long(uint32_t bar, uint32_t parity, volatile int *err, uint64_t timeout_ns) {
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        if (*err) return;
        for (int i = 0; i < 64; i++)
            if (bar_try(bar, parity)) return;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < timeout_ns);
    *err = 1;
}
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int *err, const KvqWaits &w) {
    if (!bar_try(bar, parity)) wait_long(bar, parity, err, w.timeout_ns);
}
// The same for a barrier that other blocks of the cluster arrive at.
__device__ __forceinline__ bool try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __noinline__ void wait_cluster(uint32_t bar, uint32_t parity, volatile int *err, uint64_t timeout_ns) {
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        if (*err) return;
        for (int i = 0; i < 64; i++)
            if (try_cluster(bar, parity)) return;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < timeout_ns);
    *err = 1;
}
__device__ __forceinline__ uint32_t in_block(uint32_t at, int rank) {  // a shared address of another block of the cluster
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}
__device__ __forceinline__ void arrive_in(uint32_t bar, int rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_block(bar, rank)) : "memory");
}
__device__ __forceinline__ float load_in(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void cluster_sync() {  // (by whole warps)
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 8 columns of this thread's tensor-memory lane; the values are there after tm_wait8.
__device__ __forceinline__ void tm_load8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
                 : "memory");
}
// (the values pass through the statement, so that no use of them can come before it)
__device__ __forceinline__ void tm_wait8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_store(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 8 values of a row of x from column k on, as they lie in memory, zeros past the end.
template <int XT>
struct Raw {
    static constexpr int SIZE = XT == LL_F32 ? 4 : XT == LL_BF16 ? 2 : 1, WORDS = 2 * SIZE;
    uint32_t w[WORDS];
    __device__ __forceinline__ void widen(float (&v)[8]) const {
        if constexpr (XT == LL_BF16) {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
        } else if constexpr (XT == LL_F32) {
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const float2 f = from_e4m3(w[j / 2] >> (16 * (j % 2)));
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
        }
    }
};
template <int XT>
__device__ __noinline__ Raw<XT> load_edge(const char *p, int n) {  // (rows that are not aligned, a row's end)
    Raw<XT> r;
#pragma unroll
    for (int j = 0; j < Raw<XT>::WORDS; j++) r.w[j] = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        if (j >= n) continue;
        if constexpr (XT == LL_F32) r.w[j] = reinterpret_cast<const uint32_t *>(p)[j];
        else if constexpr (XT == LL_BF16) r.w[j / 2] |= uint32_t(reinterpret_cast<const uint16_t *>(p)[j]) << (16 * (j % 2));
        else r.w[j / 4] |= uint32_t(reinterpret_cast<const uint8_t *>(p)[j]) << (8 * (j % 4));
    }
    return r;
}
template <int XT>
__device__ __forceinline__ void load_raw(const TcArgs &a, int64_t row, int k, Raw<XT> &r) {
    const char *p = static_cast<const char *>(a.x) + (row * a.x_stride + k) * Raw<XT>::SIZE;
    if (a.vec && k + 8 <= a.cols) {
        if constexpr (XT == LL_E4M3) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
            r.w[0] = u.x;
            r.w[1] = u.y;
        } else {
#pragma unroll
            for (int j = 0; j < Raw<XT>::SIZE / 2; j++) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + j);
                r.w[4 * j] = u.x; r.w[4 * j + 1] = u.y; r.w[4 * j + 2] = u.z; r.w[4 * j + 3] = u.w;
            }
        }
    } else {
        r = load_edge<XT>(p, a.cols - k);
    }
}
// e / d by 1 / d in fp32: exact for the sizes here (e below 2^16: (e + 1/2) / d is 1 / (2 d) away from any integer).
__device__ __forceinline__ int quotient(int e, float per) { return int((float(e) + 0.5f) * per); }
constexpr int BATCH = 4;  // tokens' tiles of a thread on their way at once

// HALF: a token's columns in fp16, largest values of the block's columns to [2^14, 2^15). First the largest of each
// token go round (a token's tile to 16 threads), then the values are rounded.
template <int XT, int NC, int PG>
__device__ __forceinline__ void stage_half(const TcArgs &a, uint32_t operand, int first, int tile0, int tiles) {
    using S = Shape<NC, PG, true>;
    const uint32_t scales = operand + a.slice * S::TILE, tops = scales + NC * 4;
    const int u = threadIdx.x % 16, step = THREADS / 16;
    const int held = min(a.tokens, a.n - first), items = tiles * held;
    const float per = 1.f / float(tiles);
    const unsigned mates = 0xffffu << (threadIdx.x & 16);
    for (int i = threadIdx.x; i < NC; i += THREADS) asm volatile("st.shared.u32 [%0], %1;" ::"r"(tops + 4 * i), "r"(0) : "memory");
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 2; pass++) {
#pragma unroll 1
        for (int e0 = threadIdx.x / 16; e0 < items; e0 += BATCH * step) {
            Raw<XT> raws[BATCH];
            float factor[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; i++) {
                const int e = min(e0 + i * step, items - 1), token = quotient(e, per), kt = e - token * tiles;
                load_raw(a, first + token, (tile0 + kt) * QM_TILE_COLS + 8 * u, raws[i]);
                factor[i] = XT == LL_E4M3 ? __ldg(a.scale + int64_t(first + token) * a.scale_row + (tile0 + kt) * a.scale_step) : 1.f;
            }
#pragma unroll
            for (int i = 0; i < BATCH; i++) {
                const int e = e0 + i * step;
                if (e >= items) break;  // (16 threads alike)
                const int token = quotient(e, per), kt = e - token * tiles;
                float v[8];
                raws[i].widen(v);
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] *= factor[i];
                if (pass == 0) {
                    uint32_t top = 0;  // of finite values
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const uint32_t bits = __float_as_uint(v[j]) & 0x7fffffffu;
                        top = max(top, bits < 0x7f800000u ? bits : 0u);
                    }
                    top = __reduce_max_sync(mates, top);
                    if (u == 0) asm volatile("red.shared.max.u32 [%0], %1;" ::"r"(tops + 4 * token), "r"(top) : "memory");
                } else {
                    uint32_t top;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(top) : "r"(tops + 4 * token) : "memory");
                    // by 2^(141 - top), held to normal numbers (a largest value below 2^-106: zeros)
                    const int up = 268 - int(max(top >> 23, 21u));
                    const float f = __uint_as_float(uint32_t(up) << 23);
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        // (a value that is not finite becomes a NaN: infinities would meet zeros and other signs)
                        const float p = isfinite(v[2 * j]) ? v[2 * j] * f : __uint_as_float(0x7fffffffu);
                        const float r = isfinite(v[2 * j + 1]) ? v[2 * j + 1] * f : __uint_as_float(0x7fffffffu);
                        h[j] = kvq_u32(__floats2half2_rn(p, r));
                    }
                    const uint32_t at = operand + kt * S::TILE + (u / 8) * (S::N * 128) + token * 128 + (((u & 7) ^ (token & 7)) << 4);
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
                    if (u == 0 && kt == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + 4 * token), "f"(__uint_as_float(uint32_t(254 - up) << 23)) : "memory");
                }
            }
        }
        __syncthreads();
    }
}

// 16 threads turn a token's 128 columns of a tile into the operand: thread u has columns 8 u .. 8 u + 7, 8 bytes of a row of 128 (the
// order of a word's codes as they are unpacked: columns 0, 4, 1, 5 and 2, 6, 3, 7 of the 8).
template <int XT, int NC, int PG>
__device__ __forceinline__ void stage_x(const TcArgs &a, uint32_t operand, int first, int tile0, int tiles) {
    using S = Shape<NC, PG, false>;
    const uint32_t scales = operand + a.slice * S::TILE, sums = scales + a.slice * NC * 4;
    const int u = threadIdx.x % 16, step = THREADS / 16;
    const int held = min(a.tokens, a.n - first), items = tiles * held;
    const float per = 1.f / float(tiles);
#pragma unroll 1
    for (int e0 = threadIdx.x / 16; e0 < items; e0 += BATCH * step) {
    Raw<XT> raws[BATCH];
    float factor[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; i++) {
        const int e = min(e0 + i * step, items - 1), token = quotient(e, per), kt = e - token * tiles;
        load_raw(a, first + token, (tile0 + kt) * QM_TILE_COLS + 8 * u, raws[i]);
        factor[i] = XT == LL_E4M3 ? __ldg(a.scale + int64_t(first + token) * a.scale_row + (tile0 + kt) * a.scale_step) : 1.f;
    }
#pragma unroll
    for (int i = 0; i < BATCH; i++) {
        const int e = e0 + i * step;
        if (e >= items) break;  // (16 threads alike)
        const int token = quotient(e, per), kt = e - token * tiles;
        float v[8];
        raws[i].widen(v);
        const unsigned mates = 0xffffu << (threadIdx.x & 16);
        float scale, sum = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        const int col0 = token * a.terms;
        const uint32_t tile = operand + kt * S::TILE;
        auto store = [&](int col, uint32_t w0, uint32_t w1) {  // codes of columns 0..3 and 4..7
            const uint32_t at = tile + col * 128 + ((u / 2 ^ (col & 7)) << 4) + u % 2 * 8;  // (the 128-byte swizzle)
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(__byte_perm(w0, w1, 0x5140)), "r"(__byte_perm(w0, w1, 0x7362)) : "memory");
        };
        if constexpr (XT == LL_E4M3) {
            scale = factor[i];
            store(col0, raws[i].w[0], raws[i].w[1]);
            sum *= scale;
        } else {
            uint32_t top = 0;  // the largest exponent of finite values
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const uint32_t bits = __float_as_uint(v[i]) & 0x7fffffffu;
                top = max(top, bits < 0x7f800000u ? bits : 0u);
                if (bits >= 0x7f800000u) v[i] = __uint_as_float(0x7fffffffu);
            }
            top = __reduce_max_sync(mates, top) >> 23;
            // largest values to [128, 256): by 2^(134 - top), held to what is a normal number (below 2^-113: all zeros)
            const int up = 261 - int(max(top, 14u));
            const float f = __uint_as_float(uint32_t(up) << 23);
            scale = __uint_as_float(uint32_t(254 - up) << 23);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] *= f;
            float s = scale;
            for (int term = 0; term < a.terms; term++) {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    h[i] = to_e4m3(v[2 * i], v[2 * i + 1]);
                    const float2 b = from_e4m3(h[i]);
                    v[2 * i] = (v[2 * i] - b.x) * 32.f;
                    v[2 * i + 1] = (v[2 * i + 1] - b.y) * 32.f;
                }
                store(col0 + term, h[0] | h[1] << 16, h[2] | h[3] << 16);
                if (u == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + (kt * NC + col0 + term) * 4), "f"(s) : "memory");
                s *= 1.f / 32;
            }
        }
#pragma unroll
        for (int o = 1; o < 16 / PG; o *= 2) sum += __shfl_xor_sync(mates, sum, o);
        if (XT == LL_E4M3 && u == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales + (kt * NC + col0) * 4), "f"(scale) : "memory");
        if (u % (16 / PG) == 0) {
            const uint32_t at = sums + ((kt * PG + u / (16 / PG)) * NC + col0) * 4;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(sum) : "memory");
            for (int term = 1; term < a.terms; term++) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + 4 * term), "f"(0.f) : "memory");
        }
    }
    }
}

// y of a row for up to 8 tokens, n of them held.
__device__ __forceinline__ void store_8(const TcArgs &a, int64_t row, int token, int n, const uint32_t (&y)[8]) {
    if (row >= a.rows) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = __uint_as_float(y[e]);
    if (a.add) {
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int64_t from = int64_t(token + min(e, n - 1)) * a.add_stride + row;
            v[e] += a.y_f32 ? static_cast<const float *>(a.add)[from] : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.add)[from]);
        }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
        const int64_t at = int64_t(token + e) * a.y_stride + row;
        if (e >= n) continue;
        if (a.y_f32) static_cast<float *>(a.y)[at] = v[e];
        else static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(v[e]);
    }
}

// A walk over a block's units: tile kt of its columns of its i-th row block.
struct Units {
    int tiles, rb, stride, kt = 0;
    __device__ __forceinline__ Units(int tiles_, int rb0, int stride_, int skip) : tiles(tiles_), rb(rb0), stride(stride_) { next(skip); }
    __device__ __forceinline__ void next(int by) {
        kt += by;
        while (kt >= tiles) {
            kt -= tiles;
            rb += stride;
        }
    }
};

// Pairs of codes of a word as fp16 values lo + step c. In bits 6..9 of a half, alone, a code is the subnormal number c 2^-18, so that
// with step 2^18 (while that is finite: WIDE) one operation has the value; otherwise the code becomes a number first.
template <bool WIDE>
__device__ __forceinline__ void values(uint32_t w, __half2 lo, __half2 step, uint32_t *r) {
    const uint32_t v[4] = {w << 3, w >> 1, w >> 5, __funnelshift_r(w, w, 9)};
#pragma unroll
    for (int p = 0; p < 4; p++) {
        if (WIDE) {
            r[p] = kvq_u32(__hfma2(step, kvq_h2(v[p] & 0x03c003c0u), lo));
        } else {
            const __half2 c = __hsub2(kvq_h2((v[p] & 0x03c003c0u) | 0x4c004c00u), __float2half2_rn(16.f));
            r[p] = kvq_u32(__hfma2(step, c, lo));
        }
    }
}

// NC columns of x's operand, PG parameter groups of a tile.
template <int NC, int PG, bool HALF>
__global__ void __launch_bounds__(THREADS, 1) k_qmat_tc(const __grid_constant__ TcArgs a) {
    using S = Shape<NC, PG, HALF>;
    constexpr int N = S::N, SD = S::SD, SA = S::SA;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * SA + 2 * SD + 5];
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    const uint32_t a_full = sptr(bars), a_empty = a_full + 8 * SA, d_full = a_empty + 8 * SA, d_empty = d_full + 8 * SD;
    const uint32_t ready = d_empty + 8 * SD, freed = ready + 16, drained = freed + 16;  // (ready, freed: of two shares)
    volatile int *const err = &s_err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = a.cluster, rank = int(blockIdx.x) % C, clusters = int(gridDim.x) / C, first = blockIdx.y * a.tokens;
    const int tile0 = rank * a.slice, tiles = min(a.slice, a.KT - tile0);  // (1 at least)
    const int RB = (a.RT + 7) / 8, rb0 = int(blockIdx.x) / C, blocks = (RB - rb0 + clusters - 1) / clusters;
    const int units = blocks * tiles;
    const int held = min(a.tokens, a.n - first);
    const uint32_t operand = (sptr(raw) + 1023u) & ~1023u, scales = operand + a.slice * S::TILE, sums = scales + a.slice * NC * 4;
    const uint32_t rings = operand + (S::x_bytes(a.slice) + 15) / 16 * 16, shares = rings + UNPACK * a.depth * S::SLOT;

    // the unpacking warps' copies
    const int q = warp & 3, set = warp >> 2;
    const uint32_t ring = rings + warp * (a.depth * S::SLOT);
    Units ahead(tiles, rb0, clusters, set);
    int ahead_u = set, ahead_slot = 0, aimed = -1;
    int64_t tiles_at[2];  // of the two row tiles: their first tile of the block's columns
    auto issue = [&]() {
        if (ahead_u < units) {
            if (aimed != ahead.rb) {
                aimed = ahead.rb;
#pragma unroll
                for (int r = 0; r < 2; r++) tiles_at[r] = int64_t(min(aimed * 8 + 2 * q + r, a.RT - 1)) * a.KT + tile0;  // (rows past the end: not stored)
            }
            const uint32_t to = ring + ahead_slot * S::SLOT;
            // 16 bytes a lane: row 8 i + lane / 4 of the warp's, piece lane % 4 of it, turned by the row so that a row's
            // reader meets no bank twice
            const uint32_t turned = to + lane / 4 * 64 + (((lane & 3) + (lane >> 3)) & 3) * 16;
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const uint4 *from = a.codes + (tiles_at[r] + ahead.kt) * 64 + lane;
                copy16(turned + r * 1024, from);
                copy16(turned + r * 1024 + 512, from + 32);
            }
            if (HALF) {
                if (lane < 8 * PG) copy16(to + 2048 + 16 * lane, a.params + (tiles_at[lane / (4 * PG)] + ahead.kt) * (4 * PG) + lane % (4 * PG));
            } else if (lane < 4 * PG) {  // (for the joining warps)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a.params + (tiles_at[lane / (2 * PG)] + ahead.kt) * (4 * PG) + lane % (2 * PG) * 2));
            }
            ahead.next(SETS);
            ahead_u += SETS;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead_slot = ahead_slot + 1 == a.depth ? 0 : ahead_slot + 1;
    };
    if (warp < UNPACK)
        for (int i = 0; i < a.depth - 1; i++) issue();

    if (threadIdx.x == 0) {
        for (int i = 0; i < SA; i++) {
            bar_init(a_full + 8 * i, 4);
            bar_init(a_empty + 8 * i, 1);
        }
        for (int i = 0; i < SD; i++) {
            bar_init(d_full + 8 * i, 1);
            bar_init(d_empty + 8 * i, FLUSH);
        }
        for (int i = 0; i < 2; i++) {
            bar_init(ready + 8 * i, FLUSH * C);
            bar_init(freed + 8 * i, FLUSH * C);
        }
        bar_init(drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_err = 0;
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sptr(&s_tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if constexpr (HALF) {
        if (a.x_type == LL_BF16) stage_half<LL_BF16, NC, PG>(a, operand, first, tile0, tiles);
        else stage_half<LL_E4M3, NC, PG>(a, operand, first, tile0, tiles);
    } else {
        if (a.x_type == LL_BF16) stage_x<LL_BF16, NC, PG>(a, operand, first, tile0, tiles);
        else if (a.x_type == LL_F32) stage_x<LL_F32, NC, PG>(a, operand, first, tile0, tiles);
        else stage_x<LL_E4M3, NC, PG>(a, operand, first, tile0, tiles);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    fence_before();
    if (C > 1) cluster_sync();  // (others arrive at this block's barriers)
    else __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0), tmem_a = tmem + S::TM_A;

    if (warp < UNPACK) {
        int slot = 0;
        for (int u = set; u < units; u += SETS) {
            issue();
            wait_copies(a.depth - 1);
            __syncwarp();  // (a row comes by four lanes' copies)
            const uint32_t at = ring + slot * S::SLOT;
            uint32_t w[4][4];  // [t][j]
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const uint4 v = lds16(at + lane * 64 + ((t + (lane >> 1)) & 3) * 16);
                w[t][0] = v.x; w[t][1] = v.y; w[t][2] = v.z; w[t][3] = v.w;
            }
            const int s = u % SA;
            const uint32_t to = tmem_a + S::A_COLS * s + (uint32_t(32 * q) << 16);
            if constexpr (HALF) {
                uint32_t par[PG];
#pragma unroll
                for (int g = 0; g < PG; g++)
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(par[g]) : "r"(at + 2048 + (lane / 16 * PG + g) * 64 + lane % 16 * 4) : "memory");
                bool wide = true;
                __half2 lo[PG], step[PG], step18[PG];
#pragma unroll
                for (int g = 0; g < PG; g++) {
                    lo[g] = kvq_h2(kvq_prmt(par[g], 0, 0x1010));
                    step[g] = kvq_h2(kvq_prmt(par[g], 0, 0x3232));
                    step18[g] = __hmul2(__hmul2(step[g], __float2half2_rn(512.f)), __float2half2_rn(512.f));
                    wide = wide && (kvq_u32(step18[g]) & 0x7c00u) != 0x7c00u;
                }
                wide = __all_sync(0xffffffffu, wide);
                __syncwarp();  // (before another lane's copy into this slot)
                if (u >= SA) wait(a_empty + 8 * s, (u / SA - 1) & 1, err, a.waits);
                fence_after();
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    uint32_t r[32];
                    if (wide) {
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int j = 2 * h + e / 4, t = e % 4, g = j * PG / 4;
                            values<true>(w[t][j], lo[g], step18[g], r + 4 * e);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int j = 2 * h + e / 4, t = e % 4, g = j * PG / 4;
                            values<false>(w[t][j], lo[g], step[g], r + 4 * e);
                        }
                    }
                    tm_store(to + 32 * h, r);
                }
            } else {
                uint32_t r[32];
#pragma unroll
                for (int t = 0; t < 4; t++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        r[8 * j + 2 * t] = (w[t][j] >> 3) & 0x0f0f0f0fu;
                        r[8 * j + 2 * t + 1] = __funnelshift_r(w[t][j], w[t][j], 7) & 0x0f0f0f0fu;
                    }
                __syncwarp();
                if (u >= SA) wait(a_empty + 8 * s, (u / SA - 1) & 1, err, a.waits);
                fence_after();
                tm_store(to, r);
            }
            slot = slot + 1 == a.depth ? 0 : slot + 1;
            tm_store_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) arrive(a_full + 8 * s);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else if (warp == W_MMA) {
        Units at(tiles, rb0, clusters, 0);
        int d = 0;
        for (int u = 0; u < units; u++, at.next(1)) {
            const int s = u % SA;
            wait(a_full + 8 * s, (u / SA) & 1, err, a.waits);
            const uint32_t b = operand + at.kt * S::TILE;
            if constexpr (HALF) {
                const int i = d % SD;
                if (at.kt == 0 && d >= SD) wait(d_empty + 8 * i, (d / SD - 1) & 1, err, a.waits);
                fence_after();
#pragma unroll
                for (int k = 0; k < 8; k++)
                    mma<true>(tmem + i * N, tmem_a + S::A_COLS * s + 8 * k, desc_sw128(b + k / 4 * (N * 128)) + 2 * (k % 4), IDESC<N>, (at.kt | k) != 0);
                commit(a_empty + 8 * s);
                if (at.kt + 1 == tiles) {
                    commit(d_full + 8 * i);
                    d++;
                }
            } else {
#pragma unroll
                for (int p = 0; p < PG; p++, d++) {
                    const int i = d % SD;
                    if (d >= SD) wait(d_empty + 8 * i, (d / SD - 1) & 1, err, a.waits);
                    fence_after();
#pragma unroll
                    for (int k = 0; k < 4 / PG; k++)
                        mma<false>(tmem + i * N, tmem_a + S::A_COLS * s + 8 * (p * (4 / PG) + k), desc_sw128(b) + 2 * (p * (4 / PG) + k), IDESC<N>, k != 0);
                    commit(d_full + 8 * i);
                }
                commit(a_empty + 8 * s);
            }
        }
    } else {
        const int row = 32 * q + lane;  // of the row block
        int done = 0;
        // a row block's outputs, or shares of them: begin(), put() for each token (HALF: as they come), then end()
        int64_t out = 0;
        uint32_t share = 0;
        bool lost = false;
        auto begin = [&](int rb) {
            const int half = done & 1;
            out = int64_t(rb) * 128 + row;
            share = shares + half * (a.tokens * 512) + row * 4;  // (columns past the last token: nobody's)
            if (C > 1 && done >= 2) wait_cluster(freed + 8 * half, (done / 2 - 1) & 1, err, a.waits.timeout_ns);
            lost = *err;
        };
        auto put = [&](int token, float y) {
            if (lost) y = __uint_as_float(0x7fffffffu);
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(share + token * 512), "f"(y) : "memory");
        };
        auto end = [&]() {
            const int half = done & 1;
            if (C > 1) {
                __syncwarp();
                if (lane < C) arrive_in(ready + 8 * half, lane);
                wait_cluster(ready + 8 * half, (done / 2) & 1, err, a.waits.timeout_ns);
                lost = *err;
                // this block's eighth (or so) of the tokens, 8 on their way at once
                const int mine = (held + C - 1) / C, t1 = min(held, (rank + 1) * mine);
#pragma unroll 1
                for (int t0 = rank * mine; t0 < t1; t0 += 8) {
                    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int b = 0; b < C; b++) {
                        const uint32_t at = in_block(share + t0 * 512, b);
#pragma unroll
                        for (int i = 0; i < 8; i++) y[i] += load_in(at + min(i, t1 - 1 - t0) * 512);
                    }
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) w[i] = lost ? 0x7fffffffu : __float_as_uint(y[i]);
                    store_8(a, out, first + t0, t1 - t0, w);
                }
                __syncwarp();
                if (lane < C) arrive_in(freed + 8 * half, lane);
            } else if (!HALF) {  // (a thread's own row)
#pragma unroll 1
                for (int t0 = 0; t0 < held; t0 += 8) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[e]) : "r"(share + min(t0 + e, held - 1) * 512) : "memory");
                    store_8(a, out, first + t0, held - t0, w);
                }
            }
            done++;
        };
        if constexpr (HALF) {
            for (int rb = rb0; rb < RB; rb += clusters) {
                const int i = done % SD;
                wait(d_full + 8 * i, (done / SD) & 1, err, a.waits);
                fence_after();
                begin(rb);
                const uint32_t from = tmem + i * N + (uint32_t(32 * q) << 16);
                // (a loop and not NC / 8 copies of it: code that runs once a row block comes slower than it runs)
#pragma unroll 1
                for (int c = 0; c < NC; c += 8) {
                    uint32_t w[8];
                    tm_load8(from + c, w);
                    tm_wait8(w);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        float f;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(scales + 4 * (c + e)) : "memory");
                        w[e] = __float_as_uint(lost ? __uint_as_float(0x7fffffffu) : __uint_as_float(w[e]) * f);
                    }
                    if (C > 1) {
#pragma unroll
                        for (int e = 0; e < 8; e++) asm volatile("st.shared.u32 [%0], %1;" ::"r"(share + (c + e) * 512), "r"(w[e]) : "memory");
                    } else {
                        store_8(a, out, first + c, held - c, w);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(d_empty + 8 * i);
                end();
            }
        } else {
            uint64_t tot[NC / 2];
            Units at(tiles, rb0, clusters, 0), next = at;
            uint32_t par[2][PG];
            auto fetch = [&](uint32_t (&p)[PG]) {  // (lo, step) of the row in the groups of a unit to come
                const int64_t tile = int64_t(min(next.rb * 8 + row / 16, a.RT - 1)) * a.KT + tile0 + next.kt;
#pragma unroll
                for (int g = 0; g < PG; g++) p[g] = __ldg(reinterpret_cast<const uint32_t *>(a.params) + (tile * PG + g) * 16 + row % 16);
                next.next(1);
            };
            fetch(par[0]);
            if (units > 1) fetch(par[1]);
            int d = 0;
#pragma unroll
            for (int i = 0; i < NC / 2; i++) tot[i] = 0;
            auto unit = [&](int u, uint32_t (&mine)[PG]) {
#pragma unroll
                for (int g = 0; g < PG; g++, d++) {
                    const int i = d % SD;
                    const float2 p = __half22float2(kvq_h2(mine[g]));
                    const uint64_t lo = kvq_pair(p.x, p.x), step = kvq_pair(p.y * 512.f, p.y * 512.f);
                    const uint32_t sc = scales + at.kt * (NC * 4), sum = sums + (at.kt * PG + g) * (NC * 4);
                    wait(d_full + 8 * i, (d / SD) & 1, err, a.waits);
                    fence_after();
                    const uint32_t from = tmem + i * N + (uint32_t(32 * q) << 16);
                    uint32_t v[2][8];
                    tm_load8(from, v[0]);
#pragma unroll
                    for (int c = 0; c < NC; c += 8) {
                        uint32_t (&w)[8] = v[c / 8 % 2];
                        tm_wait8(w);
                        if (c + 8 < NC) {
                            tm_load8(from + c + 8, v[(c / 8 + 1) % 2]);
                        } else {
                            fence_before();
                            __syncwarp();
                            if (lane == 0) arrive(d_empty + 8 * i);
                        }
#pragma unroll
                        for (int e = 0; e < 8; e += 4) {
                            const ulonglong2 f = lds_two_pairs(sc + 4 * (c + e)), x = lds_two_pairs(sum + 4 * (c + e));
                            uint64_t &t0 = tot[(c + e) / 2], &t1 = tot[(c + e) / 2 + 1];
                            t0 = kvq_fma2(kvq_mul2(step, f.x), kvq_pair(__uint_as_float(w[e]), __uint_as_float(w[e + 1])), kvq_fma2(lo, x.x, t0));
                            t1 = kvq_fma2(kvq_mul2(step, f.y), kvq_pair(__uint_as_float(w[e + 2]), __uint_as_float(w[e + 3])), kvq_fma2(lo, x.y, t1));
                        }
                    }
                }
                if (u + 2 < units) fetch(mine);
                if (at.kt + 1 == tiles) {
                    begin(at.rb);
#pragma unroll
                    for (int c = 0; c < NC; c += 4) {
                        float y[4];
                        kvq_split(tot[c / 2], y[0], y[1]);
                        kvq_split(tot[c / 2 + 1], y[2], y[3]);
                        tot[c / 2] = tot[c / 2 + 1] = 0;
                        if (a.terms == 1) {
#pragma unroll
                            for (int e = 0; e < 4; e++) put(c + e, y[e]);
                        } else if (a.terms == 2) {
                            put(c / 2, y[0] + y[1]);
                            put(c / 2 + 1, y[2] + y[3]);
                        } else {
                            put(c / 4, (y[0] + y[1]) + (y[2] + y[3]));
                        }
                    }
                    end();
                }
                at.next(1);
            };
            for (int u = 0; u < units; u += 2) {
                unit(u, par[0]);
                if (u + 1 < units) unit(u + 1, par[1]);
            }
        }
        fence_before();
    }
    if (C > 1) cluster_sync();  // (no block ends while others read its shares)
    __syncthreads();
    if (*err) {  // a wait has run out: products in flight end before their memory goes
        if (warp == W_MMA) {
            commit(drained);
            bar_wait_long(drained, 0, KVQ_DRAIN_NS);
        }
        __syncthreads();
    }
    if (warp == W_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

template <int NC, int PG, bool HALF>
int smem_bytes(int slice, int depth, int cluster, int tokens) {
    using S = Shape<NC, PG, HALF>;
    return 1024 + (S::x_bytes(slice) + 15) / 16 * 16 + UNPACK * depth * S::SLOT + (cluster > 1 || !HALF ? 2 * tokens * 512 : 0);
}

// Clusters of c blocks, one an SM, that the device holds at a time (c = 8: fewer than SMs / 8, by the SMs of a GPC).
int clusters_of(const void *kernel, int c, int nsm) {
    static std::atomic<int> known[4];  // (of 1, 2, 4, 8; every device is alike)
    const int at = c == 1 ? 0 : c == 2 ? 1 : c == 4 ? 2 : 3;
    if (c == 1) return nsm;
    int n = known[at].load(std::memory_order_relaxed);
    if (n) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm / c * c);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = MAX_SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(c), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        return nsm / c;
    }
    known[at].store(n, std::memory_order_relaxed);
    return n;
}

template <int NC, int PG, bool HALF>
int launch(const TcArgs &in, int nsm, cudaStream_t st) {
    const void *kernel = reinterpret_cast<const void *>(k_qmat_tc<NC, PG, HALF>);
    if (!allow_smem(kernel, MAX_SMEM)) return LL_ERR_CUDA;
    // Blocks that share the columns, by the units of the busiest block: what fits, then the fewest steps, with
    // 2 for a row block's end, 4 where shares meet.
    TcArgs a = in;
    a.cluster = 0;
    int at_once = 0;
    const int RB = (in.RT + 7) / 8;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= MAX_CLUSTER; c *= 2) {
        const int slice = (in.KT + c - 1) / c;
        if ((c - 1) * slice >= in.KT) break;  // (a block without a tile)
        int depth = 8;
        while (depth > 2 && smem_bytes<NC, PG, HALF>(slice, depth, c, in.tokens) > MAX_SMEM) depth--;
        if (smem_bytes<NC, PG, HALF>(slice, depth, c, in.tokens) > MAX_SMEM) continue;
        const int held = clusters_of(kernel, c, nsm);
        const int64_t rounds = (RB + held - 1) / held, steps = rounds * (slice + (c > 1 ? 4 : 2)) + (depth < 4 ? slice : 0);
        if (steps < best) {
            best = steps;
            a.cluster = c;
            a.slice = slice;
            a.depth = depth;
            at_once = held;
        }
    }
    if (!a.cluster) return LL_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(std::min(RB, at_once) * a.cluster, (a.n + a.tokens - 1) / a.tokens);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<NC, PG, HALF>(a.slice, a.depth, a.cluster, a.tokens);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {unsigned(a.cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_qmat_tc<NC, PG, HALF>, a) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

template <int NC, bool HALF>
int launch_pg(const TcArgs &a, int pg, int nsm, cudaStream_t st) {
    return pg == 1 ? launch<NC, 1, HALF>(a, nsm, st) : pg == 2 ? launch<NC, 2, HALF>(a, nsm, st) : launch<NC, 4, HALF>(a, nsm, st);
}
template <bool HALF>
int launch_nc(const TcArgs &a, int nc, int pg, int nsm, cudaStream_t st) {
    return nc == 64 ? launch_pg<64, HALF>(a, pg, nsm, st) : nc == 32 ? launch_pg<32, HALF>(a, pg, nsm, st) : launch_pg<16, HALF>(a, pg, nsm, st);
}

}  // namespace

// LL_ERR_SHAPE: x does not fit into shared memory (nothing was launched).
int launch_qmat_tc(const ll_qmat &m, const ll_rows &x, int n, const ll_rows *add, const ll_rows &y, int nsm, cudaStream_t st) {
    TcArgs a = {};
    a.codes = reinterpret_cast<const uint4 *>(m.codes);
    a.params = reinterpret_cast<const uint4 *>(m.params);
    a.rows = m.rows;
    a.cols = m.cols;
    a.KT = (m.cols + QM_TILE_COLS - 1) / QM_TILE_COLS;
    a.RT = (m.rows + QM_TILE_ROWS - 1) / QM_TILE_ROWS;
    a.x = x.data;
    a.x_type = x.type;
    a.x_stride = n > 1 ? x.stride : 0;
    a.scale = x.scale;
    a.scale_row = x.group ? a.KT : 1;
    a.scale_step = x.group ? 1 : 0;
    const int size = x.type == LL_F32 ? 4 : x.type == LL_BF16 ? 2 : 1, wide = size == 1 ? 8 : 16;
    a.vec = reinterpret_cast<uintptr_t>(x.data) % wide == 0 && (a.x_stride * size) % wide == 0;
    a.add = add ? add->data : nullptr;
    a.add_stride = add ? add->stride : 0;
    a.y = y.data;
    a.y_stride = y.stride;
    a.y_f32 = y.type == LL_F32;
    a.n = n;
    const bool half = !a.y_f32 && x.type != LL_F32;
    a.terms = half ? 1 : x.type == LL_F32 ? 4 : x.type == LL_BF16 ? 2 : 1;
    const int pg = QM_TILE_COLS / m.group;
    // As many columns of x a pass as there are, up to 64; fewer where they do not fit.
    for (int nc = n * a.terms <= 16 ? 16 : n * a.terms <= 32 ? 32 : 64; nc >= 16; nc /= 2) {
        a.tokens = nc / a.terms;
        const int rc = half ? launch_nc<true>(a, nc, pg, nsm, st) : launch_nc<false>(a, nc, pg, nsm, st);
        if (rc != LL_ERR_SHAPE) return rc;
    }
    return LL_ERR_SHAPE;
}

}  // namespace ll

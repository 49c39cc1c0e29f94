// qmat_mul.cu -- y = x W^T (+ add) for rows x and a matrix W in 4 bits (format in include/ll.h).
//
//   y[i][r] = sum over groups G of  step (sum_k (c - 8) x) + (lo + 8 step) (sum_k x),   k in G
//
// The integers c - 8 and the terms of x are exact in bf16, so a group's two sums are matrix products
// with exact terms and fp32 sums, the second one with a matrix of ones; lo and step meet them in fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "call.h"
#include "qmat.cuh"
#include "qmat.h"

namespace ll {
namespace {

constexpr int MV_WARPS = 8;
constexpr int MV_THREADS = 32 * MV_WARPS;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Streamed past L1: codes are read once.
__device__ __forceinline__ uint4 ld_codes(const uint4 *p) {
    uint4 u;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

struct MvArgs {
    const uint4 *codes;
    const __half2 *params;  // (lo, step)
    int rows, cols, KT, RT;
    const void *x;
    int64_t x_stride;
    const float *scale;     // e4m3: [n][scale_row], the tile's or (scale_step 0) the row's
    int scale_row, scale_step;
    bool vec;               // x's rows take 8-value loads
    const void *add;
    int64_t add_stride;
    void *y;
    int64_t y_stride;
    bool y_f32;
    int n;
    int splits;             // warps that share a row tile's columns, a divisor of MV_WARPS
};

// One column of x's fragments: a token, or one of the three bf16 terms of an fp32 one (cut, not rounded:
// 8 of its 24 bits each, so that they add up to it exactly).
template <int XT>
struct Column {
    static constexpr int TERMS = XT == LL_F32 ? 3 : 1;
    const char *row;
    int term;
    bool held;
    __device__ __forceinline__ Column(const MvArgs &a, int c, int first) {
        const int token = first + c / TERMS;
        term = c % TERMS;
        held = token < a.n;
        constexpr int SIZE = XT == LL_F32 ? 4 : XT == LL_BF16 ? 2 : 1;
        row = static_cast<const char *>(a.x) + int64_t(held ? token : 0) * a.x_stride * SIZE;
    }
    // The 8 values from column k on as four bf16 pairs.
    __device__ __forceinline__ void load(const MvArgs &a, int k, uint32_t (&b)[4]) const {
        if (!held || k >= a.cols) {
            b[0] = b[1] = b[2] = b[3] = 0;
            return;
        }
        const bool whole = a.vec && k + 8 <= a.cols;
        if constexpr (XT == LL_BF16) {
            const uint16_t *p = reinterpret_cast<const uint16_t *>(row) + k;
            if (whole) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
                b[0] = u.x; b[1] = u.y; b[2] = u.z; b[3] = u.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t lo = k + 2 * i < a.cols ? p[2 * i] : 0, hi = k + 2 * i + 1 < a.cols ? p[2 * i + 1] : 0;
                    b[i] = lo | hi << 16;
                }
            }
        } else if constexpr (XT == LL_F32) {
            const float *p = reinterpret_cast<const float *>(row) + k;
            float v[8];
            if (whole) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(p)), w = __ldg(reinterpret_cast<const float4 *>(p) + 1);
                v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w; v[4] = w.x; v[5] = w.y; v[6] = w.z; v[7] = w.w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = k + i < a.cols ? p[i] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t t[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float r = v[2 * i + e];
                    float cut = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
                    if (term > 0) {
                        r -= cut;
                        cut = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
                    }
                    if (term > 1) {
                        r -= cut;
                        cut = r;
                    }
                    t[e] = __float_as_uint(cut);
                }
                b[i] = t[0] >> 16 | (t[1] & 0xffff0000u);
            }
        } else {
            const uint8_t *p = reinterpret_cast<const uint8_t *>(row) + k;
            uint32_t w[2] = {0, 0};
            if (whole) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
                w[0] = u.x;
                w[1] = u.y;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) w[i / 4] |= (k + i < a.cols ? uint32_t(p[i]) : 0u) << (8 * (i % 4));
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {  // (e4m3 is exact in fp16 and in bf16)
                uint32_t h;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w[i / 2] >> (16 * (i % 2)))));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                b[i] = bf16_pair(f.x, f.y);
            }
        }
    }
};

// A warp takes R row tiles and the k tiles ks, ks + splits, ... of them, with up to 8 NT columns of x.
template <int XT, int NT, int R, int PG>
__global__ void __launch_bounds__(MV_THREADS) k_qmat_mv(const MvArgs a) {
    constexpr int TERMS = Column<XT>::TERMS, TOKENS = 8 * NT / TERMS;
    __shared__ float part[MV_WARPS][R * QM_TILE_ROWS][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ks = warp % a.splits, groups = MV_WARPS / a.splits;
    const int rt0 = (blockIdx.x * groups + warp / a.splits) * R;
    const int first = blockIdx.y * TOKENS;
    uint32_t magic;
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(magic));
    float tot[R][NT][4];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int i = 0; i < 4; i++) tot[r][nt][i] = 0.f;
    if (rt0 < a.RT) {
        const uint4 *codes[R];
        const __half2 *params[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int64_t tile = int64_t(min(rt0 + r, a.RT - 1)) * a.KT;  // (past the end: a tile twice, its rows not stored)
            codes[r] = a.codes + tile * 64 + lane;
            params[r] = a.params + tile * (PG * QM_TILE_ROWS) + g;
        }
        for (int kt = ks; kt < a.KT; kt += a.splits) {
            uint4 c[R][2];
            __half2 p[R][PG][2];
#pragma unroll
            for (int r = 0; r < R; r++) {
                c[r][0] = ld_codes(codes[r] + int64_t(kt) * 64);
                c[r][1] = ld_codes(codes[r] + int64_t(kt) * 64 + 32);
#pragma unroll
                for (int s = 0; s < PG; s++) {
                    p[r][s][0] = __ldg(params[r] + (int64_t(kt) * PG + s) * QM_TILE_ROWS);
                    p[r][s][1] = __ldg(params[r] + (int64_t(kt) * PG + s) * QM_TILE_ROWS + 8);
                }
            }
#pragma unroll
            for (int s = 0; s < PG; s++) {
                float acc[R][NT][4], ones[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
#pragma unroll
                    for (int i = 0; i < 4; i++) ones[nt][i] = 0.f;
#pragma unroll
                    for (int r = 0; r < R; r++)
#pragma unroll
                        for (int i = 0; i < 4; i++) acc[r][nt][i] = 0.f;
                }
#pragma unroll
                for (int jj = 0; jj < 4 / PG; jj++) {
                    const int j = s * (4 / PG) + jj;
                    uint32_t b[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        const Column<XT> col(a, nt * 8 + g, first);
                        col.load(a, kt * QM_TILE_COLS + 32 * j + 8 * t, b[nt]);
                    }
#pragma unroll
                    for (int m = 0; m < 2; m++) {
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) mma_bf16(ones[nt], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, b[nt][2 * m], b[nt][2 * m + 1]);
#pragma unroll
                        for (int r = 0; r < R; r++) {
                            const uint32_t lo = (&c[r][0].x)[j], hi = (&c[r][1].x)[j];
                            const uint32_t a0 = qm_codes(lo, 2 * m, magic), a1 = qm_codes(hi, 2 * m, magic);
                            const uint32_t a2 = qm_codes(lo, 2 * m + 1, magic), a3 = qm_codes(hi, 2 * m + 1, magic);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) mma_bf16(acc[r][nt], a0, a1, a2, a3, b[nt][2 * m], b[nt][2 * m + 1]);
                        }
                    }
                }
                float sc[NT][2];
                if constexpr (XT == LL_E4M3) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int token = first + nt * 8 + 2 * t + e;
                            sc[nt][e] = token < a.n ? __ldg(a.scale + int64_t(token) * a.scale_row + kt * a.scale_step) : 0.f;
                        }
                }
#pragma unroll
                for (int r = 0; r < R; r++) {
                    const float2 p0 = __half22float2(p[r][s][0]), p1 = __half22float2(p[r][s][1]);
                    const float z0 = fmaf(8.f, p0.y, p0.x), z1 = fmaf(8.f, p1.y, p1.x);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const float step = i < 2 ? p0.y : p1.y, z = i < 2 ? z0 : z1;
                            if constexpr (XT == LL_E4M3)
                                tot[r][nt][i] = fmaf(fmaf(step, acc[r][nt][i], z * ones[nt][i & 1]), sc[nt][i & 1], tot[r][nt][i]);
                            else
                                tot[r][nt][i] = fmaf(step, acc[r][nt][i], fmaf(z, ones[nt][i & 1], tot[r][nt][i]));
                        }
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int i = 0; i < 4; i++) part[warp][r * QM_TILE_ROWS + g + 8 * (i / 2)][nt * 8 + 2 * t + (i & 1)] = tot[r][nt][i];
    __syncthreads();
    // the splits' shares and an fp32 token's terms added up
    constexpr int ROWS = R * QM_TILE_ROWS;
    for (int e = threadIdx.x; e < groups * ROWS * TOKENS; e += MV_THREADS) {
        const int in = e % (groups * ROWS), token = e / (groups * ROWS), grp = in / ROWS;
        const int64_t row = int64_t(blockIdx.x) * groups * ROWS + in;
        if (row >= a.rows || first + token >= a.n) continue;
        float y = 0.f;
        for (int s = 0; s < a.splits; s++)
#pragma unroll
            for (int u = TERMS - 1; u >= 0; u--) y += part[grp * a.splits + s][in % ROWS][token * TERMS + u];
        const int64_t at = int64_t(first + token) * a.y_stride + row, from = int64_t(first + token) * a.add_stride + row;
        if (a.y_f32) {
            if (a.add) y += static_cast<const float *>(a.add)[from];
            static_cast<float *>(a.y)[at] = y;
        } else {
            if (a.add) y += __bfloat162float(static_cast<const __nv_bfloat16 *>(a.add)[from]);
            static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(y);
        }
    }
}

template <int XT, int NT, int R>
void launch_mv(const MvArgs &a, int pg, int nsm, cudaStream_t st) {
    constexpr int TOKENS = 8 * NT / Column<XT>::TERMS;
    MvArgs b = a;
    const int tiles = (a.RT + R - 1) / R;
    b.splits = 1;
    while (b.splits < MV_WARPS && int64_t(tiles) * b.splits < int64_t(nsm) * 16 && 2 * b.splits <= a.KT) b.splits *= 2;
    const int groups = MV_WARPS / b.splits;
    const dim3 grid((tiles + groups - 1) / groups, (a.n + TOKENS - 1) / TOKENS);
    if (pg == 1) k_qmat_mv<XT, NT, R, 1><<<grid, MV_THREADS, 0, st>>>(b);
    else if (pg == 2) k_qmat_mv<XT, NT, R, 2><<<grid, MV_THREADS, 0, st>>>(b);
    else k_qmat_mv<XT, NT, R, 4><<<grid, MV_THREADS, 0, st>>>(b);
}

template <int XT>
void launch_mv_type(const MvArgs &a, int pg, int nsm, cudaStream_t st) {
    const int columns = a.n * Column<XT>::TERMS;
    if (columns <= 8) launch_mv<XT, 1, 2>(a, pg, nsm, st);
    else if (columns <= 16) launch_mv<XT, 2, 2>(a, pg, nsm, st);
    else launch_mv<XT, 4, 1>(a, pg, nsm, st);
}

}  // namespace

int launch_qmat_mul(const ll_qmat &m, const ll_rows &x, int n, const ll_rows *add, const ll_rows &y, int nsm, cudaStream_t st) {
    MvArgs a = {};
    a.codes = reinterpret_cast<const uint4 *>(m.codes);
    a.params = reinterpret_cast<const __half2 *>(m.params);
    a.rows = m.rows;
    a.cols = m.cols;
    a.KT = (m.cols + QM_TILE_COLS - 1) / QM_TILE_COLS;
    a.RT = (m.rows + QM_TILE_ROWS - 1) / QM_TILE_ROWS;
    a.x = x.data;
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
    const int pg = QM_TILE_COLS / m.group;
    if (x.type == LL_BF16) launch_mv_type<LL_BF16>(a, pg, nsm, st);
    else if (x.type == LL_F32) launch_mv_type<LL_F32>(a, pg, nsm, st);
    else launch_mv_type<LL_E4M3>(a, pg, nsm, st);
    return launched();
}

}  // namespace ll

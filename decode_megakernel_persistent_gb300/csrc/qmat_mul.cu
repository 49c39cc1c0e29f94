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
// Tiles of a warp in flight, and blocks of an SM.
template <int NT>
struct MvGeo {
    static constexpr int UNITS = NT == 1 ? 8 : 6, BLOCKS = NT <= 2 ? 2 : 1;
};
constexpr int MV_STAGE = 1024 + 4 * 16 * 4;  // a tile's codes and (4 groups') parameters in shared memory

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
    return u;
}
__device__ __forceinline__ float2 lds_pair(uint32_t at) {  // (lo, step)
    uint32_t u;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(at) : "memory");
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
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
    int pg;                 // parameter groups of a tile
    int splits;             // warps that share a row tile's columns, a divisor of MV_WARPS
};

// One column of x's fragments: a token, or one of the three bf16 terms of an fp32 one (cut, not rounded:
// 8 of its 24 bits each, so that they add up to it exactly).
template <int XT>
struct Column {
    static constexpr int TERMS = XT == LL_F32 ? 3 : 1;
    static constexpr int SIZE = XT == LL_F32 ? 4 : XT == LL_BF16 ? 2 : 1;
    const char *row;
    int term;
    bool held;
    __device__ __forceinline__ Column(const MvArgs &a, int c, int first) {
        const int token = first + c / TERMS;
        term = c % TERMS;
        held = token < a.n;
        row = static_cast<const char *>(a.x) + int64_t(held ? token : 0) * a.x_stride * SIZE;
    }
    // The 8 values from column k on, as they lie in memory.
    struct Raw {
        uint32_t w[2 * SIZE];
    };
    __device__ __forceinline__ Raw load(const MvArgs &a, int k) const {
        Raw r;
#pragma unroll
        for (int i = 0; i < 2 * SIZE; i++) r.w[i] = 0;
        if (!held || k >= a.cols) return r;
        const char *p = row + int64_t(k) * SIZE;
        if (a.vec && k + 8 <= a.cols) {
            if constexpr (SIZE == 1) {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
                r.w[0] = u.x; r.w[1] = u.y;
            } else {
#pragma unroll
                for (int i = 0; i < SIZE / 2; i++) {
                    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                    r.w[4 * i] = u.x; r.w[4 * i + 1] = u.y; r.w[4 * i + 2] = u.z; r.w[4 * i + 3] = u.w;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                if (k + i >= a.cols) continue;
                if constexpr (SIZE == 4) r.w[i] = reinterpret_cast<const uint32_t *>(p)[i];
                else if constexpr (SIZE == 2) r.w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t *>(p)[i]) << (16 * (i % 2));
                else r.w[i / 4] |= uint32_t(reinterpret_cast<const uint8_t *>(p)[i]) << (8 * (i % 4));
            }
        }
        return r;
    }
    // The same as four bf16 pairs.
    __device__ __forceinline__ void pairs(const Raw &r, uint32_t (&b)[4]) const {
        if constexpr (XT == LL_BF16) {
#pragma unroll
            for (int i = 0; i < 4; i++) b[i] = r.w[i];
        } else if constexpr (XT == LL_F32) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                uint32_t t[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float v = __uint_as_float(r.w[2 * i + e]);
                    float cut = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
                    if (term > 0) {
                        v -= cut;
                        cut = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
                    }
                    if (term > 1) cut = v - cut;
                    t[e] = __float_as_uint(cut);
                }
                b[i] = __byte_perm(t[0], t[1], 0x7632);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {  // (e4m3 is exact in fp16 and in bf16)
                uint32_t h;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(r.w[i / 2] >> (16 * (i % 2)))));
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                b[i] = bf16_pair(f.x, f.y);
            }
        }
    }
};

// A few rows x: up to 8 NT columns. A warp takes R row tiles at a time and, of `splits` warps that share them, every
// splits-th tile of 128 columns. Its next tiles are always on their way (cp.async into a ring of its own), across
// its row tiles, so no latency shows but the first.
// EXACT: the codes as c - 8 (fp32 y: 1.4e-7 of the outputs' norm off); otherwise as 16 + c, a subtraction a pair
// less, whose sums are some six times as large, and so are their roundings (bf16 y rounds 2^-9).
template <int XT, int NT, int R, bool EXACT>
__global__ void __launch_bounds__(MV_THREADS, MvGeo<NT>::BLOCKS) k_qmat_mv(const MvArgs a) {
    constexpr int TERMS = Column<XT>::TERMS, TOKENS = 8 * NT / TERMS, UNITS = MvGeo<NT>::UNITS, DEPTH = UNITS / R;
    extern __shared__ __align__(16) uint8_t ring[];  // [warp][DEPTH][R][MV_STAGE]
    __shared__ float part[2][MV_WARPS][R * QM_TILE_ROWS][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int ks = warp % a.splits, team = warp / a.splits, teams = MV_WARPS / a.splits;
    const int groups = (a.RT + R - 1) / R, stride = gridDim.x * teams;
    const int first = blockIdx.y * TOKENS;
    const int own = (a.KT - ks + a.splits - 1) / a.splits;  // (splits <= KT: 1 at least)
    const uint32_t stages = uint32_t(__cvta_generic_to_shared(ring)) + warp * (UNITS * MV_STAGE);
    uint32_t magic;
    asm volatile("mov.b32 %0, 0x41804180;" : "=r"(magic));
    // (teams of a block are gridDim.x groups apart: with fewer groups than teams, blocks have alike many)
    const int g0 = blockIdx.x + gridDim.x * team;

    int next_group = g0, next_k = 0, next_stage = 0;
    auto issue = [&]() {
        if (next_group < groups) {
            const int kt = ks + next_k * a.splits;
#pragma unroll
            for (int r = 0; r < R; r++) {
                const int64_t tile = int64_t(min(next_group * R + r, a.RT - 1)) * a.KT + kt;  // (past the end: a tile twice, its rows not stored)
                const uint32_t to = stages + (next_stage * R + r) * MV_STAGE;
                copy16(to + 16 * lane, a.codes + tile * 64 + lane);
                copy16(to + 512 + 16 * lane, a.codes + tile * 64 + 32 + lane);
                if (lane < 4 * a.pg) copy16(to + 1024 + 16 * lane, reinterpret_cast<const uint4 *>(a.params) + tile * (4 * a.pg) + lane);
            }
            if (++next_k == own) {
                next_k = 0;
                next_group += stride;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next_stage = next_stage + 1 == DEPTH ? 0 : next_stage + 1;
    };
#pragma unroll
    for (int i = 0; i < DEPTH - 1; i++) issue();

    int stage = 0, parity = 0;
    typename Column<XT>::Raw ahead[NT][4];  // x of the next tile
    auto load_x = [&](int kt) {
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const Column<XT> col(a, nt * 8 + g, first);
#pragma unroll
            for (int j = 0; j < 4; j++) ahead[nt][j] = col.load(a, kt * QM_TILE_COLS + 32 * j + 8 * t);
        }
    };
    constexpr bool AHEAD = NT == 1 && XT != LL_F32;  // (registers)
    if (AHEAD && g0 < groups) load_x(ks);
    for (int group = g0; group < groups; group += stride) {
        float tot[R][NT][4];
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int i = 0; i < 4; i++) tot[r][nt][i] = 0.f;
        for (int k = 0; k < own; k++) {
            const int kt = ks + k * a.splits;
            uint32_t b[NT][4][4];
            if (!AHEAD) load_x(kt);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const Column<XT> col(a, nt * 8 + g, first);
#pragma unroll
                for (int j = 0; j < 4; j++) col.pairs(ahead[nt][j], b[nt][j]);
            }
            if (AHEAD) load_x(k + 1 < own ? kt + a.splits : ks);
            issue();
            asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
            __syncwarp();  // (parameters come by other lanes' copies)
            uint4 c[R][2];
#pragma unroll
            for (int r = 0; r < R; r++) {
                c[r][0] = lds16(stages + (stage * R + r) * MV_STAGE + 16 * lane);
                c[r][1] = lds16(stages + (stage * R + r) * MV_STAGE + 512 + 16 * lane);
            }
            float acc[R][NT][4], ones[NT][4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (j == 0 || (j * a.pg) % 4 == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            ones[nt][i] = 0.f;
#pragma unroll
                            for (int r = 0; r < R; r++) acc[r][nt][i] = 0.f;
                        }
                }
#pragma unroll
                for (int m = 0; m < 2; m++) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
                        mma_bf16(ones[nt], 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u, b[nt][j][2 * m], b[nt][j][2 * m + 1]);
#pragma unroll
                    for (int r = 0; r < R; r++) {
                        const uint32_t lo = (&c[r][0].x)[j], hi = (&c[r][1].x)[j];
                        const uint32_t a0 = qm_codes<EXACT>(lo, 2 * m, magic), a1 = qm_codes<EXACT>(hi, 2 * m, magic);
                        const uint32_t a2 = qm_codes<EXACT>(lo, 2 * m + 1, magic), a3 = qm_codes<EXACT>(hi, 2 * m + 1, magic);
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) mma_bf16(acc[r][nt], a0, a1, a2, a3, b[nt][j][2 * m], b[nt][j][2 * m + 1]);
                    }
                }
                if (((j + 1) * a.pg) % 4 != 0) continue;
                // the group's end: its sums meet their parameters
                const int s = j * a.pg / 4;
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
                    const uint32_t at = stages + (stage * R + r) * MV_STAGE + 1024 + (s * QM_TILE_ROWS + g) * 4;
                    const float2 p0 = lds_pair(at), p1 = lds_pair(at + 32);
                    constexpr float ZERO = EXACT ? 8.f : -16.f;
                    const float z0 = fmaf(ZERO, p0.y, p0.x), z1 = fmaf(ZERO, p1.y, p1.x);
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
            __syncwarp();  // (before another lane's copy into this stage)
            stage = stage + 1 == DEPTH ? 0 : stage + 1;
        }
        // the splits' shares and an fp32 token's terms added up
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int i = 0; i < 4; i++) part[parity][warp][r * QM_TILE_ROWS + g + 8 * (i / 2)][nt * 8 + 2 * t + (i & 1)] = tot[r][nt][i];
        // (the shares of the group before last lie in the other half: one barrier a group)
        if (a.splits == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(32 * a.splits) : "memory");
        constexpr int ROWS = R * QM_TILE_ROWS;
        for (int e = ks * 32 + lane; e < ROWS * TOKENS; e += 32 * a.splits) {
            const int in = e % ROWS, token = e / ROWS;
            const int64_t row = int64_t(group) * ROWS + in;
            if (row >= a.rows || first + token >= a.n) continue;
            float y = 0.f;
            for (int s = 0; s < a.splits; s++)
#pragma unroll
                for (int u = TERMS - 1; u >= 0; u--) y += part[parity][team * a.splits + s][in][token * TERMS + u];
            const int64_t at = int64_t(first + token) * a.y_stride + row, from = int64_t(first + token) * a.add_stride + row;
            if (a.y_f32) {
                if (a.add) y += static_cast<const float *>(a.add)[from];
                static_cast<float *>(a.y)[at] = y;
            } else {
                if (a.add) y += __bfloat162float(static_cast<const __nv_bfloat16 *>(a.add)[from]);
                static_cast<__nv_bfloat16 *>(a.y)[at] = __float2bfloat16_rn(y);
            }
        }
        parity ^= 1;
    }
}

template <int XT, int NT, int R, bool EXACT>
int launch_mv(const MvArgs &a, int nsm, cudaStream_t st) {
    constexpr int TOKENS = 8 * NT / Column<XT>::TERMS, SMEM = MV_WARPS * MvGeo<NT>::UNITS * MV_STAGE;
    if (!allow_smem(reinterpret_cast<const void *>(k_qmat_mv<XT, NT, R, EXACT>), SMEM)) return LL_ERR_CUDA;
    MvArgs b = a;
    // splits by the steps of the busiest warp: its tiles, and 2 a group for the shares' barrier
    const int tiles = (a.RT + R - 1) / R, blocks = MvGeo<NT>::BLOCKS * nsm;
    int64_t best = INT64_MAX;
    for (int splits = 1; splits <= MV_WARPS && splits <= a.KT; splits *= 2) {
        const int64_t slots = int64_t(blocks) * (MV_WARPS / splits), rounds = (tiles + slots - 1) / slots;
        const int64_t steps = rounds * ((a.KT + splits - 1) / splits * R + (splits > 1 ? 2 : 1));
        if (steps < best) {
            best = steps;
            b.splits = splits;
        }
    }
    // (fewer groups than slots: one a block before two in one)
    const dim3 grid(tiles < blocks ? tiles : blocks, (a.n + TOKENS - 1) / TOKENS);
    k_qmat_mv<XT, NT, R, EXACT><<<grid, MV_THREADS, SMEM, st>>>(b);
    return launched();
}

template <int XT>
int launch_mv_type(const MvArgs &a, int nsm, cudaStream_t st) {
    const int columns = a.n * Column<XT>::TERMS;
    // two row tiles a warp share x's fragments; one where that leaves SMs without any
    const bool two = a.RT >= 4 * nsm;
    if (a.y_f32) {
        if (columns <= 8) return two ? launch_mv<XT, 1, 2, true>(a, nsm, st) : launch_mv<XT, 1, 1, true>(a, nsm, st);
        return columns <= 16 ? launch_mv<XT, 2, 2, true>(a, nsm, st) : launch_mv<XT, 4, 1, true>(a, nsm, st);
    }
    if (columns <= 8) return two ? launch_mv<XT, 1, 2, false>(a, nsm, st) : launch_mv<XT, 1, 1, false>(a, nsm, st);
    return columns <= 16 ? launch_mv<XT, 2, 2, false>(a, nsm, st) : launch_mv<XT, 4, 1, false>(a, nsm, st);
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
    a.pg = QM_TILE_COLS / m.group;
    return x.type == LL_BF16 ? launch_mv_type<LL_BF16>(a, nsm, st) : x.type == LL_F32 ? launch_mv_type<LL_F32>(a, nsm, st) : launch_mv_type<LL_E4M3>(a, nsm, st);
}

}  // namespace ll

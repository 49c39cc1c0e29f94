// verify.cu -- drafted tokens against the target's probabilities (ll_verify in include/ll.h).
//
// A cluster of blocks has one sequence, each block a slice of the vocabulary.
//   1. Row by row: the slice's largest logit m and sum of exp((l - m) / T) in fp32, one pass; the blocks
//      give each other theirs, and every block decides alike whether the row's draft stands.
//   2. The row that draws: a draw has a border at each of some 10^5 tokens, and a residual max(p - q, 0) is
//      a difference of near numbers, so weights are taken from exponentials of two fp32 (about 2^-45 of
//      themselves) and held as integers, in units of 2^-43 of the largest: their sums are exact in any
//      order. Sums go round the cluster; the block, the warp and the lane where the sum passes u times the
//      whole one find the token.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "call.h"

namespace cg = cooperative_groups;

namespace ll {
namespace {

constexpr int VF_THREADS = 512, VF_WARPS = VF_THREADS / 32;
constexpr int VF_CLUSTER = 16;
constexpr int VF_ROWS = 8;               // rows of a step, at most
constexpr int VF_PIECES = 8 * 24;        // pieces of a step: of 1024 places, or 512 of a single row's
constexpr int VF_STEP = 4;               // neighbouring logits of a lane
constexpr int VF_MAX_VOCAB = 393216;     // a slice's weights (8 bytes each) fit in shared memory
constexpr int VF_WINDOWS = VF_MAX_VOCAB / VF_CLUSTER / VF_WARPS / 128;
constexpr double LN2 = 0.693147180559945309417232, LOG2E = 1.442695040888963407359925;

struct VfArgs {
    const void *logits;
    int64_t logits_seq, logits_row;
    const int32_t *draft, *n_draft_dev;
    const float *probs;
    int64_t probs_seq, probs_row;
    const float *u, *temperature;
    int32_t n_draft, vocab, slice;  // slice: a multiple of VF_STEP
    int32_t log_rows, piece;        // 2^this rows a step; places of a warp's piece of one
    bool vec, vec_probs;            // rows take whole-step loads
    int32_t *tokens, *accepted;
};

struct Two {  // hi + lo, |lo| at most half a unit in hi's last place (or near it)
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, bb = s - a;
    return {s, (a - (s - bb)) + (b - bb)};
}
__device__ __forceinline__ Two fast_two_sum(float a, float b) {  // |a| >= |b|
    const float s = a + b;
    return {s, b - (s - a)};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    const float p = __fmul_rn(a.hi, b.hi);
    return {p, fmaf(a.hi, b.hi, -p) + fmaf(a.hi, b.lo, a.lo * b.hi)};
}

// 2^(j / 32), j < 32, by the series of e^(j ln 2 / 32) in 64 bits, as two fp32.
struct Roots {
    float hi[32], lo[32];
};
constexpr Roots make_roots() {
    Roots r = {};
    for (int j = 0; j < 32; j++) {
        double term = 1, sum = 1;
        for (int k = 1; k < 24; k++) {  // z^24 / 24! is below 2^-90
            term *= LN2 / 32 * j / k;
            sum += term;
        }
        r.hi[j] = float(sum);
        r.lo[j] = float(sum - double(r.hi[j]));
    }
    return r;
}
__constant__ const Roots ROOTS = make_roots();

// e^((l - m) / T) for l <= m, c = log2(e) / T, off by some 2^-45 of itself: 2^(k + j / 32) from the table times
// e^z, |z| <= ln 2 / 64, of which 1, z and z^2 / 2 are held in two fp32. Below 2^-50: 0.
__device__ __forceinline__ Two exp_two(float l, float m, Two c, const float2 *roots) {
    if (l == m) return {1.f, 0.f};  // (infinities, too)
    const Two d = two_sum(l, -m);
    const float yh = __fmul_rn(d.hi, c.hi);
    if (!(yh > -50.f)) return {0.f, 0.f};
    const float yl = fmaf(d.hi, c.hi, -yh) + fmaf(d.hi, c.lo, d.lo * c.hi);
    const float r = yh + 393216.f;  // 1.5 * 2^18: to multiples of 1 / 32
    const int n = __float_as_int(r) - __float_as_int(393216.f);  // 32 k + j
    const float fh = yh - (r - 393216.f);
    constexpr float LH = float(LN2), LL = float(LN2 - double(LH));
    const float zh = __fmul_rn(fh, LH), zl = fmaf(fh, LH, -zh) + fmaf(fh, LL, yl * LH);
    const float sh = 0.5f * zh, qh = __fmul_rn(sh, zh), ql = fmaf(sh, zh, -qh) + zh * zl;
    const float t = zh * zh * zh * fmaf(zh, fmaf(zh, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f);
    const Two p = fast_two_sum(zh, qh);
    const float pl = p.lo + (zl + (ql + t));
    const float2 w = roots[n & 31];
    const float g = __fmul_rn(w.x, p.hi);
    const Two s = fast_two_sum(w.x, g);
    const float lo = s.lo + (fmaf(w.x, p.hi, -g) + fmaf(w.x, pl, fmaf(w.y, p.hi, w.y)));
    const float scale = __int_as_float(((n >> 5) + 127) << 23);
    return {s.hi * scale, lo * scale};
}

// A number in [0, 1.5] in units of 2^-43, to the nearest: its upper part in units of 2^-21 and the rest, each
// rounded by the addition of 1.5 * 2^23 of its units.
__device__ __forceinline__ int64_t fixed(Two v) {
    const float a = v.hi + 6.f;
    const int h = __float_as_int(a) - __float_as_int(6.f);
    const float rest = (v.hi - (a - 6.f)) + v.lo;
    constexpr float UNIT = 1.430511474609375e-06f;  // 1.5 * 2^23 * 2^-43
    const float b = rest + UNIT;
    return (int64_t(h) << 22) + (__float_as_int(b) - __float_as_int(UNIT));
}

template <typename T>
__device__ __forceinline__ void load_step(const T *row, int i, int end, bool vec, float none, float (&x)[VF_STEP]) {
    if (vec && i + VF_STEP <= end) {
        if constexpr (sizeof(T) == 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(row + i));
            x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(row + i));
            x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xffff0000u);
            x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < VF_STEP; e++) x[e] = i + e < end ? float(row[i + e]) : none;
    }
}
// A logit as it counts: NaN as -infinity.
__device__ __forceinline__ float logit(float x) { return fmaxf(x, -INFINITY); }

// The largest logit of some, the lowest place of it, and the sum of exp((l - m) / T).
struct Stat {
    float m, sum;
    int at;
};
__device__ __forceinline__ Stat nothing() { return {-INFINITY, 0.f, 0x7fffffff}; }
__device__ __forceinline__ float weight(float l, float m, float c) { return l == m ? 1.f : exp2f((l - m) * c); }
// The largest of a warp's numbers (no NaN): as integers of the same order.
__device__ __forceinline__ float warp_max(float x) {
    const int b = __float_as_int(x), m = __reduce_max_sync(0xffffffffu, b ^ (b >> 31 & 0x7fffffff));
    return __int_as_float(m ^ (m >> 31 & 0x7fffffff));
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// The lanes' as one.
__device__ __forceinline__ Stat warp_join(Stat a, float c) {
    const float m = warp_max(a.m);
    return {m, warp_sum(a.m > -INFINITY ? a.sum * weight(a.m, m, c) : 0.f), __reduce_min_sync(0xffffffffu, a.m == m ? a.at : 0x7fffffff)};
}

struct Shared {
    Stat piece[VF_PIECES];               // of a step's rows, by pieces of the slice
    Stat stats[2][VF_ROWS][VF_CLUSTER];  // by block (steps take turns)
    Stat row[VF_ROWS];                   // of whole rows, and whether their drafts stand
    int stands[VF_ROWS];
    int64_t window[2][VF_WARPS][VF_WINDOWS];  // sums of all weights, then of the residual's, by 128 places
    int64_t warp_sum[2][VF_WARPS];
    int64_t sums[2][VF_CLUSTER];         // by block
    float2 roots[32];
};

// Block b of a sequence's cluster has slice b of the vocabulary, and in step 2 a warp one run of it, so that sums over
// blocks, warps and windows of 128 places are sums over the vocabulary in order.
template <typename T>
__global__ void __launch_bounds__(VF_THREADS) k_verify(const VfArgs a) {
    extern __shared__ __align__(16) int64_t weights[];  // [slice]
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), blocks = int(cluster.num_blocks());
    const int s = blockIdx.x / blocks, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto begun = cluster.barrier_arrive();  // (others' memory is written to once all blocks run)
    const int V = a.vocab, D = a.n_draft;
    const int first = min(V, rank * a.slice), end = min(V, first + a.slice);
    const int n = a.n_draft_dev ? min(max(a.n_draft_dev[s], 0), D) : D;
    const float given = a.temperature ? a.temperature[s] : 1.f, temp = fminf(given, 0x1p100f);
    const bool greedy = !(given > 0x1p-100f);
    const float inv = 1.f / temp;
    const Two c = greedy ? Two{0.f, 0.f} : mul({inv, fmaf(-inv, temp, 1.f) * inv}, {float(LOG2E), float(LOG2E - double(float(LOG2E)))});
    if (warp == 0) sh.roots[lane] = make_float2(ROOTS.hi[lane], ROOTS.lo[lane]);
    const T *rows = static_cast<const T *>(a.logits) + s * a.logits_seq;

    // 1. Steps of one row or several: several where few sequences leave the device waiting for memory, one where the
    // rows behind a rejection are better not read. A warp takes pieces of a row's slice.
    constexpr int U = 8;  // loads on their way: a piece is 128 times as many places, or half of them
    const int rows_step = 1 << a.log_rows, used = a.piece / 128, pieces = (a.slice + a.piece - 1) / a.piece;
    int row = 0;
    Stat all;
    bool more = true;
    for (int step = 0; more; step++) {
        const int row0 = step << a.log_rows;
        // what warp r decides row r by
        int x = -1;
        float lx = -INFINITY, q = 1.f, uj = 0.f;
        if (warp < rows_step && row0 + warp < n) {
            const int j = row0 + warp;
            x = a.draft[int64_t(s) * D + j];
            uj = a.u[int64_t(s) * (D + 1) + j];
            if (x >= 0 && x < V) {
                lx = logit(float(rows[j * a.logits_row + x]));
                if (a.probs) q = a.probs[s * a.probs_seq + j * a.probs_row + x];
            }
        }
#pragma unroll 1
        for (int t = warp; t < pieces << a.log_rows; t += VF_WARPS) {
            const int r = t / pieces, i0 = first + (t - r * pieces) * a.piece + VF_STEP * lane;
            const T *l = rows + (row0 + r) * a.logits_row;
            Stat st = nothing();
            if (row0 + r <= n) {
                float v[U][VF_STEP];
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (u < used) load_step(l, i0 + u * 128, end, a.vec, -INFINITY, v[u]);
                float top = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; u++)
                    if (u < used)
#pragma unroll
                        for (int e = 0; e < VF_STEP; e++) top = fmaxf(top, v[u][e]);  // (a NaN is passed over)
                st.m = warp_max(top);
                if (st.m > -INFINITY) {
                    float sum = 0.f;
                    int at = 0x7fffffff;
#pragma unroll
                    for (int u = U - 1; u >= 0; u--)
                        if (u < used)
#pragma unroll
                            for (int e = VF_STEP - 1; e >= 0; e--) {
                                if (greedy) at = v[u][e] == st.m ? i0 + u * 128 + e : at;
                                else sum += weight(logit(v[u][e]), st.m, c.hi);
                            }
                    if (greedy) st.at = __reduce_min_sync(0xffffffffu, at);
                    else st.sum = warp_sum(sum);
                }
            }
            if (lane == 0) sh.piece[t] = st;
        }
        __syncthreads();
        if (step == 0) cluster.barrier_wait(std::move(begun));
        if (warp < rows_step) {
            Stat st;
            // (at most 64 pieces: two a lane)
            if (pieces > 32) {
                const Stat u = lane < pieces ? sh.piece[warp * pieces + lane] : nothing();
                const Stat w = 32 + lane < pieces ? sh.piece[warp * pieces + 32 + lane] : nothing();
                const Stat ju = warp_join(u, c.hi), jw = warp_join(w, c.hi);
                st = lane == 0 ? ju : lane == 1 ? jw : nothing();
            } else {
                st = lane < pieces ? sh.piece[warp * pieces + lane] : nothing();
            }
            st = warp_join(st, c.hi);
            if (lane < blocks) cluster.map_shared_rank(&sh, lane)->stats[step & 1][warp][rank] = st;
        }
        cluster.sync();
        if (warp < rows_step) {
            const Stat st = warp_join(lane < blocks ? sh.stats[step & 1][warp][lane] : nothing(), c.hi);
            bool stands = false;
            if (row0 + warp < n && st.m > -INFINITY) {
                if (greedy) {
                    stands = x == st.at;
                } else if (x >= 0 && x < V) {
                    // u q sum < e, all but the sum exact to some 2^-45 (by fp32 pairs: 64-bit operations are few a cycle)
                    const float uq = __fmul_rn(uj, q);
                    const Two left = mul({uq, fmaf(uj, q, -uq)}, {st.sum, 0.f});
                    const Two e = exp_two(lx, st.m, c, sh.roots);
                    stands = (left.hi - e.hi) + (left.lo - e.lo) < 0.f;
                }
            }
            if (lane == 0) {
                sh.row[warp] = st;
                sh.stands[warp] = stands;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int r = 0; r < rows_step; r++) {
            row = row0 + r;
            all = sh.row[r];
            more = sh.stands[r];
            if (!more) break;
        }
    }
    const bool none = !(all.m > -INFINITY);  // no logit to draw
    int32_t *tokens = a.tokens + int64_t(s) * (D + 1);
    if (rank == 0) {
        for (int j = tid; j <= D; j += VF_THREADS)
            if (j != row || none || greedy)
                tokens[j] = j < row ? a.draft[int64_t(s) * D + j] : j == row && !none ? all.at : -1;
        if (tid == 0) a.accepted[s] = row;
    }
    if (none || greedy) return;  // (every block of the cluster; none reads another's memory any more)

    // 2. The draw. A warp's run of the slice, in windows of 128 places, four to a lane.
    const T *l = rows + row * a.logits_row;
    const bool residual = row < n;
    const float *q = residual && a.probs ? a.probs + s * a.probs_seq + row * a.probs_row : nullptr;
    const int draft = residual ? a.draft[int64_t(s) * D + row] : -1;
    const float ud = a.u[int64_t(s) * (D + 1) + D];
    const int windows = (a.slice + VF_WARPS * 128 - 1) / (VF_WARPS * 128), from = first + warp * windows * 128 + VF_STEP * lane;
    longlong2 *const mine = reinterpret_cast<longlong2 *>(weights + warp * windows * 128 + VF_STEP * lane);  // (a lane's own)
    constexpr int W = 4;  // windows on their way
#pragma unroll 1
    for (int k0 = 0; k0 < windows; k0 += W) {
        float v[W][VF_STEP];
#pragma unroll
        for (int k = 0; k < W; k++) load_step(l, from + (k0 + k) * 128, k0 + k < windows ? end : 0, a.vec, -INFINITY, v[k]);
#pragma unroll
        for (int k = 0; k < W; k++) {
            if (k0 + k >= windows) break;
            int64_t w[VF_STEP];
#pragma unroll
            for (int e = 0; e < VF_STEP; e++) w[e] = fixed(exp_two(logit(v[k][e]), all.m, c, sh.roots));
            mine[(k0 + k) * 64] = make_longlong2(w[0], w[1]);
            mine[(k0 + k) * 64 + 1] = make_longlong2(w[2], w[3]);
            const int64_t sum = warp_sum((w[0] + w[1]) + (w[2] + w[3]));
            if (lane == 0) sh.window[0][warp][k0 + k] = sum;
        }
    }
    // sums of the warps, then of the blocks, for everyone
    auto total_of = [&](int which) {
        if (lane == 0) {
            int64_t sum = 0;
            for (int k = 0; k < windows; k++) sum += sh.window[which][warp][k];
            sh.warp_sum[which][warp] = sum;
        }
        __syncthreads();
        if (warp == 0) {
            const int64_t t = warp_sum(lane < VF_WARPS ? sh.warp_sum[which][lane] : int64_t(0));
            if (lane < blocks) cluster.map_shared_rank(&sh, lane)->sums[which][rank] = t;
        }
        cluster.sync();
        return warp_sum(lane < blocks ? sh.sums[which][lane] : int64_t(0));
    };
    int64_t total = total_of(0);
    const float zh = __ll2float_rn(total), zl = __ll2float_rn(total - __float2ll_rn(zh));
    const Two Z = {zh * 0x1p-43f, zl * 0x1p-43f};
    // the residual's weight of a place
    auto left = [&](int i, int64_t w, float p) -> int64_t {
        if (!q) return i == draft ? 0 : w;
        const float h = __fmul_rn(p, Z.hi);
        if (!(h < 1.5f)) return h >= 1.5f ? 0 : w;  // (a NaN takes nothing away)
        const int64_t d = w - (h > 0.f ? fixed({h, fmaf(p, Z.hi, -h) + p * Z.lo}) : 0);
        return d > 0 ? d : 0;
    };
    int which = 0;
    if (residual) {
#pragma unroll 1
        for (int k0 = 0; k0 < windows; k0 += W) {
            float p[W][VF_STEP];
            if (q)
#pragma unroll
                for (int k = 0; k < W; k++) load_step(q, from + (k0 + k) * 128, k0 + k < windows ? end : 0, a.vec_probs, 0.f, p[k]);
#pragma unroll
            for (int k = 0; k < W; k++) {
                if (k0 + k >= windows) break;
                const longlong2 u0 = mine[(k0 + k) * 64], u1 = mine[(k0 + k) * 64 + 1];
                const int i = from + (k0 + k) * 128;
                const int64_t sum = warp_sum((left(i, u0.x, p[k][0]) + left(i + 1, u0.y, p[k][1])) + (left(i + 2, u1.x, p[k][2]) + left(i + 3, u1.y, p[k][3])));
                if (lane == 0) sh.window[1][warp][k0 + k] = sum;
            }
        }
        const int64_t t = total_of(1);
        if (t > 0) {  // (0: nothing left, and p itself)
            total = t;
            which = 1;
        }
    }
    // floor(u total), u as 24 bits and an exponent
    int64_t target = 0;
    if (ud > 0x1p-64f) {
        const uint32_t bits = __float_as_uint(ud), mant = (bits & 0x7fffffu) | 0x800000u, shift = 150 - (bits >> 23);  // u = mant / 2^shift
        const uint64_t hi = __umul64hi(uint64_t(total), mant), lo = uint64_t(total) * mant;
        target = shift >= 64 ? int64_t(hi >> (shift - 64)) : int64_t(hi << (64 - shift) | lo >> shift);
    }
    target = min(target, total - 1);
    for (int b = 0; b < rank; b++) target -= sh.sums[which][b];
    if (target < 0 || target >= sh.sums[which][rank]) return;
    for (int w = 0; w < warp; w++) target -= sh.warp_sum[which][w];
    if (target < 0 || target >= sh.warp_sum[which][warp]) return;
    int k = 0;
    for (; k + 1 < windows && target >= sh.window[which][warp][k]; k++) target -= sh.window[which][warp][k];
    const longlong2 u0 = mine[k * 64], u1 = mine[k * 64 + 1];
    int64_t w[VF_STEP] = {u0.x, u0.y, u1.x, u1.y};
    const int i = from + k * 128;
    if (which) {
        float p[VF_STEP] = {0.f, 0.f, 0.f, 0.f};
        if (q) load_step(q, i, end, a.vec_probs, 0.f, p);
#pragma unroll
        for (int e = 0; e < VF_STEP; e++) w[e] = left(i + e, w[e], p[e]);
    }
    const int64_t own = (w[0] + w[1]) + (w[2] + w[3]);
    int64_t upto = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, upto > target);
    if (past && lane == __ffs(past) - 1) {
        target -= upto - own;
        int e = 0;
        while (e < VF_STEP - 1 && target >= w[e]) target -= w[e++];
        tokens[row] = i + e;
    }
}

template <typename T>
int launch(const VfArgs &a, int n_seq, cudaStream_t st) {
    VfArgs b = a;
    const int smem = (b.slice + VF_WARPS * 128 - 1) / (VF_WARPS * 128) * (VF_WARPS * 128) * int(sizeof(int64_t));  // (whole windows)
    // (once a device, of the 64 that check_device knows)
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LL_ERR_CUDA;
    if (!(allowed.load(std::memory_order_acquire) >> dev & 1)) {
        if (cudaFuncSetAttribute(k_verify<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaFuncSetAttribute(k_verify<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, VF_MAX_VOCAB / VF_CLUSTER * int(sizeof(int64_t))) != cudaSuccess)
            return LL_ERR_CUDA;
        allowed.fetch_or(1ull << dev, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(n_seq) * VF_CLUSTER);
    cfg.blockDim = dim3(VF_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {VF_CLUSTER, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_verify<T>, b) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

}  // namespace
}  // namespace ll

extern "C" int ll_verify(const void *logits, int32_t type, int64_t logits_seq, int64_t logits_row, const int32_t *draft, const int32_t *n_draft_dev,
                         const float *probs, int64_t probs_seq, int64_t probs_row, const float *u, const float *temperature, int32_t n_seq,
                         int32_t n_draft, int32_t vocab, int32_t *tokens, int32_t *accepted, void *stream, char *err, size_t err_len) {
    using ll::report;
    if (err && err_len) err[0] = '\0';
    if (type != LL_BF16 && type != LL_F32) return report(err, err_len, LL_ERR_ARG, "type must be LL_BF16 or LL_F32");
    if (n_seq < 1 || n_seq > 65535) return report(err, err_len, LL_ERR_SHAPE, "n_seq must be 1 to 65535");
    if (n_draft < 0 || n_draft > 1 << 20) return report(err, err_len, LL_ERR_SHAPE, "n_draft must be 0 to 2^20");
    if (vocab < 1 || vocab > ll::VF_MAX_VOCAB) return report(err, err_len, LL_ERR_SHAPE, "vocab must be 1 to %d", ll::VF_MAX_VOCAB);
    const int size = type == LL_F32 ? 4 : 2;
    if (!logits || reinterpret_cast<uintptr_t>(logits) % size) return report(err, err_len, LL_ERR_ARG, "logits is NULL or not aligned to its type");
    if (n_draft && !draft) return report(err, err_len, LL_ERR_ARG, "draft is NULL");
    if (!u || !tokens || !accepted) return report(err, err_len, LL_ERR_ARG, "u, tokens or accepted is NULL");
    for (const void *p : {static_cast<const void *>(draft), static_cast<const void *>(n_draft_dev), static_cast<const void *>(probs),
                          static_cast<const void *>(u), static_cast<const void *>(temperature), static_cast<const void *>(tokens),
                          static_cast<const void *>(accepted)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return report(err, err_len, LL_ERR_ARG, "an array of 4-byte values is not 4-byte aligned");
    int nsm = 0;
    if (int rc = ll::check_device(nsm, err, err_len)) return rc;
    ll::VfArgs a = {};
    a.logits = logits;
    a.logits_seq = n_seq > 1 ? logits_seq : 0;
    a.logits_row = n_draft ? logits_row : 0;
    a.draft = draft;
    a.n_draft_dev = n_draft ? n_draft_dev : nullptr;
    a.probs = n_draft ? probs : nullptr;
    a.probs_seq = n_seq > 1 ? probs_seq : 0;
    a.probs_row = n_draft > 1 ? probs_row : 0;
    a.u = u;
    a.temperature = temperature;
    a.n_draft = n_draft;
    a.vocab = vocab;
    a.slice = ((vocab + ll::VF_CLUSTER - 1) / ll::VF_CLUSTER + ll::VF_STEP - 1) / ll::VF_STEP * ll::VF_STEP;
    const int step = ll::VF_STEP * size;
    a.vec = reinterpret_cast<uintptr_t>(logits) % step == 0 && (a.logits_seq * size) % step == 0 && (a.logits_row * size) % step == 0;
    while (a.log_rows < 3 && 1 << a.log_rows <= n_draft && n_seq * ll::VF_CLUSTER <= nsm) a.log_rows++;
    a.piece = a.log_rows ? 1024 : 512;
    a.vec_probs = reinterpret_cast<uintptr_t>(probs) % 16 == 0 && a.probs_seq % 4 == 0 && a.probs_row % 4 == 0;
    a.tokens = tokens;
    a.accepted = accepted;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return ll::finish(type == LL_F32 ? ll::launch<float>(a, n_seq, st) : ll::launch<__nv_bfloat16>(a, n_seq, st), err, err_len);
}

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
constexpr int VF_STEP = 4;               // neighbouring logits of a lane
constexpr int VF_MAX_VOCAB = 393216;     // a slice's weights (8 bytes each) fit in shared memory
constexpr double LN2 = 0.693147180559945309417232, LOG2E = 1.442695040888963407359925;

struct VfArgs {
    const void *logits;
    int64_t logits_seq, logits_row;
    const int32_t *draft, *n_draft_dev;
    const float *probs;
    int64_t probs_seq, probs_row;
    const float *u, *temperature;
    int32_t n_draft, vocab, slice;  // slice: a multiple of VF_STEP
    bool vec;                       // rows take whole-step loads
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

// 2^(j / 32), j < 32, by the series of e^(j ln 2 / 32).
__device__ Two root_of_two(int j) {
    constexpr float H = float(LN2 / 32), L = float(LN2 / 32 - double(H));
    const Two z = mul({float(j), 0.f}, {H, L});
    Two sum = {1.f, 0.f};
    for (int k = 24; k > 0; k--) {  // 1 + z / k (1 + z / (k + 1) (...)): z^24 / 24! is below 2^-90
        const float inv = 1.f / float(k);
        const Two t = mul(mul(z, sum), {inv, fmaf(-float(k), inv, 1.f) * inv});
        const Two s = two_sum(1.f, t.hi);
        sum = fast_two_sum(s.hi, s.lo + t.lo);
    }
    return sum;
}

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
__device__ __forceinline__ float weight(float l, float m, float c) { return l == m ? 1.f : exp2f((l - m) * c); }
__device__ __forceinline__ Stat join(Stat a, Stat b, float c) {
    if (b.m > a.m || (b.m == a.m && b.at < a.at)) {
        const Stat t = a;
        a = b;
        b = t;
    }
    if (b.m > -INFINITY) a.sum += b.sum * weight(b.m, a.m, c);
    return a;
}
__device__ __forceinline__ Stat warp_join(Stat a, float c) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const Stat b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.sum, o), __shfl_xor_sync(0xffffffffu, a.at, o)};
        a = join(a, b, c);
    }
    return a;
}

struct Shared {
    Stat warp_stat[VF_WARPS];
    Stat stats[2][VF_CLUSTER];      // of a row, by block (rows take turns)
    int64_t warp_sum[VF_WARPS];
    int64_t sums[2][VF_CLUSTER];    // of all weights, then of the residual's, by block
    float2 roots[32];
};

// Block b of a sequence's cluster has slice b of the vocabulary, and in step 2 a warp one run of it, so that sums over
// blocks and warps are sums over the vocabulary in order.
template <typename T>
__global__ void __launch_bounds__(VF_THREADS) k_verify(const VfArgs a) {
    extern __shared__ int64_t weights[];
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
    if (warp == 0) {
        const Two r = root_of_two(lane);
        sh.roots[lane] = make_float2(r.hi, r.lo);
    }
    const T *rows = static_cast<const T *>(a.logits) + s * a.logits_seq;

    int row = 0;
    Stat all;
    for (;; row++) {
        const T *l = rows + row * a.logits_row;
        Stat st = {-INFINITY, 0.f, 0x7fffffff};
        for (int i = first + VF_STEP * tid; i < end; i += VF_STEP * VF_THREADS) {
            float x[VF_STEP];
            load_step(l, i, end, a.vec, -INFINITY, x);
#pragma unroll
            for (int e = 0; e < VF_STEP; e++) {
                x[e] = logit(x[e]);
                if (x[e] > st.m) {
                    st.sum *= exp2f((st.m - x[e]) * c.hi);
                    st.m = x[e];
                    st.at = i + e;
                }
            }
            if (st.m > -INFINITY)
#pragma unroll
                for (int e = 0; e < VF_STEP; e++) st.sum += weight(x[e], st.m, c.hi);
        }
        st = warp_join(st, c.hi);
        if (lane == 0) sh.warp_stat[warp] = st;
        __syncthreads();
        if (row == 0) cluster.barrier_wait(std::move(begun));
        if (warp == 0) {
            st = lane < VF_WARPS ? sh.warp_stat[lane] : Stat{-INFINITY, 0.f, 0x7fffffff};
            st = warp_join(st, c.hi);
            if (lane < blocks) cluster.map_shared_rank(&sh, lane)->stats[row & 1][rank] = st;
        }
        cluster.sync();
        all = lane < blocks ? sh.stats[row & 1][lane] : Stat{-INFINITY, 0.f, 0x7fffffff};
        all = warp_join(all, c.hi);
        if (row >= n || !(all.m > -INFINITY)) break;
        const int x = a.draft[int64_t(s) * D + row];
        bool ok = false;
        if (greedy) {
            ok = x == all.at;
        } else if (x >= 0 && x < V) {
            const float q = a.probs ? a.probs[s * a.probs_seq + row * a.probs_row + x] : 1.f;
            const Two e = exp_two(logit(float(l[x])), all.m, c, sh.roots);
            ok = double(a.u[int64_t(s) * (D + 1) + row]) * double(q) * double(all.sum) < double(e.hi) + double(e.lo);
        }
        if (!ok) break;
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

    const T *l = rows + row * a.logits_row;
    const bool residual = row < n;
    const float *q = residual && a.probs ? a.probs + s * a.probs_seq + row * a.probs_row : nullptr;
    const int draft = residual ? a.draft[int64_t(s) * D + row] : -1;
    // a warp's run of the slice, in windows of 32 steps
    const int run = ((a.slice + VF_WARPS - 1) / VF_WARPS + 32 * VF_STEP - 1) / (32 * VF_STEP) * (32 * VF_STEP);
    const int from = min(end, first + warp * run), to = min(end, from + run);
    int64_t sum = 0;
    for (int i = from + VF_STEP * lane; i < to; i += 32 * VF_STEP) {
        float x[VF_STEP];
        load_step(l, i, end, a.vec, -INFINITY, x);
#pragma unroll
        for (int e = 0; e < VF_STEP; e++) {
            const int64_t w = i + e < to ? fixed(exp_two(logit(x[e]), all.m, c, sh.roots)) : 0;
            if (i + e < to) weights[i + e - first] = w;
            sum += w;
        }
    }
    // sums of the warps, then of the blocks, for everyone
    auto total_of = [&](int64_t v, int which) {
#pragma unroll
        for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncthreads();
        if (lane == 0) sh.warp_sum[warp] = v;
        __syncthreads();
        if (warp == 0) {
            int64_t t = lane < VF_WARPS ? sh.warp_sum[lane] : 0;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane < blocks) cluster.map_shared_rank(&sh, lane)->sums[which][rank] = t;
        }
        cluster.sync();
        int64_t t = 0;
        for (int b = 0; b < blocks; b++) t += sh.sums[which][b];
        return t;
    };
    int64_t total = total_of(sum, 0);
    int which = 0;
    const double z = double(total) * 0x1p-43;
    const Two Z = {float(z), float(z - double(float(z)))};
    // the residual's weight of a place
    auto left = [&](int i, int64_t w) -> int64_t {
        if (!q) return i == draft ? 0 : w;
        const float p = q[i], h = __fmul_rn(p, Z.hi);
        if (!(h < 1.5f)) return h >= 1.5f ? 0 : w;  // (a NaN takes nothing away)
        const int64_t d = w - (h > 0.f ? fixed({h, fmaf(p, Z.hi, -h) + p * Z.lo}) : 0);
        return d > 0 ? d : 0;
    };
    bool reduced = false;
    if (residual) {
        sum = 0;
        for (int i = from + lane; i < to; i += 32) sum += left(i, weights[i - first]);
        const int64_t own = sh.warp_sum[warp];
        const int64_t t = total_of(sum, 1);
        if (t > 0) {
            total = t;
            which = 1;
            reduced = true;
        } else {  // nothing left: p itself, whose warps' sums come back
            __syncthreads();
            if (lane == 0) sh.warp_sum[warp] = own;
            __syncthreads();
        }
    }
    int64_t target = int64_t(double(a.u[int64_t(s) * (D + 1) + D]) * double(total));
    target = max(int64_t(0), min(target, total - 1));
    for (int b = 0; b < rank; b++) target -= sh.sums[which][b];
    if (target < 0 || target >= sh.sums[which][rank]) return;
    for (int w = 0; w < warp; w++) target -= sh.warp_sum[w];
    if (target < 0 || target >= sh.warp_sum[warp]) return;
    for (int base = from; base < to; base += 32) {
        const int i = base + lane;
        int64_t w = i < to ? weights[i - first] : 0;
        if (reduced && i < to) w = left(i, w);
        int64_t upto = w;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, upto > target);
        if (past) {
            if (lane == __ffs(past) - 1) tokens[row] = i;
            return;
        }
        target -= __shfl_sync(0xffffffffu, upto, 31);
    }
}

template <typename T>
int launch(const VfArgs &a, int n_seq, cudaStream_t st) {
    VfArgs b = a;
    const int smem = b.slice * int(sizeof(int64_t));
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
    a.tokens = tokens;
    a.accepted = accepted;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return ll::finish(type == LL_F32 ? ll::launch<float>(a, n_seq, st) : ll::launch<__nv_bfloat16>(a, n_seq, st), err, err_len);
}

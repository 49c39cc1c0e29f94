// kvq.cu -- the packed KV cache: writing rows (quantising K and V as they come),
// reading them back as bf16, and the C entries of the packed-cache calls. The
// format stands in include/ll.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "call.h"
#include "kvq.cuh"
#include "kvq.h"
#include "ll_internal.h"

namespace ll {
namespace {

constexpr int RW_THREADS = 256;
// Values are held within +-BOUND: far enough below fp16's largest (65504) that lo +
// step * code stays finite after lo (by 16 at most), step (by 4, or 0.25 in 8 bits,
// 15 or 255 times) and the sum are rounded.
constexpr float BOUND = 60000.f;

// r / d for r < 2^31 by one wide product: m = floor(2^(31 + l) / d) + 1 with l =
// ceil(log2 d), so that m d exceeds 2^(31 + l) by at most d <= 2^l.
struct FastDiv {
    uint32_t m, shift, d;
    explicit FastDiv(uint32_t div = 1) : d(div) {
        uint32_t l = 0;
        while ((1ull << l) < div) l++;
        m = uint32_t((1ull << (31 + l)) / div + 1);
        shift = 31 + l;
    }
    __device__ __forceinline__ uint32_t div(uint32_t r) const { return uint32_t((uint64_t(r) * m) >> shift); }
};

struct RwArgs {
    ll_kvq_rows rows[2];   // K, V
    uint8_t *codes[2];
    uint32_t *params[2];   // (lo, step) as fp16 pairs
    int64_t seq_rows;
    int32_t max_seq, nkv, n_rows;  // n_rows = n_tok * nkv
    FastDiv heads;  // nkv
    KvqLens l;
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A thread's 8 values of a row, as they are stored.
__device__ __forceinline__ void load8(const float *p, uint32_t (&w)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *reinterpret_cast<const uint4 *>(p + 4);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, uint32_t (&w)[4]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
}
__device__ __forceinline__ void widen8(const uint32_t (&w)[8], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void widen8(const uint32_t (&w)[4], float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

// Smallest and largest of values as (min, -max), so that one kind of minimum joins
// ranges; NaN if any value is. bf16: both in a word.
struct Range32 {
    float mn, neg_mx;
};
__device__ __forceinline__ Range32 join(Range32 a, Range32 b) { return {min_nan(a.mn, b.mn), min_nan(a.neg_mx, b.neg_mx)}; }
__device__ __forceinline__ Range32 from_lane(Range32 a, int o) {
    return {__shfl_xor_sync(0xffffffffu, a.mn, o), __shfl_xor_sync(0xffffffffu, a.neg_mx, o)};
}
__device__ __forceinline__ float2 ends(Range32 a) { return make_float2(a.mn, -a.neg_mx); }
__device__ __forceinline__ Range32 range8(const uint32_t (&w)[8]) {
    float mn = __uint_as_float(w[0]), mx = mn;
#pragma unroll
    for (int i = 1; i < 8; i++) {
        mn = min_nan(mn, __uint_as_float(w[i]));
        mx = max_nan(mx, __uint_as_float(w[i]));
    }
    return {mn, -mx};
}
struct Range16 {
    uint32_t v;
};
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ Range16 join(Range16 a, Range16 b) { return {min2_nan(a.v, b.v)}; }
__device__ __forceinline__ Range16 from_lane(Range16 a, int o) { return {__shfl_xor_sync(0xffffffffu, a.v, o)}; }
__device__ __forceinline__ float2 ends(Range16 a) { return make_float2(__uint_as_float(a.v << 16), -__uint_as_float(a.v & 0xffff0000u)); }
__device__ __forceinline__ Range16 range8(const uint32_t (&w)[4]) {
    const uint32_t lo = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3]));
    const uint32_t hi = max2_nan(max2_nan(w[0], w[1]), max2_nan(w[2], w[3])) ^ 0x80008000u;
    return {min2_nan(kvq_prmt(lo, hi, 0x5410), kvq_prmt(lo, hi, 0x7632))};
}
// The ranges of U rows over the four lanes of a group (lane a of them): of row a % U.
// Lanes that differ in a bit hand each other the rows that are not theirs.
template <typename R>
__device__ __forceinline__ R group_range(const R (&r)[4], int a) {
    const R x = join(a & 1 ? r[1] : r[0], from_lane(a & 1 ? r[0] : r[1], 1));
    const R y = join(a & 1 ? r[3] : r[2], from_lane(a & 1 ? r[2] : r[3], 1));
    return join(a & 2 ? y : x, from_lane(a & 2 ? x : y, 2));
}
template <typename R>
__device__ __forceinline__ R group_range(const R (&r)[2], int a) {
    const R x = join(a & 1 ? r[1] : r[0], from_lane(a & 1 ? r[0] : r[1], 1));
    return join(x, from_lane(x, 2));
}

// The integer n nearest to each t / step, t = x[i] - lo in fp32, ties to even, within
// [0, TOP], as the bits of 1.5 * 2^23 + n (whose lowest 16 are n).
//
// It is the rounded quotient rounded again: a border b between two integers has 9 bits
// and step 11, so b step is an fp32 number, and a t that is not b step differs from it by
// so much that the quotient misses b by more than half of b's last place (times 1 +
// 2^-11 or more): rounding to fp32 cannot take it onto or past the border. The
// quotient is t inv, corrected once by its residue times inv (Markstein), with inv
// within 2^-22 of 1 / step: then it is off by 2^-43 of itself before its rounding, which
// is within that margin. inside: no t is so far outside that n might be outside [0, TOP].
//
// (16 layers of 32768 positions, 8 heads of 64 dims, written in 4 bits and read again: 1,257
// us with an IEEE division for every value; 534 with the product t inv rounded to an integer and
// compared with half a step, whose comparisons kept the ALU pipe busy; 518 this way.)
template <int TOP>
__device__ __forceinline__ void nearest8(float (&x)[8], float lo, float step, float inv, bool inside, uint32_t (&n)[8]) {
    constexpr float MAGIC = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    if (!inside) {  // (finite, so that the quotients are)
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = fminf(fmaxf(x[i], -BOUND), BOUND);
    }
    const uint64_t magic = kvq_pair(MAGIC, MAGIC), l = kvq_pair(-lo, -lo), inv2 = kvq_pair(inv, inv), step2 = kvq_pair(-step, -step);
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t t = kvq_add2(kvq_pair(x[i], x[i + 1]), l), q = kvq_mul2(t, inv2);
        kvq_split(kvq_add2(kvq_fma2(kvq_fma2(q, step2, t), inv2, q), magic), m[i], m[i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) n[i] = __float_as_uint(inside ? m[i] : fminf(fmaxf(m[i], MAGIC), MAGIC + float(TOP)));
}

// Where a thread's rows are. FAR (many tokens): a block takes one head, K or V, and
// neighbouring rows are neighbouring positions (the packed rows of a head are one
// run). Otherwise the heads of a token are neighbours.
__host__ __device__ constexpr int rw_rows(bool far) { return far ? 4 : 2; }  // rows a thread has in flight

template <bool FAR, int RPB, int U>
struct RowWalk {
    int kv;
    uint32_t valid = 0;    // bit u: there is something to do
    int64_t row[U], at[U]; // row in the cache, and the token's row in the call's tensor
    __device__ __forceinline__ RowWalk(const RwArgs &a, int s, int row0) {
        const int n = a.l.n(s), first = a.l.len(s) - n;
        if (FAR) {  // neighbouring rows in both: one address each, and steps from it
            kv = blockIdx.y & 1;
            const int h = blockIdx.y >> 1, j = blockIdx.x * (RPB * U) + row0;
            const ll_kvq_rows &t = a.rows[kv];
            row[0] = s * a.seq_rows + int64_t(h) * a.max_seq + first + j;
            at[0] = s * t.seq + h * t.head + j * t.token;
#pragma unroll
            for (int u = 0; u < U; u++) {
                row[u] = row[0] + u * RPB;
                at[u] = at[0] + u * (RPB * t.token);
                // (j < n, and the position first + j in [0, max_seq))
                if (j + u * RPB < n && uint32_t(first + j + u * RPB) < uint32_t(a.max_seq)) valid |= 1u << u;
            }
        } else {
            kv = blockIdx.y;
            const ll_kvq_rows &t = a.rows[kv];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int r = blockIdx.x * (RPB * U) + row0 + u * RPB;
                const int j = int(a.heads.div(uint32_t(min(r, a.n_rows)))), h = min(r, a.n_rows) - j * a.nkv;
                row[u] = s * a.seq_rows + int64_t(h) * a.max_seq + first + j;
                at[u] = s * t.seq + h * t.head + j * t.token;
                if (r < a.n_rows && j < n && uint32_t(first + j) < uint32_t(a.max_seq)) valid |= 1u << u;
            }
        }
    }
    __device__ __forceinline__ bool has(int u) const { return valid >> u & 1; }
    __device__ __forceinline__ int64_t row_of(int u) const {  // (u not a constant)
        if (FAR) return row[0] + u * RPB;
        int64_t r = row[0];
#pragma unroll
        for (int i = 1; i < U; i++)
            if (u == i) r = row[i];
        return r;
    }
};

// Lanes of a row: lane e takes dims 8 e .. 8 e + 7, which is cells g = 2 a and 2 a
// + 1 (a = e % 4) of group gr = e / 4; the four lanes of a group share its min
// and max by shuffles. Cells of one g and neighbouring groups are neighbours in
// the row, so lanes e and e ^ 4 exchange a cell and each stores a whole word (two
// cells): the row leaves the warp as one run of bytes.
//
// What bounds it: from bf16 the instructions, from fp32 the memory. 4 layers of 32768 positions, 8
// heads of 64 dims to 4 bits: 79 us from bf16 (352 MB, 66 % of the copy rate), 97 us from fp32
// (621 MB, 95 %); one token: 3 us, a launch.
template <typename T, int BITS, int HD, bool FAR>
__global__ void __launch_bounds__(RW_THREADS) k_kvq_write(const __grid_constant__ RwArgs a) {
    constexpr int LPR = HD / 8, GR = HD / 32, RPB = RW_THREADS / LPR, U = rw_rows(FAR);
    const int s = blockIdx.z, e = threadIdx.x % LPR, gr = e / 4, ga = e % 4;
    const RowWalk<FAR, RPB, U> w(a, s, threadIdx.x / LPR);
    uint32_t raw[U][2 * sizeof(T)];
    const T *src = static_cast<const T *>(a.rows[w.kv].data) + 8 * e;
#pragma unroll
    for (int u = 0; u < U; u++) {
        if (w.has(u)) {
            load8(src + w.at[u], raw[u]);
        } else {
#pragma unroll
            for (int i = 0; i < int(2 * sizeof(T)); i++) raw[u][i] = 0;
        }
    }
    // lo and step of a group's rows, a row to a lane (all four lanes computing every row's: 518 us where this is
    // 494); handed round as one word, whose top bit (step is not negative) says that a value lies far outside
    // of lo .. lo + TOP step
    constexpr int TOP = (1 << BITS) - 1;
    decltype(range8(raw[0])) ranges[U];
#pragma unroll
    for (int u = 0; u < U; u++) ranges[u] = range8(raw[u]);
    uint32_t par;
    {
        const int mine = ga % U;
        const float2 e2 = ends(group_range(ranges, ga));
        // (values past the bound need no clamp of their own: their codes are clamped)
        const float low = min_nan(max_nan(e2.x, -BOUND), BOUND), high = min_nan(max_nan(e2.y, -BOUND), BOUND);
        const __half lo = __float2half_rn(low);
        const float lof = __half2float(lo), d = __fsub_rn(high, lof);
        constexpr float R = 1.f / float(TOP);
        const __half step = __float2half_rn(max_nan(__fmul_rn(d, R), 0.f));
        const float stf = __half2float(step);
        const bool inside = e2.x - lof > -0.25f * stf && e2.y - lof < (float(TOP) + 0.25f) * stf;
        par = uint32_t(__half_as_ushort(lo)) | uint32_t(__half_as_ushort(step)) << 16;
        if (ga < U && (w.valid >> mine & 1)) a.params[w.kv][w.row_of(mine) * GR + gr] = par;
        par = (par & 0x7fffffffu) | (inside ? 0u : 0x80000000u);
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        float x[8];
        widen8(raw[u], x);
        const uint32_t p = __shfl_sync(0xffffffffu, par, (threadIdx.x & 28) + u);
        const float lof = __half2float(__ushort_as_half(uint16_t(p))), stf = __half2float(__ushort_as_half(uint16_t(p >> 16 & 0x7fffu)));
        const bool inside = int32_t(p) >= 0;
        uint32_t c[2] = {0, 0};  // cells 2 ga, 2 ga + 1
        if (stf > 0.f) {
            float inv;
            uint32_t q[8];
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(stf));
            nearest8<TOP>(x, lof, stf, inv, inside, q);
            // the codes of a cell as one number (two, in 8 bits), the low 16 bits of a sum: those of 1.5 * 2^23 are zero
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t *v = q + 4 * i;
                if (BITS == 4)
                    c[i] = ((v[3] * 16 + v[2]) * 16 + v[1]) * 16 + v[0];
                else
                    c[i] = kvq_prmt(v[1] * 256 + v[0], v[3] * 256 + v[2], 0x5410);
            }
        }
        const uint32_t got = __shfl_xor_sync(0xffffffffu, gr & 1 ? c[0] : c[1], 4);
        if (!w.has(u)) continue;
        const int64_t row = w.row[u];
        const int word = (2 * ga + (gr & 1)) * (GR / 2) + gr / 2;
        const uint32_t first = gr & 1 ? got : c[0], second = gr & 1 ? c[1] : got;  // groups gr & ~1, gr | 1
        if (BITS == 4)
            reinterpret_cast<uint32_t *>(a.codes[w.kv])[row * (HD / 8) + word] = kvq_prmt(first, second, 0x5410);
        else
            reinterpret_cast<uint2 *>(a.codes[w.kv])[row * (HD / 8) + word] = make_uint2(first, second);
    }
}

// The same walk backwards: each lane loads a word (two cells), exchanges one with
// its partner and stores 8 dims as bf16. Bound by the memory: the cache of the write
// above in 58 us, 89 % of the copy rate (rows of 128 dims: 96 %).
template <int BITS, int HD, bool FAR>
__global__ void __launch_bounds__(RW_THREADS) k_kvq_read(const __grid_constant__ RwArgs a) {
    constexpr int LPR = HD / 8, GR = HD / 32, RPB = RW_THREADS / LPR, U = rw_rows(FAR);
    const int s = blockIdx.z, e = threadIdx.x % LPR, gr = e / 4, ga = e % 4;
    const RowWalk<FAR, RPB, U> at(a, s, threadIdx.x / LPR);
    const KvqConsts consts;
    const int word = (2 * ga + (gr & 1)) * (GR / 2) + gr / 2;
    uint2 w[U];
    uint32_t par[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        w[u] = make_uint2(0, 0);
        par[u] = 0;
        if (at.has(u)) {
            const int64_t row = at.row[u];
            if (BITS == 4)
                w[u].x = reinterpret_cast<const uint32_t *>(a.codes[at.kv])[row * (HD / 8) + word];
            else
                w[u] = reinterpret_cast<const uint2 *>(a.codes[at.kv])[row * (HD / 8) + word];
            par[u] = a.params[at.kv][row * GR + gr];
        }
    }
    __nv_bfloat16 *const dst = static_cast<__nv_bfloat16 *>(a.rows[at.kv].data) + 8 * e;
#pragma unroll
    for (int u = 0; u < U; u++) {
        // the word is cell (2 ga + gr % 2) of groups gr & ~1 (first) and gr | 1: keep
        // this lane's group, hand the partner its own; v = pairs (dim i, dim 4 + i)
        __half2 v[4];
        if (BITS == 4) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, w[u].x, 4);
            kvq_codes4(gr & 1 ? kvq_prmt(got, w[u].x, 0x7632) : kvq_prmt(w[u].x, got, 0x5410), consts, v);
        } else {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, gr & 1 ? w[u].x : w[u].y, 4);
            kvq_codes8(gr & 1 ? got : w[u].x, gr & 1 ? w[u].y : got, consts, v);
        }
        if (!at.has(u)) continue;
        const __half2 lo = kvq_h2(kvq_prmt(par[u], 0, 0x1010)), st = kvq_h2(kvq_prmt(par[u], 0, 0x3232));
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = __half22float2(__hfma2(st, v[i], lo));
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(f[2 * i].x, f[2 * i + 1].x);
            const __nv_bfloat162 b1 = __floats2bfloat162_rn(f[2 * i].y, f[2 * i + 1].y);
            o[i] = *reinterpret_cast<const uint32_t *>(&b0);
            o[2 + i] = *reinterpret_cast<const uint32_t *>(&b1);
        }
        *reinterpret_cast<uint4 *>(dst + at.at[u]) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

RwArgs rw_args(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, const KvqLens &l) {
    RwArgs a;
    a.rows[0] = k;
    a.rows[1] = v;
    a.codes[0] = c.k_codes;
    a.codes[1] = c.v_codes;
    a.params[0] = reinterpret_cast<uint32_t *>(c.k_params);
    a.params[1] = reinterpret_cast<uint32_t *>(c.v_params);
    a.seq_rows = c.seq_rows;
    a.max_seq = c.max_seq;
    a.nkv = c.n_kv_heads;
    a.n_rows = l.n_tok * c.n_kv_heads;
    a.heads = FastDiv(uint32_t(c.n_kv_heads));
    a.l = l;
    return a;
}

// The walk by whole heads pays once a head's tokens fill a block's rows.
bool rw_far(const ll_kvq_cache &c, const KvqLens &l) { return l.n_tok >= RW_THREADS / (c.head_dim / 8); }

dim3 rw_grid(const ll_kvq_cache &c, const KvqLens &l, bool far) {
    const int rows = far ? l.n_tok : l.n_tok * c.n_kv_heads, per_block = RW_THREADS / (c.head_dim / 8) * rw_rows(far);
    return dim3((rows + per_block - 1) / per_block, far ? 2 * c.n_kv_heads : 2, c.n_seq);
}

}  // namespace

int launch_kvq_write(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, int type, const KvqLens &l,
                     cudaStream_t st) {
    const RwArgs a = rw_args(c, k, v, l);
    const bool far = rw_far(c, l);
    const dim3 g = rw_grid(c, l, far);
    kvq_dispatch(c, [&](auto bits, auto hd) {
        constexpr int B = bits.value, H = hd.value;
        if (type == LL_F32)
            far ? k_kvq_write<float, B, H, true><<<g, RW_THREADS, 0, st>>>(a)
                : k_kvq_write<float, B, H, false><<<g, RW_THREADS, 0, st>>>(a);
        else
            far ? k_kvq_write<__nv_bfloat16, B, H, true><<<g, RW_THREADS, 0, st>>>(a)
                : k_kvq_write<__nv_bfloat16, B, H, false><<<g, RW_THREADS, 0, st>>>(a);
    });
    return launched();
}

int launch_kvq_read(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, const KvqLens &l, cudaStream_t st) {
    const RwArgs a = rw_args(c, k, v, l);
    const bool far = rw_far(c, l);
    const dim3 g = rw_grid(c, l, far);
    kvq_dispatch(c, [&](auto bits, auto hd) {
        constexpr int B = bits.value, H = hd.value;
        far ? k_kvq_read<B, H, true><<<g, RW_THREADS, 0, st>>>(a) : k_kvq_read<B, H, false><<<g, RW_THREADS, 0, st>>>(a);
    });
    return launched();
}

int kvq_check_cache(const ll_kvq_cache *c, const char *&msg) {
    auto bad = [&](int code, const char *why) {
        msg = why;
        return code;
    };
    if (!c) return bad(LL_ERR_ARG, "the packed cache is NULL");
    if (c->bits != 4 && c->bits != 8) return bad(LL_ERR_SHAPE, "bits must be 4 or 8");
    if (c->head_dim != 64 && c->head_dim != 128) return bad(LL_ERR_SHAPE, "head_dim must be 64 or 128");
    if (c->n_seq < 1 || c->n_seq > 65535) return bad(LL_ERR_SHAPE, "n_seq must be 1 to 65535");
    if (c->n_kv_heads < 1 || c->n_kv_heads > 32767) return bad(LL_ERR_SHAPE, "n_kv_heads must be 1 to 32767");
    if (c->max_seq < 1 || c->max_seq > 1 << 30) return bad(LL_ERR_SHAPE, "max_seq must be 1 to 2^30");
    if (c->n_seq > 1 && c->seq_rows < int64_t(c->n_kv_heads) * c->max_seq)
        return bad(LL_ERR_ARG, "seq_rows is less than n_kv_heads * max_seq");
    const void *p[4] = {c->k_codes, c->v_codes, c->k_params, c->v_params};
    for (const void *q : p)
        if (!q || (reinterpret_cast<uintptr_t>(q) & 15u)) return bad(LL_ERR_ARG, "a packed cache array is NULL or not 16-byte aligned");
    return LL_OK;
}

}  // namespace ll

namespace {

using ll::check_device;
using ll::check_rows;
using ll::finish;
using ll::report;

int check_call(const ll_kvq_cache *c, int32_t n_tok, const int32_t *len_dev, const int32_t *n_tok_dev, int64_t heads, char *err,
               size_t err_len) {
    if (err && err_len) err[0] = '\0';
    const char *msg = "";
    if (const int rc = ll::kvq_check_cache(c, msg)) return report(err, err_len, rc, "%s", msg);
    if (n_tok < 1) return report(err, err_len, LL_ERR_ARG, "n_tok must be at least 1");
    if (int64_t(n_tok) * heads >= int64_t(1) << 30) return report(err, err_len, LL_ERR_SHAPE, "n_tok * heads must be below 2^30");
    if (!len_dev) return report(err, err_len, LL_ERR_ARG, "len_dev is NULL");
    if ((reinterpret_cast<uintptr_t>(len_dev) & 3u) || (reinterpret_cast<uintptr_t>(n_tok_dev) & 3u))
        return report(err, err_len, LL_ERR_ARG, "len_dev or n_tok_dev is not 4-byte aligned");
    return LL_OK;
}

}  // namespace

extern "C" {

int ll_kvq_write(const ll_kvq_cache *c, const ll_kvq_rows *k, const ll_kvq_rows *v, int32_t type, int32_t n_tok,
                 const int32_t *len_dev, const int32_t *n_tok_dev, void *stream, char *err, size_t err_len) {
    if (int rc = check_call(c, n_tok, len_dev, n_tok_dev, c ? c->n_kv_heads : 1, err, err_len)) return rc;
    if (type != LL_BF16 && type != LL_F32) return report(err, err_len, LL_ERR_ARG, "type must be LL_BF16 or LL_F32");
    const int size = type == LL_F32 ? 4 : 2;
    if (int rc = check_rows(k, "k", c->n_seq, n_tok, c->n_kv_heads, size, false, err, err_len)) return rc;
    if (int rc = check_rows(v, "v", c->n_seq, n_tok, c->n_kv_heads, size, false, err, err_len)) return rc;
    int nsm = 0;
    if (int rc = check_device(nsm, err, err_len)) return rc;
    const ll::KvqLens l = {len_dev, n_tok_dev, 0, n_tok};
    return finish(ll::launch_kvq_write(*c, *k, *v, type, l, static_cast<cudaStream_t>(stream)), err, err_len);
}

int ll_kvq_read(const ll_kvq_cache *c, const ll_kvq_rows *k, const ll_kvq_rows *v, int32_t n_tok, const int32_t *len_dev,
                const int32_t *n_tok_dev, void *stream, char *err, size_t err_len) {
    if (int rc = check_call(c, n_tok, len_dev, n_tok_dev, c ? c->n_kv_heads : 1, err, err_len)) return rc;
    if (int rc = check_rows(k, "k", c->n_seq, n_tok, c->n_kv_heads, 2, true, err, err_len)) return rc;
    if (int rc = check_rows(v, "v", c->n_seq, n_tok, c->n_kv_heads, 2, true, err, err_len)) return rc;
    int nsm = 0;
    if (int rc = check_device(nsm, err, err_len)) return rc;
    const ll::KvqLens l = {len_dev, n_tok_dev, 0, n_tok};
    return finish(ll::launch_kvq_read(*c, *k, *v, l, static_cast<cudaStream_t>(stream)), err, err_len);
}

int ll_kvq_attention(const ll_kvq_cache *c, const ll_kvq_rows *q, int32_t n_q_heads, int32_t n_tok, const int32_t *len_dev,
                     const int32_t *n_tok_dev, int32_t max_len, float scale, const ll_kvq_rows *out, void *stream, char *err,
                     size_t err_len) {
    if (int rc = check_call(c, n_tok, len_dev, n_tok_dev, n_q_heads > 0 ? n_q_heads : 1, err, err_len)) return rc;
    if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || n_q_heads / c->n_kv_heads > ll::MAX_GQA)
        return report(err, err_len, LL_ERR_SHAPE, "n_q_heads must be a multiple (at most 8x) of n_kv_heads");
    if (!(scale >= 0.f) || !isfinite(scale)) return report(err, err_len, LL_ERR_ARG, "scale must be finite and not negative");
    if (max_len < 0) return report(err, err_len, LL_ERR_ARG, "max_len must not be negative");
    if (int rc = check_rows(q, "q", c->n_seq, n_tok, n_q_heads, 2, false, err, err_len)) return rc;
    if (int rc = check_rows(out, "out", c->n_seq, n_tok, n_q_heads, 2, true, err, err_len)) return rc;
    int nsm = 0;
    if (int rc = check_device(nsm, err, err_len)) return rc;
    const ll::KvqLens l = {len_dev, n_tok_dev, 0, n_tok};
    ll::KvqOut o = {};
    o.t[0] = static_cast<uint16_t *>(out->data);
    o.seq = out->seq;
    o.token = out->token;
    o.head = out->head;
    return finish(ll::launch_kvq_attention(*c, *q, LL_BF16, n_q_heads, l, max_len, scale, o, {}, nsm,
                                           static_cast<cudaStream_t>(stream)),
                  err, err_len);
}

}  // extern "C"

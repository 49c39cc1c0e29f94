// kvq.cu -- the packed KV cache: writing rows (quantising K and V as they come),
// reading them back as bf16, and the C entries of the packed-cache calls. The
// format stands in include/ll.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <mutex>

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
    int32_t token_fast;    // row index r: 1 = head * n_tok + token, 0 = token * nkv + head
    FastDiv inner;         // n_tok or nkv
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

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

// A thread's row of the call: token and head of row number r, and its position,
// or -1 where there is nothing to do.
__device__ __forceinline__ int row_of(const RwArgs &a, int r, int n, int len, int &j, int &h) {
    if (r >= a.n_rows) return -1;
    const int o = int(a.inner.div(uint32_t(r))), i = r - o * int(a.inner.d);
    j = a.token_fast ? i : o;
    h = a.token_fast ? o : i;
    const int pos = len - n + j;
    return j < n && pos >= 0 && pos < a.max_seq ? pos : -1;
}

// Lanes of a row: lane e takes dims 8 e .. 8 e + 7, which is cells g = 2 a and 2 a
// + 1 (a = e % 4) of group gr = e / 4; the four lanes of a group share its min
// and max by shuffles. Cells of one g and neighbouring groups are neighbours in
// the row, so lanes e and e ^ 4 exchange a cell and each stores a whole word (two
// cells): the row leaves the warp as one run of bytes.
template <typename T, int BITS, int HD>
__global__ void __launch_bounds__(RW_THREADS) k_kvq_write(const __grid_constant__ RwArgs a) {
    constexpr int LPR = HD / 8, GR = HD / 32, RPB = RW_THREADS / LPR, U = 2;
    const int s = blockIdx.z, kv = blockIdx.y, e = threadIdx.x % LPR, gr = e / 4, ga = e % 4;
    const int n = a.l.n(s), len = a.l.len(s);
    const ll_kvq_rows &in = a.rows[kv];
    const int r0 = blockIdx.x * (RPB * U) + threadIdx.x / LPR;
    float x[U][8];
    int pos[U], h[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        int j = 0;
        h[u] = 0;
        pos[u] = row_of(a, r0 + u * RPB, n, len, j, h[u]);
        if (pos[u] >= 0) {
            load8(static_cast<const T *>(in.data) + s * in.seq + j * in.token + h[u] * in.head + 8 * e, x[u]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) x[u][i] = 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        float mn = x[u][0], mx = x[u][0];
#pragma unroll
        for (int i = 1; i < 8; i++) {
            mn = min_nan(mn, x[u][i]);
            mx = max_nan(mx, x[u][i]);
        }
#pragma unroll
        for (int o = 1; o <= 2; o *= 2) {
            mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        // (values past the bound need no clamp of their own: their codes are clamped)
        mn = min_nan(max_nan(mn, -BOUND), BOUND);
        mx = min_nan(max_nan(mx, -BOUND), BOUND);
        constexpr float TOP = float((1 << BITS) - 1);
        const __half lo = __float2half_rn(mn);
        const float lof = __half2float(lo);
        const __half step = __float2half_rn(max_nan(__fdiv_rn(mx - lof, TOP), 0.f));
        const float stf = __half2float(step);
        uint32_t c[2] = {0, 0};  // cells 2 ga, 2 ga + 1
        if (stf > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float q = fminf(fmaxf(rintf(__fdiv_rn(x[u][i] - lof, stf)), 0.f), TOP);
                c[i / 4] |= uint32_t(int(q)) << (BITS * (i % 4));
            }
        }
        const uint32_t got = __shfl_xor_sync(0xffffffffu, gr & 1 ? c[0] : c[1], 4);
        if (pos[u] < 0) continue;
        const int64_t row = s * a.seq_rows + int64_t(h[u]) * a.max_seq + pos[u];
        const int word = (2 * ga + (gr & 1)) * (GR / 2) + gr / 2;
        const uint32_t first = gr & 1 ? got : c[0], second = gr & 1 ? c[1] : got;  // groups gr & ~1, gr | 1
        if (BITS == 4)
            reinterpret_cast<uint32_t *>(a.codes[kv])[row * (HD / 8) + word] = first | second << 16;
        else
            reinterpret_cast<uint2 *>(a.codes[kv])[row * (HD / 8) + word] = make_uint2(first, second);
        if (ga == 0)
            a.params[kv][row * GR + gr] = uint32_t(__half_as_ushort(lo)) | uint32_t(__half_as_ushort(step)) << 16;
    }
}

// The same walk backwards: each lane loads a word (two cells), exchanges one with
// its partner and stores 8 dims as bf16.
template <int BITS, int HD>
__global__ void __launch_bounds__(RW_THREADS) k_kvq_read(const __grid_constant__ RwArgs a) {
    constexpr int LPR = HD / 8, GR = HD / 32, RPB = RW_THREADS / LPR, U = 2;
    const int s = blockIdx.z, kv = blockIdx.y, e = threadIdx.x % LPR, gr = e / 4, ga = e % 4;
    const int n = a.l.n(s), len = a.l.len(s);
    const ll_kvq_rows &out = a.rows[kv];
    const int r0 = blockIdx.x * (RPB * U) + threadIdx.x / LPR;
    const int word = (2 * ga + (gr & 1)) * (GR / 2) + gr / 2;
    uint2 w[U];
    uint32_t par[U];
    int pos[U], h[U], j[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        j[u] = h[u] = 0;
        pos[u] = row_of(a, r0 + u * RPB, n, len, j[u], h[u]);
        w[u] = make_uint2(0, 0);
        par[u] = 0;
        if (pos[u] >= 0) {
            const int64_t row = s * a.seq_rows + int64_t(h[u]) * a.max_seq + pos[u];
            if (BITS == 4) {
                const uint32_t v = reinterpret_cast<const uint32_t *>(a.codes[kv])[row * (HD / 8) + word];
                w[u] = make_uint2(v & 0xffffu, v >> 16);
            } else {
                w[u] = reinterpret_cast<const uint2 *>(a.codes[kv])[row * (HD / 8) + word];
            }
            par[u] = a.params[kv][row * GR + gr];
        }
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        // the word is cell (2 ga + gr % 2) of groups gr & ~1 (x) and gr | 1 (y): keep
        // this lane's group, hand the partner its own
        const uint32_t got = __shfl_xor_sync(0xffffffffu, gr & 1 ? w[u].x : w[u].y, 4);
        if (pos[u] < 0) continue;
        const uint32_t c0 = gr & 1 ? got : w[u].x, c1 = gr & 1 ? w[u].y : got;  // cells 2 ga, 2 ga + 1
        __half2 v[4];  // (dim i, dim 4 + i)
        if (BITS == 4)
            kvq_codes4(c0 | c1 << 16, v);
        else
            kvq_codes8(c0, c1, v);
        const __half2 lo = kvq_h2(kvq_prmt(par[u], 0, 0x1010)), st = kvq_h2(kvq_prmt(par[u], 0, 0x3232));
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 p = __half22float2(__hfma2(st, v[i], lo));
            f[i] = p.x;
            f[4 + i] = p.y;
        }
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(out.data) + s * out.seq + j[u] * out.token +
                                   h[u] * out.head + 8 * e) = make_uint4(o[0], o[1], o[2], o[3]);
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
    // many tokens: neighbouring threads take neighbouring positions of one head (the
    // packed rows of a head are one run); few: the heads of a token
    a.token_fast = l.n_tok >= 32;
    a.inner = FastDiv(uint32_t(a.token_fast ? l.n_tok : c.n_kv_heads));
    a.l = l;
    return a;
}

dim3 rw_grid(const ll_kvq_cache &c, const RwArgs &a) {
    const int per_block = RW_THREADS / (c.head_dim / 8) * 2;
    return dim3((a.n_rows + per_block - 1) / per_block, 2, c.n_seq);
}

int launched() { return cudaGetLastError() == cudaSuccess ? LL_OK : LL_ERR_CUDA; }

}  // namespace

int launch_kvq_write(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, int type, const KvqLens &l,
                     cudaStream_t st) {
    const RwArgs a = rw_args(c, k, v, l);
    const dim3 g = rw_grid(c, a);
    kvq_dispatch(c, [&](auto bits, auto hd) {
        if (type == LL_F32)
            k_kvq_write<float, bits.value, hd.value><<<g, RW_THREADS, 0, st>>>(a);
        else
            k_kvq_write<__nv_bfloat16, bits.value, hd.value><<<g, RW_THREADS, 0, st>>>(a);
    });
    return launched();
}

int launch_kvq_read(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, const KvqLens &l, cudaStream_t st) {
    const RwArgs a = rw_args(c, k, v, l);
    const dim3 g = rw_grid(c, a);
    kvq_dispatch(c, [&](auto bits, auto hd) { k_kvq_read<bits.value, hd.value><<<g, RW_THREADS, 0, st>>>(a); });
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
    if (c->max_seq < 1) return bad(LL_ERR_SHAPE, "max_seq must be positive");
    if (c->n_seq > 1 && c->seq_rows < int64_t(c->n_kv_heads) * c->max_seq)
        return bad(LL_ERR_ARG, "seq_rows is less than n_kv_heads * max_seq");
    const void *p[4] = {c->k_codes, c->v_codes, c->k_params, c->v_params};
    for (const void *q : p)
        if (!q || (reinterpret_cast<uintptr_t>(q) & 15u)) return bad(LL_ERR_ARG, "a packed cache array is NULL or not 16-byte aligned");
    return LL_OK;
}

}  // namespace ll

namespace {

int report(char *err, size_t err_len, int code, const char *fmt, ...) {
    if (err && err_len) {
        va_list ap;
        va_start(ap, fmt);
        std::vsnprintf(err, err_len, fmt, ap);
        va_end(ap);
    }
    return code;
}

// Once per device: is it the one this library is built for, and its SM count.
struct Dev {
    int state = 0;  // 0 unknown, 1 fits, 2 another architecture
    int nsm = 0, sm = 0;
};
constexpr int MAX_DEVICES = 64;
std::mutex g_dev_mu;
Dev g_dev[MAX_DEVICES];

int check_device(int &nsm, char *err, size_t err_len) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return report(err, err_len, LL_ERR_CUDA, "no CUDA device");
    if (dev < 0 || dev >= MAX_DEVICES) return report(err, err_len, LL_ERR_DEVICE, "device ordinal %d out of range", dev);
    std::lock_guard<std::mutex> lock(g_dev_mu);
    Dev &d = g_dev[dev];
    if (!d.state) {
        int major = 0, minor = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&d.nsm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return report(err, err_len, LL_ERR_CUDA, "cannot query device %d", dev);
        d.sm = 10 * major + minor;
        d.state = d.sm == 103 ? 1 : 2;
    }
    if (d.state == 2) return report(err, err_len, LL_ERR_DEVICE, "device is sm_%d, this library is built for sm_103a", d.sm);
    nsm = d.nsm;
    return LL_OK;
}

// Rows of head_dim elements of `size` bytes each over (n_seq, n_tok, heads);
// written: they are outputs, so no two may share their place by a stride of 0.
int check_rows(const ll_kvq_rows *r, const char *name, int64_t n_seq, int64_t n_tok, int64_t heads, int size, bool written,
               char *err, size_t err_len) {
    if (!r || !r->data) return report(err, err_len, LL_ERR_ARG, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(r->data) & 15u) return report(err, err_len, LL_ERR_ARG, "%s is not 16-byte aligned", name);
    const int64_t stride[3] = {r->seq, r->token, r->head}, extent[3] = {n_seq, n_tok, heads};
    for (int i = 0; i < 3; i++) {
        if (extent[i] <= 1) continue;
        if ((stride[i] * size) % 16) return report(err, err_len, LL_ERR_ARG, "a stride of %s is not a multiple of 16 bytes", name);
        if (written && stride[i] == 0) return report(err, err_len, LL_ERR_ARG, "%s is written and has a stride of 0", name);
    }
    return LL_OK;
}

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

int finish(int rc, char *err, size_t err_len) {
    if (rc == LL_OK) return rc;
    const cudaError_t e = cudaGetLastError();
    return report(err, err_len, rc, "kernel launch failed: %s", cudaGetErrorString(e));
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
    return finish(ll::launch_kvq_attention(*c, *q, LL_BF16, n_q_heads, l, max_len, scale, o, nsm,
                                           static_cast<cudaStream_t>(stream)),
                  err, err_len);
}

}  // extern "C"

// rmsnorm.cu -- the residual's addition and the RMS norm of rows (ll_rmsnorm in include/ll.h).
//
//   r = round(x + residual),   out = r / sqrt(mean(r^2) + eps) * gain,   e4m3: out / scale, scale = max|out| / 448
//
// One pass: a row's values stay in the registers of the threads that loaded them (units of 8, one 16-byte
// load of bf16) while its sum of squares goes round.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "call.h"
#include "rows.cuh"

namespace ll {
namespace {

struct NormArgs {
    const void *x, *res;
    void *res_out, *out;
    int64_t x_stride, res_stride, res_out_stride, out_stride;
    const __nv_bfloat16 *gain;
    float *scale;
    int group, scale_row;  // columns of a scale (0: the row), scales of a row
    float eps;
    int n, width;
    bool vec;              // every row takes 8-value loads and stores
};

// A row's sum or largest over its TEAM threads (a power of two; of one warp up to 32).
template <int TEAM, bool MAX>
__device__ __forceinline__ float team_reduce(float v, float *red) {
#pragma unroll
    for (int o = (TEAM < 32 ? TEAM : 32) / 2; o > 0; o /= 2) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    if constexpr (TEAM > 32) {
        constexpr int WARPS = TEAM / 32;
        const int warp = threadIdx.x / 32, first = warp / WARPS * WARPS;
        if (threadIdx.x % 32 == 0) red[warp] = v;
        __syncthreads();
        v = red[first + threadIdx.x % WARPS];  // (every lane one of the team's, over and over)
#pragma unroll
        for (int o = WARPS / 2; o > 0; o /= 2) {
            const float w = __shfl_xor_sync(0xffffffffu, v, o);
            v = MAX ? fmaxf(v, w) : v + w;
        }
    }
    return v;
}

// TEAM threads a row, up to UNITS units of 8 values each.
template <typename TX, typename TR, typename TO, int TEAM, int UNITS, bool RES>
__global__ void __launch_bounds__(TEAM < 256 ? 256 : TEAM) k_rmsnorm_rows(const NormArgs a) {
    constexpr int THREADS = TEAM < 256 ? 256 : TEAM, ROWS = THREADS / TEAM;
    __shared__ float red[2][THREADS / 32];
    const int in = threadIdx.x % TEAM;
    const int64_t row = int64_t(blockIdx.x) * ROWS + threadIdx.x / TEAM;
    const bool held = row < a.n;
    const TX *x = static_cast<const TX *>(a.x) + (held ? row : 0) * a.x_stride;
    float v[UNITS][8];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < UNITS; u++) {
        const int k = 8 * (in + u * TEAM);
        if (held) load8(x, k, a.width, a.vec, v[u]);
        else
#pragma unroll
            for (int i = 0; i < 8; i++) v[u][i] = 0.f;
    }
    if constexpr (RES) {
        const TR *res = static_cast<const TR *>(a.res) + (held ? row : 0) * a.res_stride;
        TR *res_out = static_cast<TR *>(a.res_out) + (held ? row : 0) * a.res_out_stride;
        float w[UNITS][8];
#pragma unroll
        for (int u = 0; u < UNITS; u++)
            if (held) load8(res, 8 * (in + u * TEAM), a.width, a.vec, w[u]);
#pragma unroll
        for (int u = 0; u < UNITS; u++)
            if (held) {
#pragma unroll
                for (int i = 0; i < 8; i++) v[u][i] = rounded<TR>(v[u][i] + w[u][i]);
                store8(res_out, 8 * (in + u * TEAM), a.width, a.vec, v[u]);
            }
    }
#pragma unroll
    for (int u = 0; u < UNITS; u++)
#pragma unroll
        for (int i = 0; i < 8; i++) ss = fmaf(v[u][i], v[u][i], ss);
    ss = team_reduce<TEAM, false>(ss, red[0]);
    const float r = 1.f / sqrtf(ss / float(a.width) + a.eps);
    float mx[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; u++) {
        float gain[8];
        load8(a.gain, 8 * (in + u * TEAM), a.width, a.vec, gain);
        mx[u] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[u][i] = v[u][i] * r * gain[i];
            mx[u] = fmaxf(mx[u], fabsf(v[u][i]));
        }
    }
    TO *out = static_cast<TO *>(a.out) + (held ? row : 0) * a.out_stride;
    if constexpr (sizeof(TO) == 1) {
        float row_max = 0.f;
        if (a.group == 0) {
#pragma unroll
            for (int u = 0; u < UNITS; u++) row_max = fmaxf(row_max, mx[u]);
            row_max = team_reduce<TEAM, true>(row_max, red[1]);
        }
#pragma unroll
        for (int u = 0; u < UNITS; u++) {
            const int k = 8 * (in + u * TEAM);
            float m = row_max;
            if (a.group) {  // 16 threads share 128 columns
                m = mx[u];
#pragma unroll
                for (int o = 8; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            // (2^-126: a scale whose reciprocal is finite)
            const float scale = fmaxf(m / 448.f, 1.17549435e-38f), inv = 1.f / scale;
            if (held && k < a.width && (a.group ? k % 128 == 0 : k == 0)) a.scale[row * a.scale_row + (a.group ? k / 128 : 0)] = scale;
#pragma unroll
            for (int i = 0; i < 8; i++) v[u][i] *= inv;
            if (held) store8(out, k, a.width, a.vec, v[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < UNITS; u++)
            if (held) store8(out, 8 * (in + u * TEAM), a.width, a.vec, v[u]);
    }
}

template <typename TX, typename TR, typename TO, bool RES>
void launch_norm(const NormArgs &a, cudaStream_t st) {
    const int units = (a.width + 7) / 8;
    auto go = [&](auto kernel, int team) {
        const int threads = team < 256 ? 256 : team, rows = threads / team;
        kernel<<<(a.n + rows - 1) / rows, threads, 0, st>>>(a);
    };
    if (units <= 16) go(k_rmsnorm_rows<TX, TR, TO, 16, 1, RES>, 16);
    else if (units <= 32) go(k_rmsnorm_rows<TX, TR, TO, 32, 1, RES>, 32);
    else if (units <= 64) go(k_rmsnorm_rows<TX, TR, TO, 64, 1, RES>, 64);
    else if (units <= 128) go(k_rmsnorm_rows<TX, TR, TO, 128, 1, RES>, 128);
    else if (units <= 256) go(k_rmsnorm_rows<TX, TR, TO, 256, 1, RES>, 256);
    else if (units <= 512) go(k_rmsnorm_rows<TX, TR, TO, 512, 1, RES>, 512);
    else if (units <= 1024) go(k_rmsnorm_rows<TX, TR, TO, 1024, 1, RES>, 1024);
    else if (units <= 2048) go(k_rmsnorm_rows<TX, TR, TO, 1024, 2, RES>, 1024);
    else go(k_rmsnorm_rows<TX, TR, TO, 1024, 4, RES>, 1024);
}

template <typename TX, typename TR, bool RES>
void launch_norm_out(const NormArgs &a, int type, cudaStream_t st) {
    if (type == LL_BF16) launch_norm<TX, TR, __nv_bfloat16, RES>(a, st);
    else if (type == LL_F32) launch_norm<TX, TR, float, RES>(a, st);
    else launch_norm<TX, TR, e4m3, RES>(a, st);
}

}  // namespace

int launch_rmsnorm(const ll_rows &x, const ll_rows *res, const ll_rows *res_out, const uint16_t *gain, float eps, int n, int width,
                   const ll_rows &out, cudaStream_t st) {
    NormArgs a = {};
    a.x = x.data;
    a.out = out.data;
    a.gain = reinterpret_cast<const __nv_bfloat16 *>(gain);
    a.scale = out.scale;
    a.group = out.group;
    a.scale_row = out.group ? (width + 127) / 128 : 1;
    a.eps = eps;
    a.n = n;
    a.width = width;
    a.vec = reinterpret_cast<uintptr_t>(gain) % 16 == 0;
    auto rows = [&](const ll_rows &r, int64_t &stride) {
        stride = n > 1 ? r.stride : 0;
        const int size = r.type == LL_F32 ? 4 : r.type == LL_BF16 ? 2 : 1, wide = size == 1 ? 8 : 16;
        a.vec = a.vec && reinterpret_cast<uintptr_t>(r.data) % wide == 0 && (stride * size) % wide == 0;
    };
    rows(x, a.x_stride);
    rows(out, a.out_stride);
    if (res) {
        a.res = res->data;
        a.res_out = res_out->data;
        rows(*res, a.res_stride);
        rows(*res_out, a.res_out_stride);
    }
    using B = __nv_bfloat16;
    if (!res)
        x.type == LL_F32 ? launch_norm_out<float, float, false>(a, out.type, st) : launch_norm_out<B, B, false>(a, out.type, st);
    else if (res->type == LL_F32)
        x.type == LL_F32 ? launch_norm_out<float, float, true>(a, out.type, st) : launch_norm_out<B, float, true>(a, out.type, st);
    else
        x.type == LL_F32 ? launch_norm_out<float, B, true>(a, out.type, st) : launch_norm_out<B, B, true>(a, out.type, st);
    return launched();
}

}  // namespace ll

extern "C" int ll_rmsnorm(const ll_rows *x, const ll_rows *residual, const ll_rows *residual_out, const uint16_t *gain, float eps, int32_t n,
                          int32_t width, const ll_rows *out, void *stream, char *err, size_t err_len) {
    using ll::report;
    if (err && err_len) err[0] = '\0';
    if (n < 1) return report(err, err_len, LL_ERR_ARG, "n must be at least 1");
    if (width < 1 || width > 32768) return report(err, err_len, LL_ERR_SHAPE, "width must be 1 to 32768");
    if (!(eps >= 0.f) || !isfinite(eps)) return report(err, err_len, LL_ERR_ARG, "eps must be finite and not negative");
    if (!gain || reinterpret_cast<uintptr_t>(gain) % 2) return report(err, err_len, LL_ERR_ARG, "gain is NULL or not aligned to its type");
    if (int rc = ll::check_matrix_rows(x, "x", n, width, false, false, err, err_len)) return rc;
    if (int rc = ll::check_matrix_rows(out, "out", n, width, true, true, err, err_len)) return rc;
    if (!residual != !residual_out) return report(err, err_len, LL_ERR_ARG, "residual and residual_out go together");
    if (residual) {
        if (int rc = ll::check_matrix_rows(residual, "residual", n, width, false, false, err, err_len)) return rc;
        if (int rc = ll::check_matrix_rows(residual_out, "residual_out", n, width, false, true, err, err_len)) return rc;
        if (residual->type != residual_out->type) return report(err, err_len, LL_ERR_ARG, "residual_out must be of residual's type");
        if (residual_out->data == out->data) return report(err, err_len, LL_ERR_ARG, "out and residual_out are the same rows");
    }
    int nsm = 0;
    if (int rc = ll::check_device(nsm, err, err_len)) return rc;
    return ll::finish(ll::launch_rmsnorm(*x, residual, residual_out, gain, eps, n, width, *out, static_cast<cudaStream_t>(stream)), err, err_len);
}

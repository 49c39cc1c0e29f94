// kvq_attn.cuh -- what the attention kernels over the packed KV cache share
// (kvq_attn.cu: few query rows and chunks; kvq_prompt.cu: prompts).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "kvq.cuh"
#include "kvq.h"

namespace ll {

struct KvqAttnArgs {
    const uint8_t *kc, *vc;
    const uint32_t *kp, *vp;
    int64_t seq_rows;
    int32_t max_seq, group, nkv;
    KvqLens l;
    const void *q;
    int64_t q_seq, q_tok, q_head;
    float scale_log2;  // scale * log2(e): scores in log2 units, probabilities by exp2
    KvqOut out;
    KvqWaits waits;
};

// A row's reference m is its running maximum less KVQ_ROOM (log2 units), and moves only once
// a score passes it by KVQ_ROOM + KVQ_HOLD: until then neither l nor O needs rescaling.
// Probabilities are taken against m, so the largest score's is 2^7 to 2^15. They enter the products as
// fp16 (the matrix rate of its 11 bits; K and V themselves come with 4 or 8), whose range
// that uses up: the smallest that is not lost is 2^-32 of the largest or less, where
// it would be 2^-25 with the maximum itself as the reference.
constexpr float KVQ_HOLD = 8.f, KVQ_ROOM = 7.f;
// A score (a product s times its row's factor) above m, rounded before m is taken off, as m was. With one rounding for
// s * fac - m, scores past 2^25 log2 units stood above the largest of them by their own last place, and their
// probabilities past fp16's range (one rounding: 32 sequences of 32768 positions 1 % faster, a prompt of 8192 5 %; the
// prompt kernel takes it and does such rows again).
__device__ __forceinline__ float kvq_above(float s, float fac, float m) { return __fsub_rn(__fmul_rn(s, fac), m); }
// Whether a row's largest score (rounded) moves m.
__device__ __forceinline__ bool kvq_passes(float top, float m) { return __fsub_rn(top, m) > KVQ_ROOM + KVQ_HOLD; }

__device__ __forceinline__ uint32_t sptr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// A run of bytes to shared memory by the copy engine (both addresses and the size
// multiples of 16), counted by an mbarrier.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// Waits for a phase for at most timeout_ns: false when it has not come by then.
static __device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        for (int i = 0; i < 64; i++)
            if (bar_try(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < timeout_ns);
    return false;
}
// The same for a warp's copies, with what a lane found in *lost: false when this or an earlier one has not come. Each lane looks
// at its own clock, so a limit may pass for some lanes alone; the warp goes on whole all the same, with what the memory
// holds and without further waits (its rows become NaN).
static __device__ __noinline__ bool copy_wait(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int *lost) {
    if (!*lost && bar_wait_long(bar, parity, timeout_ns)) return true;
    *lost = 1;
    return false;
}
constexpr uint64_t KVQ_DRAIN_NS = 1000000000ull;  // what is in flight when a wait has run out is given this long to land

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return kvq_u32(__floats2half2_rn(lo, hi)); }

__device__ __forceinline__ void load_q8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load_q8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}
__device__ __forceinline__ float4 load_q4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load_q4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float q_at(const float *p) { return *p; }
__device__ __forceinline__ float q_at(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// The power of two that brings a row whose largest magnitude is mx into [1, 2)
// (fp16 then holds 11 bits of every value that matters to a product; a bf16 q is
// exact but for values 2^-14 of the largest), and its inverse.
__device__ __forceinline__ void row_scale(float mx, float &down, float &up) {
    int e = int((__float_as_uint(mx) >> 23) & 255u) - 127;
    e = mx > 0.f ? min(max(e, -126), 126) : 0;
    down = __uint_as_float(uint32_t(127 - e) << 23);
    up = __uint_as_float(uint32_t(127 + e) << 23);
}

// Two neighbouring values (dims d, d + 1) of a token's head.
__device__ __forceinline__ void put_out(const KvqOut &o, int s, int j, int head, int d, float a, float b) {
    const int64_t at = s * o.seq + j * o.token + head * o.head + d;
    if (o.f32) {
        *reinterpret_cast<float2 *>(o.f32 + at) = make_float2(a, b);
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; i++) {
        if (!o.t[i]) break;
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        *reinterpret_cast<__nv_bfloat162 *>(o.t[i] + at) = v;
        a -= __low2float(v);
        b -= __high2float(v);
    }
}

// 32 values from dim d on, each times f.
__device__ __forceinline__ void put_out32(const KvqOut &o, int s, int j, int head, int d, const uint32_t (&x)[32], float f) {
    if (o.f32 || o.t[1]) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) put_out(o, s, j, head, d + i, __uint_as_float(x[i]) * f, __uint_as_float(x[i + 1]) * f);
        return;
    }
    uint4 *const to = reinterpret_cast<uint4 *>(o.t[0] + s * o.seq + j * o.token + head * o.head + d);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(x[8 * i + 2 * k]) * f, __uint_as_float(x[8 * i + 2 * k + 1]) * f);
            w[k] = *reinterpret_cast<const uint32_t *>(&v);
        }
        to[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Once per kernel and device (the current one): its shared memory, and clusters of up to 16.
template <auto kernel>
bool prepared(int smem, int dev) {
    static std::atomic<uint64_t> done{0};
    if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return true;
}

template <typename K, typename... Args>
int kvq_launch(K kernel, dim3 grid, int threads, int smem, int cluster, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? LL_OK : LL_ERR_CUDA;
}

// Blocks of `kernel` that are resident at once in clusters of each size (a cluster's
// blocks have to fit in one group of SMs, so larger clusters leave some SMs out: with
// one block to an SM, 152 of them in ones and 112 in sixteens), asked once per device.
constexpr int KVQ_CLUSTERS[] = {1, 2, 4, 6, 8, 12, 16}, KVQ_CLUSTER_SIZES = 7;
struct KvqSlots {
    int n[KVQ_CLUSTER_SIZES];
};
template <auto kernel>
const KvqSlots &kvq_slots(int threads, int smem, int nsm, int dev) {
    static KvqSlots slots[64];
    static std::atomic<uint64_t> known{0};
    static std::mutex mu;
    dev &= 63;
    if (known.load(std::memory_order_acquire) >> dev & 1) return slots[dev];
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < KVQ_CLUSTER_SIZES; i++) {
        const unsigned size = unsigned(KVQ_CLUSTERS[i]);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = size_t(smem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            clusters = i ? 0 : nsm;
        }
        slots[dev].n[i] = clusters * int(size);
    }
    known.fetch_or(uint64_t(1) << dev, std::memory_order_release);
    return slots[dev];
}

// The kernel for prompts (kvq_prompt.cu): 256 query rows of a KV head to a block.
constexpr int KVQ_PROMPT_ROWS = 256;
// longest: the longest length it is laid out for; dev: the current device.
int launch_kvq_prompt(const ll_kvq_cache &c, const KvqAttnArgs &a, int type, int longest, int nsm, int dev, cudaStream_t st);

}  // namespace ll

// kvq_prompt.cu -- attention of many query rows over the packed KV cache, on the
// fifth-generation tensor cores.
//
// A block takes 256 query rows of a KV head (row = token * group + head), as two
// tiles A and B of 128, and walks the keys in tiles of 128. Four warps unpack
// tiles of K and four tiles of V into fp16 in shared memory, two stages deep or
// more (once for both row tiles: unpacking costs about as much as one row
// tile's softmax); one warp issues tcgen05.mma, S = Q K^T and O += P V, both in tensor memory; and four warps
// per row tile, a row to a thread, read S, take P = exp(S - m) back into the first
// half of S's columns as fp16 (the A operand of P V), and move the running
// maximum where a score passes it. While one row tile is in its softmax, the
// other is in its products.
//
// Where there are too few blocks for the device, a cluster of them shares the keys
// of its rows: each keeps O, m and l of its part in its own shared memory, and
// merges a share of the rows from all of them.
//
// What bounds it: at 128 dims the products of a key tile take 2,048 cycles of the
// tensor cores for the two row tiles, the softmax and unpacking about 1,800 issue
// slots per scheduler; at 64 dims the products are half of that, and the softmax
// bounds. A prompt of 8192 with 32 query heads over 8 packed in 4 bits: 538 us at 128
// dims (1.02 PFLOP/s of causal products, 54 % of the measured matrix rate; the products
// alone, without softmax and unpacking, took 420 us), 380 us at 64.
#include <cooperative_groups.h>

#include "kvq_attn.cuh"
#include "ll_internal.h"

namespace ll {
namespace {

constexpr int THREADS = 20 * 32;  // softmax A, softmax B, K, V (4 warps each), products (a warp of four)
constexpr int W_MMA = 16;  // the warp, or two, that issue products
// Registers a thread: 96 at launch, then as the roles need them (a softmax thread
// holds P of its row, 64, beside the scores on their way; a V thread up to 64 packed
// words). The groups' shares add up to the launch's.
constexpr int R_LAUNCH = 96, R_SOFTMAX = 112, R_K = 72, R_V = 136, R_MMA = 48;
static_assert(2 * R_SOFTMAX + R_K + R_V + R_MMA == 5 * R_LAUNCH && 5 * 128 * R_LAUNCH <= 65536, "registers");
template <int N>
__device__ __forceinline__ void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int KEYS = 128;

template <int HD>
struct Shape {
    static constexpr uint32_t QT = 128 * HD * 2, KT = KEYS * HD * 2;  // a row tile; a K or V tile
    // K/V stages and S buffers: at 64 dims there is room for three S (512 columns of tensor memory with the two O),
    // so that a row tile's next scores are there when its softmax ends; the products then run two steps ahead,
    // which takes four stages.
    static constexpr int ST = HD == 64 ? 4 : 2, NB = HD == 64 ? 3 : 2;
    // With three buffers two warps issue the products, one S and one P V, so that one's waits and address work lie under
    // the other's products (a prompt of 8192 at 64 dims 404 -> 357 us). With two, S has to follow the P V of its
    // buffer, and one warp issues them in an order that keeps the two row tiles out of step (two warps at 128 dims, one
    // for S and one for P V or one per row tile: 537 -> 611 and 635 us).
    static constexpr bool ONE_WARP = NB == 2;
    static constexpr uint32_t SMEM = 2 * QT + ST * 2 * KT + 1024;     // (from a 1,024-byte border)
    static constexpr uint32_t TM_O = 128 * NB;                        // tensor memory: S buffers, O of A and B
    static_assert(TM_O + 2 * HD <= 512, "tensor memory");
};

// The order of the block's steps (row tile t, key tile i): A and B in turn, then
// what the longer walk has left. Step j uses S buffer j % NB.
struct Steps {
    int na, nb;
    __device__ __forceinline__ int both() const { return min(na, nb); }
    __device__ __forceinline__ int count() const { return na + nb; }
    __device__ __forceinline__ int tile(int j) const { return j < 2 * both() ? j >> 1 : j - both(); }
    __device__ __forceinline__ int row(int j) const { return j < 2 * both() ? j & 1 : int(nb > na); }
    __device__ __forceinline__ int step(int t, int i) const { return i < both() ? 2 * i + t : both() + i; }
};

// Shared-memory matrix descriptor of a K-major tile in the 128-byte swizzle (rows
// of 128 bytes, 8-row groups 1,024 bytes apart); 16 elements along K are 32 bytes.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t addr) {
    return uint64_t((addr >> 4) & 0x3fffu) | uint64_t(1u) << 16 | uint64_t(1024u >> 4) << 32 | uint64_t(1u) << 46 |
           uint64_t(2u) << 61;
}
// Instruction descriptor of kind::f16: fp16 A and B, both K-major, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int m, int n) {
    return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// The products are issued by a whole warp, of which one elected lane (the same at every
// call) carries them out: in a branch for one lane the compiler has to move every
// operand into a uniform register first, which took as long as the products
// (prompt of 8192: 617 us, and 564 this way).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {  // arrives once all products issued so far are done
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Bounded wait: once the limit passes, with *err and the status word set, or once another's has, the block goes on without
// waits to its end, as if all had come: its loops and whole-warp instructions stay together, and its rows become NaN.
__device__ __forceinline__ void wait_long(uint32_t bar, uint32_t parity, volatile int *err, const KvqWaits &w) {
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    do {
        if (*err) return;
        for (int i = 0; i < 64; i++)
            if (bar_try(bar, parity)) return;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    } while (t - t0 < w.timeout_ns);
    *err = 1;
    if (w.status) atomicCAS(w.status, 0, LL_ERR_DEP_TIMEOUT);
}
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile int *err, const KvqWaits &w) {
    if (!bar_try(bar, parity)) wait_long(bar, parity, err, w);
}

// 32 columns of this thread's tensor-memory lane; the values are there after tm_wait.
__device__ __forceinline__ void tm_load(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
// (16 columns)
__device__ __forceinline__ void tm_load16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
// (the values pass through the statement, so that no use of them can come before it)
__device__ __forceinline__ void tm_wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
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
__device__ __forceinline__ void tm_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync() {  // (by whole warps)
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The dim of element p of a K or Q row in shared memory: a packed word (cells g of
// groups 2 gp and 2 gp + 1) becomes one 16-byte chunk, in the order its
// unpacking leaves it.
template <int HD>
__device__ __forceinline__ int dim_at(int p) {
    constexpr int GP = HD / 64;
    const int q = p >> 3;
    return 32 * (2 * (q % GP) + (p & 1)) + 4 * (q / GP) + ((p & 7) >> 1);
}

// Byte of 16-byte chunk c (8 fp16) of row r in a K-major tile of `rows` rows: 64
// columns (8 chunks) after 64 columns, each in the 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int rows, int r, int c) {
    return uint32_t((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The product of a row of Q (in shared memory, as it is multiplied) and a K row of the cache.
template <int BITS, int HD>
__device__ __forceinline__ float product(const uint8_t *qs, int row, const uint8_t *codes, const uint32_t *params) {
    float sum = 0.f;
#pragma unroll 1
    for (int e = 0; e < HD; e++) {
        const int d = dim_at<HD>(e), gr = d / 32;
        const __half q = *reinterpret_cast<const __half *>(qs + chunk_at(128, row, e >> 3) + 2 * (e & 7));
        sum = fmaf(__half2float(q), __half2float(kvq_value<BITS, HD>(codes, params[gr], gr, d % 32)), sum);
    }
    return sum;
}

// What the walk could not do, for rows like that are rare: a row to a thread of whole warps, its O in tensor memory (to) and its
// m and l, over the keys k0 .. last. `flags`: REDO, scores so large that the walk's one rounding may have lost them
// (kvq_above): all of it again, by the row itself. A group's bit: O lacks those keys from k on whose V in the group may not be
// finite; they are added, NaN where a value is not. (A function of its own, and its arguments by value: a prompt of 8192 554 us,
// 558 to 564 as part of the kernel or with the arguments' address.)
constexpr uint32_t REDO = 0x80000000u;
template <int BITS, int HD>
__device__ __noinline__ float2 finish_rows(const uint8_t *kc, const uint8_t *vc, const uint32_t *kp, const uint32_t *vp, int k0, int k, int last,
                                           uint32_t flags, const uint8_t *qs, int row, float fac, float2 ml, uint32_t to) {
    constexpr int GR = HD / 32, RB = HD * BITS / 8;
    const bool redo = flags & REDO;
    if (redo) {
        ml = make_float2(-INFINITY, 0.f);
#pragma unroll 1
        for (int i = k0; i <= last; i++) ml.x = fmaxf(ml.x, __fmul_rn(product<BITS, HD>(qs, row, kc + int64_t(i) * RB, kp + int64_t(i) * GR), fac));
    }
#pragma unroll 1
    for (int gr = 0; gr < GR; gr++) {
        uint32_t x[32];
        tm_load(to + 32 * gr, x);
        tm_wait(x);
        if (redo) {
            ml.y = 0.f;
#pragma unroll
            for (int d = 0; d < 32; d++) x[d] = 0;
        }
#pragma unroll 1
        for (int i = redo ? k0 : flags >> gr & 1 ? k : last + 1; i <= last; i++) {
            const uint32_t par = vp[int64_t(i) * GR + gr];
            if (!redo && !kvq_not_finite<BITS>(par)) continue;
            const float p = ex2(kvq_above(product<BITS, HD>(qs, row, kc + int64_t(i) * RB, kp + int64_t(i) * GR), fac, ml.x));
            if (redo) ml.y += p;
#pragma unroll
            for (int d = 0; d < 32; d++) {
                const float v = __half2float(kvq_value<BITS, HD>(vc + int64_t(i) * RB, par, gr, d));
                x[d] = __float_as_uint(isfinite(v) ? fmaf(p, v, __uint_as_float(x[d])) : __uint_as_float(0x7fffffffu));
            }
        }
        __syncwarp();
        tm_store(to + 32 * gr, x);
    }
    tm_store_wait();
    return ml;
}

template <int BITS, int HD, typename QT>
__global__ void __launch_bounds__(THREADS, 1) k_kvq_prompt(const __grid_constant__ KvqAttnArgs a, int C) {
    using S = Shape<HD>;
    constexpr int GR = HD / 32, GP = HD / 64, RB = HD * BITS / 8;
    extern __shared__ uint8_t raw[];
    uint8_t *const smem = raw + ((1024u - (sptr(raw) & 1023u)) & 1023u);
    constexpr int ST = S::ST, NB = S::NB;
    __shared__ uint64_t bars[4 * ST + 4 * NB + 6];
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    __shared__ float2 s_ml[256];
    __shared__ __align__(16) uint8_t s_bad[ST][GR][16];  // [stage][group][keys of 8]: keys of the tile whose V may not be finite
    const uint32_t bar0 = sptr(bars);
    // per K/V stage; per S buffer (p_full for the two halves of its keys); per row tile (its products with the first
    // half of a tile's V, and with all of it, are done)
    const uint32_t k_full = bar0, k_empty = k_full + 8 * ST, v_full = k_empty + 8 * ST, v_empty = v_full + 8 * ST,
                   s_full = v_empty + 8 * ST, p_full = s_full + 8 * NB, s_free = p_full + 16 * NB, o_half = s_free + 8 * NB, o_done = o_half + 16, drained = o_done + 16;
    volatile int *const err = &s_err;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (row tiles slowest, last ones first: the blocks with the most keys of every head start first)
    const int nkv = a.nkv, s = blockIdx.z, unit = int(blockIdx.x) / C, rank = int(blockIdx.x) % C, h = unit % nkv;
    const int n = a.l.n(s), len = a.l.len(s), rows = n * a.group, first = len - n;
    const int r0 = (int(gridDim.x) / C - 1 - unit) / nkv * KVQ_PROMPT_ROWS;
    if (r0 >= rows) return;
    // keys that a row tile's last row sees, in tiles; a row tile past the last row sees none
    auto seen = [&](int t) {
        const int lo = r0 + 128 * t, hi = min(lo + 128, rows) - 1;
        return lo < rows ? max(0, min(min(len, a.max_seq), first + hi / a.group + 1)) : 0;
    };
    const int seen_a = seen(0), seen_b = seen(1), limit = max(seen_a, seen_b);
    // this block's key tiles: `tiles` of them from tile0 on, of which row tile A or B may see fewer
    const int all = (limit + KEYS - 1) / KEYS, tile0 = int(int64_t(all) * rank / C);
    const int tiles = int(int64_t(all) * (rank + 1) / C) - tile0;
    const Steps steps = {min(max((seen_a + KEYS - 1) / KEYS - tile0, 0), tiles), min(max((seen_b + KEYS - 1) / KEYS - tile0, 0), tiles)};
    const int first_last = first + r0 / a.group;           // the last position that the block's first row sees
    const int edge_from = min(first_last + 1, limit);      // tiles that reach past it are masked
    const uint32_t q_at0 = sptr(smem), kv0 = q_at0 + 2 * S::QT;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; i++) {
            bar_init(k_full + 8 * i, 4);
            bar_init(k_empty + 8 * i, 1);
            bar_init(v_full + 8 * i, 4);
            bar_init(v_empty + 8 * i, 1);
        }
        for (int i = 0; i < NB; i++) {
            bar_init(s_full + 8 * i, 1);
            bar_init(p_full + 16 * i, 4);
            bar_init(p_full + 16 * i + 8, 4);
            bar_init(s_free + 8 * i, 1);
        }
        for (int i = 0; i < 6; i++) bar_init(o_half + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_err = 0;
    }
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sptr(&s_tmem)), "n"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    float fac = 0.f;
    if (warp < 8) {  // this thread's row of Q: scaled to fp16, in the order of K's unpacking
        const int r = r0 + int(threadIdx.x), row = threadIdx.x & 127;
        float mx = 0.f, down, up;
        const QT *q = static_cast<const QT *>(a.q) + s * a.q_seq + int64_t(r / a.group) * a.q_tok +
                      int64_t(h * a.group + r % a.group) * a.q_head;
        if (r < rows)
            for (int d = 0; d < HD; d += 8) {
                float v[8];
                load_q8(q + d, v);
#pragma unroll
                for (int i = 0; i < 8; i++) mx = fmaxf(mx, fabsf(v[i]));
            }
        row_scale(mx, down, up);
        fac = up * a.scale_log2;
        uint8_t *const qs = smem + (threadIdx.x >> 7) * S::QT;
        for (int gp = 0; gp < GP; gp++)
            for (int g = 0; g < 8; g++) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
                if (r < rows) {
                    x = load_q4(q + 64 * gp + 4 * g);
                    y = load_q4(q + 64 * gp + 32 + 4 * g);
                }
                *reinterpret_cast<uint4 *>(qs + chunk_at(128, row, g * GP + gp)) =
                    make_uint4(pack_h2(x.x * down, y.x * down), pack_h2(x.y * down, y.y * down),
                               pack_h2(x.z * down, y.z * down), pack_h2(x.w * down, y.w * down));
            }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);

    if (warp >= W_MMA) {
        fewer_regs<R_MMA>();
    }
    if (warp > W_MMA + (S::ONE_WARP ? 0 : 1)) {
    } else if (warp >= W_MMA) {
        constexpr uint32_t id_s = idesc_f16(128, KEYS), id_o = idesc_f16(128, HD);
        const int count = steps.count();
        int kready = 0, vready = 0;  // key tiles whose K, V is known to be unpacked
        // the last of the steps that use a key tile
        auto last = [&](int j, int i) { return j + 1 == count || steps.tile(j + 1) != i; };
        auto scores = [&](int j) {  // S of step j
            const int i = steps.tile(j), b = j % NB;
            const uint32_t q = q_at0 + steps.row(j) * S::QT, k = kv0 + (i % ST) * 2 * S::KT;
            if (i >= kready) {
                wait(k_full + 8 * (i % ST), (i / ST) & 1, err, a.waits);
                kready = i + 1;
                fence_after();
            }
#pragma unroll
            for (int d = 0; d < HD / 16; d++)
                mma_ss(tmem + 128 * b, desc_sw128(q + (d >> 2) * 128 * 128) + 2 * (d & 3),
                       desc_sw128(k + (d >> 2) * KEYS * 128) + 2 * (d & 3), id_s, d != 0);
            commit(s_full + 8 * b);
            if (last(j, i)) commit(k_empty + 8 * (i % ST));
        };
        auto values = [&](int j) {  // O += P V of step j, in two halves of the keys
            const int i = steps.tile(j), t = steps.row(j), b = j % NB;
            const uint32_t v = kv0 + (i % ST) * 2 * S::KT + S::KT;
            if (i >= vready) {
                wait(v_full + 8 * (i % ST), (i / ST) & 1, err, a.waits);
                vready = i + 1;
            }
#pragma unroll
            for (int f = 0; f < 2; f++) {
                wait(p_full + 16 * b + 8 * f, (j / NB) & 1, err, a.waits);
                fence_after();
#pragma unroll
                for (int k = 4 * f; k < 4 * f + 4; k++)
                    mma_ts(tmem + S::TM_O + HD * t, tmem + 128 * b + 8 * k, desc_sw128(v + f * HD * 128) + 2 * (k & 3), id_o,
                           (i | k) != 0);
                commit((f ? o_done : o_half) + 8 * t);
            }
            if (last(j, i)) commit(v_empty + 8 * (i % ST));
        };
        if (S::ONE_WARP) {
            for (int j = 0; j < min(NB, count); j++) scores(j);
            for (int j = 0; j < count; j++) {
                values(j);
                if (j + NB < count) scores(j + NB);
            }
        } else if (warp == W_MMA) {
            for (int j = 0; j < count; j++) {
                if (j >= NB) {
                    wait(s_free + 8 * (j % NB), (j / NB - 1) & 1, err, a.waits);
                    fence_after();
                }
                scores(j);
            }
        } else {
            for (int j = 0; j < count; j++) {
                values(j);
                commit(s_free + 8 * (j % NB));
            }
        }
    } else if (warp >= 8) {
        const KvqConsts consts;
        const int t = threadIdx.x & 127, w = t >> 5;
        const int64_t row0 = s * a.seq_rows + int64_t(h) * a.max_seq;
        auto words = [](const void *p, auto &to) {
            constexpr int N = sizeof(to) / 4;
            if constexpr (N >= 4) {
#pragma unroll
                for (int j = 0; j < N / 4; j++) {
                    const uint4 u = static_cast<const uint4 *>(p)[j];
                    to[4 * j] = u.x;
                    to[4 * j + 1] = u.y;
                    to[4 * j + 2] = u.z;
                    to[4 * j + 3] = u.w;
                }
            } else if constexpr (N == 2) {
                const uint2 u = *static_cast<const uint2 *>(p);
                to[0] = u.x;
                to[1] = u.y;
            } else {
                to[0] = *static_cast<const uint32_t *>(p);
            }
        };
        auto zero = [](auto &to) {
#pragma unroll
            for (int j = 0; j < int(sizeof(to) / 4); j++) to[j] = 0;
        };
        if (warp < 12) {  // K: a thread is a key
            fewer_regs<R_K>();
            uint32_t kw[RB / 4], kpar[GR];
            auto load = [&](int i) {
                const int key = i * KEYS + t;
                if (key < limit) {
                    words(a.kc + (row0 + key) * RB, kw);
                    words(a.kp + (row0 + key) * GR, kpar);
                } else {
                    zero(kw);
                    zero(kpar);
                }
            };
            for (int i = 0; i < tiles; i++) {
                const int stage = i % ST;
                load(tile0 + i);
                if (i >= ST) wait(k_empty + 8 * stage, (i / ST - 1) & 1, err, a.waits);
                uint8_t *const ks = smem + 2 * S::QT + stage * 2 * S::KT;
#pragma unroll
                for (int gp = 0; gp < GP; gp++) {
                    const __half2 lo = kvq_h2(kvq_prmt(kpar[2 * gp], kpar[2 * gp + 1], 0x5410));
                    const __half2 st = kvq_h2(kvq_prmt(kpar[2 * gp], kpar[2 * gp + 1], 0x7632));
#pragma unroll
                    for (int c = 0; c < 8; c++) {
                        const int q = c * GP + gp;  // the chunk: cell c of this pair of groups
                        __half2 v[4];
                        if (BITS == 4)
                            kvq_codes4(kw[q], consts, v);
                        else
                            kvq_codes8(kw[(2 * q) % (RB / 4)], kw[(2 * q + 1) % (RB / 4)], consts, v);
                        *reinterpret_cast<uint4 *>(ks + chunk_at(KEYS, t, q)) =
                            make_uint4(kvq_u32(__hfma2(st, v[0], lo)), kvq_u32(__hfma2(st, v[1], lo)),
                                       kvq_u32(__hfma2(st, v[2], lo)), kvq_u32(__hfma2(st, v[3], lo)));
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(k_full + 8 * stage);
            }
        } else {
            more_regs<R_V>();
            // V: a thread is 8 keys of a cell, which leave as 16-byte runs of the transposed
            // tile's rows (a row a dim). Lanes 0..7 take 8 runs of 8 keys: their stores
            // fall in different banks.
            const int oct = (lane & 7) | (w & 1) << 3, g = lane >> 3 | (w >> 1) << 2;
            constexpr int VW = GR * BITS / 8;  // words of a cell's groups: 4-bit cells sit two groups to a word
            uint32_t vw[8][VW], vpar[8][GR];
            for (int i = 0; i < tiles; i++) {
                const int k0 = (tile0 + i) * KEYS, stage = i % ST;
                const bool edge = k0 + KEYS > edge_from;
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const int key = k0 + 8 * oct + j;
                    if (key < limit) {
                        words(a.vc + (row0 + key) * RB + g * (RB / 8), vw[j]);
                        words(a.vp + (row0 + key) * GR, vpar[j]);
                    } else {
                        zero(vw[j]);
                        zero(vpar[j]);
                    }
                }
                if (i >= ST) wait(v_empty + 8 * stage, (i / ST - 1) & 1, err, a.waits);
                uint8_t *const vs = smem + 2 * S::QT + stage * 2 * S::KT + S::KT;
                if (edge) {  // V that is not finite must reach only the rows that see it: its group enters as zeros, the rows
                             // are told (taking out single values here cost a prompt of 8192 1 to 2 %)
#pragma unroll
                    for (int gr = 0; gr < GR; gr++) {
                        uint32_t bits = 0;
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            if (kvq_not_finite<BITS>(vpar[j][gr])) {
                                bits |= 1u << j;
                                vpar[j][gr] = 0;
                            }
                        if (g == 0) s_bad[stage][gr][oct] = uint8_t(bits);
                    }
                }
#pragma unroll
                for (int gr = 0; gr < GR; gr++) {
                    uint32_t x[4][4];  // [dim][pair of keys]
#pragma unroll
                    for (int p = 0; p < 4; p++) {
                        __half2 v[4];
                        if (BITS == 4)
                            kvq_codes4(kvq_prmt(vw[2 * p][gr / 2], vw[2 * p + 1][gr / 2], gr & 1 ? 0x7632 : 0x5410), consts, v);
                        else
                            kvq_codes8(vw[2 * p][gr % VW], vw[2 * p + 1][gr % VW], consts, v);
                        const __half2 lo = kvq_h2(kvq_prmt(vpar[2 * p][gr], vpar[2 * p + 1][gr], 0x5410));
                        const __half2 st = kvq_h2(kvq_prmt(vpar[2 * p][gr], vpar[2 * p + 1][gr], 0x7632));
#pragma unroll
                        for (int d = 0; d < 4; d++) x[d][p] = kvq_u32(__hfma2(st, v[d], lo));
                    }
#pragma unroll
                    for (int d = 0; d < 4; d++)
                        *reinterpret_cast<uint4 *>(vs + chunk_at(HD, 32 * gr + 4 * g + d, oct)) =
                            make_uint4(x[d][0], x[d][1], x[d][2], x[d][3]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive(v_full + 8 * stage);
            }
        }
    } else {
        more_regs<R_SOFTMAX>();
        const int t = warp >> 2, r = r0 + int(threadIdx.x), mine = t ? steps.nb : steps.na;
        const uint32_t lanes = uint32_t(warp & 3) << 21;  // this warp's 32 tensor-memory lanes
        const uint32_t to = tmem + lanes + S::TM_O + HD * t;
        const int last = r < rows ? min(first + r / a.group, limit - 1) : -1;  // the last key this row sees
        float m = -INFINITY, l = 0.f;
        uint32_t flags = 0;  // groups of V of which this row sees one that may not be finite, and REDO
        for (int i = 0; i < mine; i++) {
            const int j = steps.step(t, i), b = j % NB;
            const uint32_t ts = tmem + lanes + 128 * b;
            wait(s_full + 8 * b, (j / NB) & 1, err, a.waits);
            fence_after();
            const int k0 = (tile0 + i) * KEYS;
            const bool edge = k0 + KEYS > edge_from;
            const int valid = last - k0 + 1;  // keys of the tile that this row sees
            // O is this thread's once the products of its tile before are done. (Waited for at
            // every tile: a phase that nobody waits for could be taken for the one after next.)
            if (i > 0) wait(o_done + 8 * t, (i - 1) & 1, err, a.waits);
            if (edge) {
                wait(v_full + 8 * (i % ST), (i / ST) & 1, err, a.waits);  // (V is unpacked: what of it may not be finite is known)
#pragma unroll
                for (int gr = 0; gr < GR; gr++) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(s_bad[i % ST][gr]);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        if (u[q] && 32 * q + __ffs(u[q]) - 1 < valid) flags |= 1u << gr;
                }
            }
            // The keys in two halves, each with its own look at the maximum: the products with
            // the first half of V run under the softmax of the second.
#pragma unroll 1
            for (int f = 0; f < 2; f++) {
                uint32_t p[32];  // P, fp16 pairs
                float top, sum;
                auto pass = [&](float m_use, auto masked) {  // P against m_use, its sum, the largest score
                    const uint64_t f2 = kvq_pair(fac, fac), m2 = kvq_pair(-m_use, -m_use);
                    uint64_t acc = kvq_pair(0.f, 0.f);
                    uint32_t c[2][16];
                    float mx = -INFINITY;
                    tm_load16(ts + 64 * f, c[0]);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        uint32_t(&x)[16] = c[q & 1];
                        tm_wait16(x);
                        if (q < 3) tm_load16(ts + 64 * f + 16 * (q + 1), c[(q + 1) & 1]);
                        if (masked.value) {
#pragma unroll
                            for (int j = 0; j < 16; j++)
                                if (64 * f + 16 * q + j >= valid) x[j] = 0xff800000u;
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float s0 = __uint_as_float(x[j]), s1 = __uint_as_float(x[j + 1]);
                            mx = fmaxf(mx, fmaxf(s0, s1));
                            float e0, e1;
                            kvq_split(kvq_fma2(kvq_pair(s0, s1), f2, m2), e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            acc = kvq_add2(acc, kvq_pair(e0, e1));
                            p[8 * q + j / 2] = pack_h2(e0, e1);
                        }
                    }
                    float u, v;
                    kvq_split(acc, u, v);
                    sum = u + v;
                    top = __fmul_rn(mx, fac);
                };
                auto both = [&](float m_use) {
                    if (edge)
                        pass(m_use, KvqConst<1>{});
                    else
                        pass(m_use, KvqConst<0>{});
                };
                both(m == -INFINITY ? 0.f : m);
                const bool grow = kvq_passes(top, m);
                if (__any_sync(0xffffffffu, grow)) {
                    const float to_m = grow ? top - KVQ_ROOM : m, al = !grow ? 1.f : m == -INFINITY ? 0.f : ex2(m - to_m);
                    m = to_m;
                    if (fabsf(m) > 8388608.f && fabsf(m) < INFINITY) flags |= REDO;  // (up to 2^23 no place is more than 1/2)
                    both(m == -INFINITY ? 0.f : m);
                    l *= al;
                    if (f) wait(o_half + 8 * t, i & 1, err, a.waits);
                    fence_after();
                    if (i + f > 0) {
#pragma unroll 1
                        for (int q = 0; q < HD / 16; q++) {
                            uint32_t x[16];
                            tm_load16(to + 16 * q, x);
                            tm_wait16(x);
#pragma unroll
                            for (int j = 0; j < 16; j++) x[j] = __float_as_uint(__uint_as_float(x[j]) * al);
                            tm_store16(to + 16 * q, x);
                        }
                    }
                }
                l += sum;
                tm_store(ts + 32 * f, p);
                tm_store_wait();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive(p_full + 16 * b + 8 * f);
            }
        }
        if (mine > 0) wait(o_done + 8 * t, (mine - 1) & 1, err, a.waits);
        fence_after();
        if (__any_sync(0xffffffffu, flags)) {
            const int64_t row0 = s * a.seq_rows + int64_t(h) * a.max_seq;
            const float2 ml = finish_rows<BITS, HD>(a.kc + row0 * RB, a.vc + row0 * RB, a.kp + row0 * GR, a.vp + row0 * GR, tile0 * KEYS,
                                                    max(tile0, edge_from / KEYS) * KEYS, min(last, (tile0 + mine) * KEYS - 1), flags,
                                                    smem + t * S::QT, threadIdx.x & 127, fac, make_float2(m, l), to);
            m = ml.x;
            l = ml.y;
        }
        // (every lane takes part in the loads; a tile without keys has no O)
        const float inv = *err ? __uint_as_float(0x7fffffffu) : C > 1 ? 1.f : m == -INFINITY ? 0.f : 1.f / l;
        const int j = r / a.group, head = h * a.group + r % a.group;
        float *const part = reinterpret_cast<float *>(smem + 2 * S::QT);  // [256][HD], 16-byte chunk c of row x at c ^ x
        if (C > 1) {
            // the block's products are done, so its K and V stages are free
            asm volatile("bar.sync 1, 256;" ::: "memory");
            s_ml[threadIdx.x] = make_float2(m, l);
        }
#pragma unroll 1
        for (int q = 0; q < HD / 32; q++) {
            uint32_t x[32];
#pragma unroll
            for (int e = 0; e < 32; e++) x[e] = 0;
            if (mine > 0) {
                tm_load(to + 32 * q, x);
                tm_wait(x);
            }
            if (C > 1) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    *reinterpret_cast<float4 *>(part + threadIdx.x * HD + 4 * ((8 * q + e) ^ (threadIdx.x & (HD / 4 - 1)))) =
                        make_float4(__uint_as_float(x[4 * e]) * inv, __uint_as_float(x[4 * e + 1]) * inv,
                                    __uint_as_float(x[4 * e + 2]) * inv, __uint_as_float(x[4 * e + 3]) * inv);
            } else if (r < rows) {
                put_out32(a.out, s, j, head, 32 * q, x, inv);
            }
        }
        fence_before();
        if (C > 1) {
            cluster_sync();
            const cooperative_groups::cluster_group cl = cooperative_groups::this_cluster();
            const int share = 256 / C, live = min(share, rows - r0 - rank * share);
            for (int e = threadIdx.x; e < live * (HD / 4); e += 256) {
                const int row = rank * share + e / (HD / 4), c = e % (HD / 4), R = r0 + row;
                float M = -INFINITY, L = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < C; k++) M = fmaxf(M, cl.map_shared_rank(&s_ml[row], k)->x);
#pragma unroll 4
                for (int k = 0; k < C; k++) {
                    const float2 ml = *cl.map_shared_rank(&s_ml[row], k);
                    const float4 v = *reinterpret_cast<const float4 *>(
                        cl.map_shared_rank(part + row * HD + 4 * (c ^ (row & (HD / 4 - 1))), k));
                    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
                    L = fmaf(ml.y, f, L);
                    o = make_float4(fmaf(v.x, f, o.x), fmaf(v.y, f, o.y), fmaf(v.z, f, o.z), fmaf(v.w, f, o.w));
                }
                const float g = M == -INFINITY ? 0.f : 1.f / L;
                put_out(a.out, s, R / a.group, h * a.group + R % a.group, 4 * c, o.x * g, o.y * g);
                put_out(a.out, s, R / a.group, h * a.group + R % a.group, 4 * c + 2, o.z * g, o.w * g);
            }
            cluster_sync();  // no block leaves while another reads its memory
        }
    }
    if (C > 1 && warp >= 8) {
        cluster_sync();
        cluster_sync();
    }
    __syncthreads();
    if (*err) {  // a wait has run out: products in flight end before their memory goes
        if (warp == W_MMA || warp == W_MMA + 1) {
            commit(drained + 8 * (warp - W_MMA));
            bar_wait_long(drained + 8 * (warp - W_MMA), 0, KVQ_DRAIN_NS);
        }
        __syncthreads();
    }
    if (warp == W_MMA) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512) : "memory");
}

}  // namespace

namespace {

// Blocks that share the keys of a block's rows: for `units` blocks whose longest
// walk has `steps` key tiles, the number with the fewest steps in a row. A block's
// start and end take as long as 6 steps, the merge of a cluster 4 more.
int prompt_splits(int64_t units, const KvqSlots &slots, double steps) {
    int best = 1;
    double least = 0;
    for (int i = 0; i < KVQ_CLUSTER_SIZES; i++) {
        const int c = KVQ_CLUSTERS[i];
        if (KVQ_PROMPT_ROWS % c || slots.n[i] < 1) continue;  // (the merge's shares are whole)
        const int64_t rounds = (units * c + slots.n[i] - 1) / slots.n[i];
        const double time = double(rounds) * (steps / c + 6 + (c > 1 ? 4 : 0));
        if (c == 1 || time < least) {
            least = time;
            best = c;
        }
    }
    return best;
}

}  // namespace

int launch_kvq_prompt(const ll_kvq_cache &c, const KvqAttnArgs &a, int type, int longest, int nsm, int dev, cudaStream_t st) {
    const int64_t rows = int64_t(a.l.n_tok) * a.group, tiles = (rows + KVQ_PROMPT_ROWS - 1) / KVQ_PROMPT_ROWS * c.n_kv_heads;
    int rc = LL_OK;
    kvq_dispatch(c, [&](auto bits, auto hd) {
        auto go = [&](auto qt) {
            constexpr auto kernel = k_kvq_prompt<bits.value, hd.value, decltype(qt)>;
            constexpr int SMEM = Shape<hd.value>::SMEM;
            if (!prepared<kernel>(SMEM, dev)) {
                rc = LL_ERR_CUDA;
                return;
            }
            const int C = prompt_splits(tiles * c.n_seq, kvq_slots<kernel>(THREADS, SMEM, nsm, dev), double(longest) / KEYS);
            rc = kvq_launch(kernel, dim3(unsigned(tiles * C), 1, c.n_seq), THREADS, SMEM, C, st, a, C);
        };
        if (type == LL_F32)
            go(float{});
        else
            go(__nv_bfloat16{});
    });
    return rc;
}

}  // namespace ll

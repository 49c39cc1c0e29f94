// kvq_attn.cu -- attention over the packed KV cache.
//
// One pass over the positions with the running maximum and sum of a softmax: a
// tile of keys gives scores S = Q K^T, the reference m grows where they pass it (KVQ_HOLD),
// P = exp(S - m) adds to the sum l and to O = P V, and O / l is the output. K and
// V rows come packed; they become fp16 numbers in registers, exactly the values
// the format defines, on their way to the tensor cores.
//
// Three kernels share the work by the number of query rows a KV head has (its
// query heads times the call's tokens): k_kvq_decode for up to 16, where the
// packed bytes bound the time; for more, k_kvq_chunk, and k_kvq_prompt (a file of its own)
// once there is enough to compute for blocks of 256 rows.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "kvq_attn.cuh"
#include "ll_internal.h"

namespace ll {
namespace {

namespace cg = cooperative_groups;

// D += A B: A 16 x 16 (row), B 16 x 8 (col), fp16 in, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values held as an mma fragment, transposed.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// ---- few query rows: one warp per run of keys --------------------------------------
//
// Grid (splits, KV heads, sequences), the splits of a (sequence, KV head) one
// cluster. A block's keys are cut into tiles; its warps take them in turn, each
// with a ring of its own in shared memory, which one lane fills by bulk copies
// (a tile of a head's codes is one run of bytes, its parameters another), and its
// own m, l and O: no block barriers. At the end the warps of a block merge, then the
// blocks of the cluster: each owns a share of the outputs, and sends the others their
// shares of its own (stores into their shared memory, one cluster barrier).
//
// A tile of 16 keys is the A operand of S^T = K Q^T (keys x rows, 8 query rows per
// product) and, transposed, of O^T = V^T P^T (dims x rows): with the keys as the
// operand's 16 rows, every code is unpacked once whatever the number of query
// rows, and few rows cost few products. A group of 4 dims by 8 lanes is how the
// format lays a row out: lane (g, t) finds the dims of its K fragment (k = 2t, 2t +
// 1, 2t + 8, 2t + 9 of each product, in an order of our own that Q's fragment
// shares) in cells 2t and 2t + 1, and those of its V fragment in cell g. What a
// pair of a K fragment holds are the same dim of two neighbouring groups, which
// share a packed word; of a V fragment, one dim of two keys.
//
// What bounds it: where blocks fill the device, the unpacking (8 sequences of 32768, 128 dims in
// 4 bits: the schedulers issue in 58 % of the cycles, the ALU pipe is busy in 48 %); 32 of
// them take 270 us for 1.34 GB, 73 % of the copy rate. Where few do, each
// warp's chain of a tile (0.7 us alone) and start and merge (3 to 5 us): one
// sequence of 32768 positions of 64 dims 12.9 us, of 1024 4.8 us. With two blocks of query
// rows (NC = 2) at 128 dims 260 to 400 bytes a thread are spilled: 4 tokens of 8 ragged
// sequences up to 4097 27 us in 4 bits, 12 at 64 dims.
template <int BITS, int HD, int WARPS>
struct DecodeShape {
    // Blocks of 4, 8 or 16 warps, 16 to an SM: many units of work run best as small blocks (one's start and merge run
    // under the others' tiles: 32 sequences at 32768 positions of 128 dims 266 us, in blocks of 8 warps 271), few as large
    // ones, whose warps a cluster cannot otherwise bring to an SM (decode_plan has the figures).
    static constexpr int NW = WARPS, PER_SM = 16 / WARPS;
    static constexpr int RB = HD * BITS / 8, PB = HD / 8;        // bytes of a row's codes and parameters
    static constexpr int TILE = RB == 128 ? 16 : 32;             // keys
    static constexpr int PAR = TILE * PB + 16;                   // a tile's parameters, from an even row on
    static constexpr int STAGE = 2 * (TILE * RB + PAR);
    static constexpr int ROOM = 208 * 1024 / PER_SM / (NW * STAGE), STAGES = ROOM < 4 ? ROOM : 4;
    static constexpr int SMEM = NW * STAGES * STAGE;
    static_assert(STAGES >= 2, "a ring needs two stages");
};

// The key of a block of 8 that is row r of the operand: rows 2t are keys 0..3 and
// rows 2t + 1 keys 7..4, which spreads both the K reads (rows g) and the V reads
// (rows 2t, then 2t + 1) over the banks (32-byte rows: no conflicts; 64: K none, V
// two to a bank; 128: two and four, with the shared-memory pipe half idle).
__device__ __forceinline__ int key_of(int r) { return r & 1 ? 7 - (r >> 1) : r >> 1; }

template <int BITS, int HD, int WARPS, int NC, typename QT>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) k_kvq_decode(const __grid_constant__ KvqAttnArgs a) {
    using S = DecodeShape<BITS, HD, WARPS>;
    constexpr int NW = S::NW, RB = S::RB, PB = S::PB, TILE = S::TILE, NT = TILE / 16, GR = HD / 32, COLS = 8 * NC;
    constexpr int GP = GR / 2, PAR = S::PAR;  // pairs of groups
    static_assert(NW * COLS * HD * 4 <= S::SMEM, "the merge fits in the ring's memory");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_ml[NW][COLS][2];  // the warps' m and l
    __shared__ __align__(8) float s_recv[COLS * HD + 32];  // the cluster's sums of this block's share of the outputs, by rank (16 shares, rounded up)
    __shared__ __align__(8) float s_rml[16][COLS][2]; // and the ranks' m and l
    __shared__ uint64_t s_full[NW][S::STAGES];
    __shared__ int s_lost[NW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const KvqConsts consts;
    const int s = blockIdx.z, h = blockIdx.y, C = gridDim.x, rank = blockIdx.x;
    // q first, while the lengths are on their way: (nc) row 8 nc + g, this lane's dims 32 gr + 8 t .. (Rows of padded
    // tokens may not exist, so with counts of tokens q waits for its sequence's.)
    const int n = a.l.n(s), len = a.l.len(s), rows = n * a.group;  // rows: of queries
    if (a.l.n_dev && n == 0) return;
    float qv[NC][GR][8];
#pragma unroll
    for (int nc = 0; nc < NC; nc++) {
        const int r = 8 * nc + g;
        const bool ok = r < rows;
        const QT *q = static_cast<const QT *>(a.q) + s * a.q_seq + (ok ? r / a.group : 0) * a.q_tok +
                      (h * a.group + (ok ? r % a.group : 0)) * a.q_head + 8 * t;
#pragma unroll
        for (int gr = 0; gr < GR; gr++) load_q8(q + 32 * gr, qv[nc][gr]);
        if (!ok) {
#pragma unroll
            for (int gr = 0; gr < GR; gr++)
#pragma unroll
                for (int i = 0; i < 8; i++) qv[nc][gr][i] = 0.f;
        }
    }
    const int first = len - n;                      // the first token's position
    const int limit = min(len, a.max_seq);          // no token sees a position from here on
    const int64_t row0 = s * a.seq_rows + int64_t(h) * a.max_seq;
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before the first remote store)

    // this block's tiles
    const int tiles = (limit + TILE - 1) / TILE;
    const int t0 = int(int64_t(tiles) * rank / C), t1 = int(int64_t(tiles) * (rank + 1) / C);
    uint8_t *const ring = smem + warp * (S::STAGES * S::STAGE);
    const uint32_t full = sptr(s_full[warp]);
    // rows of 8 bytes of parameters are copied from a 16-byte border on (skew: the first one's place. By its address, as
    // the arrays of one layer of a handle's cache may begin at an odd row); the row behind the last position of all
    // may not exist, so one in the middle of 16 bytes is fetched when its tile is used
    const int skew = PB == 8 ? int((row0 + int64_t(reinterpret_cast<uintptr_t>(a.kp) / 8)) & 1) : 0;
    const bool odd_end = PB == 8 && limit == a.max_seq && ((skew + limit) & 1);
    const int edge_from = min(first + 1, limit) - int(odd_end);
    // (lane 0; tiles come in order, NW apart: the addresses move by constants)
    const uint8_t *kc = a.kc + (row0 + (t0 + warp) * TILE) * RB, *vc = a.vc + (row0 + (t0 + warp) * TILE) * RB;
    const uint32_t *kp = a.kp + (row0 + (t0 + warp) * TILE - skew) * GR, *vp = a.vp + (row0 + (t0 + warp) * TILE - skew) * GR;
    auto load = [&](int ti, uint32_t dst, uint32_t bar) {
        const int count = min(TILE, limit - ti * TILE);
        uint32_t par = (count + skew) * PB;
        if (PB == 8) par = (odd_end && ti * TILE + count == limit ? par : par + 8) & ~15u;
        bar_expect(bar, 2 * (count * RB + par));
        bulk_copy(dst, kc, count * RB, bar);
        bulk_copy(dst + TILE * RB, vc, count * RB, bar);
        if (PB != 8 || par) {
            bulk_copy(dst + 2 * TILE * RB, kp, par, bar);
            bulk_copy(dst + 2 * TILE * RB + PAR, vp, par, bar);
        }
        kc += NW * TILE * RB;
        vc += NW * TILE * RB;
        kp += NW * TILE * GR;
        vp += NW * TILE * GR;
    };
    const uint32_t ring0 = sptr(ring);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < S::STAGES; i++) bar_init(full + 8 * i, 1);
        s_lost[warp] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n\tfence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; i++)
            if (t0 + warp + i * NW < t1) load(t0 + warp + i * NW, ring0 + i * S::STAGE, full + 8 * i);
    }
    __syncwarp();

    // q as B fragments: (gp, b, i) the pair of dims 64 gp + 4 (2 t + b) + i and 32 on, of row 8 nc + g
    uint32_t qf[NC][GP][2][4];
    float fac[NC][2];  // log2 score units per product unit, of rows 8 nc + 2 t and + 1
    int last[NC][2];   // the last position those rows see
#pragma unroll
    for (int nc = 0; nc < NC; nc++) {
        const float(&v)[GR][8] = qv[nc];
        float mx = 0.f;
#pragma unroll
        for (int gr = 0; gr < GR; gr++)
#pragma unroll
            for (int i = 0; i < 8; i++) mx = fmaxf(mx, fabsf(v[gr][i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float down, up;
        row_scale(mx, down, up);
        up *= a.scale_log2;
        fac[nc][0] = __shfl_sync(0xffffffffu, up, 8 * t);
        fac[nc][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4);
        last[nc][0] = first + (8 * nc + 2 * t) / a.group;
        last[nc][1] = first + (8 * nc + 2 * t + 1) / a.group;
#pragma unroll
        for (int gp = 0; gp < GP; gp++)
#pragma unroll
            for (int i = 0; i < 8; i++) qf[nc][gp][i >> 2][i & 3] = pack_h2(v[2 * gp][i] * down, v[2 * gp + 1][i] * down);
    }

    float o[NC][2 * GR][4], m[NC][2], l[NC][2];
#pragma unroll
    for (int nc = 0; nc < NC; nc++) {
#pragma unroll
        for (int i = 0; i < 2 * GR; i++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[nc][i][e] = 0.f;
        m[nc][0] = m[nc][1] = -INFINITY;
        l[nc][0] = l[nc][1] = 0.f;
    }

    int stage = 0;
    uint32_t phase = 0;  // the parity that the ring's stages complete next
    int load_end = t1;
    bool bad_seen = false;
    for (int ti = t0 + warp; ti < t1; ti += NW) {
        __syncwarp();  // every lane is done with the tile before: its stage is free
        if (lane == 0 && ti + (S::STAGES - 1) * NW < load_end) {
            const int to = stage == 0 ? S::STAGES - 1 : stage - 1;
            load(ti + (S::STAGES - 1) * NW, ring0 + to * S::STAGE, full + 8 * to);
        }
        if (!bar_try(full + 8 * stage, phase) && !copy_wait(full + 8 * stage, phase, a.waits.timeout_ns, &s_lost[warp]))
            load_end = min(load_end, ti + (S::STAGES - 1) * NW + 1);  // (no more copies are made)
        const uint8_t *kt = ring + stage * S::STAGE, *vt = kt + TILE * RB;
        const uint32_t *kpar = reinterpret_cast<const uint32_t *>(vt + TILE * RB) + skew * GR, *vpar = kpar + PAR / 4;
        if (++stage == S::STAGES) {
            stage = 0;
            phase ^= 1;
        }

        // A tile in which some row's last position lies (or the sequence ends). Its keys
        // past the end become zeros. V values there that are not finite must reach only the
        // rows that see them: others enter the product in their place, and the rows that
        // see them get NaN behind the walk.
        const int k0 = ti * TILE;
        const bool edge = k0 + TILE > edge_from;
        if (edge) {
            uint32_t *const ks = const_cast<uint32_t *>(kpar), *const vs = const_cast<uint32_t *>(vpar);
            uint8_t *const vr = const_cast<uint8_t *>(vt) + lane * RB;
            const int valid = limit - k0;
            if (odd_end && valid <= TILE && lane < GR) {
                ks[(valid - 1) * GR + lane] = a.kp[(row0 + limit - 1) * GR + lane];
                vs[(valid - 1) * GR + lane] = a.vp[(row0 + limit - 1) * GR + lane];
            }
            __syncwarp();
            bool bad = false;
            if (lane < TILE) {
#pragma unroll
                for (int gr = 0; gr < GR; gr++) {
                    if (lane < valid)
                        bad |= kvq_not_finite<BITS>(vs[lane * GR + gr]);
                    else
                        ks[lane * GR + gr] = vs[lane * GR + gr] = 0u;
                }
            }
            if (__builtin_expect(__any_sync(0xffffffffu, bad), 0)) {
                bad_seen = true;
#pragma unroll 1
                for (int gr = 0; gr < GR && bad; gr++)
                    if (kvq_not_finite<BITS>(vs[lane * GR + gr])) vs[lane * GR + gr] = kvq_make_finite<BITS, HD>(vr, vs[lane * GR + gr], gr);
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // (the stage is copied into again)
            __syncwarp();
        }

        float sc[NT][NC][4];
#pragma unroll
        for (int mt = 0; mt < NT; mt++) {
#pragma unroll
            for (int nc = 0; nc < NC; nc++)
#pragma unroll
                for (int e = 0; e < 4; e++) sc[mt][nc][e] = 0.f;
            // this lane's quarter of rows g and g + 8: cells 2t and 2t + 1, GR groups each
            uint32_t w[2][RB / 16], par[2][GR];
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                const int r = 16 * mt + 8 * hf + key_of(g);
                if (RB == 32) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(kt + r * RB + 8 * t);
                    w[hf][0] = u.x;
                    w[hf][1] = u.y;
                } else {
#pragma unroll
                    for (int i = 0; i < RB / 64; i++) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(kt + r * RB + RB / 4 * t + 16 * i);
                        w[hf][4 * i] = u.x;
                        w[hf][4 * i + 1] = u.y;
                        w[hf][4 * i + 2] = u.z;
                        w[hf][4 * i + 3] = u.w;
                    }
                }
#pragma unroll
                for (int gr = 0; gr < GR; gr++) par[hf][gr] = kpar[r * GR + gr];
            }
#pragma unroll
            for (int gp = 0; gp < GP; gp++) {
                __half2 lo[2], st[2];
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    lo[hf] = kvq_h2(kvq_prmt(par[hf][2 * gp], par[hf][2 * gp + 1], 0x5410));
                    st[hf] = kvq_h2(kvq_prmt(par[hf][2 * gp], par[hf][2 * gp + 1], 0x7632));
                }
#pragma unroll
                for (int b = 0; b < 2; b++) {
                    __half2 c[2][4];
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        if (BITS == 4)
                            kvq_codes4(w[hf][b * GP + gp], consts, c[hf]);
                        else
                            kvq_codes8(w[hf][b * GR + 2 * gp], w[hf][b * GR + 2 * gp + 1], consts, c[hf]);
#pragma unroll
                        for (int i = 0; i < 4; i++) c[hf][i] = __hfma2(st[hf], c[hf][i], lo[hf]);
                    }
#pragma unroll
                    for (int ks = 0; ks < 2; ks++) {
                        const uint32_t af[4] = {kvq_u32(c[0][2 * ks]), kvq_u32(c[1][2 * ks]), kvq_u32(c[0][2 * ks + 1]),
                                                kvq_u32(c[1][2 * ks + 1])};
#pragma unroll
                        for (int nc = 0; nc < NC; nc++) mma(sc[mt][nc], af, qf[nc][gp][b][2 * ks], qf[nc][gp][b][2 * ks + 1]);
                    }
                }
            }
        }
        // scores of keys past a row's last position leave (the tile's tail holds zeros)
        if (edge) {
#pragma unroll
            for (int mt = 0; mt < NT; mt++)
#pragma unroll
                for (int nc = 0; nc < NC; nc++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int k = k0 + 16 * mt + 8 * (e >> 1) + key_of(g);
                        if (k > last[nc][e & 1] || k >= limit) sc[mt][nc][e] = -INFINITY;
                    }
        }
        bool grow = false;
        float top[NC][2];
#pragma unroll
        for (int nc = 0; nc < NC; nc++)
#pragma unroll
            for (int b = 0; b < 2; b++) {
                float x = sc[0][nc][b];
                x = fmaxf(x, sc[0][nc][2 + b]);
#pragma unroll
                for (int mt = 1; mt < NT; mt++) x = fmaxf(x, fmaxf(sc[mt][nc][b], sc[mt][nc][2 + b]));
                top[nc][b] = __fmul_rn(x, fac[nc][b]);
                grow |= kvq_passes(top[nc][b], m[nc][b]);
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nc = 0; nc < NC; nc++)
#pragma unroll
                for (int b = 0; b < 2; b++) {
                    float x = top[nc][b];
#pragma unroll
                    for (int d = 4; d <= 16; d *= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                    x = fmaxf(m[nc][b], x - KVQ_ROOM);
                    const float al = m[nc][b] == -INFINITY ? 0.f : ex2(m[nc][b] - x);
                    m[nc][b] = x;
                    l[nc][b] *= al;
#pragma unroll
                    for (int i = 0; i < 2 * GR; i++) {
                        o[nc][i][b] *= al;
                        o[nc][i][2 + b] *= al;
                    }
                }
        }
        uint32_t pf[NT][NC][2];  // P^T as B fragments
#pragma unroll
        for (int nc = 0; nc < NC; nc++) {
            const float m0 = m[nc][0] == -INFINITY ? 0.f : m[nc][0], m1 = m[nc][1] == -INFINITY ? 0.f : m[nc][1];
#pragma unroll
            for (int mt = 0; mt < NT; mt++)
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    const float p0 = ex2(kvq_above(sc[mt][nc][2 * hf], fac[nc][0], m0));
                    const float p1 = ex2(kvq_above(sc[mt][nc][2 * hf + 1], fac[nc][1], m1));
                    l[nc][0] += p0;
                    l[nc][1] += p1;
                    pf[mt][nc][hf] = movmatrix(pack_h2(p0, p1));
                }
        }
#pragma unroll
        for (int mt = 0; mt < NT; mt++) {
            // cell g of keys 2t, 2t + 1 (first half) and 2t + 8, 2t + 9 of the operand's order
            uint32_t w[4][RB / 32], par[4][GR];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int r = 16 * mt + 8 * (i >> 1) + key_of(2 * t + (i & 1));
                const uint8_t *p = vt + r * RB;
                if (RB == 32) {
                    w[i][0] = *reinterpret_cast<const uint32_t *>(p + 4 * g);
                } else if (RB == 64) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(p + 8 * g);
                    w[i][0] = u.x;
                    w[i][1 % (RB / 32)] = u.y;
                } else {
                    const uint4 u = *reinterpret_cast<const uint4 *>(p + 16 * g);
                    w[i][0] = u.x;
                    w[i][1 % (RB / 32)] = u.y;
                    w[i][2 % (RB / 32)] = u.z;
                    w[i][3 % (RB / 32)] = u.w;
                }
#pragma unroll
                for (int gr = 0; gr < GR; gr++) par[i][gr] = vpar[r * GR + gr];
            }
#pragma unroll
            for (int gr = 0; gr < GR; gr++) {
                __half2 c[2][4];
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    if (BITS == 4)
                        kvq_codes4(kvq_prmt(w[2 * hf][gr / 2], w[2 * hf + 1][gr / 2], gr & 1 ? 0x7632 : 0x5410), consts, c[hf]);
                    else
                        kvq_codes8(w[2 * hf][gr], w[2 * hf + 1][gr], consts, c[hf]);
                    const __half2 lo = kvq_h2(kvq_prmt(par[2 * hf][gr], par[2 * hf + 1][gr], 0x5410));
                    const __half2 st = kvq_h2(kvq_prmt(par[2 * hf][gr], par[2 * hf + 1][gr], 0x7632));
#pragma unroll
                    for (int i = 0; i < 4; i++) c[hf][i] = __hfma2(st, c[hf][i], lo);
                }
#pragma unroll
                for (int b = 0; b < 2; b++) {  // dims 32 gr + 4 g + 2 b and + 1
                    const uint32_t af[4] = {kvq_u32(c[0][2 * b]), kvq_u32(c[0][2 * b + 1]), kvq_u32(c[1][2 * b]),
                                            kvq_u32(c[1][2 * b + 1])};
#pragma unroll
                    for (int nc = 0; nc < NC; nc++) mma(o[nc][2 * gr + b], af, pf[mt][nc][0], pf[mt][nc][1]);
                }
            }
        }
    }
    if (__builtin_expect(bad_seen, 0)) {  // NaN in the rows that see them (once, behind the walk: in it, 32 sequences of 32768 took 282 us for 271)
#pragma unroll 1
        for (int ti = t0 + warp; ti < t1; ti += NW) {
            if ((ti + 1) * TILE <= edge_from) continue;
            const int k0 = ti * TILE, k_mine = k0 + lane;
#pragma unroll
            for (int gr = 0; gr < GR; gr++) {
                const bool bad = lane < TILE && k_mine < limit && kvq_not_finite<BITS>(a.vp[(row0 + k_mine) * GR + gr]);
#pragma unroll 1
                for (uint32_t keys = __ballot_sync(0xffffffffu, bad); keys; keys &= keys - 1) {
                    const int k = k0 + __ffs(keys) - 1;
                    const uint32_t dims = kvq_not_finite_dims<BITS, HD>(a.vc + (row0 + k) * RB, a.vp[(row0 + k) * GR + gr], gr) >> (4 * g);
#pragma unroll
                    for (int nc = 0; nc < NC; nc++)
#pragma unroll
                        for (int b = 0; b < 2; b++)
#pragma unroll
                            for (int i = 0; i < 4; i++)  // dim 32 gr + 4 g + i
                                if (k <= last[nc][b] && (dims >> i & 1)) o[nc][2 * gr + (i >> 1)][2 * (i & 1) + b] = __uint_as_float(0x7fffffffu);
                }
            }
        }
    }
    __syncwarp();
    if (__builtin_expect(s_lost[warp], 0)) {  // a copy that did not come in time: the rows have no result, and what is in flight lands first
        if (lane == 0) {
            const int end = (load_end - t0 - warp + NW - 1) / NW;  // copies that were made, of this warp's tiles
            for (int i = max(0, end - S::STAGES); i < end; i++) bar_wait_long(full + 8 * (i % S::STAGES), i / S::STAGES & 1, KVQ_DRAIN_NS);
            if (a.waits.status) atomicCAS(a.waits.status, 0, LL_ERR_DEP_TIMEOUT);
        }
#pragma unroll
        for (int nc = 0; nc < NC; nc++)
#pragma unroll
            for (int i = 0; i < 2 * GR; i++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[nc][i][e] = __uint_as_float(0x7fffffffu);
    }
    __syncthreads();  // every ring is read: its memory takes the warps' results

    float *const red = reinterpret_cast<float *>(smem);  // [NW][COLS][HD]
#pragma unroll
    for (int nc = 0; nc < NC; nc++) {
#pragma unroll
        for (int b = 0; b < 2; b++) {
            float x = l[nc][b];
#pragma unroll
            for (int d = 4; d <= 16; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
            const int col = 8 * nc + 2 * t + b;
            if (g == 0) {
                s_ml[warp][col][0] = m[nc][b];
                s_ml[warp][col][1] = x;
            }
#pragma unroll
            for (int i = 0; i < 2 * GR; i++)
                *reinterpret_cast<float2 *>(&red[(warp * COLS + col) * HD + 32 * (i >> 1) + 4 * g + 2 * (i & 1)]) =
                    make_float2(o[nc][i][b], o[nc][i][2 + b]);
        }
    }
    __syncthreads();
    // the block's warps: pairs of dims, NW partial sums each, against the largest m
    const int head0 = h * a.group, pairs = rows * (HD / 2), share = (pairs + C - 1) / C;
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the cluster's blocks have all begun
    cg::cluster_group cl = cg::this_cluster();
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int col = i / (HD / 2), d = 2 * (i % (HD / 2));
        float M = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < NW; w++) M = fmaxf(M, s_ml[w][col][0]);
#pragma unroll
        for (int w = 0; w < NW; w++) {
            // (a warp that saw nothing adds its zeros; a NaN in it stays one)
            const float mw = s_ml[w][col][0], f = mw == -INFINITY ? 0.f : ex2(mw - M);
            const float2 v = *reinterpret_cast<const float2 *>(&red[(w * COLS + col) * HD + d]);
            L = fmaf(s_ml[w][col][1], f, L);
            x = fmaf(v.x, f, x);
            y = fmaf(v.y, f, y);
        }
        if (C == 1) {
            const float inv = M == -INFINITY ? 0.f : 1.f / L;
            put_out(a.out, s, col / a.group, head0 + col % a.group, d, x * inv, y * inv);
        } else {
            const int owner = i / share;
            float2 *to = reinterpret_cast<float2 *>(s_recv) + rank * share + (i - owner * share);
            *cl.map_shared_rank(to, owner) = make_float2(x, y);
        }
    }
    if (C == 1) return;
    for (int i = threadIdx.x; i < rows * C; i += blockDim.x) {  // every block gets every row's m and l
        const int col = i / C;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < NW; w++) M = fmaxf(M, s_ml[w][col][0]);
#pragma unroll
        for (int w = 0; w < NW; w++)
            L = fmaf(s_ml[w][col][1], s_ml[w][col][0] == -INFINITY ? 0.f : ex2(s_ml[w][col][0] - M), L);
        *reinterpret_cast<float2 *>(cl.map_shared_rank(&s_rml[rank][col][0], i % C)) = make_float2(M, L);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    for (int k = threadIdx.x; k < share && rank * share + k < pairs; k += blockDim.x) {
        const int i = rank * share + k, col = i / (HD / 2), d = 2 * (i % (HD / 2));
        float M = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
        for (int c = 0; c < C; c++) M = fmaxf(M, s_rml[c][col][0]);
#pragma unroll 4
        for (int c = 0; c < C; c++) {
            const float mc = s_rml[c][col][0], f = mc == -INFINITY ? 0.f : ex2(mc - M);
            const float2 v = reinterpret_cast<const float2 *>(s_recv)[c * share + k];
            L = fmaf(s_rml[c][col][1], f, L);
            x = fmaf(v.x, f, x);
            y = fmaf(v.y, f, y);
        }
        const float inv = M == -INFINITY ? 0.f : 1.f / L;
        put_out(a.out, s, col / a.group, head0 + col % a.group, d, x * inv, y * inv);
    }
}

// ---- many query rows ---------------------------------------------------------------
//
// Grid (splits x row tiles, KV heads, sequences). A block takes 64 query rows of
// a KV head (row = token * group + head), 16 to a warp, and walks the keys in
// tiles of 64: all four warps unpack a tile of K and V into fp16 in shared
// memory, then each takes it to the tensor cores as B operands (S = Q K^T, O = P V).
// A packed word (pair of cells of neighbouring groups) becomes one 16-byte chunk
// of a shared-memory row, its dims in the order the unpacking leaves them; q is
// read in the same order, and O leaves through it. Its calls are short: start, merge and the
// unpacking of each tile before its products bound it (8 heads of 64 dims, 128 rows
// by 4096 keys: 15.5 us).
constexpr int CK_ROWS = 64, CK_KEYS = 64, CK_THREADS = 128;

// dim of element p (0..HD) of a shared-memory row
template <int HD>
__device__ __forceinline__ int dim_of(int p) {
    constexpr int GP = HD / 64;  // pairs of groups
    const int q = p >> 3;
    return 32 * (2 * (q % GP) + (p & 1)) + 4 * (q / GP) + ((p & 7) >> 1);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <int BITS, int HD, typename QT>
__global__ void __launch_bounds__(CK_THREADS) k_kvq_chunk(const __grid_constant__ KvqAttnArgs a, int C) {
    constexpr int GR = HD / 32, GP = HD / 64, CH = HD / 8, KS = HD / 16;  // 16-byte chunks of a row, k-steps
    constexpr int PER = CK_KEYS * CH / CK_THREADS;                        // chunks a thread unpacks, of K and of V
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const ks = smem, *const vs = smem + CK_KEYS * HD * 2;  // [key][HD] fp16, chunk c of row r at c ^ (r & 7)
    __shared__ float s_ml[CK_ROWS][2];
    __shared__ uint32_t s_bad[GR][2];  // keys of the tile whose V may not be finite, per group
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const KvqConsts consts;
    const int s = blockIdx.z, h = blockIdx.y, rank = blockIdx.x % C;
    const int n = a.l.n(s), len = a.l.len(s), rows = n * a.group, first = len - n;
    // the row tiles with the most keys come first
    const int r0 = (int(gridDim.x) / C - 1 - int(blockIdx.x) / C) * CK_ROWS;
    if (r0 >= rows) return;
    const int row_hi = min(r0 + CK_ROWS, rows) - 1;
    const int limit = max(0, min(min(len, a.max_seq), first + row_hi / a.group + 1));  // the tile's rows see keys below
    const int first_last = first + r0 / a.group;                                       // the last position the first row sees
    const int64_t krow = s * a.seq_rows + int64_t(h) * a.max_seq;
    const int tiles = (limit + CK_KEYS - 1) / CK_KEYS;
    const int t0 = int(int64_t(tiles) * rank / C), t1 = int(int64_t(tiles) * (rank + 1) / C);

    // q as A fragments of this warp's rows g and g + 8
    uint32_t qf[KS][4];
    float fac[2];
    int last[2];
#pragma unroll
    for (int b = 0; b < 2; b++) {
        const int r = r0 + warp * 16 + 8 * b + g;
        const int j = r / a.group;
        last[b] = first + j;
        float v[KS][4], mx = 0.f;
        const QT *q = static_cast<const QT *>(a.q) + s * a.q_seq + int64_t(j) * a.q_tok + int64_t(h * a.group + r % a.group) * a.q_head;
#pragma unroll
        for (int k = 0; k < KS; k++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                v[k][e] = r < rows ? q_at(q + dim_of<HD>(16 * k + 2 * t + (e & 1) + 8 * (e >> 1))) : 0.f;
                mx = fmaxf(mx, fabsf(v[k][e]));
            }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float down, up;
        row_scale(mx, down, up);
        fac[b] = up * a.scale_log2;
#pragma unroll
        for (int k = 0; k < KS; k++) {
            qf[k][b] = pack_h2(v[k][0] * down, v[k][1] * down);
            qf[k][2 + b] = pack_h2(v[k][2] * down, v[k][3] * down);
        }
    }
    float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < HD / 8; d++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[d][e] = 0.f;

    // a tile's packed words, in registers one tile ahead
    uint2 w[2][PER];
    uint32_t par[2][PER][2];
    auto fetch = [&](int ti) {
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int at = threadIdx.x + i * CK_THREADS, r = at / CH, c = at % CH, key = ti * CK_KEYS + r;
            const bool ok = key < limit;
            const int64_t row = krow + (ok ? key : 0);
#pragma unroll
            for (int kv = 0; kv < 2; kv++) {
                const uint8_t *codes = kv ? a.vc : a.kc;
                const uint32_t *pp = (kv ? a.vp : a.kp) + row * GR + 2 * (c % GP);
                w[kv][i] = make_uint2(0, 0);
                par[kv][i][0] = par[kv][i][1] = 0;
                if (ok) {
                    if (BITS == 4)
                        w[kv][i].x = reinterpret_cast<const uint32_t *>(codes)[row * CH + c];
                    else
                        w[kv][i] = reinterpret_cast<const uint2 *>(codes)[row * CH + c];
                    const uint2 u = *reinterpret_cast<const uint2 *>(pp);
                    par[kv][i][0] = u.x;
                    par[kv][i][1] = u.y;
                }
            }
        }
    };
    if (t0 < t1) fetch(t0);
    for (int ti = t0; ti < t1; ti++) {
        const int k0 = ti * CK_KEYS;
        const bool edge = k0 + CK_KEYS > min(first_last + 1, limit);
        __syncthreads();  // every warp is done with the tile before
        if (edge && threadIdx.x < 2 * GR) s_bad[threadIdx.x >> 1][threadIdx.x & 1] = 0;
        if (edge) __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int at = threadIdx.x + i * CK_THREADS, r = at / CH, c = at % CH;
#pragma unroll
            for (int kv = 0; kv < 2; kv++) {
                const uint32_t p0 = par[kv][i][0], p1 = par[kv][i][1];
                bool bad = false;
                if (kv && edge) {  // (see k_kvq_decode: V that is not finite reaches only the rows that see it)
                    const bool b0 = kvq_not_finite<BITS>(p0), b1 = kvq_not_finite<BITS>(p1);
                    if (b0) atomicOr(&s_bad[2 * (c % GP)][r >> 5], 1u << (r & 31));
                    if (b1) atomicOr(&s_bad[2 * (c % GP) + 1][r >> 5], 1u << (r & 31));
                    bad = b0 || b1;
                }
                __half2 v[4];
                if (BITS == 4)
                    kvq_codes4(w[kv][i].x, consts, v);
                else
                    kvq_codes8(w[kv][i].x, w[kv][i].y, consts, v);
                const __half2 lo = kvq_h2(kvq_prmt(p0, p1, 0x5410)), st = kvq_h2(kvq_prmt(p0, p1, 0x7632));
                uint4 u;
                u.x = kvq_u32(__hfma2(st, v[0], lo));
                u.y = kvq_u32(__hfma2(st, v[1], lo));
                u.z = kvq_u32(__hfma2(st, v[2], lo));
                u.w = kvq_u32(__hfma2(st, v[3], lo));
                if (bad) u = make_uint4(kvq_finite2(u.x), kvq_finite2(u.y), kvq_finite2(u.z), kvq_finite2(u.w));
                *reinterpret_cast<uint4 *>((kv ? vs : ks) + (r * CH + (c ^ (r & 7))) * 16) = u;
            }
        }
        if (ti + 1 < t1) fetch(ti + 1);
        __syncthreads();

        float sc[CK_KEYS / 8][4];
#pragma unroll
        for (int nb = 0; nb < CK_KEYS / 8; nb++)
#pragma unroll
            for (int e = 0; e < 4; e++) sc[nb][e] = 0.f;
#pragma unroll
        for (int nb = 0; nb < CK_KEYS / 16; nb++) {
            const int r = 16 * nb + 8 * (lane >> 4) + (lane & 7);
#pragma unroll
            for (int k = 0; k < KS; k++) {
                uint32_t b[4];
                const int c = 2 * k + ((lane >> 3) & 1);
                ldsm4(sptr(ks + (r * CH + (c ^ (r & 7))) * 16), b);
                mma(sc[2 * nb], qf[k], b[0], b[1]);
                mma(sc[2 * nb + 1], qf[k], b[2], b[3]);
            }
        }
        if (edge) {
#pragma unroll
            for (int nb = 0; nb < CK_KEYS / 8; nb++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int k = k0 + 8 * nb + 2 * t + (e & 1);
                    if (k > last[e >> 1] || k >= limit) sc[nb][e] = -INFINITY;
                }
        }
        bool grow = false;
        float top[2];
#pragma unroll
        for (int b = 0; b < 2; b++) {
            float x = -INFINITY;
#pragma unroll
            for (int nb = 0; nb < CK_KEYS / 8; nb++) x = fmaxf(x, fmaxf(sc[nb][2 * b], sc[nb][2 * b + 1]));
            top[b] = __fmul_rn(x, fac[b]);
            grow |= kvq_passes(top[b], m[b]);
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int b = 0; b < 2; b++) {
                float x = top[b];
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                x = fmaxf(m[b], x - KVQ_ROOM);
                const float al = m[b] == -INFINITY ? 0.f : ex2(m[b] - x);
                m[b] = x;
                l[b] *= al;
#pragma unroll
                for (int d = 0; d < HD / 8; d++) {
                    o[d][2 * b] *= al;
                    o[d][2 * b + 1] *= al;
                }
            }
        }
        const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int nb = 0; nb < CK_KEYS / 8; nb++) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                sc[nb][e] = ex2(kvq_above(sc[nb][e], fac[e >> 1], e < 2 ? m0 : m1));
                l[e >> 1] += sc[nb][e];
            }
        }
#pragma unroll
        for (int nb = 0; nb < CK_KEYS / 16; nb++) {
            const uint32_t pf[4] = {pack_h2(sc[2 * nb][0], sc[2 * nb][1]), pack_h2(sc[2 * nb][2], sc[2 * nb][3]),
                                    pack_h2(sc[2 * nb + 1][0], sc[2 * nb + 1][1]), pack_h2(sc[2 * nb + 1][2], sc[2 * nb + 1][3])};
            const int r = 16 * nb + 8 * ((lane >> 3) & 1) + (lane & 7);
#pragma unroll
            for (int d = 0; d < HD / 16; d++) {
                uint32_t b[4];
                const int c = 2 * d + (lane >> 4);
                ldsm4t(sptr(vs + (r * CH + (c ^ (r & 7))) * 16), b);
                mma(o[2 * d], pf, b[0], b[1]);
                mma(o[2 * d + 1], pf, b[2], b[3]);
            }
        }
        if (edge) {  // element 8 d + 2 t + e of a row is dim 4 (d / GP) + t of group 2 (d % GP) + e
#pragma unroll
            for (int gr = 0; gr < GR; gr++)
                for (uint64_t keys = uint64_t(s_bad[gr][1]) << 32 | s_bad[gr][0]; keys; keys &= keys - 1) {
                    const int k = k0 + __ffsll(keys) - 1;
                    const uint32_t dims = kvq_not_finite_dims<BITS, HD>(a.vc + (krow + k) * (HD * BITS / 8), a.vp[(krow + k) * GR + gr], gr) >> t;
#pragma unroll
                    for (int d = gr / 2; d < HD / 8; d += GP)
#pragma unroll
                        for (int b = 0; b < 2; b++)
                            if (k <= last[b] && (dims >> (4 * (d / GP)) & 1)) o[d][2 * b + (gr & 1)] = __uint_as_float(0x7fffffffu);
                }
        }
    }
#pragma unroll
    for (int b = 0; b < 2; b++) {
        l[b] += __shfl_xor_sync(0xffffffffu, l[b], 1);
        l[b] += __shfl_xor_sync(0xffffffffu, l[b], 2);
    }
    const int head0 = h * a.group;
    float *const red = reinterpret_cast<float *>(smem);  // [CK_ROWS][HD], dims in their own order
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 2; b++) {
        const int r = warp * 16 + 8 * b + g;
        const float f = C > 1 ? 1.f : m[b] == -INFINITY ? 0.f : 1.f / l[b];
#pragma unroll
        for (int d = 0; d < HD / 8; d++)
#pragma unroll
            for (int e = 0; e < 2; e++) red[r * HD + dim_of<HD>(8 * d + 2 * t + e)] = o[d][2 * b + e] * f;
        if (t == 0) {
            s_ml[r][0] = m[b];
            s_ml[r][1] = l[b];
        }
    }
    const int live = min(CK_ROWS, rows - r0) * (HD / 2);
    if (C == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < live; i += CK_THREADS) {
            const int r = i / (HD / 2), d = 2 * (i % (HD / 2)), R = r0 + r;
            put_out(a.out, s, R / a.group, head0 + R % a.group, d, red[r * HD + d], red[r * HD + d + 1]);
        }
        return;
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    for (int i = rank * CK_THREADS + int(threadIdx.x); i < live; i += C * CK_THREADS) {
        const int r = i / (HD / 2), d = 2 * (i % (HD / 2)), R = r0 + r;
        float M = -INFINITY, L = 0.f, x = 0.f, y = 0.f;
        for (int c = 0; c < C; c++) {
            const float *ml = cl.map_shared_rank(&s_ml[r][0], c);
            const float mc = ml[0], lc = ml[1];
            const float2 v = *reinterpret_cast<const float2 *>(cl.map_shared_rank(&red[r * HD + d], c));
            const float Mn = fmaxf(M, mc);
            const float f0 = M == -INFINITY ? 0.f : ex2(M - Mn), f1 = mc == -INFINITY ? 0.f : ex2(mc - Mn);
            L = L * f0 + lc * f1;
            x = x * f0 + v.x * f1;
            y = y * f0 + v.y * f1;
            M = Mn;
        }
        const float inv = M == -INFINITY ? 0.f : 1.f / L;
        put_out(a.out, s, R / a.group, head0 + R % a.group, d, x * inv, y * inv);
    }
    cl.sync();
}

// ---- launches ----------------------------------------------------------------------

// The chunk kernel's splits of one unit of work (a power of two, at most 16: a cluster) for
// `units` units whose longest walk has `steps` key tiles, with `slots` blocks on the device:
// the fewest of a block's own steps and the device's share of all blocks' steps
// together. A block's start and merge take as long as EXTRA steps, and a step on
// a full SM twice as long as on one that holds a single block. Of 22 layouts measured (64 to
// 256 rows by 512 to 20000 keys) it was within 13 % of the best of 1, 2, 4, 8 and 16 in all,
// within 5 % in 17.
int splits_for(int64_t units, int slots, double steps) {
    constexpr double EXTRA = 4;
    int best = 1;
    double least = 0;
    for (int c = 1; c <= 16; c *= 2) {
        const double time = steps / c + EXTRA + 2.0 * double(units) * (steps + EXTRA * c) / slots;
        if (c == 1 || time < least) {
            least = time;
            best = c;
        }
    }
    return best;
}

// How the decode kernel cuts `seqs` x `heads` units of up to `keys` keys: warps of a
// block, and blocks that share a unit. slots: the blocks that the device holds at once
// with one, two and four of them (of 16, 8 and 4 warps) to an SM.
//
// The fewest microseconds, by what was measured: a warp's step (a tile) takes 0.45 +
// 0.06 x the warps that its SM holds where it is 32 keys of 64 dims or 16 of 128, 0.62 +
// 0.107 x for 32 of 128; start and merge 3.4 + 0.07 a warp, and 0.9 more where SMs hold
// several blocks; more blocks than fit run in rounds, the last of them with what is left. As
// lengths may differ, half of that is added, or the time of one long sequence alone if that is
// more. Of 128 layouts measured (2 to 1024 units of 512 to 131072 keys, uniform and ragged, one
// token and a few) it was within 10 % of the best of all warps and splits in 123, 18 % off at worst. A sequence of 32768 keys, 8 heads of 64 dims in 4
// bits: 12.6 us in 12 splits of 16 warps (18.1 in 16 of 4: a device of 152 SMs holds only
// seven clusters of 16 without two blocks on an SM); 32 of them, 128 dims in 8 bits: 373 us in 4 splits
// of 4 warps (397 in 16, 481 in one).
struct DecodePlan {
    int warps, splits;
};
DecodePlan decode_plan(int seqs, int heads, const KvqSlots *const (&slots)[3], int keys, int tile, int tile_values) {
    const double fixed = tile_values > 2048 ? 0.62 : 0.45, per_warp = tile_values > 2048 ? 0.107 : 0.06;
    const int64_t units = int64_t(seqs) * heads;
    const int tiles = (keys + tile - 1) / tile;
    DecodePlan best = {4, 1};
    double least = 0;
    for (int v = 2; v >= 0; v--)
        for (int i = 0; i < KVQ_CLUSTER_SIZES; i++) {
            const int c = KVQ_CLUSTERS[i], warps = 16 >> v, room = slots[v]->n[i];
            if (room < 1) continue;
            const int steps = ((tiles + c - 1) / c + warps - 1) / warps;
            const double start = 3.4 + 0.07 * warps, full = start + steps * (fixed + per_warp * 16);
            auto time = [&](int64_t n) {
                const int64_t rounds = n * c < room ? 0 : n * c / room;
                const int rest = int(n * c - rounds * room);
                if (!rest) return rounds * full;
                const int per_sm = rest <= slots[0]->n[i] ? 1 : rest <= slots[1]->n[i] ? 2 : 4 * rest <= 3 * slots[2]->n[i] ? 3 : 4;
                return rounds * full + start + (per_sm > 1 ? 0.9 : 0.) + steps * (fixed + per_warp * warps * per_sm);
            };
            const double all = time(units), t = all + std::max(all / 2, time(heads));
            if (least == 0 || t < least) {
                least = t;
                best = {warps, c};
            }
        }
    return best;
}

template <int BITS, int HD, int WARPS, int NC, typename QT>
const KvqSlots &decode_slots(int nsm, int dev) {
    constexpr auto kernel = k_kvq_decode<BITS, HD, WARPS, NC, QT>;
    constexpr int SMEM = DecodeShape<BITS, HD, WARPS>::SMEM;
    static const KvqSlots none = {};
    return prepared<kernel>(SMEM, dev) ? kvq_slots<kernel>(WARPS * 32, SMEM, nsm, dev) : none;
}
template <int BITS, int HD, int WARPS, int NC, typename QT>
int decode_launch(const ll_kvq_cache &c, const KvqAttnArgs &a, int splits, int dev, cudaStream_t st) {
    constexpr auto kernel = k_kvq_decode<BITS, HD, WARPS, NC, QT>;
    constexpr int SMEM = DecodeShape<BITS, HD, WARPS>::SMEM;
    if (!prepared<kernel>(SMEM, dev)) return LL_ERR_CUDA;
    return kvq_launch(kernel, dim3(splits, c.n_kv_heads, c.n_seq), WARPS * 32, SMEM, splits, st, a);
}

}  // namespace

int launch_kvq_attention(const ll_kvq_cache &c, const ll_kvq_rows &q, int type, int n_q_heads, const KvqLens &l,
                         int max_len, float scale, const KvqOut &out, const KvqWaits &waits, int nsm, cudaStream_t st) {
    KvqAttnArgs a;
    a.kc = c.k_codes;
    a.vc = c.v_codes;
    a.kp = reinterpret_cast<const uint32_t *>(c.k_params);
    a.vp = reinterpret_cast<const uint32_t *>(c.v_params);
    a.seq_rows = c.seq_rows;
    a.max_seq = c.max_seq;
    a.group = n_q_heads / c.n_kv_heads;
    a.nkv = c.n_kv_heads;
    a.l = l;
    a.q = q.data;
    a.q_seq = q.seq;
    a.q_tok = q.token;
    a.q_head = q.head;
    a.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(float(c.head_dim))) * 1.4426950408889634f;
    a.out = out;
    a.waits = waits;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return LL_ERR_CUDA;
    const int longest = max_len > 0 ? std::min(max_len, c.max_seq) : c.max_seq;
    const int rows = l.n_tok * a.group;
    const int64_t pairs = int64_t(c.n_seq) * c.n_kv_heads;
    // The prompt kernel does a pair of row and key in a quarter of the chunk kernel's time but takes 7 us longer to start
    // and merge: at 64 dims 4 to 16 million pairs take as long either way (8 heads, 128 rows by 4096 keys: 15.5 us and
    // 15.8; 512 by 4096: 37 and 25), at 128 dims half as many.
    if (rows > 16 && double(pairs) * rows * longest * (c.head_dim / 64) >= double(8 << 20))
        return launch_kvq_prompt(c, a, type, longest, nsm, dev, st);
    int rc = LL_OK;
    kvq_dispatch(c, [&](auto bits, auto hd) {
        constexpr int B = bits.value, H = hd.value;
        auto typed = [&](auto qt) {
            using QT = decltype(qt);
            if (rows <= 16) {
                auto go = [&](auto nc) {
                    constexpr int tile = DecodeShape<B, H, 4>::TILE;
                    const KvqSlots *const slots[3] = {&decode_slots<B, H, 16, nc.value, QT>(nsm, dev), &decode_slots<B, H, 8, nc.value, QT>(nsm, dev),
                                                &decode_slots<B, H, 4, nc.value, QT>(nsm, dev)};
                    const DecodePlan plan = decode_plan(c.n_seq, c.n_kv_heads, slots, longest, tile, H * tile);
                    if (plan.warps == 16)
                        rc = decode_launch<B, H, 16, nc.value, QT>(c, a, plan.splits, dev, st);
                    else if (plan.warps == 8)
                        rc = decode_launch<B, H, 8, nc.value, QT>(c, a, plan.splits, dev, st);
                    else
                        rc = decode_launch<B, H, 4, nc.value, QT>(c, a, plan.splits, dev, st);
                };
                if (rows <= 8)
                    go(KvqConst<1>{});
                else
                    go(KvqConst<2>{});
            } else {
                constexpr int SMEM = 2 * CK_KEYS * H * 2;
                static_assert(CK_ROWS * H * 4 <= SMEM, "the merge fits in the tiles' memory");
                const int rt = (rows + CK_ROWS - 1) / CK_ROWS;
                const int C = splits_for(pairs * rt, 2 * nsm, double(longest) / CK_KEYS);
                constexpr auto kernel = k_kvq_chunk<B, H, QT>;
                rc = prepared<kernel>(SMEM, dev)
                         ? kvq_launch(kernel, dim3(rt * C, c.n_kv_heads, c.n_seq), CK_THREADS, SMEM, C, st, a, C)
                         : LL_ERR_CUDA;
            }
        };
        if (type == LL_F32)
            typed(float{});
        else
            typed(__nv_bfloat16{});
    });
    return rc;
}

}  // namespace ll

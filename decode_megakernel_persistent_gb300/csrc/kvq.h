// kvq.h -- the packed KV cache's structures and launchers inside libll.so
// (kvq.cu: writing and reading rows, and the C entries; kvq_attn.cu: attention
// over the rows). include/ll.h describes the format and the calls.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ll.h"

namespace ll {

// Which rows a call is about: sequence s holds len(s) positions with the call's
// n(s) <= n_tok tokens as the last of them, token j at position len - n + j.
// len_dev / n_dev are device arrays, or null for len_host / n_tok in every sequence.
struct KvqLens {
    const int32_t *len_dev;
    const int32_t *n_dev;
    int32_t len_host;
    int32_t n_tok;
#ifdef __CUDACC__
    __device__ __forceinline__ int n(int s) const { return n_dev ? min(max(n_dev[s], 0), n_tok) : n_tok; }
    __device__ __forceinline__ int len(int s) const { return max(len_dev ? len_dev[s] : len_host, 0); }
#endif
};

// Where an attention call's output goes: bf16 rows, or (the prefill) fp32 values
// as three bf16 terms each, for the O projection's GEMM.
struct KvqOut {
    uint16_t *t[3];
    int64_t seq, token, head;
    float *f32;  // fp32 rows instead, or null
};

// How long a kernel waits for a copy or a product of its own, and the handle's status word that
// records LL_ERR_DEP_TIMEOUT when one has not come by then (null: the rows' NaN are all that tells).
struct KvqWaits {
    uint64_t timeout_ns = 1000000000ull;
    int32_t *status = nullptr;
};

// f(bits, head_dim) with both as compile-time constants.
template <int V>
struct KvqConst {
    static constexpr int value = V;
};
template <typename F>
void kvq_dispatch(const ll_kvq_cache &c, F &&f) {
    if (c.bits == 4)
        c.head_dim == 64 ? f(KvqConst<4>{}, KvqConst<64>{}) : f(KvqConst<4>{}, KvqConst<128>{});
    else
        c.head_dim == 64 ? f(KvqConst<8>{}, KvqConst<64>{}) : f(KvqConst<8>{}, KvqConst<128>{});
}

// All return LL_OK or LL_ERR_CUDA; arguments are already checked.
int launch_kvq_write(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, int type, const KvqLens &l,
                     cudaStream_t st);
int launch_kvq_read(const ll_kvq_cache &c, const ll_kvq_rows &k, const ll_kvq_rows &v, const KvqLens &l, cudaStream_t st);
// q: bf16 (type LL_BF16) or fp32 rows. max_len: the longest length the launch is laid out for.
int launch_kvq_attention(const ll_kvq_cache &c, const ll_kvq_rows &q, int type, int n_q_heads, const KvqLens &l,
                         int max_len, float scale, const KvqOut &out, const KvqWaits &waits, int nsm, cudaStream_t st);

// Sequence s of the cache alone. Its parameters may begin 8 bytes off a 16-byte border (64 dims, an odd row).
inline ll_kvq_cache kvq_sequence(const ll_kvq_cache &c, int s) {
    ll_kvq_cache one = c;
    const int64_t row = s * c.seq_rows, codes = row * (c.head_dim * c.bits / 8), params = row * (c.head_dim / 16);
    one.n_seq = 1;
    one.k_codes += codes;
    one.v_codes += codes;
    one.k_params += params;
    one.v_params += params;
    return one;
}

// The cache's own checks (shape, pointers), as every entry point makes them:
// LL_OK, or the code with a reason in msg.
int kvq_check_cache(const ll_kvq_cache *c, const char *&msg);

}  // namespace ll

"""Attention over the packed KV cache at the edges of its contract: what a call may not
read, values that are not finite, long contexts whose every key has to count."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll
import kvq_ref
from test_gpu_kvq import check_attention, gen, i32, make_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_megakernel_persistent_gb300 import build
    build.build()


@pytest.mark.parametrize("T,group,cap", [(1, 4, 300), (4, 4, 300), (2, 5, 40000), (40, 2, 300), (300, 4, 9000)])
@pytest.mark.parametrize("hd", [64, 128])
def test_query_storage_that_ends_with_the_last_token(T, group, cap, hd):
    """Rows of padded tokens and free places need not exist: q holds what the sequences have, and
    out is written there alone. (What lies around it, in the same allocation, is marked.)"""
    KV, M, S = 2, 300, 4
    H = KV * group
    n, lens = [0, T, (T + 1) // 2, 0], [0, M, 200, 0]
    c, kv, vv = make_cache(31, S, KV, M, hd, 4, lens, cap)
    q = torch.randn(S, T, H, hd, generator=gen(1), device="cuda").bfloat16()
    row = H * hd
    first, end = T * row, (T + n[1] + n[2]) * row  # sequence 1's tokens, then sequence 2's: places 0 and 3 have nothing
    store, got = (torch.full((end + 4 * T * row,), x, dtype=torch.bfloat16, device="cuda") for x in (float("nan"), 5.0))
    for s, at in ((1, first), (2, first + T * row)):
        store[at:at + n[s] * row] = q[s, :n[s]].flatten()
    rows = [ll.ll_kvq_rows(t.data_ptr(), T * row, row, hd) for t in (store, got)]
    lens_dev, n_dev = i32(lens), i32(n)
    err = ctypes.create_string_buffer(200)
    rc = ll.lib().ll_kvq_attention(c.ref, ctypes.byref(rows[0]), H, T, lens_dev.data_ptr(), n_dev.data_ptr(), 0, 0.0, ctypes.byref(rows[1]),
                                   torch.cuda.current_stream().cuda_stream, err, 200)
    assert rc == ll.LL_OK, err.value
    out = torch.full_like(q, 9.0)
    for s, at in ((1, first), (2, first + T * row)):
        out[s, :n[s]] = got[at:at + n[s] * row].view(n[s], H, hd)
    check_attention(c, kv, vv, q, lens, n, out, mark=9.0)
    assert bool((got[:first] == 5).all()) and bool((got[end:] == 5).all())


@pytest.mark.parametrize("T,group,L,cap", [(1, 4, 1, 32), (1, 4, 40, 40), (1, 4, 5000, 5000), (2, 8, 600, 600), (40, 2, 700, 700), (24, 4, 900, 60000),
                                           (300, 4, 5000, 5000), (300, 4, 5000, 40000)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("x", [12, 20, 26, 30])
def test_many_small_weights_behind_a_dominant_key(T, group, L, cap, hd, x):
    """The first key outweighs each of the others 2^x times, and only the others have a V: the output is
    what they add up to. K and V are values that the packed rows hold exactly, the scores 0 and x log2 units."""
    KV, M = 2, L + T
    c = ll.KVQCache.empty(1, KV, max(M, cap), hd, 4)
    k, v = torch.zeros(1, M, KV, hd, device="cuda"), torch.ones(1, M, KV, hd, device="cuda")
    k[0, 0, :, :32] = 1.0
    v[0, 0] = 0.0
    c.write(k, v, i32([M]))
    q = torch.ones(1, T, KV * group, hd, device="cuda").bfloat16()
    out = c.attention(q, i32([M]), scale=x * 0.6931471805599453 / 32).double()
    others = (L + torch.arange(T, device="cuda", dtype=torch.float64)) * 2.0 ** -x  # (token t sees L + t of them)
    want = (others / (1 + others))[None, :, None, None]
    # bf16's rounding; a probability's to fp16, 2^-11 of it or half of fp16's smallest step, where the first key's is
    # 2^7 at least; scores (exact products, one fp32 factor) and exp2 within 2^-18 at 30 log2 units
    tol = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** (x - 32) + 2.0 ** -18
    off = (out - want).abs() / want
    assert float(off.max()) <= tol, float(off.max())

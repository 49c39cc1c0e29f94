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

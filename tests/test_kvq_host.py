"""The packed KV cache without a GPU: the structures' layout, what the C entries
and the binding refuse before anything is launched, and the definition's own
closed forms."""
import ctypes
import os
import subprocess

import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import build as llbuild
from decode_megakernel_persistent_gb300 import ll
import kvq_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    llbuild.build()
    return ll.lib()


def test_struct_layout_matches_c(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text(r'''
#include <stdio.h>
#include <stddef.h>
#include "ll.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu\n", sizeof(ll_kvq_cache), offsetof(ll_kvq_cache, seq_rows), offsetof(ll_kvq_cache, bits),
         sizeof(ll_kvq_rows), offsetof(ll_kvq_rows, head));
  return 0;
}
''')
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    want = [ctypes.sizeof(ll.ll_kvq_cache), ll.ll_kvq_cache.seq_rows.offset, ll.ll_kvq_cache.bits.offset,
            ctypes.sizeof(ll.ll_kvq_rows), ll.ll_kvq_rows.head.offset]
    assert got == want
    want = ll.ll_kvq_rows(4096, 3, -5, 1 << 40)  # as the binding packs it
    assert ll._rows_bytes(4096, 3, -5, 1 << 40) == ctypes.string_at(ctypes.addressof(want), ctypes.sizeof(want))


def cache(**k):
    d = dict(k_codes=4096, v_codes=8192, k_params=16384, v_params=32768, seq_rows=64, n_seq=2, n_kv_heads=2, head_dim=64,
             max_seq=32, bits=4)
    d.update(k)
    return ll.ll_kvq_cache(**d)


def rows(**k):
    d = dict(data=65536, seq=1024, token=128, head=64)
    d.update(k)
    return ll.ll_kvq_rows(**d)


def call(lib, name, c, r=None, r2=None, n_tok=1, lens=64, n_toks=None, kind=0, heads=4, scale=0.0, max_len=0, err=True):
    r, r2 = r if r is not None else rows(), r2 if r2 is not None else rows()
    buf = ctypes.create_string_buffer(200) if err else None
    tail = (None, buf, 200 if err else 0)
    cp = ctypes.byref(c) if c is not None else None
    a, b = ctypes.byref(r), ctypes.byref(r2)
    if name == "write":
        rc = lib.ll_kvq_write(cp, a, b, kind, n_tok, lens, n_toks, *tail)
    elif name == "read":
        rc = lib.ll_kvq_read(cp, a, b, n_tok, lens, n_toks, *tail)
    else:
        rc = lib.ll_kvq_attention(cp, a, heads, n_tok, lens, n_toks, max_len, scale, b, *tail)
    return rc, buf.value.decode() if err else ""


CALLS = ("write", "read", "attention")


@pytest.mark.parametrize("name", CALLS)
def test_caches_that_are_refused(lib, name):
    assert call(lib, name, None)[0] == ll.LL_ERR_ARG
    for k in (dict(bits=3), dict(bits=16), dict(head_dim=96), dict(n_seq=0), dict(n_seq=65536), dict(n_kv_heads=0),
              dict(n_kv_heads=32768), dict(max_seq=0)):
        rc, msg = call(lib, name, cache(**k))
        assert rc == ll.LL_ERR_SHAPE and list(k)[0] in msg, (k, rc, msg)
    for k in (dict(seq_rows=63), dict(k_codes=None), dict(v_codes=8200), dict(k_params=16388), dict(v_params=None)):
        rc, msg = call(lib, name, cache(**k))
        assert rc == ll.LL_ERR_ARG and msg, (k, rc)
    assert call(lib, name, cache(bits=5), err=False)[0] == ll.LL_ERR_SHAPE  # no buffer for the reason


@pytest.mark.parametrize("name", CALLS)
def test_arguments_that_are_refused(lib, name):
    c = cache()
    assert call(lib, name, c, n_tok=0)[0] == ll.LL_ERR_ARG
    assert call(lib, name, c, n_tok=1 << 29)[0] == ll.LL_ERR_SHAPE
    assert call(lib, name, c, lens=None)[0] == ll.LL_ERR_ARG
    assert call(lib, name, c, lens=66)[0] == ll.LL_ERR_ARG
    assert call(lib, name, c, n_toks=67)[0] == ll.LL_ERR_ARG
    for bad in (dict(data=None), dict(data=65544), dict(seq=1025), dict(head=66)):
        assert call(lib, name, c, r=rows(**bad))[0] == ll.LL_ERR_ARG, bad
        assert call(lib, name, c, r2=rows(**bad))[0] == ll.LL_ERR_ARG, bad
    assert call(lib, name, c, n_tok=2, r=rows(token=129))[0] == ll.LL_ERR_ARG
    for zero in (dict(seq=0), dict(head=0)):  # an output's rows must not share their place
        if name != "write":
            rc, msg = call(lib, name, c, r2=rows(**zero))
            assert rc == ll.LL_ERR_ARG and "stride of 0" in msg
    if not torch.cuda.is_available():  # a good call gets as far as the device, and there is none
        rc, msg = call(lib, name, c, r=rows(token=3))
        assert rc == ll.LL_ERR_CUDA and msg


def test_write_and_attention_refusals(lib):
    c = cache()
    assert call(lib, "write", c, kind=2)[0] == ll.LL_ERR_ARG
    for heads in (0, 1, 3, 18, -2):
        assert call(lib, "attention", c, heads=heads)[0] == ll.LL_ERR_SHAPE, heads
    for scale in (-1.0, float("inf"), float("nan")):
        assert call(lib, "attention", c, scale=scale)[0] == ll.LL_ERR_ARG, scale
    assert call(lib, "attention", c, max_len=-1)[0] == ll.LL_ERR_ARG


@pytest.mark.parametrize("name", CALLS)
def test_longest_cache(lib, name):
    """Positions are 32-bit numbers in the kernels, rounded up to tiles: 2^30 is the last size that is taken."""
    rc, msg = call(lib, name, cache(max_seq=(1 << 30) + 1, seq_rows=1 << 40))
    assert rc == ll.LL_ERR_SHAPE and "max_seq" in msg
    if not torch.cuda.is_available():
        assert call(lib, name, cache(max_seq=1 << 30, seq_rows=1 << 40))[0] == ll.LL_ERR_CUDA


def init_kvq(lib, c, out=True, **k):
    d = dict(n_layers=2, hidden=256, n_q_heads=4, n_kv_heads=2, head_dim=64, inter=512, vocab=64, max_seq=32, tied=1,
             backend=ll.LL_BACKEND_CHAIN, rms_eps=1e-5, rope_theta=1e4)
    d.update(k)
    cfg, w, h = ll.ll_config(**d), ll.ll_weights(), ctypes.c_void_p(1)
    rc = lib.ll_init_kvq(ctypes.byref(cfg), ctypes.byref(w), ctypes.byref(c) if c is not None else None, None,
                         ctypes.byref(h) if out else None)
    return rc, h.value, lib.ll_init_error().decode()


def test_handles_that_are_refused(lib):
    """The packed cache is checked before the weights' pointers (NULL here) are looked at."""
    rc, h, msg = init_kvq(lib, None)
    assert rc == ll.LL_ERR_ARG and h is None and "cache" in msg
    assert init_kvq(lib, cache(), out=False)[0] == ll.LL_ERR_ARG
    for k in (dict(bits=3), dict(max_seq=0), dict(n_seq=0)):
        rc, h, msg = init_kvq(lib, cache(**k))
        assert rc == ll.LL_ERR_SHAPE and h is None and msg, k
    for k in (dict(n_seq=3), dict(n_kv_heads=1), dict(head_dim=128), dict(max_seq=31), dict(seq_rows=63), dict(v_codes=None)):
        rc, h, msg = init_kvq(lib, cache(**k))
        assert rc == ll.LL_ERR_ARG and h is None and msg, k
    rc, h, msg = init_kvq(lib, cache(), backend=ll.LL_BACKEND_MEGAKERNEL)
    assert rc == ll.LL_ERR_ARG and h is None and "LL_BACKEND_CHAIN" in msg
    rc, h, msg = init_kvq(lib, cache())  # the cache is taken, the weights are not
    assert rc == ll.LL_ERR_ARG and h is None and "embed" in msg


def test_scale_as_the_call_gets_it():
    c, q, lens = fake_cache(), _Fake((2, 1, 2, 64), torch.bfloat16, "cuda:0"), _Fake((2,), torch.int32, "cuda:0")
    for scale in (0.0, -0.5, float("nan"), 1e-60):
        with pytest.raises(ll.LLError, match="scale"):
            ll.ll_kvq_attention(c, q, lens, scale=scale)


def test_binding_refuses_host_tensors_and_bits():
    codes = torch.zeros(1, 1, 8, 32, dtype=torch.uint8)
    params = torch.zeros(1, 1, 8, 2, 2, dtype=torch.float16)
    with pytest.raises(ll.LLError):
        ll.KVQCache(codes, params, codes, params, 4)
    with pytest.raises(ll.LLError):
        ll.KVQCache(codes, params, codes, params, 5)
    with pytest.raises(ll.LLError):
        ll.KVQCache.empty(1, 1, 8, 96, 4, device="cpu")
    with pytest.raises(ll.LLError):
        ll.KVQCache.empty(1, 1, 8, 64, 4, device="cpu")


class _Fake:
    """A tensor's description, as the binding's checks see it."""
    is_cuda = True

    def __init__(self, shape, dtype, device, strides=None):
        self.shape, self.dtype, self.device = tuple(shape), dtype, torch.device(device)
        self.ndim = len(self.shape)
        st, n = [], 1
        for x in reversed(self.shape):
            st.insert(0, n)
            n *= x
        self._st = tuple(strides or st)

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._st if i is None else self._st[i]

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def is_contiguous(self):
        return self._st == _Fake(self.shape, self.dtype, self.device)._st

    def data_ptr(self):
        return 4096

    def __getitem__(self, i):
        d = len(i) if isinstance(i, tuple) else 1
        return _Fake(self.shape[d:], self.dtype, self.device, self._st[d:] or None)


def fake_cache(S=2, KV=2, M=16, hd=64, bits=4, strides=None, dev="cuda:0"):
    codes = _Fake((S, KV, M, hd * bits // 8), torch.uint8, dev, strides)
    params = _Fake((S, KV, M, hd // 32, 2), torch.float16, dev)
    return ll.KVQCache(codes, params, codes, params, bits)


def test_binding_cache_checks():
    c = fake_cache()
    assert (c.n_seq, c.n_kv_heads, c.max_seq, c.head_dim, c.struct.seq_rows) == (2, 2, 16, 64, 32)
    with pytest.raises(ll.LLError):  # sequences of codes and parameters not equally far apart
        fake_cache(strides=(64 * 32, 16 * 32, 32, 1))
    with pytest.raises(ll.LLError):  # rows apart from each other
        fake_cache(strides=(32 * 32, 16 * 32, 64, 1))
    with pytest.raises(ll.LLError):  # sequences that share their rows
        S, KV, M = 2, 2, 16
        codes = _Fake((S, KV, M, 32), torch.uint8, "cuda:0", (0, 512, 32, 1))
        params = _Fake((S, KV, M, 2, 2), torch.float16, "cuda:0", (0, 64, 4, 2, 1))
        ll.KVQCache(codes, params, codes, params, 4)


def test_binding_rows_checks():
    c = fake_cache()
    good = _Fake((2, 3, 2, 64), torch.bfloat16, "cuda:0")
    assert c._rows(good, "k", torch.bfloat16, 2, written=True)[1] == 3
    lens = _Fake((2,), torch.int32, "cuda:0")
    for bad in (_Fake((2, 3, 2, 64), torch.float16, "cuda:0"), _Fake((2, 3, 2, 64), torch.bfloat16, "cuda:1"),
                _Fake((3, 3, 2, 64), torch.bfloat16, "cuda:0"), _Fake((2, 3, 4, 64), torch.bfloat16, "cuda:0"),
                _Fake((2, 3, 2, 128), torch.bfloat16, "cuda:0"), _Fake((2, 3, 128), torch.bfloat16, "cuda:0"),
                _Fake((2, 3, 2, 64), torch.bfloat16, "cuda:0", (768, 256, 128, 2)), torch.zeros(2, 3, 2, 64).bfloat16(), None):
        with pytest.raises(ll.LLError):
            c._rows(bad, "k", torch.bfloat16, 2)
        with pytest.raises(ll.LLError):
            ll.ll_kvq_write(c, bad, good, lens)
        with pytest.raises(ll.LLError):
            ll.ll_kvq_read(c, bad, good, lens)
    for overlap in ((0, 128, 64, 1), (384, 0, 64, 1), (384, 128, 32, 1), (384, 64, 64, 1)):
        t = _Fake((2, 3, 2, 64), torch.bfloat16, "cuda:0", overlap)
        c._rows(t, "k", torch.bfloat16, 2)  # (an input may be broadcast)
        with pytest.raises(ll.LLError):
            c._rows(t, "out", torch.bfloat16, 2, written=True)
    for t in (None, _Fake((1,), torch.int32, "cuda:0"), _Fake((2,), torch.int64, "cuda:0"), _Fake((2,), torch.int32, "cuda:1"),
              torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ll.LLError):
            c._lens(t, "lens")
        with pytest.raises(ll.LLError):
            ll.ll_kvq_write(c, good, good, t)
        with pytest.raises(ll.LLError):
            ll.ll_kvq_read(c, good, good, t)
        with pytest.raises(ll.LLError):
            ll.ll_kvq_attention(c, good, t)
    with pytest.raises(ll.LLError):
        ll.ll_kvq_attention(c, None, lens)
    with pytest.raises(ll.LLError):
        ll.ll_kvq_attention(c, good, lens, scale=-1.0)
    with pytest.raises(ll.LLError):
        ll.ll_kvq_attention(c, good, None)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_definition_closed_forms(hd, bits):
    """Of the tests' own definition: every dim has a place of its own; a ramp of 2^bits
    levels reads back exactly; a constant is held to fp16; bytes hold the codes."""
    assert sorted(kvq_ref.place(hd).tolist()) == list(range(hd))
    top = 2 ** bits - 1
    ramp = (torch.arange(hd) % 32).float().clamp(max=top)
    ramp[::32], ramp[31::32] = 0.0, float(top)
    lo, step, code = kvq_ref.quantise(ramp[None], bits)
    assert bool((lo == 0).all()) and bool((step == 1).all())
    assert torch.equal(kvq_ref.values(lo, step, code)[0].float(), ramp)
    codes, params = kvq_ref.pack(lo, step, code, bits)
    assert codes.shape == (1, hd * bits // 8) and params.shape == (1, hd // 32, 2)
    assert int(codes[0, 0]) == (int(ramp[0]) + 16 * int(ramp[1]) if bits == 4 else int(ramp[0]))
    lo, step, code = kvq_ref.quantise(torch.full((1, hd), 0.3), bits)
    assert torch.equal(kvq_ref.values(lo, step, code)[0].half(), torch.full((hd,), 0.3).half())

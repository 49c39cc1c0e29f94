"""Handles over packed caches whose layers lie at every kind of row number: odd numbers
of rows apart (at 64 dims a row of parameters is 8 bytes, so an odd row starts in the
middle of 16), with rows between them that are not the cache's, and prefills long
enough for every attention kernel."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll, synth
from helpers import check_token, compare_logits
from test_gpu_kvq_model import Reference

pytestmark = pytest.mark.gpu

ONE_KV = synth.ModelShape("one-kv", 3, 256, 4, 1, 64, 512, 1000, True)
THREE_KV = synth.ModelShape("three-kv", 3, 768, 12, 3, 64, 512, 1000, True)
ONE_KV_128 = synth.ModelShape("one-kv-128", 3, 512, 4, 1, 128, 512, 1000, True)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_megakernel_persistent_gb300 import build
    build.build()


def spread_cache(shape, max_seq, bits, gap):
    """A cache whose layers are n_kv_heads * max_seq + gap rows apart, and its four flat arrays of marks."""
    L, KV, hd = shape.n_layers, shape.n_kv_heads, shape.head_dim
    rows, cb, pb = KV * max_seq + gap, hd * bits // 8, hd // 16
    flat = [torch.full((L * rows * cb,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2)]
    flat += [torch.full((L * rows * pb,), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]
    kc, vc = (t.as_strided((L, KV, max_seq, cb), (rows * cb, max_seq * cb, cb, 1)) for t in flat[:2])
    kp, vp = (t.as_strided((L, KV, max_seq, hd // 32, 2), (rows * pb, max_seq * pb, pb, 2, 1)) for t in flat[2:])
    return ll.KVQCache(kc, kp, vc, vp, bits), flat


def gaps_are_marked(shape, max_seq, gap, flat):
    rows = shape.n_layers, shape.n_kv_heads * max_seq + gap
    for t in flat:
        rest = t.view(*rows, -1)[:, shape.n_kv_heads * max_seq:]
        assert bool((torch.isnan(rest) if t.dtype == torch.float16 else rest == 0xA5).all())


def pair(shape, bits, max_seq, gap=0):
    w = synth.make_weights(shape, seed=0, device="cuda", gain_jitter=0.25, std=0.05)
    cache, flat = spread_cache(shape, max_seq, bits, gap)
    return ll.KVQDecoder(shape, w, cache), Reference(shape, w, cache), flat


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape,max_seq,gap", [(ONE_KV, 23, 0), (THREE_KV, 23, 0), (ONE_KV, 24, 1), (synth.TINY, 24, 3), (ONE_KV_128, 23, 0)],
                         ids=["1x23", "3x23", "1x24+1", "2x24+3", "1x23-128"])
@pytest.mark.parametrize("n", [0, 2, 4, 9])
def test_layers_an_odd_number_of_rows_apart(shape, max_seq, gap, bits, n):
    """Steps up to the cache's last row, behind a prefill of n tokens (up to 16 query rows a KV head and more)."""
    dec, ref, flat = pair(shape, bits, max_seq, gap)
    logits, nxt = torch.empty(shape.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    tok = 17
    if n:
        prompt = synth.make_tokens(shape.vocab, n, seed=3)
        dec.prefill(torch.tensor(prompt, dtype=torch.int32, device="cuda"), 0, logits, nxt)
        dec.synchronize()
        for pos in range(n):
            want = ref.step(prompt[pos], pos)
        compare_logits(logits.cpu().numpy(), want, "prefill")
        check_token(int(nxt), want, "prefill")
        tok = int(np.argmax(want))
    for pos in range(n, max_seq):
        got = dec.step(tok, pos, logits)
        want = ref.step(tok, pos)
        compare_logits(logits.cpu().numpy(), want, f"pos {pos}")
        check_token(got, want, f"pos {pos}")
        tok = int(np.argmax(want))
    gaps_are_marked(shape, max_seq, gap, flat)
    dec.close()

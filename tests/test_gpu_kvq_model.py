"""Handles with a packed KV cache (ll_init_kvq): decode steps and prefill against
the forward pass written out in 64 bits. The logits' bar is the framework's: max
|delta| within 2e-2 of the largest, relative L2 within 1e-2, and the same greedy
token unless the top two are within 1e-2.

Rounding to a code is not continuous: a value within fp32 noise of the border
between two codes may take either, and in 4 bits the two are a fifteenth of the
group's range apart, far more than any logits' bar. So the reference attends to the rows that
the cache holds, after checking that every one of them is a right rounding of its
own K or V: within half a step, and the noise that those may carry."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll, synth
from helpers import check_token, compare_logits
import kvq_ref

pytestmark = pytest.mark.gpu

SMALL = synth.ModelShape("small-128", 2, 512, 8, 2, 128, 512, 1000, False)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_megakernel_persistent_gb300 import build
    build.build()


class Reference:
    """The forward pass in double on the same bf16 weights, over the rows that `cache` holds."""

    def __init__(self, shape, w, cache):
        self.s, self.cache = shape, cache
        self.w = {k: ([t.double() for t in v] if isinstance(v, list) else None if v is None else v.double()) for k, v in w.items()}

    def held(self, which, l, pos, x):
        """The rows 0..pos of layer l that the cache holds, the one at pos a right rounding of x [n_kv, hd]."""
        c = self.cache
        codes, params = (getattr(c, f"{which}_{kind}")[l, :, :pos + 1] for kind in ("codes", "params"))
        el = codes.long() if c.bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        code = el[..., kvq_ref.place(c.head_dim).cuda()].unflatten(-1, (c.head_dim // 32, 32))
        val = kvq_ref.values(params[..., 0].cpu(), params[..., 1].cpu(), code.cpu()).cuda()
        lo, step = (params[:, pos, :, i].double().repeat_interleave(32, -1) for i in (0, 1))
        # half a step; the roundings to fp16 of step (times the code), lo and the value; the fp32 noise of x, at
        # a tenth of the logits' bar
        tol = step * (0.5 + 2 ** c.bits * 2.0 ** -11) + (lo.abs() + val[:, pos].abs()) * 2.0 ** -11 + 2e-3 * x.abs().max()
        off = (val[:, pos] - x).abs()
        assert bool((off <= tol).all()), (which, l, pos, float((off / tol).max()))
        return val

    def norm(self, x, g):
        return x / torch.sqrt((x * x).mean() + self.s.rms_eps) * g

    def rope(self, x, pos):
        half = self.s.head_dim // 2
        a = pos * self.s.rope_theta ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / self.s.head_dim)
        p, q = x[:, :half], x[:, half:]
        return torch.cat([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()], 1)

    def step(self, token, pos):
        """The logits of the token at pos, once the handle has run it."""
        s, w = self.s, self.w
        x = w["embed"][token]
        G = s.n_q_heads // s.n_kv_heads
        for l in range(s.n_layers):
            h = self.norm(x, w["attn_norm"][l])
            q = self.rope((w["wq"][l] @ h).view(-1, s.head_dim), pos)
            k = self.rope((w["wk"][l] @ h).view(-1, s.head_dim), pos)
            v = (w["wv"][l] @ h).view(-1, s.head_dim)
            k, v = self.held("k", l, pos, k), self.held("v", l, pos, v)
            qg = q.view(s.n_kv_heads, G, s.head_dim)
            p = torch.softmax(qg @ k.transpose(1, 2) / s.head_dim ** 0.5, -1)
            x = x + w["wo"][l] @ (p @ v).reshape(-1)
            h = self.norm(x, w["mlp_norm"][l])
            x = x + w["wd"][l] @ (torch.nn.functional.silu(w["wg"][l] @ h) * (w["wu"][l] @ h))
        head = w["embed"] if s.tied else w["lm_head"]
        return (head @ self.norm(x, w["final_norm"])).cpu().numpy()


def build_pair(shape, bits, max_seq):
    w = synth.make_weights(shape, seed=0, device="cuda", gain_jitter=0.25, std=0.05)
    cache = ll.KVQCache.empty(shape.n_layers, shape.n_kv_heads, max_seq, shape.head_dim, bits)
    for t in (cache.k_params, cache.v_params):
        t.fill_(float("nan"))  # what no step has written must not matter
    return ll.KVQDecoder(shape, w, cache), Reference(shape, w, cache)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape", [synth.TINY, SMALL], ids=lambda s: s.name)
def test_steps_match_the_definition(shape, bits):
    dec, ref = build_pair(shape, bits, 24)
    logits = torch.empty(shape.vocab, device="cuda")
    tok = 17
    for pos in range(12):
        nxt = dec.step(tok, pos, logits)
        want = ref.step(tok, pos)
        compare_logits(logits.cpu().numpy(), want, f"pos {pos}")
        check_token(nxt, want, f"pos {pos}")
        tok = int(np.argmax(want))
    assert dec.query(ll.LL_Q_KV_BITS) == bits
    dec.close()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape", [synth.TINY, SMALL], ids=lambda s: s.name)
@pytest.mark.parametrize("n0,n1", [(1, 2), (70, 0), (40, 37)])
def test_prefill_then_steps(shape, bits, n0, n1):
    """A prompt (in one or two calls), then greedy steps chained on the device."""
    n, steps = n0 + n1, 3
    dec, ref = build_pair(shape, bits, n + steps)
    prompt = synth.make_tokens(shape.vocab, n, seed=3)
    dev = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    logits, nxt = torch.empty(shape.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dec.prefill(dev[:n0], 0, logits, nxt)
    if n1:
        dec.prefill(dev[n0:], n0, logits, nxt)
    dec.synchronize()
    for pos in range(n):
        want = ref.step(prompt[pos], pos)
    compare_logits(logits.cpu().numpy(), want, "prefill")
    check_token(int(nxt), want, "prefill")
    nxt.fill_(int(np.argmax(want)))
    toks, all_logits = torch.zeros(steps, dtype=torch.int32, device="cuda"), torch.empty(steps, shape.vocab, device="cuda")
    dec.steps(nxt, n, steps, all_logits, toks)
    dec.synchronize()
    tok = int(nxt)
    for i in range(steps):
        want = ref.step(tok, n + i)
        compare_logits(all_logits[i].cpu().numpy(), want, f"step {i}")
        check_token(int(toks[i]), want, f"step {i}")
        if int(toks[i]) != int(np.argmax(want)):
            break
        tok = int(toks[i])
    dec.close()


def test_steps_equal_chained_single_steps():
    shape, n = synth.TINY, 5
    a, _ = build_pair(shape, 4, 8)
    b, _ = build_pair(shape, 4, 8)
    t0 = torch.tensor([3], dtype=torch.int32, device="cuda")
    toks, la = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.empty(n, shape.vocab, device="cuda")
    a.steps(t0, 0, n, la, toks)
    a.synchronize()
    cur, lb = t0.clone(), torch.empty(n, shape.vocab, device="cuda")
    for i in range(n):
        b.step_async(cur, i, lb[i], cur)
    b.synchronize()
    assert torch.equal(la, lb) and int(toks[-1]) == int(cur)
    assert torch.equal(a.cache.k_codes, b.cache.k_codes)
    a.close()
    b.close()


def test_packed_from_a_bf16_cache_and_back():
    """A bf16 cache (of a prompt that another handle ran) packed into a decoder's, which goes on
    from it; and the packed rows read back give a bf16 cache that an ordinary handle goes on from."""
    shape, n, M = synth.TINY, 48, 64
    w = synth.make_weights(shape, seed=0, device="cuda", std=0.05)
    k, v = synth.make_kv(shape, M, 0, device="cuda")
    prompt = torch.tensor(synth.make_tokens(shape.vocab, n, seed=5), dtype=torch.int32, device="cuda")
    logits, nxt = torch.empty(shape.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dec = ll.Decoder(shape, w, k, v, M)
    dec.prefill(prompt, 0, logits, nxt)
    dec.synchronize()
    tok = int(nxt)
    cache = ll.KVQCache.empty(shape.n_layers, shape.n_kv_heads, M, shape.head_dim, 8)
    lens = torch.full((shape.n_layers,), n, dtype=torch.int32, device="cuda")
    cache.write(k[:, :, :n].transpose(1, 2), v[:, :, :n].transpose(1, 2), lens)
    k2, v2 = synth.make_kv(shape, M, 0, device="cuda")
    cache.read(k2[:, :, :n].transpose(1, 2), v2[:, :, :n].transpose(1, 2), lens)
    assert float((k2 - k).abs().max()) < 0.05 * float(k.abs().max())
    back, packed = ll.Decoder(shape, w, k2, v2, M), ll.KVQDecoder(shape, w, cache)
    got = []
    for d in (dec, back, packed):
        d.step(tok, n, logits)
        got.append(logits.cpu().numpy().copy())
    # the same held rows on both sides (their bf16 and fp16 roundings apart), and 8 bits near the bf16 cache
    compare_logits(got[2], got[1], "packed against read back")
    compare_logits(got[2], got[0], "packed against bf16")
    for d in (dec, back, packed):
        d.close()


def test_handles_that_are_refused():
    shape = synth.TINY
    w = synth.make_weights(shape, seed=0, device="cuda")

    def cache(**k):
        d = dict(n_seq=shape.n_layers, n_kv_heads=shape.n_kv_heads, max_seq=16, head_dim=shape.head_dim, bits=4)
        d.update(k)
        return ll.KVQCache.empty(**d)

    good = cache()
    for other in (dict(n_seq=1), dict(n_kv_heads=1), dict(head_dim=128)):
        with pytest.raises(ll.LLError):
            ll.KVQDecoder(shape, w, cache(**other))
    for kw in (dict(backend=ll.LL_BACKEND_MEGAKERNEL, max_seq=16), dict(backend=ll.LL_BACKEND_CHAIN, max_seq=17)):
        with pytest.raises(ll.LLError) as e:
            ll.ll_init_kvq(ll.make_config(shape, **kw), w, good)
        assert e.value.code == ll.LL_ERR_ARG
    dec = ll.KVQDecoder(shape, w, good)
    with pytest.raises(ll.LLError):
        dec.step(0, 16)
    tok = torch.tensor([shape.vocab], dtype=torch.int32, device="cuda")
    dec.step_async(tok, 0, None, torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ll.LLError) as e:
        dec.synchronize()
    assert e.value.code == ll.LL_ERR_ARG
    assert dec.step(0, 0) >= 0
    dec.close()

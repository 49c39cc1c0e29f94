"""Handles over packed caches whose layers lie at every kind of row number: odd numbers
of rows apart (at 64 dims a row of parameters is 8 bytes, so an odd row starts in the
middle of 16), with rows between them that are not the cache's, and prefills long
enough for every attention kernel."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll, synth
from helpers import check_token, compare_logits
import kvq_ref
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


WIDE = synth.ModelShape("wide-64", 2, 512, 32, 8, 64, 512, 1000, True)
WIDE_128 = synth.ModelShape("wide-128", 2, 512, 32, 8, 128, 512, 1000, True)


class Forward:
    """Reference's forward pass of many positions at once, over the rows that the cache holds, checked as there."""

    def __init__(self, ref):
        self.s, self.c, self.w = ref.s, ref.cache, ref.w

    def held(self, which, l, pos0, x):
        """The rows of layer l up to those of x [n, n_kv, hd] (positions pos0 on), which are right roundings of it."""
        c, end = self.c, pos0 + x.shape[0]
        codes, params = (getattr(c, f"{which}_{kind}")[l, :, :end] for kind in ("codes", "params"))
        el = codes.long() if c.bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        code = el[..., kvq_ref.place(c.head_dim).cuda()].unflatten(-1, (c.head_dim // 32, 32))
        val = kvq_ref.values(params[..., 0].cpu(), params[..., 1].cpu(), code.cpu()).cuda()  # [n_kv, end, hd]
        lo, step = (params[:, pos0:, :, i].double().repeat_interleave(32, -1)[:, :x.shape[0]] for i in (0, 1))
        x, got = x.transpose(0, 1), val[:, pos0:]
        # (as Reference.held bounds it; the noise by the position's own largest value)
        tol = step * (0.5 + 2 ** c.bits * 2.0 ** -11) + (lo.abs() + got.abs()) * 2.0 ** -11 + 2e-3 * x.abs().amax((0, 2), keepdim=True)
        off = (got - x).abs()
        assert bool((off <= tol).all()), (which, l, float((off / tol).max()))
        return val

    def norm(self, x, g):
        return x / torch.sqrt((x * x).mean(-1, keepdim=True) + self.s.rms_eps) * g

    def rope(self, x, pos0):
        half = self.s.head_dim // 2
        pos = pos0 + torch.arange(x.shape[0], dtype=torch.float64, device="cuda")
        a = pos[:, None, None] * self.s.rope_theta ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / self.s.head_dim)
        p, q = x[..., :half], x[..., half:]
        return torch.cat([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()], -1)

    def logits(self, tokens, pos0):
        """Those of the last of `tokens`, at positions pos0 on, once the handle has run them."""
        s, w, n = self.s, self.w, len(tokens)
        x = w["embed"][torch.tensor(tokens, device="cuda")]
        G = s.n_q_heads // s.n_kv_heads
        unseen = torch.arange(pos0 + n, device="cuda") > pos0 + torch.arange(n, device="cuda")[:, None]
        for l in range(s.n_layers):
            h = self.norm(x, w["attn_norm"][l])
            q, k, v = ((h @ w[m][l].view(-1, s.hidden).T).view(n, -1, s.head_dim) for m in ("wq", "wk", "wv"))
            k, v = self.held("k", l, pos0, self.rope(k, pos0)), self.held("v", l, pos0, v)
            q = self.rope(q, pos0).view(n, s.n_kv_heads, G, s.head_dim).permute(1, 2, 0, 3)  # [n_kv, G, n, hd]
            p = torch.softmax((q @ k[:, None].transpose(-1, -2) / s.head_dim ** 0.5).masked_fill_(unseen, float("-inf")), -1)
            x = x + (p @ v[:, None]).permute(2, 0, 1, 3).reshape(n, -1) @ w["wo"][l].view(s.hidden, -1).T
            h = self.norm(x, w["mlp_norm"][l])
            g, u = (h @ w[m][l].view(-1, s.hidden).T for m in ("wg", "wu"))
            x = x + (torch.nn.functional.silu(g) * u) @ w["wd"][l].view(s.hidden, -1).T
        head = (w["embed"] if s.tied else w["lm_head"]).view(s.vocab, s.hidden)
        return (head @ self.norm(x[-1], w["final_norm"])).cpu().numpy()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape,calls", [(WIDE, (530,)), (WIDE, (200, 600)), (WIDE_128, (400,)), (WIDE_128, (130, 401)), (synth.TINY, (1500,)),
                                         (synth.TINY, (700, 1301)), (ONE_KV_128, (1101,)), (ONE_KV_128, (300, 1001))],
                         ids=lambda x: x.name if hasattr(x, "name") else "+".join(map(str, x)))
def test_prefill_of_prompts(shape, calls, bits):
    """Prompts long enough for the kernel of 256 query rows to a block (rows x positions x KV heads past 8 million at 64 dims,
    half as many at 128): blocks on their own (the wide shapes) and clusters that share the keys, fp32 queries, outputs
    as three bf16 terms, behind a prefix too. What attention gives shows in the next layer's rows, and in the logits."""
    n = sum(calls)
    dec, ref, flat = pair(shape, bits, n + 3, gap=1)
    fwd = Forward(ref)
    prompt = synth.make_tokens(shape.vocab, n, seed=3)
    dev = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    logits, nxt = torch.empty(shape.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    at = 0
    for m in calls:
        dec.prefill(dev[at:at + m], at, logits, nxt)
        dec.synchronize()
        want = fwd.logits(prompt[at:at + m], at)
        compare_logits(logits.cpu().numpy(), want, f"prefill up to {at + m}")
        check_token(int(nxt), want, f"prefill up to {at + m}")
        at += m
    tok = int(np.argmax(want))
    for pos in range(n, n + 3):
        got = dec.step(tok, pos, logits)
        want = fwd.logits([tok], pos)
        compare_logits(logits.cpu().numpy(), want, f"pos {pos}")
        check_token(got, want, f"pos {pos}")
        tok = int(np.argmax(want))
    gaps_are_marked(shape, n + 3, 1, flat)
    dec.close()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("shape", [synth.TINY, ONE_KV_128], ids=lambda s: s.name)
def test_steps_at_long_contexts(shape, bits):
    """fp32 queries over rows enough for many splits and large blocks."""
    n, M = 3000, 20001
    dec, ref, flat = pair(shape, bits, M, gap=3)
    fwd = Forward(ref)
    prompt = synth.make_tokens(shape.vocab, n, seed=4)
    logits, nxt = torch.empty(shape.vocab, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dec.prefill(torch.tensor(prompt, dtype=torch.int32, device="cuda"), 0, logits, nxt)
    dec.synchronize()
    want = fwd.logits(prompt, 0)
    tok = int(np.argmax(want))
    for pos in range(n, n + 4):
        got = dec.step(tok, pos, logits)
        want = fwd.logits([tok], pos)
        compare_logits(logits.cpu().numpy(), want, f"pos {pos}")
        check_token(got, want, f"pos {pos}")
        tok = int(np.argmax(want))
    gaps_are_marked(shape, M, 3, flat)
    dec.close()

"""The operators around the attention together, as a model's steps use them: each stage against its formula in 64 bits on what
the stage before it gave, whole steps captured and replayed, two at once, and sizes past 32 bits."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll
import kvq_ref
import step_ref
from step_ref import HALF_STEP, gen, i32

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_megakernel_persistent_gb300 import build
    build.build()


class Model:
    """Two layers with 4-bit matrices, a packed cache, rotary positions; rows of `tokens` a sequence, in buffers of its own."""
    H, HEADS, KV, HD, INTER, V = 256, 8, 2, 64, 640, 1000

    def __init__(self, S, T, group, norm, bits, scaling, seed=0):
        g = gen(seed)
        self.S, self.T, self.norm = S, T, norm
        self.scaling = scaling
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        q4 = lambda r, c: ll.Q4Matrix.quantised(rand(r, c) * c ** -0.5, group)
        gain = lambda: (1 + 0.1 * rand(self.H)).bfloat16()
        self.layers = [dict(qkv=q4((self.HEADS + 2 * self.KV) * self.HD, self.H), o=q4(self.H, self.HEADS * self.HD), gate=q4(self.INTER, self.H),
                            up=q4(self.INTER, self.H), down=q4(self.H, self.INTER), first=gain(), second=gain()) for _ in range(2)]
        self.embed, self.last, self.head = rand(self.V, self.H).bfloat16(), gain(), q4(self.V, self.H)
        self.caches = [ll.KVQCache.empty(S, self.KV, 100, self.HD, bits) for _ in self.layers]
        self.rope = ll.Rope(self.HD, 10000.0, scaling=scaling)

    def buffers(self):
        z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")
        return dict(ids=z(self.S, self.T), lens=z(self.S), n=z(self.S), drafts=z(self.S, self.T - 1), u=z(self.S, self.T, d=torch.float32),
                    temperature=z(self.S, d=torch.float32))

    def step(self, b, see=lambda *a, **k: None):
        """Tokens b["ids"] (the last of each sequence): verified against b["drafts"]. see: is shown each call."""
        S, T = self.S, self.T
        res = self.embed[b["ids"].long()].view(S * T, self.H)
        delta = None

        def norm(gain, dtype):
            before = res.clone()
            out = ll.ll_rmsnorm(res if delta is None else delta, gain, 1e-5, residual=None if delta is None else res, out_dtype=dtype,
                                group=128 if dtype == E4M3 else 0)
            out, scale = out if dtype == E4M3 else (out, None)
            see("norm", before, delta, res, gain, out, scale)
            return out, scale

        def product(m, x, scale=None, dtype=torch.bfloat16):
            y = m.matvec(x, scale=scale, out_dtype=dtype)
            see("product", m, x, scale, y)
            return y

        for w, cache in zip(self.layers, self.caches):
            x, scale = norm(w["first"], self.norm)
            qkv = product(w["qkv"], x, scale).view(S, T, -1, self.HD)
            before = qkv.clone()
            q, k, v = qkv.split([self.HEADS, self.KV, self.KV], 2)
            self.rope.apply(q, k, b["lens"], b["n"])
            see("rope", before, qkv, b)
            cache.write(k, v, b["lens"], b["n"])
            att = cache.attention(q, b["lens"], b["n"])
            see("attention", cache, q, att, b)
            delta = product(w["o"], att.view(S * T, -1))
            x, scale = norm(w["second"], self.norm)
            gate, up = product(w["gate"], x, scale), product(w["up"], x, scale)
            delta = product(w["down"], (torch.nn.functional.silu(gate.float()) * up.float()).bfloat16())
        x, _ = norm(self.last, torch.bfloat16)
        logits = product(self.head, x, dtype=torch.float32).view(S, T, self.V)
        tokens, accepted = ll.ll_verify(logits, b["drafts"], b["u"], n_drafts=b["n"] - 1, temperature=b["temperature"])
        see("verify", logits, tokens, accepted, b)
        return logits, tokens, accepted


class Check:
    """Each call against its formula in 64 bits, on its own inputs."""

    def __init__(self, model):
        self.m = model

    def __call__(self, what, *a):
        getattr(self, what)(*a)

    def norm(self, before, delta, res, gain, out, scale):
        r = before if delta is None else (delta.float() + before.float()).bfloat16()
        assert torch.equal(r, res)
        v = r.double()
        v = v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt() * gain.double()
        tol = 30 * 2.0 ** -24 * v.abs()
        if scale is None:
            assert bool(((out.double() - v).abs() <= tol + HALF_STEP[out.dtype] * (v.abs() + tol)).all())
        else:  # half a step of three mantissa bits, or of the smallest step, 2^-9
            wide = scale.double().repeat_interleave(128, 1)[:, :v.shape[1]]
            z = v / wide
            assert bool(((out.double() - z).abs() <= (z.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 2.0 ** -18) + z.abs() * 34 * 2.0 ** -24).all())

    def product(self, m, x, scale, y):
        wide = x.double()
        if scale is not None:
            wide = wide * scale.double().repeat_interleave(128, 1)[:, :x.shape[1]]
        want, tol = step_ref.product(m, wide.cpu(), None, y.dtype)
        assert bool(((y.cpu().double() - want).abs() <= tol).all())

    def rope(self, before, after, b):
        S, T = before.shape[:2]
        j = torch.arange(T, device="cuda")
        held = (j < b["n"][:, None])
        pos = (b["lens"] - b["n"])[:, None] + j
        turned = before.shape[2] - self.m.KV
        want, size = step_ref.rotated(before.double(), pos, self.m.HD, 10000.0, self.m.scaling, False)
        tol = 2.0 ** -21 * size
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
        ok = (after.double() - want).abs() <= tol
        assert bool(ok[:, :, :turned][held].all())
        assert torch.equal(after[:, :, turned:], before[:, :, turned:]) and torch.equal(after[~held], before[~held])

    def attention(self, c, q, out, b):
        vals = []
        for params, codes in ((c.k_params, c.k_codes), (c.v_params, c.v_codes)):
            el = codes.long() if c.bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
            code = el[..., kvq_ref.place(c.head_dim).cuda()].unflatten(-1, (c.head_dim // 32, 32))
            vals.append(kvq_ref.values(params[..., 0].cpu(), params[..., 1].cpu(), code.cpu()).cuda())
        G = self.m.HEADS // self.m.KV
        for s in range(self.m.S):
            L, n = int(b["lens"][s]), int(b["n"][s])
            last = (L - n + torch.arange(n, device="cuda")).repeat_interleave(G)
            for h in range(self.m.KV):
                o, tol = kvq_ref.attend(q[s, :n, h * G:(h + 1) * G].double().reshape(-1, c.head_dim), vals[0][s, h, :L], vals[1][s, h, :L], last)
                got = out[s, :n, h * G:(h + 1) * G].double().reshape(-1, c.head_dim)
                assert bool(((got - o).abs() <= tol).all())
            assert bool((out[s, n:] == 0).all())

    def verify(self, logits, tokens, accepted, b):
        want = step_ref.verified(logits.cpu(), b["drafts"].cpu(), b["u"].cpu(), None, (b["n"] - 1).cpu(), b["temperature"].cpu())
        assert want[2] > 1e-6  # (no decision so near its border that fp32 sums could turn it)
        assert torch.equal(tokens.cpu(), want[0]) and torch.equal(accepted.cpu(), want[1])


def set_step(b, ids, lens, n, seed, temperature):
    b["ids"].copy_(ids)
    b["lens"].copy_(i32(lens))
    b["n"].copy_(i32(n))
    b["drafts"].copy_(ids[:, 1:])
    b["u"].copy_(torch.rand(b["u"].shape, generator=gen(seed), device="cuda"))
    b["temperature"].copy_(torch.tensor(temperature, device="cuda"))


@pytest.mark.parametrize("norm", [torch.bfloat16, E4M3])
@pytest.mark.parametrize("group,bits,scaling", [(128, 8, None), (32, 4, dict(kind="bands", factor=32.0, low=1.0, high=4.0, length=64))])
def test_a_models_steps(norm, group, bits, scaling):
    """A prompt with padded rows, steps that verify drafts (the model's own greedy tokens at first, so that some stand), and
    a single token: every stage as its formula has it."""
    m = Model(3, 7, group, norm, bits, scaling)
    check = Check(m)
    b = m.buffers()
    ids = torch.randint(0, m.V, (3, 7), generator=gen(1), device="cuda").int()
    lens, n, temperature = [7, 5, 1], [7, 5, 1], [0.0, 1.0, 0.7]
    set_step(b, ids, lens, n, 2, temperature)
    logits, tokens, accepted = m.step(b, check)
    stood = 0
    for turn in range(4):
        # each sequence goes on behind what stood: its new token, then drafts: the greedy tokens of this step's logits (what a
        # draft model would offer does not matter here)
        kept = [lens[s] - n[s] + int(accepted[s]) + 1 for s in range(3)]
        new = [int(tokens[s, int(accepted[s])]) for s in range(3)]
        assert all(0 <= t < m.V for t in new)
        n = [1 + (turn + s) % 4 for s in range(3)]
        ids = torch.randint(0, m.V, (3, 7), generator=gen(10 + turn), device="cuda").int()
        for s in range(3):
            ids[s, 0] = new[s]
        lens = [kept[s] + n[s] for s in range(3)]
        if turn % 2:  # the greedy sequence's first draft as it will be
            set_step(b, ids, [kept[s] + 1 for s in range(3)], [1, 1, 1], 0, [0.0] * 3)
            ids[:, 1] = m.step(b)[1][:, 0]
        set_step(b, ids, lens, n, 20 + turn, temperature)
        logits, tokens, accepted = m.step(b, check)
        stood += int(accepted.sum())
    assert stood > 0


def test_captured_steps():
    """A step captured into a graph and replayed with other tokens, lengths, drafts and random numbers gives the plain step's bits."""
    plain, captured = (Model(2, 4, 64, E4M3, 8, None) for _ in range(2))
    bufs = [m.buffers() for m in (plain, captured)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = captured.step(bufs[1])
    for turn in range(3):
        ids = torch.randint(0, plain.V, (2, 4), generator=gen(turn), device="cuda").int()
        for b in bufs:
            set_step(b, ids, [4 + 3 * turn, 4 + 3 * turn], [4, 1 + turn], turn, [0.9, 0.0])
        want = plain.step(bufs[0])
        g.replay()
        assert all(torch.equal(x, y) for x, y in zip(want, out))


def test_steps_at_once():
    """Two models' steps on two streams, plain and as graphs replayed at once."""
    models = [Model(2, 4, 64, E4M3, 8, None, seed) for seed in (1, 2)]
    bufs = [m.buffers() for m in models]
    for i, (m, b) in enumerate(zip(models, bufs)):
        set_step(b, torch.randint(0, m.V, (2, 4), generator=gen(i), device="cuda").int(), [4, 3], [4, 3], i, [0.9, 0.0])
    want = [[t.clone() for t in m.step(b)] for m, b in zip(models, bufs)]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in models], []
    for g, m, b in zip(graphs, models, bufs):
        with torch.cuda.graph(g):
            outs.append(m.step(b))
    streams = [torch.cuda.Stream() for _ in models]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(want, outs) for a, b in zip(x, y))
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(models[i].step(bufs[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i in range(2) for out in got[i] for a, b in zip(want[i], out))


def test_first_calls_of_a_process_may_be_captured():
    code = """
import torch
from decode_megakernel_persistent_gb300 import ll
torch.manual_seed(1)
w = torch.randn(17100, 300, device="cuda").bfloat16()
m = ll.Q4Matrix.empty(17100, 300, 64)
x = torch.randn(40, 300, device="cuda").bfloat16()
gain = torch.ones(300, device="cuda").bfloat16()
rope, lens = ll.Rope(64), torch.tensor([9], dtype=torch.int32, device="cuda")
q, k = torch.randn(1, 5, 4, 64, device="cuda").bfloat16(), torch.randn(1, 5, 2, 64, device="cuda").bfloat16()
drafts, u = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.rand(2, 4, device="cuda")
outs = [torch.zeros(s, dtype=t, device="cuda") for s, t in (((40, 300), torch.bfloat16), ((40, 17100), torch.bfloat16), ((8, 17100), torch.float32),
        ((17100, 300), torch.float32), (q.shape, torch.bfloat16), (k.shape, torch.bfloat16), ((2, 4), torch.int32), ((2,), torch.int32))]
def run():
    m.write(w)
    ll.ll_rmsnorm(x, gain, out=outs[0])
    m.matvec(outs[0], out=outs[1])
    m.matvec(outs[0][:8], out=outs[2])
    m.read(out=outs[3])
    rope.apply(q, k, lens, q_out=outs[4], k_out=outs[5])
    ll.ll_verify(outs[2].view(2, 4, 17100), drafts, u, tokens=outs[6], accepted=outs[7])
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
for t in outs:
    t.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
assert all(bool((t != 0).any()) for t in got[:7])
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_most_rows(kind):
    """2^18 rows x, the most that a product takes, each as the same row in a small call."""
    m = ll.Q4Matrix.quantised(torch.randn(3, 40, generator=gen(1), device="cuda"), 32)
    some = torch.randint(-3, 4, (1 << 10, 40), generator=gen(2), device="cuda").to(kind)
    y = m.matvec(some.repeat(1 << 8, 1), out_dtype=torch.float32)
    want = torch.cat([m.matvec(r, out_dtype=torch.float32) for r in some.split(16)])
    assert bool(((y.view(1 << 8, 1 << 10, 3) - want).abs() <= 1e-5 * want.abs() + 1e-5).all())
    with pytest.raises(ll.LLError):
        m.matvec(some.repeat((1 << 8) + 1, 1))


def test_rows_far_apart():
    """Rows more than 2^31 elements (and 2^32 bytes) from each other, read and written."""
    far = (1 << 31) + 64
    stores = [torch.empty(2 * far, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    view = lambda i, width: stores[i].as_strided((2, width), (far, 1))
    g = gen(1)
    x = torch.randn(2, 640, generator=g, device="cuda").bfloat16()
    src, dst = view(0, 640), view(1, 640)
    src.copy_(x)
    gain = torch.randn(640, generator=g, device="cuda").bfloat16()
    assert torch.equal(ll.ll_rmsnorm(src, gain, out=dst), ll.ll_rmsnorm(x, gain))
    m = ll.Q4Matrix.quantised(torch.randn(500, 640, generator=g, device="cuda"), 128)
    assert torch.equal(m.matvec(src, out=view(1, 500)), m.matvec(x))
    wide = view(0, 640)
    back = ll.Q4Matrix.quantised(wide, 64)
    near = ll.Q4Matrix.quantised(x, 64)
    assert torch.equal(back.codes, near.codes) and torch.equal(back.read(out=dst), near.read())
    rope = ll.Rope(64)
    heads = lambda i: stores[i].as_strided((2, 1, 10, 64), (far, 640, 64, 1))
    lens = i32([5, 9])
    near = torch.empty(2, 1, 10, 64, dtype=torch.bfloat16, device="cuda")
    rope.apply(x.view(2, 1, 10, 64), None, lens, q_out=near)
    rope.apply(heads(0), None, lens, q_out=heads(1))
    assert torch.equal(heads(1), near)
    u = torch.rand(2, 1, generator=g, device="cuda")
    none = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    assert torch.equal(ll.ll_verify(stores[0].as_strided((2, 1, 640), (far, far, 1)), none, u)[0], ll.ll_verify(x.view(2, 1, 640), none, u)[0])


@pytest.mark.parametrize("n", [1, 20])
def test_a_matrix_past_32_bits(n):
    """8.6 GB of codes: the last rows' outputs (and values, 34 GB of them) are those of a matrix of these rows alone."""
    rows, cols = 1 << 20, 1 << 14
    g = gen(3)
    codes = torch.randint(0, 256, (rows // 16, cols // 128, 1024), generator=g, device="cuda", dtype=torch.uint8)
    params = torch.rand(rows // 16, cols // 128, 1, 16, 2, generator=g, device="cuda").half()
    m, last = ll.Q4Matrix(codes, params, rows, cols), ll.Q4Matrix(codes[-4:].clone(), params[-4:].clone(), 64, cols)
    x = torch.randn(n, cols, generator=g, device="cuda").bfloat16()
    y = m.matvec(x)[:, -64:]
    want, tol = step_ref.product(last, x.double().cpu(), None, torch.bfloat16)
    assert bool(((y.cpu().double() - want).abs() <= tol).all())
    if n == 1:
        assert torch.equal(m.read(dtype=torch.bfloat16)[-64:], last.read())

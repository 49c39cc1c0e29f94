"""Attention over the packed KV cache at the edges of its contract: what a call may not
read, values that are not finite, long contexts whose every key has to count."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll
import kvq_keys
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


@pytest.mark.parametrize("T,group,cap", [(1, 4, 333), (4, 4, 333), (5, 1, 333), (24, 4, 333), (200, 2, 333), (24, 4, 60000),
                                         (200, 2, 60000), (200, 4, 20000), (300, 4, 9000)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lo,step", [(float("inf"), 0.5), (-1.0, float("inf")), (float("-inf"), 0.0), (60000.0, None), (-60000.0, None)])
def test_infinite_values_reach_only_rows_that_see_them(T, group, cap, hd, bits, lo, step):
    """V groups of the caller's own whose parameters are infinite, or whose larger codes pass fp16's range
    (step None: from about the middle code on): such a value makes its dim infinite or NaN where it
    is seen. Its group's finite values count as any others, and rows that do not see it are as before."""
    KV, M = 1, 333
    lens = [M]
    c, kv, vv = make_cache(12, 1, KV, M, hd, bits, lens, cap)
    q = torch.randn(1, T, group, hd, generator=gen(6), device="cuda").bfloat16()
    base = c.attention(q, i32(lens))
    if step is None:
        step = (1 if lo > 0 else -1) * 11000.0 / 2 ** bits
    gr = hd // 32 - 1
    codes = c.v_codes[0, 0].long() if bits == 8 else torch.stack([c.v_codes[0, 0] & 15, c.v_codes[0, 0] >> 4], -1).flatten(-2).long()
    codes = codes[:, kvq_ref.place(hd).cuda()].unflatten(-1, (hd // 32, 32))[:, gr]  # [positions, 32]
    # one seen by the later half of the tokens, two by the last alone
    places = [M - (T + 1) // 2, M - 1] if T > 1 else [M - 1]
    bad = torch.zeros(M, 32, dtype=torch.bool, device="cuda")
    vv = vv.clone()
    for at in places:
        c.v_params[0, 0, at, gr, 0], c.v_params[0, 0, at, gr, 1] = lo, step
        p = c.v_params[0, 0, at, gr].cpu()
        val = kvq_ref.values(p[None, 0], p[None, 1], codes[at].cpu()[None])  # (numpy's infinities past fp16's range)
        bad[at] = ~torch.isfinite(val).cuda()
        vv[0, 0, at, 32 * gr:32 * gr + 32] = torch.where(bad[at], torch.zeros_like(bad[at], dtype=torch.float64), val.cuda())
    assert bool(bad[places[-1]].any()) and (lo in (60000.0, -60000.0)) == (not bool(bad[places[-1]].all()))
    out = c.attention(q, i32(lens))
    last = M - T + torch.arange(T, device="cuda")
    blind = last < min(places)
    assert torch.equal(out[0, blind], base[0, blind])
    assert torch.equal(out[0, :, :, :32 * gr], base[0, :, :, :32 * gr])
    seen = torch.stack([bad[:p + 1].any(0) for p in last.tolist()])  # [tokens, 32]: a value that is not finite is seen
    got = out[0, :, :, 32 * gr:]
    assert torch.equal(~torch.isfinite(got.float()), seen[:, None].expand_as(got))
    # the finite ones: the formula's, with zeros in the places that it leaves out
    o, tol = kvq_ref.attend(q[0].double().reshape(-1, hd), kv[0, 0], vv[0, 0], last.repeat_interleave(group))
    o, tol = (x.view(T, group, hd)[..., 32 * gr:] for x in (o, tol))
    fin = ~seen[:, None].expand_as(got)
    assert bool(((got.double() - o).abs() <= tol)[fin].all())


def test_a_launch_that_fails_says_why():
    """A stream whose capture was made invalid (by waiting for it while it captures) takes no launches: each call reports
    LL_ERR_CUDA with CUDA's reason, and works again once the capture has ended. In a process of its own."""
    code = """
import ctypes, torch
from decode_megakernel_persistent_gb300 import ll
c = ll.KVQCache.empty(1, 2, 5000, 64, 4)
x = torch.randn(1, 600, 2, 64, device="cuda").bfloat16()
qs = [torch.randn(1, t, 16, 64, device="cuda").bfloat16() for t in (1, 12, 600)]
outs = [torch.empty_like(q) for q in qs]
back = [torch.empty_like(x) for _ in range(2)]
lens = torch.tensor([600], dtype=torch.int32, device="cuda")
calls = [lambda: c.write(x, x, lens), lambda: c.read(back[0], back[1], lens)]
calls += [lambda q=q, o=o: c.attention(q, lens, out=o) for q, o in zip(qs, outs)]
torch.cuda.synchronize()
st = torch.cuda.Stream()
cu = ctypes.CDLL("libcuda.so.1")
s, graph = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p()
assert cu.cuStreamBeginCapture_v2(s, 2) == 0  # (relaxed: the first calls of the process may look things up)
assert cu.cuStreamSynchronize(s) != 0
with torch.cuda.stream(st):
    for f in calls:
        try:
            f()
        except ll.LLError as e:
            assert e.code == ll.LL_ERR_CUDA and "captur" in str(e) and "no error" not in str(e), str(e)
        else:
            raise AssertionError("launched into an invalid capture")
cu.cuStreamEndCapture(s, ctypes.byref(graph))
for f in calls:
    f()
torch.cuda.synchronize()
print("told")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "told" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("T,group,KV,lens,cap", [
    (1, 4, 1, [70001], 70001), (1, 4, 8, [32768], 32768), (1, 8, 2, [4099, 32768, 1000], 32768), (1, 1, 1, [333] * 300, 333), (1, 4, 1, [333], 60000),
    (4, 4, 1, [70001, 4099], 70001), (2, 8, 8, [1000], 32768), (3, 4, 2, [333, 40], 333),
    (17, 1, 1, [32768], 32768), (32, 4, 1, [4099, 333], 4099), (5, 4, 2, [32768], 32768),
    (64, 4, 1, [70001], 70001), (300, 4, 1, [32768, 4099], 32768), (600, 2, 2, [4099], 4099), (300, 4, 1, [1000], 9000)])
def test_every_run_of_keys_counts(T, group, KV, lens, cap, bits, hd):
    """Keys that all weigh alike, each run of 16 in a dim of its own (as far as the dims go): a tile or a split
    left out, or counted twice, is far outside of the bound (the CPU tests of the bound show it)."""
    S, M = len(lens), max(lens)
    g = torch.Generator()
    g.manual_seed(T + M)
    c = ll.KVQCache.empty(S, KV, max(M, cap), hd, bits)
    k, v = (torch.zeros(S, M, KV, hd) for _ in range(2))
    for s, n in enumerate(lens):
        for h in range(KV):
            k[s, :n, h], v[s, :n, h] = kvq_keys.key_values(n, hd, g)
    c.write(k.cuda(), v.cuda(), i32(lens), i32(lens))
    q = torch.randn(S, T, KV * group, hd, generator=gen(2), device="cuda").bfloat16()
    out = c.attention(q, i32(lens))
    for s in range(S) if S < 10 else (0, 151, S - 1):
        last = (lens[s] - T + torch.arange(T, device="cuda")).repeat_interleave(group)
        for h in range(KV):
            vals = []
            for codes, params in ((c.k_codes, c.k_params), (c.v_codes, c.v_params)):
                codes, params = codes[s, h, :lens[s]], params[s, h, :lens[s]].cpu()
                el = codes.long() if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
                code = el[:, kvq_ref.place(hd).cuda()].unflatten(-1, (hd // 32, 32)).cpu()
                vals.append(kvq_ref.values(params[..., 0], params[..., 1], code).cuda())
            o, tol = kvq_keys.attend(q[s, :, h * group:(h + 1) * group].double().reshape(-1, hd), vals[0], vals[1], last)
            off = (out[s, :, h * group:(h + 1) * group].double().reshape(-1, hd) - o).abs()
            assert bool((off <= tol).all()), (s, h, float((off / tol).max()))


@pytest.mark.parametrize("T,group,M,cap", [(1, 4, 333, 333), (1, 1, 3000, 40000), (4, 4, 333, 333), (40, 2, 333, 333), (24, 4, 500, 60000), (300, 4, 2000, 2000),
                                           (300, 4, 2000, 9000)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("mag", [1e4, 1e6, 3e7, 1e8, 1e9, 1e12, 1e25])
def test_scores_far_apart(T, group, M, cap, hd, mag):
    """Queries so large that the largest score wins outright, at any magnitude: what a row gives is its best key's V. The keys
    are whole numbers that the packed rows hold exactly, and queries small whole numbers times a power of
    two, so that the scores of a row (before scale) are exact, and the best and the next far apart or equal."""
    KV = 2
    g = gen(T + M)
    k = torch.randint(-7, 9, (1, M, KV, hd), generator=g, device="cuda").float()
    k[..., ::32], k[..., 1::32] = -7.0, 8.0  # every group's codes 0 and 15, step 1
    v = torch.randint(0, 16, (1, M, KV, hd), generator=g, device="cuda").float()
    v[..., ::32], v[..., 1::32] = 0.0, 15.0
    c = ll.KVQCache.empty(1, KV, max(M, cap), hd, 4)
    c.write(k, v, i32([M]))
    q = torch.randint(-3, 4, (1, T, KV * group, hd), generator=g, device="cuda").float()
    e = int(torch.log2(torch.tensor(mag)))
    out = c.attention((q * 2.0 ** e).bfloat16(), i32([M]), scale=1.0)
    for h in range(KV):
        s = q[0, :, h * group:(h + 1) * group].double() @ k[0, :, h].double().T  # [T, group, M]
        s.masked_fill_(torch.arange(M, device="cuda") > M - T + torch.arange(T, device="cuda")[:, None, None], float("-inf"))
        best = (s == s.amax(-1, keepdim=True)).double()  # (the others are 2^13 log2 units and more behind)
        want = (best @ v[0, :, h].double()) / best.sum(-1, keepdim=True)
        got = out[0, :, h * group:(h + 1) * group].double()
        # bf16's rounding, the weights' to fp16 and sums of few of them; and, where several keys are best, their weights against each
        # other: a score is s * fac - m in fp32, in one rounding or in two of 2^-24 of it each (kvq_above), so that equal
        # scores of different blocks or tiles may come out u = |score| 2^-23 log2 units apart. Weights that are off by factors of
        # at most 2^u move a mean by at most 2^u - 1 of the values' spread, and never out of it.
        vb = torch.where(best[..., None] > 0, v[0, :, h].double(), torch.nan)
        spread = torch.nan_to_num(vb, nan=-1e9).amax(-2) - torch.nan_to_num(vb, nan=1e9).amin(-2)
        u = s.amax(-1, keepdim=True).abs() * 2.0 ** e * 1.4427 * 2.0 ** -23
        tol = want.abs() * (2.0 ** -8 + 2.0 ** -11) + 2.0 ** -20 + spread * (2.0 ** u.clamp(max=1.0) - 1.0)
        assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())

"""The packed KV cache's calls on the GPU against their definition (kvq_ref): the
bytes a write leaves and the rows a read gives, bit for bit; attention over packed
rows in 64 bits, within the bound of its roundings."""
import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll
import kvq_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_megakernel_persistent_gb300 import build
    build.build()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows_of(g, S, T, H, hd, dtype, layout):
    """[S, T, H, hd] values in one of the layouts a program has them in."""
    if layout == "fused":  # the rows of a projection: other columns on both sides
        return torch.randn(S, T, 3 * H + 2, hd, generator=g, device="cuda", dtype=torch.float32).to(dtype)[:, :, H + 1:2 * H + 1]
    if layout == "cache":
        return torch.randn(S, H, T, hd, generator=g, device="cuda", dtype=torch.float32).to(dtype).transpose(1, 2)
    return torch.randn(S, T, H, hd, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def filled_cache(S, KV, M, hd, bits):
    """A cache whose every byte is a mark."""
    c = ll.KVQCache.empty(S, KV, M, hd, bits)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    for t in (c.k_params, c.v_params):
        t.view(torch.int16).fill_(0x7E5A)  # a NaN
    return c


def expect_rows(x, bits):
    lo, step, code = kvq_ref.quantise(x, bits)
    codes, params = kvq_ref.pack(lo, step, code, bits)
    return codes, params, kvq_ref.values(lo, step, code)


def same_params(a, b):
    """Equal bit patterns, but that a NaN is any NaN."""
    ai, bi = a.contiguous().view(torch.int16), b.contiguous().view(torch.int16)
    return bool(((ai == bi) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,T,KV,layout,ragged", [(1, 1, 1, "plain", False), (1, 1, 8, "fused", False), (3, 5, 2, "fused", True),
                                                  (2, 33, 3, "cache", False), (4, 70, 8, "plain", True)])
def test_write_and_read_back(bits, hd, dtype, S, T, KV, layout, ragged):
    M = T + 9
    g = gen(7 * S + T)
    k, v = rows_of(g, S, T, KV, hd, dtype, layout), rows_of(g, S, T, KV, hd, dtype, layout) * 3 + 1
    n = [T] * S
    lens = [min(M, T + 2 * s) for s in range(S)]
    if ragged:
        n = [(T * (s + 1)) // S if s != 1 else 0 for s in range(S)]
        lens[2] = n[2] - 1  # its first token is at position -1: skipped
        lens[0] = M + 1     # its last token is past the end: skipped
    c = filled_cache(S, KV, M, hd, bits)
    c.write(k, v, i32(lens), i32(n) if ragged else None)
    ko, vo = (torch.full((S, T, KV, hd), 77.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(ko, vo, i32(lens), i32(n) if ragged else None)
    torch.cuda.synchronize()
    for x, codes, params, out in ((k, c.k_codes, c.k_params, ko), (v, c.v_codes, c.v_params, vo)):
        wc, wp, val = expect_rows(x, bits)
        want_codes = torch.full_like(codes.cpu(), 0xA5)
        want_params = torch.full_like(params.cpu().view(torch.int16), 0x7E5A).view(torch.float16)
        want_out = torch.full((S, T, KV, hd), 77.0, dtype=torch.bfloat16)
        for s in range(S):
            for j in range(n[s]):
                p = lens[s] - n[s] + j
                if 0 <= p < M:
                    want_codes[s, :, p] = wc[s, j]
                    want_params[s, :, p] = wp[s, j]
                    want_out[s, j] = val[s, j].float().bfloat16()
        assert torch.equal(codes.cpu(), want_codes)
        assert same_params(params.cpu(), want_params)
        assert torch.equal(out.cpu(), want_out)


@pytest.mark.parametrize("bits", [4, 8])
def test_write_within_half_a_step(bits):
    """A value is read back within half a step, the roundings of lo, step and the value beside it."""
    g = gen(3)
    x = (torch.randn(1, 64, 2, 128, generator=g, device="cuda") * 2).bfloat16()
    c = ll.KVQCache.empty(1, 2, 64, 128, bits)
    c.write(x, x, i32([64]))
    lo, step = (c.k_params[..., i].float().transpose(1, 2).repeat_interleave(32, -1) for i in (0, 1))
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    c.read(ko, vo, i32([64]))
    assert torch.equal(ko, vo)
    # half a step; the top code's step rounding; lo, the fp16 value and the bf16 output
    tol = step * (0.5 + (2 ** bits - 1) * 2.0 ** -11) + lo.abs() * 2.0 ** -11 + ko.float().abs() * (2.0 ** -11 + 2.0 ** -8)
    assert bool(((ko.float() - x.float()).abs() <= tol).all())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_write_special_values(bits, dtype):
    inf, nan = float("inf"), float("nan")
    x = torch.randn(1, 16, 1, 64, generator=gen(5), device="cuda")
    x[0, 0] = 0.0
    x[0, 1] = -0.0
    x[0, 2] = 3.25
    x[0, 3, 0, :32] = 1e-30
    x[0, 4, 0, 5] = nan
    x[0, 5, 0, 40] = inf
    x[0, 6, 0, 3] = -inf
    x[0, 7, 0, 2] = 3e38
    x[0, 8, 0, :32] = -1e6
    x[0, 9] = torch.linspace(-70000, 70000, 64, device="cuda")
    x[0, 10] = torch.linspace(0, 1e-6, 64, device="cuda")  # steps among fp16's smallest numbers
    x[0, 11, 0, ::2] = 60000.0
    x[0, 11, 0, 1::2] = -60000.0
    x[0, 12, 0, :32] = 1000.0 + torch.arange(32, device="cuda") * 1e-4  # a range far below lo's rounding
    x = x.to(dtype)
    c = ll.KVQCache.empty(1, 1, 16, 64, bits)
    c.write(x, x, i32([16]))
    ko, vo = (torch.empty(1, 16, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(ko, vo, i32([16]))
    wc, wp, val = expect_rows(x, bits)
    bad = torch.isnan(wp[..., 0, 0]) | torch.isnan(wp[..., 1, 0])
    assert same_params(c.k_params.cpu()[0, 0], wp[0, :, 0])
    want = val.float().bfloat16()
    got = ko.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and int(torch.isnan(got).sum()) == 32 and int(bad.sum()) == 1
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok]) and bool(torch.isfinite(got[ok].float()).all())
    assert torch.equal(ko.view(torch.int16), vo.view(torch.int16))


def make_cache(seed, S, KV, M, hd, bits, lens, cap=None):
    """A cache (of cap positions, M unless given) of M random rows; what lies past a sequence's length is NaN. Also the
    rows' values [S, KV, M, hd], float64."""
    g = gen(seed)
    k = torch.randn(S, M, KV, hd, generator=g, device="cuda").bfloat16()
    k[..., ::16] *= 4
    v = torch.randn(S, M, KV, hd, generator=g, device="cuda").bfloat16()
    c = filled_cache(S, KV, cap or M, hd, bits)
    full = i32([M] * S)
    c.write(k, v, full)
    vals = []
    for params, codes in ((c.k_params[:, :, :M], c.k_codes[:, :, :M]), (c.v_params[:, :, :M], c.v_codes[:, :, :M])):
        el = codes.long() if bits == 8 else torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
        code = el[..., kvq_ref.place(hd).cuda()].unflatten(-1, (hd // 32, 32))
        vals.append(kvq_ref.values(params[..., 0].cpu(), params[..., 1].cpu(), code.cpu()).cuda())
    for s, n in enumerate(lens):
        n = max(n, 0)
        for t in (c.k_codes, c.v_codes):
            t[s, :, n:] = 0xFF
        for t in (c.k_params, c.v_params):
            t[s, :, n:] = float("nan")
    return c, vals[0], vals[1]


def check_attention(c, kv, vv, q, lens, n, out, scale=None, mark=None):
    S, T, H, hd = q.shape
    KV, M = c.n_kv_heads, c.max_seq
    G = H // KV
    for s in range(S):
        if mark is not None and n[s] < T:
            assert bool((out[s, n[s]:] == mark).all())
        if n[s] == 0:
            continue
        L = max(0, min(lens[s], M))
        last = (lens[s] - n[s] + torch.arange(n[s], device="cuda")).repeat_interleave(G)
        for h in range(KV):
            qs = q[s, :n[s], h * G:(h + 1) * G].double().reshape(-1, hd)
            o, tol = kvq_ref.attend(qs, kv[s, h, :L], vv[s, h, :L], last, scale)
            got = out[s, :n[s], h * G:(h + 1) * G].double().reshape(-1, hd)
            off = (got - o).abs()
            assert bool((off <= tol).all()), (s, h, float((off / tol).max()), float(off.max()))
            assert bool((got[last < 0] == 0).all())


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 255, 256, 257, 511, 512, 513, 700]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,KV", [(1, 3), (2, 2), (3, 1), (4, 8), (7, 1), (8, 2)])
@pytest.mark.parametrize("max_len", [0, 1])
def test_decode_attention(bits, hd, group, KV, max_len):
    S, M = len(LENS), 701
    c, kv, vv = make_cache(11 + hd + group, S, KV, M, hd, bits, LENS)
    q = torch.randn(S, 1, KV * group, hd, generator=gen(2), device="cuda").bfloat16() * 2
    out = c.attention(q, i32(LENS), max_len=max_len)
    check_attention(c, kv, vv, q, LENS, [1] * S, out)
    assert torch.equal(out, c.attention(q, i32(LENS), max_len=max_len))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("cap", [460, 60000])  # laid out for short lengths (few splits), and for long ones (many, most empty)
@pytest.mark.parametrize("T,group", [(2, 4), (3, 3), (2, 8), (4, 4), (16, 1), (5, 4), (17, 1), (33, 2), (70, 4), (129, 3), (150, 8)])
def test_chunk_attention(bits, hd, T, group, cap):
    KV, M = 2, 460
    # (the last two reach before the start, and past the end where there is one)
    lens = [T, T + 1, 460, 300, 0, 64 + T, T // 2, 461 if cap == M else 459]
    n = [T, 1, T, T // 2, T, 0, T, T]
    S = len(lens)
    c, kv, vv = make_cache(5 + T, S, KV, M, hd, bits, lens, cap)
    q = torch.randn(S, T, KV * group, hd, generator=gen(4), device="cuda").bfloat16()
    out = torch.full_like(q, 9.0)
    c.attention(q, i32(lens), i32(n), out=out)
    check_attention(c, kv, vv, q, lens, n, out, mark=9.0)
    again = torch.full_like(q, 9.0)
    c.attention(q, i32(lens), i32(n), out=again)
    assert torch.equal(out, again)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,group,M,cap", [(300, 4, 2100, 2100), (513, 2, 600, 600), (1000, 1, 1000, 1000), (600, 4, 2100, 2100),
                                           (1000, 1, 1000, 9000), (1025, 8, 1100, 1100), (70, 4, 5000, 5000), (64, 2, 9001, 70001)])
@pytest.mark.parametrize("hd", [64, 128])
def test_long_chunk_attention(bits, hd, T, group, M, cap):
    lens = [M, M - 3]
    c, kv, vv = make_cache(8, 2, 1, M, hd, bits, lens, cap)
    q = torch.randn(2, T, group, hd, generator=gen(6), device="cuda").bfloat16()
    out = c.attention(q, i32(lens), scale=0.21)
    check_attention(c, kv, vv, q, lens, [T, T], out, scale=0.21)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_long_decode(hd, bits):
    lens = [70001, 40000]
    c, kv, vv = make_cache(9, 2, 1, 70001, hd, bits, lens)
    q = torch.randn(2, 1, 4, hd, generator=gen(6), device="cuda").bfloat16()
    check_attention(c, kv, vv, q, lens, [1, 1], c.attention(q, i32(lens)))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,group", [(1, 4), (2, 5), (2, 8)])
@pytest.mark.parametrize("KV,lens,cap", [(8, [1], 32768), (8, [385], 32768), (8, [4099], 32767), (8, [2000], 8192), (1, [3001], 60001),
                                         (2, [777], 9000), (8, [1500, 64], 32768), (3, [3000, 1, 0], 20001), (7, [5003], 5003)])
def test_decode_attention_of_few_sequences(bits, hd, T, group, KV, lens, cap):
    """Laid out for few units of long rows: blocks of 8 and 16 warps, 6 and 12 splits, most of them with little to do."""
    S, M = len(lens), max(lens)
    c, kv, vv = make_cache(21 + KV, S, KV, M, hd, bits, lens, cap)
    q = torch.randn(S, T, KV * group, hd, generator=gen(2), device="cuda").bfloat16() * 2
    out = c.attention(q, i32(lens))
    check_attention(c, kv, vv, q, lens, [T] * S, out)
    assert torch.equal(out, c.attention(q, i32(lens)))


@pytest.mark.parametrize("T,group,cap", [(1, 4, 200), (3, 4, 200), (40, 2, 200), (40, 2, 70000)])
@pytest.mark.parametrize("mag", [1e-30, 1e-3, 60.0, 1e30])
def test_query_magnitudes(T, group, cap, mag):
    """Queries far outside fp16's range: each row is scaled by a power of two."""
    M, KV, hd = 200, 2, 64
    c, kv, vv = make_cache(10, 1, KV, M, hd, 4, [M], cap)
    q = (torch.randn(1, T, KV * group, hd, generator=gen(6), device="cuda") * mag).bfloat16()
    q[0, 0, 0] = 0  # a row of zeros attends evenly
    scale = 0.125 if mag < 1e3 else 1e-31
    out = c.attention(q, i32([M]), scale=scale)
    check_attention(c, kv, vv, q, [M], [T], out, scale=scale)


@pytest.mark.parametrize("T,group,cap", [(1, 4, 333), (4, 4, 333), (5, 1, 333), (24, 4, 333), (200, 2, 333), (24, 4, 60000),
                                         (200, 2, 60000), (200, 4, 20000)])
@pytest.mark.parametrize("bits", [4, 8])
def test_nan_reaches_only_rows_that_see_it(T, group, cap, bits):
    KV, hd, M = 1, 128, 333
    lens = [M]
    c, kv, vv = make_cache(12, 1, KV, M, hd, bits, lens, cap)
    q = torch.randn(1, T, group, hd, generator=gen(6), device="cuda").bfloat16()
    at = M - (T + 1) // 2  # seen by the later half of the tokens
    base = c.attention(q, i32(lens))
    saved = c.v_params.clone()
    c.v_params[0, 0, at, 2] = float("nan")  # group 2 of a V row
    out = c.attention(q, i32(lens))
    sees = (M - T + torch.arange(T, device="cuda")) >= at
    assert bool(torch.isnan(out[0, sees][..., 64:96]).all())
    assert torch.equal(out[0, ~sees], base[0, ~sees])
    assert torch.equal(out[0, sees][..., :64], base[0, sees][..., :64])
    assert torch.equal(out[0, sees][..., 96:], base[0, sees][..., 96:])
    c.v_params.copy_(saved)
    c.k_params[0, 0, at, 1] = float("nan")  # a K row: the rows that see it have no softmax
    out = c.attention(q, i32(lens))
    assert bool(torch.isnan(out[0, sees]).all()) and torch.equal(out[0, ~sees], base[0, ~sees])


def test_strided_sequences_past_32_bits():
    """Sequences far apart in one allocation: byte offsets past 2^32."""
    KV, M, hd, bits, S = 2, 50, 128, 8, 3
    gap = 1 << 24  # rows from sequence to sequence: 2 GB of codes
    codes = [torch.empty(S * gap * hd, dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.empty(S * gap * hd // 16, dtype=torch.float16, device="cuda") for _ in range(2)]
    kc, vc = (t.as_strided((S, KV, M, hd), (gap * hd, M * hd, hd, 1)) for t in codes)
    kp, vp = (t.as_strided((S, KV, M, hd // 32, 2), (gap * hd // 16, M * hd // 16, hd // 16, 2, 1)) for t in params)
    c = ll.KVQCache(kc, kp, vc, vp, bits)
    near = ll.KVQCache.empty(S, KV, M, hd, bits)
    k, v = (torch.randn(S, M, KV, hd, generator=gen(i), device="cuda").bfloat16() for i in (1, 2))
    q = torch.randn(S, 1, 8, hd, generator=gen(3), device="cuda").bfloat16()
    q2 = torch.randn(S, 20, 8, hd, generator=gen(3), device="cuda").bfloat16()
    lens = i32([50, 49, 50])
    for x in (c, near):
        x.write(k, v, i32([50] * 3))
    assert torch.equal(kc, near.k_codes) and torch.equal(vp, near.v_params)
    assert torch.equal(c.attention(q, lens), near.attention(q, lens))
    assert torch.equal(c.attention(q2, lens), near.attention(q2, lens))
    outs = [torch.empty(S, M, KV, hd, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    c.read(outs[0], outs[1], i32([50] * 3))
    near.read(outs[2], outs[3], i32([50] * 3))
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


@pytest.mark.parametrize("T,cap", [(1, 400), (4, 400), (40, 400), (300, 400), (1, 40000), (300, 40000)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_bad_queries_stay_in_their_rows(T, cap, hd, value):
    """A query row with a NaN or an infinity has no softmax: NaN, and the other rows as they are without it."""
    M, KV, group = 400, 2, 4
    c, kv, vv = make_cache(17, 1, KV, M, hd, 4, [M], cap)
    q = torch.randn(1, T, KV * group, hd, generator=gen(6), device="cuda").bfloat16()
    base = c.attention(q, i32([M]))
    bad = torch.zeros(1, T, KV * group, dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (T // 2, 3), (T - 1, KV * group - 1)):
        q[0, t, h, (7 * t + h) % hd] = value
        bad[0, t, h] = True
    out = c.attention(q, i32([M]))
    assert bool(torch.isnan(out[bad]).all())
    assert torch.equal(out[~bad], base[~bad])


def test_rows_past_32_bits():
    """One sequence whose codes reach past 2^31 bytes. Every position holds the same K and V row but three (the first, one in
    the middle, the last), whose K rows win by far in turn: each query row gives its key's V."""
    M, hd, bits = (1 << 24) + 5, 128, 8
    c = ll.KVQCache.empty(1, 1, M, hd, bits)
    g = gen(31)
    k = torch.randn(1, 1, 1, hd, generator=g, device="cuda").bfloat16() * 0.01
    v = torch.randn(1, 1, 1, hd, generator=g, device="cuda").bfloat16()
    c.write(k.expand(1, M, 1, hd), v.expand(1, M, 1, hd), i32([M]))
    at = [0, M // 2 + 1, M - 1 - 400]
    rows = torch.zeros(3, hd, device="cuda")
    for i, p in enumerate(at):
        rows[i, 32 * i:32 * i + 32] = 16.0 * torch.randn(32, generator=g, device="cuda").sign()
        vi = torch.randn(1, 1, 1, hd, generator=g, device="cuda").bfloat16()
        c.write(rows[i].bfloat16().view(1, 1, 1, hd), vi, i32([p + 1]))
    back = [torch.empty(1, 1, 1, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = []
    for p in at:
        c.read(back[0], back[1], i32([p + 1]))
        want.append(back[1].flatten().clone())
    for T in (1, 4, 40, 400):
        q = rows.bfloat16()[torch.arange(4 * T, device="cuda") % 3].view(1, T, 4, hd)
        out = c.attention(q, i32([M])).view(4 * T, hd)
        for r in range(4 * T):
            # (its key's score is 16 * 16 * 32 / sqrt(128) = 724 above the others': their weights are zeros; the product with
            # q is exact but for the K codes, whose group is +-16 alone, and V comes back as it is read)
            assert torch.equal(out[r], want[r % 3]), (T, r)


@pytest.mark.parametrize("S,KV", [(65535, 1), (1, 32767), (300, 200)])
@pytest.mark.parametrize("T", [1, 17])
def test_many_sequences_and_heads(S, KV, T):
    """The largest counts of sequences and heads. With one position per token, each row attends to those before it."""
    M, hd, bits = 17, 64, 4
    c = ll.KVQCache.empty(S, KV, M, hd, bits)
    k, v = (torch.randn(S, T, KV, hd, generator=gen(i), device="cuda").bfloat16() for i in (1, 2))
    q = torch.randn(S, T, KV, hd, generator=gen(3), device="cuda").bfloat16()
    lens = torch.full((S,), T, dtype=torch.int32, device="cuda")
    c.write(k, v, lens)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    c.read(kb, vb, lens)
    out = c.attention(q, lens)
    for s, h in ((0, 0), (S - 1, KV - 1), (S // 2, KV // 3), (S // 3, KV // 2)):
        one = ll.KVQCache(c.k_codes[s:s + 1, h:h + 1], c.k_params[s:s + 1, h:h + 1], c.v_codes[s:s + 1, h:h + 1],
                          c.v_params[s:s + 1, h:h + 1], bits)
        vals = []
        for x, codes, params, b in ((k, one.k_codes, one.k_params, kb), (v, one.v_codes, one.v_params, vb)):
            wc, wp, val = expect_rows(x[s, :, h], bits)
            assert torch.equal(codes[0, 0, :T].cpu(), wc) and same_params(params[0, 0, :T].cpu(), wp)
            assert torch.equal(b[s, :, h].cpu(), val.float().bfloat16())
            vals.append(val.cuda()[None, None])
        check_attention(one, vals[0], vals[1], q[s:s + 1, :, h:h + 1], [T], [T], out[s:s + 1, :, h:h + 1])


@pytest.mark.parametrize("T,cap", [(1, 100), (3, 100), (30, 100), (30, 20000)])
def test_strided_queries_and_outputs(T, cap):
    """q as columns of a fused projection, out as columns of a wider buffer: the rest of it stays."""
    S, KV, group, hd, M = 3, 2, 4, 64, 100
    lens = [100, 37, 64]
    c, kv, vv = make_cache(15, S, KV, M, hd, 4, lens, cap)
    H = KV * group
    q = torch.randn(S, T, H + 2 * KV, hd, generator=gen(1), device="cuda").bfloat16()[:, :, :H]
    wide = torch.full((S, T, H + 3, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    c.attention(q, i32(lens), out=wide[:, :, 1:H + 1])
    check_attention(c, kv, vv, q, lens, [T] * S, wide[:, :, 1:H + 1])
    assert bool((wide[:, :, 0] == 5).all()) and bool((wide[:, :, H + 1:] == 5).all())
    # one query row broadcast to every token
    qb = q[:, :1].expand(S, T, H, hd)
    check_attention(c, kv, vv, qb, lens, [T] * S, c.attention(qb, i32(lens)))


def test_decode_loop_captured_and_on_a_side_stream():
    """A decode loop's calls together: a token written, then attention over all so far,
    captured once and replayed with new tokens and lengths, on a stream of its own."""
    S, KV, group, hd, M, bits = 3, 2, 4, 64, 40, 4
    c = filled_cache(S, KV, M, hd, bits)
    k, v = (torch.empty(S, 1, KV, hd, device="cuda") for _ in range(2))
    q = torch.empty(S, 1, KV * group, hd, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")

    def step():
        c.write(k, v, lens)
        c.attention(q, lens, out=out)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step()
    torch.cuda.current_stream().wait_stream(st)
    hist = []
    for i in range(M):
        kn, vn = (torch.randn(S, 1, KV, hd, generator=gen(100 * j + i), device="cuda") for j in (1, 2))
        q.copy_(torch.randn(S, 1, KV * group, hd, generator=gen(300 + i), device="cuda").bfloat16())
        k.copy_(kn)
        v.copy_(vn)
        lens += i32([1, 1, 0])  # the third place of the batch stays free
        g.replay()
        hist.append((kn, vn))
        if i in (0, 1, 17, M - 1):
            torch.cuda.synchronize()
            kk, vv = (torch.cat([x[j] for x in hist], 1) for j in (0, 1))
            kq, vq = (kvq_ref.values(*kvq_ref.quantise(x, bits)).transpose(1, 2).cuda() for x in (kk, vv))
            check_attention(c, kq, vq, q, [i + 1, i + 1, 0], [1] * S, out)


def test_calls_at_once_on_two_streams():
    """Single tokens, chunks and prompts over one cache, on two streams at once and as two graphs replayed at once,
    while a third writes another cache."""
    KV, M, hd = 4, 3000, 64
    c, kv, vv = make_cache(23, 2, KV, M, hd, 4, [M, M - 7])
    other = ll.KVQCache.empty(2, KV, M, hd, 8)
    rows = torch.randn(2, M, KV, hd, generator=gen(1), device="cuda").bfloat16()
    lens = i32([M, M - 7])
    qs = [[torch.randn(2, t, 4 * KV, hd, generator=gen(40 + i), device="cuda").bfloat16() for t in (1, 9, 700)] for i in range(2)]
    want = [[c.attention(q, lens) for q in x] for x in qs]
    outs = [[torch.zeros_like(q) for q in x] for x in qs]
    streams = [torch.cuda.Stream() for _ in range(3)]

    def run(i):
        for q, o in zip(qs[i], outs[i]):
            c.attention(q, lens, out=o)

    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            run(i)
    for how in range(2):
        for x in outs:
            for o in x:
                o.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay() if how else run(i)
            with torch.cuda.stream(streams[2]):
                other.write(rows, rows, lens)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(outs, want) for a, b in zip(x, y))
    last = ll.KVQCache.empty(2, KV, M, hd, 8)
    last.write(rows, rows, lens)
    assert torch.equal(other.k_codes, last.k_codes) and torch.equal(other.v_params, last.v_params)


def test_first_calls_of_a_process_may_be_captured():
    """No call needs one before it outside a graph: a new process captures its first write, read and attention (of
    one token, a few and many), replays them and gets what the plain calls give."""
    code = """
import torch
from decode_megakernel_persistent_gb300 import ll
c = ll.KVQCache.empty(1, 2, 5000, 64, 4)
x = torch.randn(1, 2200, 2, 64, device="cuda").bfloat16()
qs = [torch.randn(1, t, 16, 64, device="cuda").bfloat16() for t in (1, 12, 2200)]
outs = [torch.full_like(q, 7.0) for q in qs]
back = [torch.empty_like(x) for _ in range(2)]
lens = torch.tensor([2200], dtype=torch.int32, device="cuda")
def run():
    c.write(x, x, lens)
    c.read(back[0], back[1], lens)
    for q, o in zip(qs, outs):
        c.attention(q, lens, out=o)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs + back]
for t in outs + back:
    t.zero_()
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs + back))
assert all(bool((t != 7).any()) and bool(torch.isfinite(t.float()).all()) for t in got)
print("same")
"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_prompt_then_tokens_equals_one_chunk():
    """A prompt written and attended in pieces gives what the whole prompt gives."""
    KV, group, hd, n = 2, 4, 64, 90
    k, v = (torch.randn(1, n, KV, hd, generator=gen(i), device="cuda").bfloat16() for i in (1, 2))
    q = torch.randn(1, n, KV * group, hd, generator=gen(3), device="cuda").bfloat16()
    one, parts = (ll.KVQCache.empty(1, KV, n, hd, 4) for _ in range(2))
    one.write(k, v, i32([n]))
    whole = one.attention(q, i32([n]))
    got, at = [], 0
    for step in (50, 1, 3, 30, 6):
        sl = slice(at, at + step)
        at += step
        parts.write(k[:, sl], v[:, sl], i32([at]))
        got.append(parts.attention(q[:, sl], i32([at])))
    assert torch.equal(parts.k_codes, one.k_codes) and torch.equal(parts.v_params, one.v_params)
    kq, vq = (kvq_ref.values(*kvq_ref.quantise(x, 4)).transpose(1, 2).cuda() for x in (k, v))
    check_attention(one, kq, vq, q, [n], [n], whole)
    check_attention(one, kq, vq, q, [n], [n], torch.cat(got, 1))

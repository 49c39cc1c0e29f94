"""The packed KV cache's operators in their plain form, and the cases they are measured on.

A packed cache holds K and V rows of (sequence, KV head, position) in 4 or 8
bits. A row is cut into groups of 32 dims; a group keeps lo and step in fp16,
and a code c stands for the value fp16(lo + step * c). Byte order within a row:
dim d = 32 * gr + 4 * g + i (gr the group, g < 8, i < 4) is the row's element
(g * (head_dim / 32) + gr) * 4 + i; 4-bit elements sit two to a byte, the even
one in the low half.

  * "roundtrip": the cache's write of new tokens (rows of a projection's output,
    or of a whole bf16 cache) and the read of the same positions back as bf16
    (token j of a sequence's n tokens at position len - n + j, as below);
  * "attention": softmax(q k^T / sqrt(head_dim)) v over the packed positions
    0..p of each query token, with one query token a sequence (a decode step) or
    a chunk of them (a prompt, or drafted tokens to check), causal. Token j of a
    sequence's n tokens is at position len - n + j; a row with no position to
    look at gives zeros, and rows past a sequence's n tokens are left alone.
"""
import math

import torch

own = False

# Head layouts of the framework's models: 32 query heads on 8 KV heads of 64
# dims, 24 on 8 and 32 on 8 of 128, 4 on 2 of 64 in the small test model.


def listed():
    def rt(name, **k):
        return dict(dict(name=name, op="roundtrip", bits=4, seqs=1, tokens=1, kv=8, hd=64, fp32=False, fused=False, ragged=False, cap=1024), **k)

    def at(name, **k):
        return dict(dict(name=name, op="attention", bits=4, seqs=1, tokens=1, heads=32, kv=8, hd=64, length=1024, ragged=False), **k)

    return [
        # one sequence's new token in a decode step (fp32 rows of the projection's output): latency
        rt("append one token", fp32=True, fused=True),
        # a batch's new tokens
        rt("append 64 sequences, 8 bits", bits=8, seqs=64, hd=128, cap=256),
        # prompts of several sequences, padded to the longest, in the projection's rows
        rt("prompts of 3, ragged", seqs=3, tokens=1023, hd=128, fp32=True, fused=True, ragged=True, cap=2048),
        # a whole bf16 cache packed: 16 layers of 32768 positions
        rt("pack a cache of 16 layers", seqs=16, tokens=32768, cap=32768),
        # a decode step's attention in the 1B shape at context 1024 and 32768
        at("decode at 1024"),
        at("decode at 32768", length=32768),
        # a batch of decode steps at context 8192 in the 8B shape, lengths of every size
        at("decode 8 ragged", seqs=8, hd=128, length=8192, ragged=True),
        at("decode 64 ragged, 8 bits", bits=8, seqs=64, length=8191, ragged=True),
        # the largest: 32 sequences of 32768 positions, 128 dims
        at("decode 32 at 32768", seqs=32, hd=128, length=32768),
        # four drafted tokens a sequence, checked at once
        at("check 4 drafted tokens", seqs=8, tokens=4, length=4097, ragged=True),
        # a prompt of an odd length behind a cached prefix, in 8 bits
        at("prompt of 1001 behind 500", bits=8, tokens=1001, length=1501),
        # a long prompt in the 8B shape
        at("prompt of 8192", tokens=8192, hd=128, length=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    bits, hd = rng.choice([4, 4, 8]), rng.choice([64, 128])
    kv = rng.choice([1, 2, 8, 8])
    if rng.random() < 0.35:
        seqs = _log(rng, 1, 64)
        tokens = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, min(32768, (1 << 22) // (seqs * kv * (hd // 64)))))
        return dict(op="roundtrip", bits=bits, seqs=seqs, tokens=tokens, kv=kv, hd=hd, fp32=rng.random() < 0.5,
                    fused=rng.random() < 0.5, ragged=rng.random() < 0.5, cap=tokens + rng.randrange(0, 64))
    group = rng.choice([1, 2, 3, 4, 4, 8] if hd == 64 else [1, 2, 3, 4, 4])
    if rng.random() < 0.6:  # one token a sequence
        seqs = _log(rng, 1, 64)
        length = _log(rng, 1, min(32768, (32 * 32768) // seqs))
        tokens = 1
    else:
        seqs = _log(rng, 1, 8)
        tokens = _log(rng, 2, 4096 // seqs)
        length = tokens + rng.choice([0, _log(rng, 1, 4096)])
    return dict(op="attention", bits=bits, seqs=seqs, tokens=tokens, heads=kv * group, kv=kv, hd=hd, length=length, ragged=rng.random() < 0.5)


def _lengths(c, g):
    """Each sequence's length after the call, and its tokens in the call."""
    S, T = c["seqs"], c["tokens"]
    most = c["length"] if c["op"] == "attention" else c["cap"]
    if not c["ragged"]:
        return [most] * S, [T] * S
    r = torch.rand(2, S, generator=g).tolist()
    n = [max(1, min(T, int(x * (T + 1)))) for x in r[1]]
    n[0] = T
    lens = [max(n[s], min(most, int(r[0][s] * (most + 1)))) for s in range(S)]
    lens[0] = most
    if S > 2 and c["op"] == "attention":
        lens[1], n[1] = 0, min(1, T)  # a free place in the batch
    return lens, n


def _groups(x):
    return x.unflatten(-1, (x.shape[-1] // 32, 32))


def _quantise(x, bits, wide=torch.float32):
    """lo and step (as fp16 numbers) and codes of x [..., hd], each by group of 32, in `wide` arithmetic."""
    x = _groups(x.to(wide)).clamp(-60000.0, 60000.0)
    lo = x.amin(-1, keepdim=True).half().to(wide)
    step = ((x.amax(-1, keepdim=True) - lo) / (2 ** bits - 1)).half().to(wide)
    code = torch.where(step > 0, (x - lo) / step, torch.zeros_like(x)).round().clamp(0, 2 ** bits - 1)
    return lo, step, code


def _pack(x, bits):
    """The packed rows of x [..., hd]: codes uint8 [..., hd * bits / 8], params fp16 [..., hd / 32, 2]."""
    lo, step, code = _quantise(x, bits)
    code = code.to(torch.uint8).unflatten(-1, (8, 4)).transpose(-3, -2).flatten(-3)
    if bits == 4:
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    return code.contiguous(), torch.cat([lo, step], -1).half().contiguous()


def _unpack(codes, params, bits, wide=torch.float32):
    """The values the packed rows stand for, [..., hd]."""
    if bits == 4:
        codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    groups = params.shape[-2]
    c = codes.unflatten(-1, (8, groups, 4)).transpose(-3, -2).flatten(-2)
    # (fp32 holds step * c exactly; the sum is rounded to fp16, as the format says)
    return (params[..., 1:2].to(wide) * c.to(wide) + params[..., 0:1].to(wide)).half().to(wide).flatten(-2)


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    S, T, KV, HD, bits = c["seqs"], c["tokens"], c["kv"], c["hd"], c["bits"]
    lens, n = _lengths(c, cpu)
    st = dict(case=c, bits=bits, lens=torch.tensor(lens, dtype=torch.int32, device=dev),
              n=torch.tensor(n, dtype=torch.int32, device=dev) if c["ragged"] else None)
    cap = c["cap"] if c["op"] == "roundtrip" else c["length"]

    def normal(*shape, dtype):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    if c["op"] == "roundtrip":
        dt = torch.float32 if c["fp32"] else torch.bfloat16
        if c["fused"]:  # rows of a fused projection: 4 * KV query heads, then K, then V
            rows = normal(S, T, 6 * KV, HD, dtype=dt)
            st["k"], st["v"] = rows[:, :, 4 * KV:5 * KV], rows[:, :, 5 * KV:]
        else:  # a cache [sequence or layer][KV head][position][dim]
            st["k"], st["v"] = (normal(S, KV, T, HD, dtype=dt).transpose(1, 2) for _ in range(2))
        for x in ("k", "v"):
            st[x + "_codes"] = torch.zeros(S, KV, cap, HD * bits // 8, dtype=torch.uint8, device=dev)
            st[x + "_params"] = torch.zeros(S, KV, cap, HD // 32, 2, dtype=torch.float16, device=dev)
            st[x + "_out"] = torch.zeros(S, KV, T, HD, dtype=torch.bfloat16, device=dev).transpose(1, 2)
        return st
    for x in ("k", "v"):  # keys with some channels larger than the others, as rotary caches have them
        rows = normal(S, KV, cap, HD, dtype=torch.bfloat16)
        if x == "k":
            rows[..., ::16] *= 2
        st[x + "_codes"], st[x + "_params"] = _pack(rows, bits)
    st["q"] = normal(S, T, c["heads"], HD, dtype=torch.bfloat16)
    st["out"] = torch.zeros_like(st["q"])
    return st


def _roundtrip(x, n, bits, wide):
    """The tokens x [S, T, KV, HD] as they are read back, zeros past each sequence's n, in `wide` arithmetic."""
    lo, step, code = _quantise(x, bits, wide)
    val = (lo + step * code).half().to(wide).flatten(-2)
    if n is None:
        return val
    held = torch.arange(x.shape[1], device=x.device) < n[:, None]
    return torch.where(held[..., None, None], val, torch.zeros_like(val))


def run(st):
    c = st["case"]
    if own:
        from decode_megakernel_persistent_gb300 import ll
        if "cache" not in st:  # the cache object a program keeps for as long as the buffers
            st["cache"] = ll.KVQCache(st["k_codes"], st["k_params"], st["v_codes"], st["v_params"], c["bits"])
        cache = st["cache"]
        if c["op"] == "roundtrip":
            cache.write(st["k"], st["v"], st["lens"], st["n"])
            cache.read(st["k_out"], st["v_out"], st["lens"], st["n"])
            return {"k": st["k_out"], "v": st["v_out"]}
        cache.attention(st["q"], st["lens"], st["n"], out=st["out"])
        return st["out"]
    if c["op"] == "roundtrip":
        return {x: _roundtrip(st[x], st["n"], c["bits"], torch.float32).bfloat16() for x in ("k", "v")}
    k = _unpack(st["k_codes"], st["k_params"], c["bits"])
    v = _unpack(st["v_codes"], st["v_params"], c["bits"])
    S, T, HD, KV = c["seqs"], c["tokens"], c["hd"], c["kv"]
    G = c["heads"] // KV
    lens = st["lens"].long()
    n = st["n"].long() if st["n"] is not None else torch.full_like(lens, T)
    j = torch.arange(T, device=lens.device)
    last = (lens - n)[:, None] + j  # each token's own position [S, T]
    q = st["q"].float().unflatten(2, (KV, G)).permute(0, 2, 1, 3, 4).reshape(S, KV, T * G, HD)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(HD)).view(S, KV, T, G, -1)
    seen = torch.arange(s.shape[-1], device=s.device) <= last[..., None]  # [S, T, len]
    s.masked_fill_(~seen[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(S, KV, T * G, -1), v).view(S, KV, T, G, HD) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 2, 1, 3, 4).reshape(S, T, c["heads"], HD)
    return torch.where((j < n[:, None])[..., None, None], o, torch.zeros_like(o)).bfloat16()


def exact(c, seed):
    """The same from the definition in 64 bits, one sequence and KV head at a time."""
    st = prepare(c, seed)
    S, T, KV, HD, bits = c["seqs"], c["tokens"], c["kv"], c["hd"], c["bits"]
    lens = st["lens"].tolist()
    n = st["n"].tolist() if st["n"] is not None else [T] * S
    dev = st["lens"].device
    if c["op"] == "roundtrip":
        res = {}
        for x in ("k", "v"):
            out = torch.zeros(S, T, KV, HD, dtype=torch.float64, device=dev)
            for s in range(S):
                r = st[x][s, :n[s]].double().reshape(n[s], KV, HD // 32, 32)
                lo = r.min(-1).values.half().double()
                step = ((r.max(-1).values - lo) / (2 ** bits - 1)).half().double()
                code = torch.floor((r - lo[..., None]) / step[..., None] + 0.5)
                half = ((r - lo[..., None]) / step[..., None] + 0.5 == code) & (code % 2 == 1)  # ties go to the even code
                code = (code - half.double()).clamp(0, 2 ** bits - 1)
                out[s, :n[s]] = (lo[..., None] + step[..., None] * code).half().double().reshape(n[s], KV, HD)
            res[x] = out
        return res
    G, GR = c["heads"] // KV, HD // 32
    d = torch.arange(HD, device=dev)
    place = ((d % 32 // 4) * GR + d // 32) * 4 + d % 4  # the element of a row that holds dim d
    out = torch.zeros(S, T, c["heads"], HD, dtype=torch.float64, device=dev)

    def rows(codes, params, m):
        b = codes[:m].long()
        e = b[:, place] if bits == 8 else (b[:, place // 2] >> (4 * (place % 2))) & 15
        p = params[:m].double()
        return (p[:, d // 32, 0] + p[:, d // 32, 1] * e.double()).half().double()

    for s in range(S):
        for h in range(KV):
            if not lens[s]:
                continue
            k = rows(st["k_codes"][s, h], st["k_params"][s, h], lens[s])
            v = rows(st["v_codes"][s, h], st["v_params"][s, h], lens[s])
            q = st["q"][s, :n[s], h * G:(h + 1) * G].double()  # [n, G, HD]
            sc = torch.einsum("ngd,ld->ngl", q, k) / math.sqrt(HD)
            pos = lens[s] - n[s] + torch.arange(n[s], device=dev)
            sc = sc.masked_fill(torch.arange(lens[s], device=dev) > pos[:, None, None], float("-inf"))
            out[s, :n[s], h * G:(h + 1) * G] = torch.einsum("ngl,ld->ngd", torch.softmax(sc, -1), v)
    return out


def work(c):
    """Every input read once and every output written once; two flops a multiply-add of the products."""
    g = torch.Generator()
    g.manual_seed(0)
    lens, n = _lengths(c, g)
    row = c["hd"] * c["bits"] // 8 + c["hd"] // 8  # a packed row: codes, and 4 bytes a group
    if c["op"] == "roundtrip":
        rows = 2 * c["kv"] * sum(n)
        return {"bytes": rows * (c["hd"] * (4 if c["fp32"] else 2) + 2 * row + 2 * c["hd"]), "flops": 4 * rows * c["hd"]}
    pairs = sum(m * (m + 1) // 2 - (m - k) * (m - k + 1) // 2 for m, k in zip(lens, n) if m)
    return {"bytes": 2 * c["kv"] * sum(lens) * row + 4 * c["heads"] * c["hd"] * sum(n), "flops": 4 * pairs * c["heads"] * c["hd"]}

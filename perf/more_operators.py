"""What a decode step does around the packed cache's attention, in plain form, and the cases it is measured on.

  * "matvec": y = W x (+ add) for a few rows x and a matrix W held in 4 bits: W[r][k] = lo + step * code, with
    one fp16 pair (lo, step) for each row and group of 32, 64 or 128 inputs. x is bf16, fp32, or e4m3 with a
    scale a row or a 128 inputs.
  * "pack": a bf16 matrix quantised into that form, and read back.
  * "norm": the residual's addition and the RMS norm of the sum, out in bf16, fp32 or e4m3 with scales.
  * "rope": rotary positions of the query and key heads of each sequence's last tokens, in both layouts, on the
    whole head or its first dims, with the frequencies scaled for long contexts or not.
  * "verify": drafted tokens accepted or rejected against the target's probabilities, and the token behind the
    last accepted one drawn, all from given random numbers; with no drafts, plain sampling.

The 4-bit matrix in memory: tiles of 16 rows by 128 inputs, tile (r / 16, k / 128) holding 256 words of 8 codes.
Word (r % 16 / 8) * 128 + (r % 8) * 16 + (k % 32 / 8) * 4 + k % 128 / 32 has inputs k..k+7 (k a multiple of 8); the
i-th of them is at bits (4 f + 3) % 32 and up (turned round at bit 31), f = i / 2 + 4 * (i % 2). Parameters:
[tile row][tile column][group of the tile][row of the tile][lo, step]. What lies past the matrix is 0.
"""
import math

import torch

own = False

TILE = 128


def listed():
    def mv(name, **k):
        return dict(dict(name=name, op="matvec", rows=4096, cols=4096, group=128, tokens=1, x="bf16", scales=0, y="bf16", add=False), **k)

    def norm(name, **k):
        return dict(dict(name=name, op="norm", rows=1, width=2048, fp32=False, residual=True, y="bf16", group=0), **k)

    def rope(name, **k):
        return dict(dict(name=name, op="rope", seqs=1, tokens=1, heads=32, kv=8, hd=64, rot=64, cap=1024, interleaved=False,
                         scaling="none", fp32=False, ragged=False), **k)

    def verify(name, **k):
        return dict(dict(name=name, op="verify", seqs=1, drafts=4, vocab=128256, probs=True, ragged=False, bf16=False, temperature=1.0), **k)

    return [
        # the K projection of one token in the 1B shape: latency
        mv("matvec 512x2048, 1 token", rows=512, cols=2048),
        # gate and up of one token in the 8B shape, stacked
        mv("matvec 28672x4096, 1 token", rows=28672),
        # the logits of four drafted tokens and the one before them, 1B shape, in fp32
        mv("matvec 128256x2048, 5 tokens, logits", rows=128256, cols=2048, group=64, tokens=5, y="fp32"),
        # down of a batch of 64 in the 8B shape, from e4m3 rows, added to the residual
        mv("matvec 4096x14336, 64 tokens, e4m3", cols=14336, tokens=64, x="e4m3", scales=128, add=True),
        # gate's weights of one 8B layer, quantised and read back
        dict(name="pack 14336x4096", op="pack", rows=14336, cols=4096, group=128),
        # the norm in front of a layer's projections, one token in the 1B shape: latency
        norm("norm of one token"),
        # the same for a prompt in the 8B shape, into e4m3 rows for the products
        norm("norm of 8192 tokens, e4m3", rows=8192, width=4096, y="e4m3", group=128),
        # one token's query and key heads in the 1B shape: latency
        rope("rope of one token"),
        # a prompt of 8192 in the 8B shape behind a cached prefix, frequencies scaled
        rope("rope of 8192 tokens, scaled", tokens=8192, hd=128, rot=128, cap=40000, scaling="bands"),
        # four drafted tokens of one sequence: latency
        verify("verify 4 drafts"),
        # a batch with up to seven drafted tokens each
        verify("verify 64 sequences, up to 7 drafts", seqs=64, drafts=7, ragged=True, temperature=0.8),
        # no drafts: a batch's next tokens sampled from bf16 logits
        verify("sample 64 sequences", seqs=64, drafts=0, probs=False, bf16=True, temperature=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["matvec", "matvec", "matvec", "pack", "norm", "rope", "verify", "verify"])
    if op in ("matvec", "pack"):
        group = rng.choice([32, 64, 128, 128])
        rows = _log(rng, 1, 32768)
        cols = _log(rng, 32, min(16384, (1 << 27) // rows))
        if rng.random() < 0.7:  # most matrices are whole tiles
            rows, cols = -(-rows // 16) * 16, -(-cols // TILE) * TILE
        if op == "pack":
            return dict(op=op, rows=rows, cols=cols, group=group)
        x = rng.choice(["bf16", "bf16", "fp32", "e4m3"])
        return dict(op=op, rows=rows, cols=cols, group=group, tokens=rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 2, 64)]), x=x,
                    scales=rng.choice([0, 128]) if x == "e4m3" else 0, y=rng.choice(["bf16", "bf16", "fp32"]), add=rng.random() < 0.3)
    if op == "norm":
        width = rng.choice([64, 128, 256, 2048, 4096, 8192, _log(rng, 1, 16384)])
        y = rng.choice(["bf16", "fp32", "e4m3", "e4m3"])
        return dict(op=op, rows=_log(rng, 1, (1 << 25) // width), width=width, fp32=rng.random() < 0.4, residual=rng.random() < 0.7, y=y,
                    group=rng.choice([0, 128]) if y == "e4m3" else 0)
    if op == "rope":
        hd = rng.choice([64, 64, 128, 128, 80, 96, 256])
        kv = rng.choice([1, 2, 8, 8])
        seqs = _log(rng, 1, 64)
        heads = kv * rng.choice([1, 3, 4, 4, 8])
        tokens = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, min(8192, (1 << 25) // (seqs * (heads + kv) * hd))))
        return dict(op=op, seqs=seqs, tokens=tokens, heads=heads, kv=kv, hd=hd, rot=rng.choice([hd, hd, hd // 2, hd // 4 * 2 - 8]),
                    cap=tokens + _log(rng, 1, 1 << 20), interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "none", "linear", "bands", "ramp"]),
                    fp32=rng.random() < 0.3, ragged=rng.random() < 0.5)
    seqs, drafts = _log(rng, 1, 64), rng.choice([0, 1, rng.randrange(1, 9), rng.randrange(1, 9)])
    return dict(op=op, seqs=seqs, drafts=drafts, vocab=rng.choice([128256, 32000, _log(rng, 2, 128256), _log(rng, 1000, 200000)]),
                probs=drafts > 0 and rng.random() < 0.7, ragged=rng.random() < 0.5, bf16=rng.random() < 0.3,
                temperature=rng.choice([1.0, 1.0, 0.7, 1.3, 0.0]))


def _tiles(n, by):
    return -(-n // by)


def _pack_codes(code):
    """Codes [16 R, 128 K] (whole tiles) as the words' bytes [R, K, 1024]."""
    c = code.to(torch.int64).view(code.shape[0] // 16, 2, 8, code.shape[1] // TILE, 4, 4, 4, 2)  # R, r/8, r%8, K, k%128/32, k%32/8, i/2, i%2
    f = torch.arange(4, device=code.device)[:, None] + 4 * torch.arange(2, device=code.device)
    w = (c << (4 * f)).sum((-1, -2))  # nibble f of the word, before it is turned by 3 bits
    w = ((w << 3) | (w >> 29)) & 0xFFFFFFFF
    w = w.permute(0, 3, 1, 2, 5, 4).contiguous()  # R, K, r/8, r%8, k%32/8, k%128/32
    w = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
    return w.view(w.shape[0], w.shape[1], 256).view(torch.uint8)


def _unpack_codes(codes):
    """The codes [16 R, 128 K] of the words' bytes [R, K, 1024]."""
    R, K, _ = codes.shape
    w = codes.view(torch.int32).view(R, K, 2, 8, 4, 4).permute(0, 2, 3, 1, 5, 4)  # R, r/8, r%8, K, k%128/32, k%32/8
    f = torch.arange(4, device=codes.device, dtype=torch.int32)[:, None] + 4 * torch.arange(2, device=codes.device, dtype=torch.int32)
    turned = ((w >> 3) & 0x1FFFFFFF) | (w << 29)
    return ((turned[..., None, None] >> (4 * f)) & 15).to(torch.uint8).reshape(16 * R, TILE * K)


def _quantise(w, group):
    """lo and step (fp16) [rows, groups, 1] and codes [rows, groups, group] of whole groups w."""
    w = w.float().clamp(-60000.0, 60000.0).unflatten(-1, (w.shape[-1] // group, group))
    lo = w.amin(-1, keepdim=True).half()
    step = ((w.amax(-1, keepdim=True) - lo.float()) / 15).half()
    s = step.float()
    code = torch.where(s > 0, (w - lo.float()) / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(w)).round().clamp(0, 15)
    return lo, step, code


def _pack(w, group):
    """codes and params of a matrix w [rows, cols] of whole groups (or one short group at the end, whose missing inputs are the last one's)."""
    rows, cols = w.shape
    R, K = _tiles(rows, 16), _tiles(cols, TILE)
    whole = torch.cat([w, w[:, -1:].expand(rows, -cols % group)], 1) if cols % group else w
    lo, step, code = _quantise(whole, group)
    c = torch.zeros(16 * R, TILE * K, dtype=torch.uint8, device=w.device)
    c[:rows, :cols] = code.flatten(1)[:, :cols].to(torch.uint8)
    p = torch.zeros(16 * R, K * TILE // group, 2, dtype=torch.float16, device=w.device)
    p[:rows, :lo.shape[1]] = torch.cat([lo, step], -1)
    p = p.view(R, 16, K, TILE // group, 2).permute(0, 2, 3, 1, 4).contiguous()
    return _pack_codes(c), p


def _matrix(codes, params, rows, cols, wide=torch.float32):
    """The matrix that the packed tiles stand for."""
    R, K, per = params.shape[:3]
    p = params.permute(0, 3, 1, 2, 4).reshape(16 * R, K * per, 1, 2).to(wide)
    c = _unpack_codes(codes).view(16 * R, K * per, TILE // per).to(wide)
    return (p[..., 0] + p[..., 1] * c).flatten(1)[:rows, :cols]


TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _to_e4m3(v, group):
    """v [n, width] (fp32) as e4m3 codes and their scales, one for each row (group 0) or group of columns."""
    n, width = v.shape
    g = group or width
    pad = torch.nn.functional.pad(v, (0, -width % g)).view(n, -1, g)
    scale = pad.abs().amax(-1, keepdim=True) / 448
    code = (pad / torch.where(scale > 0, scale, torch.ones_like(scale))).to(torch.float8_e4m3fn)
    return code.view(n, -1)[:, :width].contiguous(), scale[..., 0].contiguous()


def _lengths(c, seed):
    S, T = c["seqs"], c["tokens"]
    if not c["ragged"]:
        return [c["cap"]] * S, [T] * S
    g = torch.Generator()
    g.manual_seed(seed)
    r = torch.rand(2, S, generator=g).tolist()
    n = [max(1, min(T, int(x * (T + 1)))) for x in r[1]]
    return [max(m, min(c["cap"], int(x * (c["cap"] + 1)))) for x, m in zip(r[0], n)], n


SCALING = {"none": None, "linear": dict(kind="linear", factor=4.0), "bands": dict(kind="bands", factor=32.0, low=1.0, high=4.0, length=8192),
           "ramp": dict(kind="ramp", factor=16.0, fast=32.0, slow=1.0, length=4096)}
THETA = 500000.0


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=dtype)

    st = dict(case=c)
    if c["op"] in ("matvec", "pack"):
        R, K = _tiles(c["rows"], 16), _tiles(c["cols"], TILE)
        w = normal(c["rows"], c["cols"], dtype=torch.bfloat16).mul_(0.02)
        if c["op"] == "pack":
            st["w"] = w
            st["codes"] = torch.zeros(R, K, 1024, dtype=torch.uint8, device=dev)
            st["params"] = torch.zeros(R, K, TILE // c["group"], 16, 2, dtype=torch.float16, device=dev)
            st["out"] = torch.zeros_like(w)
            return st
        st["codes"], st["params"] = _pack(w, c["group"])
        x = normal(c["tokens"], c["cols"])
        st["scale"] = None
        if c["x"] == "e4m3":
            st["x"], st["scale"] = _to_e4m3(x, c["scales"])
        else:
            st["x"] = x.to(TYPES[c["x"]])
        st["add"] = normal(c["tokens"], c["rows"]).to(TYPES[c["y"]]) if c["add"] else None
        st["out"] = torch.zeros(c["tokens"], c["rows"], dtype=TYPES[c["y"]], device=dev)
        return st
    if c["op"] == "norm":
        dt = torch.float32 if c["fp32"] else torch.bfloat16
        st["x"] = normal(c["rows"], c["width"]).to(dt)
        st["residual"] = (4 * normal(c["rows"], c["width"])).to(dt) if c["residual"] else None
        st["gain"] = (1 + 0.1 * normal(c["width"])).bfloat16()
        st["new"] = torch.zeros_like(st["x"]) if c["residual"] else None
        st["out"] = torch.zeros(c["rows"], c["width"], dtype=TYPES[c["y"]], device=dev)
        return st
    if c["op"] == "rope":
        lens, n = _lengths(c, seed)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["n"] = torch.tensor(n, dtype=torch.int32, device=dev) if c["ragged"] else None
        rows = normal(c["seqs"], c["tokens"], c["heads"] + 2 * c["kv"], c["hd"], dtype=torch.float32 if c["fp32"] else torch.bfloat16)
        st["q"], st["k"] = rows[:, :, :c["heads"]], rows[:, :, c["heads"]:c["heads"] + c["kv"]]  # of a fused projection
        st["q_out"] = torch.zeros(c["seqs"], c["tokens"], c["heads"], c["hd"], dtype=rows.dtype, device=dev)
        st["k_out"] = torch.zeros(c["seqs"], c["tokens"], c["kv"], c["hd"], dtype=rows.dtype, device=dev)
        return st
    S, D, V = c["seqs"], c["drafts"], c["vocab"]
    logits = normal(S, D + 1, V).mul_(2)
    few = torch.randint(0, V, (S, D + 1, 16), generator=g, device=dev)  # the words that fit: a model's logits are peaked
    logits.scatter_add_(2, few, 8 + 3 * normal(S, D + 1, 16))
    st["logits"] = logits.bfloat16() if c["bf16"] else logits
    T = c["temperature"] or 1.0
    st["u"] = torch.rand(S, D + 1, generator=g, device=dev)
    st["temperature"] = torch.full((S,), c["temperature"], device=dev)
    st["n"], st["probs"] = None, None
    st["drafts"] = torch.zeros(S, D, dtype=torch.int32, device=dev)
    if D:
        guess = (logits[:, :D] + 0.7 * normal(S, D, V)) / T  # a smaller model's
        if c["ragged"]:
            st["n"] = torch.randint(0, D + 1, (S,), generator=g, device=dev, dtype=torch.int32)
        if c["probs"]:
            st["probs"] = torch.softmax(guess, -1)
            gumbel = torch.rand(S, D, V, generator=g, device=dev).clamp_(min=1e-30).log_().neg_().log_().neg_()
            guess = guess + gumbel
        st["drafts"] = guess.argmax(-1).int()
    st["tokens"] = torch.full((S, D + 1), -1, dtype=torch.int32, device=dev)
    st["accepted"] = torch.zeros(S, dtype=torch.int32, device=dev)
    return st


def _run_own(st):
    from decode_megakernel_persistent_gb300 import ll
    c = st["case"]
    if c["op"] in ("matvec", "pack"):
        if "matrix" not in st:  # the object a program keeps for as long as the buffers
            st["matrix"] = ll.Q4Matrix(st["codes"], st["params"], c["rows"], c["cols"])
        if c["op"] == "pack":
            st["matrix"].write(st["w"])
            return st["matrix"].read(out=st["out"])
        return st["matrix"].matvec(st["x"], scale=st["scale"], add=st["add"], out=st["out"])
    if c["op"] == "norm":
        got = ll.ll_rmsnorm(st["x"], st["gain"], 1e-5, residual=st["residual"], residual_out=st["new"], out=st["out"], group=c["group"])
        res = {"out": st["out"]}
        if c["y"] == "e4m3":
            res["scale"] = got[1]
        if c["residual"]:
            res["residual"] = st["new"]
        return res
    if c["op"] == "rope":
        if "rope" not in st:
            st["rope"] = ll.Rope(c["hd"], THETA, rot_dims=c["rot"], interleaved=c["interleaved"], scaling=SCALING[c["scaling"]])
        st["rope"].apply(st["q"], st["k"], st["lens"], st["n"], q_out=st["q_out"], k_out=st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"]}
    ll.ll_verify(st["logits"], st["drafts"], st["u"], probs=st["probs"], n_drafts=st["n"], temperature=st["temperature"],
                 tokens=st["tokens"], accepted=st["accepted"])
    return {"tokens": st["tokens"], "accepted": st["accepted"]}


def _spread(scale, width, group):
    """Scales [n, groups] for each column."""
    return scale.repeat_interleave(group or width, 1)[:, :width]


def _frequencies(c, dev):
    """The angle of a position's step for each pair, in 64 bits, and what cos and sin are multiplied by."""
    rot, s = c["rot"], SCALING[c["scaling"]]
    i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
    f = THETA ** (-2 * i / rot)
    if s is None:
        return f, 1.0
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "bands":
        turns = s["length"] * f / (2 * math.pi)  # over the original length
        smooth = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        return f * smooth + f / s["factor"] * (1 - smooth), 1.0

    def pair(beta):  # the pair (a fraction of one) that turns beta times over the original length
        return rot * math.log(s["length"] / (2 * math.pi * beta)) / (2 * math.log(THETA))

    lo, hi = max(math.floor(pair(s["fast"])), 0), min(math.ceil(pair(s["slow"])), rot - 1)
    ramp = ((i - lo) / (hi - lo if hi != lo else 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / s["factor"] * ramp, 0.1 * math.log(s["factor"]) + 1


def _rotate(x, cos, sin, c):
    """x [S, T, heads, hd] turned by angles [S, T, 1, rot / 2]."""
    rot = c["rot"]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _positions(st):
    """Each token's position [S, T], and whether the sequence has it."""
    T = st["case"]["tokens"]
    lens = st["lens"].long()[:, None]
    n = st["n"].long()[:, None] if st["n"] is not None else torch.full_like(lens, T)
    j = torch.arange(T, device=lens.device)
    return lens - n + j, j < n


def run(st):
    c = st["case"]
    if own:
        return _run_own(st)
    if c["op"] == "pack":
        codes, params = _pack(st["w"], c["group"])
        return _matrix(codes, params, c["rows"], c["cols"]).bfloat16()
    if c["op"] == "matvec":
        w = _matrix(st["codes"], st["params"], c["rows"], c["cols"])
        x = st["x"].float()
        if st["scale"] is not None:
            x = x * _spread(st["scale"], c["cols"], c["scales"])
        y = x @ w.t()
        return (y + st["add"].float() if c["add"] else y).to(TYPES[c["y"]])
    if c["op"] == "norm":
        r = st["x"]
        if c["residual"]:
            r = (r.float() + st["residual"].float()).to(r.dtype)
        v = r.float()
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5) * st["gain"].float()
        res = {}
        if c["y"] == "e4m3":
            res["out"], res["scale"] = _to_e4m3(v, c["group"])
        else:
            res["out"] = v.to(TYPES[c["y"]])
        if c["residual"]:
            res["residual"] = r
        return res
    if c["op"] == "rope":
        f, size = _frequencies(c, st["lens"].device)
        pos, held = _positions(st)
        angle = pos[..., None, None].double() * f  # (far positions: a 32-bit angle has no digits left)
        cos, sin = (angle.cos() * size).float(), (angle.sin() * size).float()
        held = held[..., None, None]
        return {x: torch.where(held, _rotate(st[x].float(), cos, sin, c), 0.0).to(st[x].dtype) for x in ("q", "k")}
    D, V = c["drafts"], c["vocab"]
    l = st["logits"].double()  # (a draw has a border at every token: 32-bit sums decide some of them wrongly)
    best = l.argmax(-1)  # the lowest of equals
    if c["temperature"] > 0:
        p = l - l.amax(-1, keepdim=True)
        p = p.div_(st["temperature"].double()[:, None, None]).exp_()
        p /= p.sum(-1, keepdim=True)
    else:
        p = torch.zeros_like(l).scatter_(2, best[..., None], 1.0)
    n = st["n"].long() if st["n"] is not None else torch.full((c["seqs"],), D, device=l.device)
    j = torch.arange(D + 1, device=l.device)
    x = st["drafts"].long()
    px = p[:, :D].gather(2, x[..., None])[..., 0]
    qx = st["probs"].gather(2, x[..., None])[..., 0].double() if st["probs"] is not None else torch.ones_like(px)
    ok = st["u"][:, :D].double() * qx < px if c["temperature"] > 0 else x == best[:, :D]
    ok &= j[:D] < n[:, None]
    acc = ok.int().cumprod(-1).sum(-1) if D else torch.zeros_like(n)
    pr = p[torch.arange(c["seqs"], device=l.device), acc]
    w = pr
    if D:
        at = acc.clamp(max=D - 1)[:, None]
        q = st["probs"].gather(1, at[..., None].expand(-1, -1, V))[:, 0].double() if st["probs"] is not None else torch.zeros_like(pr).scatter_(
            1, x.gather(1, at), 1.0)
        w = torch.where((acc < n)[:, None], (pr - q).clamp(min=0), pr)
        w = torch.where(w.sum(-1, keepdim=True) > 0, w, pr)
    cum = w.cumsum(-1)
    new = (cum <= st["u"][:, D:].double() * cum[:, -1:]).sum(-1)
    if c["temperature"] == 0:
        new = best.gather(1, acc[:, None])[:, 0]
    drafts = torch.cat([x, new[:, None]], 1)
    tokens = torch.where(j < acc[:, None], drafts, torch.where(j == acc[:, None], new[:, None], -1))
    return {"tokens": tokens.int(), "accepted": acc.int()}


def _code_of(codes, r, k):
    """The codes of rows r [m, 1] and inputs k [1, cols], each looked up where it lies."""
    word = (r % 16 // 8) * 128 + (r % 8) * 16 + (k % 32 // 8) * 4 + k % 128 // 32
    b = codes.view(torch.int32)[r // 16, k // 128, word].long() & 0xFFFFFFFF
    f = k % 8 // 2 + 4 * (k % 2)
    at = (4 * f + 3) % 32
    return ((b >> at) | torch.where(at > 28, b << (32 - at), torch.zeros_like(b))) & 15


def _exact_rows(st, c, y=None):
    """Blocks of the matrix's rows in 64 bits: their first and last row, and the block."""
    k = torch.arange(c["cols"], device=st["codes"].device)[None]
    by = max(16, (1 << 25) // c["cols"])
    for a in range(0, c["rows"], by):
        b = min(c["rows"], a + by)
        r = torch.arange(a, b, device=k.device)[:, None]
        p = st["params"][r // 16, k // TILE, k % TILE // c["group"], r % 16].double()
        yield a, b, p[..., 0] + p[..., 1] * _code_of(st["codes"], r, k).double()


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "pack":
        w = st["w"].double()
        out = torch.empty_like(w)
        for a in range(0, c["cols"], c["group"]):
            x = w[:, a:a + c["group"]]
            lo = x.min(1, keepdim=True).values.half().double()
            step = ((x.max(1, keepdim=True).values - lo) / 15).half().double()
            z = (x - lo) / step
            code = torch.floor(z)
            code = torch.where((z - code > 0.5) | ((z - code == 0.5) & (code % 2 == 1)), code + 1, code).clamp(0, 15)
            out[:, a:a + c["group"]] = torch.where(step > 0, lo + step * code, lo.expand_as(x))
        return out
    if c["op"] == "matvec":
        x = st["x"].double()
        if st["scale"] is not None:
            for a in range(0, c["cols"], c["scales"] or c["cols"]):
                b = a + (c["scales"] or c["cols"])
                x[:, a:b] *= st["scale"][:, a // (b - a)].double()[:, None]
        y = torch.empty(c["tokens"], c["rows"], dtype=torch.float64, device=x.device)
        for a, b, w in _exact_rows(st, c):
            y[:, a:b] = torch.einsum("nk,rk->nr", x, w)
        return y + st["add"].double() if c["add"] else y
    if c["op"] == "norm":
        res = {}
        r = st["x"].double()
        if c["residual"]:
            r = r + st["residual"].double()
            res["residual"] = r
            r = r.to(st["x"].dtype).double()  # the norm is of the sum as it is stored
        v = r / torch.sqrt((r * r).sum(-1, keepdim=True) / c["width"] + 1e-5) * st["gain"].double()
        res["out"] = v
        if c["y"] == "e4m3":
            g = c["group"] or c["width"]
            scale = torch.stack([v[:, a:a + g].abs().max(1).values / 448 for a in range(0, c["width"], g)], 1)
            res["scale"] = scale
            wide = _spread(scale, c["width"], c["group"])
            res["out"] = v / torch.where(wide > 0, wide, 1.0)
        return res
    if c["op"] == "rope":
        f, size = _frequencies(c, st["lens"].device)
        lens = st["lens"].tolist()
        n = st["n"].tolist() if st["n"] is not None else [c["tokens"]] * c["seqs"]
        rot, half = c["rot"], c["rot"] // 2
        first = torch.arange(half, device=f.device) * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else half)
        res = {}
        for x in ("q", "k"):
            out = torch.zeros(st[x].shape, dtype=torch.float64, device=f.device)
            for s in range(c["seqs"]):
                y = st[x][s, :n[s]].double()
                pos = torch.arange(lens[s] - n[s], lens[s], device=f.device, dtype=torch.float64)
                z = torch.polar(torch.full((n[s], half), size, dtype=torch.float64, device=f.device), pos[:, None] * f)[:, None]
                z = torch.complex(y[..., first], y[..., second]) * z
                out[s, :n[s]] = y
                out[s, :n[s], :, first] = z.real
                out[s, :n[s], :, second] = z.imag
            res[x] = out
        return res
    S, D = c["seqs"], c["drafts"]
    tokens, accepted = torch.full((S, D + 1), -1, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    n = st["n"].tolist() if st["n"] is not None else [D] * S
    u, drafts, T = st["u"].tolist(), st["drafts"].tolist(), c["temperature"]
    for s in range(S):
        for j in range(n[s] + 1):
            l = st["logits"][s, j].double()
            if T == 0:
                new = int(torch.nonzero(l == l.max())[0, 0])
                go = j < n[s] and drafts[s][j] == new
            else:
                p = torch.softmax(l / float(st["temperature"][s]), 0)
                x = drafts[s][j] if j < n[s] else -1
                q = st["probs"][s, j].double() if st["probs"] is not None and x >= 0 else None
                go = x >= 0 and u[s][j] * (float(q[x]) if q is not None else 1.0) < float(p[x])
                if not go:
                    if q is not None:
                        p = torch.clamp(p - q, min=0)
                    elif x >= 0:
                        p[x] = 0
                    new = int(torch.searchsorted(torch.cumsum(p, 0), u[s][D] * float(p.sum()), right=True))
            tokens[s, j] = drafts[s][j] if go else new
            if not go:
                break
            accepted[s] += 1
    return {"tokens": tokens, "accepted": accepted}


def work(c):
    """Every input read once and every output written once; two flops a multiply-add of the products."""
    size = {"bf16": 2, "fp32": 4, "e4m3": 1}
    if c["op"] in ("matvec", "pack"):
        packed = c["rows"] * (c["cols"] // 2 + 4 * _tiles(c["cols"], c["group"]))
        if c["op"] == "pack":
            return {"bytes": 2 * packed + 4 * c["rows"] * c["cols"], "flops": 8 * c["rows"] * c["cols"]}
        y = c["tokens"] * c["rows"] * size[c["y"]] * (2 if c["add"] else 1)
        scales = 4 * c["tokens"] * _tiles(c["cols"], c["scales"] or c["cols"]) if c["x"] == "e4m3" else 0
        return {"bytes": packed + c["tokens"] * c["cols"] * size[c["x"]] + scales + y, "flops": 2 * c["tokens"] * c["rows"] * c["cols"]}
    if c["op"] == "norm":
        x = 4 if c["fp32"] else 2
        return {"bytes": c["rows"] * c["width"] * (x * (3 if c["residual"] else 1) + size[c["y"]]) + 2 * c["width"], "flops": 4 * c["rows"] * c["width"]}
    if c["op"] == "rope":
        tokens = sum(_lengths(c, 0)[1])
        return {"bytes": 2 * tokens * (c["heads"] + c["kv"]) * c["hd"] * (4 if c["fp32"] else 2), "flops": 3 * tokens * (c["heads"] + c["kv"]) * c["rot"]}
    # the rows up to the first rejection, here taken as half of the drafts, and the draft's probabilities there
    rows = c["drafts"] / 2 * (0.5 if c["ragged"] else 1) + 1
    return {"bytes": c["seqs"] * c["vocab"] * (rows * (2 if c["bf16"] else 4) + (4 if c["probs"] else 0)), "flops": 4 * c["seqs"] * rows * c["vocab"]}

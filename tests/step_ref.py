"""The operators around the attention in 64 bits, written from include/ll.h, and how far fp32 kernels may be off."""
import math

import torch


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- 4-bit matrices -----------------------------------------------------------------------------

def place(r, k):
    """Where the code of row r and column k lies: its word in the tile and the word's bit."""
    i = k % 8
    return (r % 16 // 8) * 128 + (r % 8) * 16 + (k % 32 // 8) * 4 + k % 128 // 32, (4 * (i // 2 + 4 * (i % 2)) + 3) % 32


def pack(code, lo, step, group):
    """codes and params tensors (on the CPU) of code [rows, cols] and lo, step [rows, groups]."""
    rows, cols = code.shape
    R, K = -(-rows // 16), -(-cols // 128)
    words = torch.zeros(R * K * 256, dtype=torch.int64)
    r, k = torch.meshgrid(torch.arange(rows), torch.arange(cols), indexing="ij")
    word, bit = place(r, k)
    at = ((r // 16) * K + k // 128) * 256 + word
    c = code.to(torch.int64)
    bits = ((c << bit) | (c >> (32 - bit))) & 0xFFFFFFFF  # (a code at bit 31 goes on at bit 0)
    words.index_put_((at.flatten(),), bits.flatten(), accumulate=True)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    per = 128 // group
    params = torch.zeros(R, K, per, 16, 2, dtype=torch.float16)
    r, g = torch.meshgrid(torch.arange(rows), torch.arange(lo.shape[1]), indexing="ij")
    params[r // 16, g // per, g % per, r % 16, 0] = lo.half()
    params[r // 16, g // per, g % per, r % 16, 1] = step.half()
    return words.view(R, K, 256).view(torch.uint8), params


def unpack(codes, params, rows, cols):
    """(code, lo, step) [rows, cols] in 64 bits (on the CPU)."""
    codes, params = codes.cpu(), params.cpu()
    K, per = codes.shape[1], params.shape[2]
    group = 128 // per
    r, k = torch.meshgrid(torch.arange(rows), torch.arange(cols), indexing="ij")
    word, bit = place(r, k)
    w = codes.view(torch.int32).view(-1, K, 256)[r // 16, k // 128, word].to(torch.int64) & 0xFFFFFFFF
    code = ((w >> bit) | (w << (32 - bit))) & 15
    p = params[r // 16, k // 128, k % 128 // group, r % 16].double()
    return code.double(), p[..., 0], p[..., 1]


def quantised(w, group):
    """What w [rows, cols] reads back as, in 64 bits: the format's two fp16 roundings, the nearest code; and
    half a step, how far a value may be from that where the quotient's own rounding decides a border."""
    w = w.double().clamp(-60000, 60000)
    out, steps = torch.empty_like(w), torch.empty_like(w)
    for a in range(0, w.shape[1], group):
        x = w[:, a:a + group]
        lo = x.amin(1, keepdim=True).half().double()
        step = ((x.amax(1, keepdim=True) - lo).clamp(min=0).float() / 15).half().double()  # (lo may round past the largest)
        z = (x - lo) / torch.where(step > 0, step, 1.0)
        out[:, a:a + group] = lo + step * torch.where(step > 0, z.round().clamp(0, 15), 0.0)
        steps[:, a:a + group] = step
    return out, steps


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11}


def product(m, x, add, dtype):
    """x W^T + add in 64 bits and how far a kernel's may be off. x [n, cols] in 64 bits (on the CPU).
    A group of 128 columns is at most 8 matrix instructions with fp32 sums of exact products: each adds
    16 products to a sum, in an order and with a cut that are not documented: 2^-21 of the sum of their sizes
    is allowed. lo and step join in one fp32 operation each, (2 for e4m3 scales), and sums go over the groups,
    8 warps and 3 terms of fp32 x, and add: a rounding of 2^-24 for each. bf16 outputs may take W and x rounded to
    fp16's 11 bits (half a step is 2^-11 of a value, both (1 + 2^-11)^2 - 1; below 2^-14 of W, 2^-25; of x 2^-39 of its
    row's largest)."""
    code, lo, step = unpack(m.codes, m.params, m.rows, m.cols)
    y = x @ (lo + step * code).t()
    size = x.abs() @ (step.abs() * (code - 8).abs() + (lo + 8 * step).abs()).t()
    groups = -(-m.cols // 128) * (128 // m.group)
    tol = (8 * 2.0 ** -21 + (2 * groups + 16) * 2.0 ** -24) * size
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -10 * 1.001 * (x.abs() @ (lo + step * code).abs().t()) + 2.0 ** -25 * x.abs().sum(1, keepdim=True)
        tol = tol + 2.0 ** -39 * x.abs().amax(1, keepdim=True) * (lo.abs() + 15 * step.abs()).sum(1)
    if add is not None:
        y = y + add
        tol = tol + 2.0 ** -24 * (y.abs() + add.abs())
    return y, tol + HALF_STEP[dtype] * (y.abs() + tol) + 1e-37


# ---- rotary positions -----------------------------------------------------------------------------

def frequencies(rot, theta, scaling):
    f = [theta ** (-2 * i / rot) for i in range(rot // 2)]
    size = 1.0
    s = scaling or {"kind": "plain"}
    if s["kind"] == "linear":
        f = [x / s["factor"] for x in f]
    elif s["kind"] == "bands":
        def band(x):
            wave = 2 * math.pi / x
            if wave < s["length"] / s["high"]:
                return x
            if wave > s["length"] / s["low"]:
                return x / s["factor"]
            k = (s["length"] / wave - s["low"]) / (s["high"] - s["low"])
            return (1 - k) * x / s["factor"] + k * x
        f = [band(x) for x in f]
    elif s["kind"] == "ramp":
        def pair(turns):
            return rot * math.log(s["length"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(pair(s["fast"])), 0), min(math.ceil(pair(s["slow"])), rot - 1)
        k = [min(max((i - lo) / ((hi - lo) or 0.001), 0), 1) for i in range(rot // 2)]
        f = [x * (1 - a) + x / s["factor"] * a for x, a in zip(f, k)]
        size = 0.1 * math.log(s["factor"]) + 1
    return torch.tensor(f, dtype=torch.float64), size


def rotated(x, pos, rot, theta, scaling, interleaved, inverse=False):
    """x [..., heads, hd] (64 bits) at positions pos [...], and the sizes |a| + |b| of its pairs."""
    f, size = frequencies(rot, theta, scaling)
    t = pos.double()[..., None, None] * f.to(x.device)
    c, s = t.cos() * size, t.sin() * size * (-1 if inverse else 1)
    y, w = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    w[..., a] = w[..., b] = (x[..., a].abs() + x[..., b].abs()) * size
    return y, w


# ---- verification ---------------------------------------------------------------------------------

def verified(logits, drafts, u, probs=None, n_drafts=None, temperature=None):
    """ll_verify from its definition, one sequence, row and token at a time, in 64 bits (tensors on the CPU). Also how near the
    nearest border each decision was (relative), so that a test can tell that none is closer than the kernel's own bounds."""
    S, rows, V = logits.shape
    D = rows - 1
    tokens, accepted, near = torch.full((S, rows), -1, dtype=torch.int32), torch.zeros(S, dtype=torch.int32), 1.0
    for s in range(S):
        n = D if n_drafts is None else max(0, min(D, int(n_drafts[s])))
        T = 1.0 if temperature is None else float(temperature[s])
        for j in range(n + 1):
            l = logits[s, j].double()
            l = torch.where(torch.isnan(l), -math.inf, l)
            m = float(l.max())
            if m == -math.inf:
                tokens[s, j] = -1
                break
            x = int(drafts[s, j]) if j < n else -1
            if not T > 2.0 ** -100:
                best = int((l == m).nonzero()[0, 0])
                if x != best or j == n:
                    tokens[s, j] = best
                    break
            else:
                if m == math.inf:
                    w = (l == m).double()
                else:
                    w = torch.exp((l - m) / T)
                p = w / w.sum()
                q = None
                if j < n:
                    q = probs[s, j].double() if probs is not None else torch.zeros(V, dtype=torch.float64).index_fill_(0, torch.tensor([x]), 1.0) \
                        if 0 <= x < V else torch.zeros(V, dtype=torch.float64)
                    if 0 <= x < V:
                        left, right = float(u[s, j]) * float(q[x]), float(p[x])
                        near = min(near, abs(left - right) / max(left, right, 1e-300) if left != right else 1.0)
                        if left < right:
                            tokens[s, j] = x
                            accepted[s] += 1
                            continue
                    r = (p - q).clamp(min=0)
                    p = r if float(r.sum()) > 0 else p
                cum = p.cumsum(0)
                at = float(u[s, D]) * float(cum[-1])
                new = int((cum > at).nonzero()[0, 0])
                near = min(near, abs(float(cum[new]) - at) / float(cum[-1]), abs(at - (float(cum[new - 1]) if new else -1.0)) / float(cum[-1]))
                tokens[s, j] = new
                break
            tokens[s, j] = x
            accepted[s] += 1
    return tokens, accepted, near

"""The packed KV cache's definition in plain tensor operations, for the tests:
quantising rows, the bytes they pack to, the values they stand for, and attention
over them in 64 bits with the bound its roundings allow."""
from __future__ import annotations

import numpy as np
import torch

BOUND = 60000.0


def quantise(x, bits):
    """(lo, step) fp16 and codes int64 of x [..., hd] (fp32 or bf16), the definition's fp32 arithmetic, on the CPU."""
    top = float(2 ** bits - 1)
    x = x.detach().float().cpu()
    x = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32).clamp(-BOUND, BOUND)  # (keeps NaN)
    lo = x.amin(-1).half()  # (NaN if any is)
    step = ((x.amax(-1) - lo.float()) * torch.tensor(1.0 / top)).clamp(min=0).half()  # (1 / top rounded to fp32)
    # the integer nearest to (x - lo) / step: the difference in fp32, its quotient in fp64, where
    # 24 bits by 11 cannot round onto a border between two integers
    t, sf = (x - lo.float()[..., None]).double(), step.double()[..., None]
    code = torch.where(sf > 0, (t / sf).round().clamp(0, top), torch.zeros_like(t))
    return lo, step, torch.nan_to_num(code, nan=0.0).long()


def values(lo, step, code):
    """fp16(lo + step * code) in one rounding (numpy rounds a double to half once), as float64 [..., hd]."""
    v = lo.double()[..., None] + step.double()[..., None] * code.double()
    return torch.from_numpy(v.numpy().astype(np.float16).astype(np.float64)).flatten(-2)


def place(hd):
    """The element of a packed row that holds dim d."""
    d = torch.arange(hd)
    return ((d % 32 // 4) * (hd // 32) + d // 32) * 4 + d % 4


def pack(lo, step, code, bits):
    """codes uint8 [..., hd * bits / 8] and params fp16 [..., hd / 32, 2]."""
    flat = code.flatten(-2)
    el = torch.empty_like(flat)
    el[..., place(flat.shape[-1])] = flat
    if bits == 4:
        el = el[..., 0::2] + 16 * el[..., 1::2]
    return el.to(torch.uint8), torch.stack([lo, step], -1)


def attend(q, k, v, last, scale=None):
    """Attention of rows q [R, hd] over positions 0..last[r] of k, v [L, hd] (float64),
    and how far a kernel may be from it: with A = sum p |v|,
      * the probabilities' fp16 rounding is 2^-11 of each, or 2^-25 of the largest for small ones;
      * the scores: products of exact fp16 numbers summed in fp32 (at most 2^-21
        of sum |q k| over these widths), exp2 and its argument within 2^-21;
      * the output is rounded to bf16 (2^-9, taken as 2^-8 of |o|)."""
    R, hd = q.shape
    L = k.shape[0]
    scale = scale or hd ** -0.5
    s = (q @ k.T) * scale
    seen = torch.arange(L, device=q.device)[None] <= last[:, None]
    s = s.masked_fill(~seen, float("-inf"))
    m = s.amax(-1, keepdim=True) if L else s.new_full((R, 1), float("-inf"))
    e = torch.where(seen, (s - torch.where(torch.isinf(m), torch.zeros_like(m), m)).exp(), torch.zeros_like(s))
    tot = e.sum(-1, keepdim=True)
    p = e / torch.where(tot == 0, torch.ones_like(tot), tot)
    vs = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v)) if L else v
    o = p @ vs
    A = p @ vs.abs()
    score = ((q.abs() @ k.abs().T) * scale).masked_fill(~seen, 0.0)
    err = score.amax(-1, keepdim=True) * 2.0 ** -21 * 2 + 2.0 ** -20 if L else s.new_zeros((R, 1))
    vmax = vs.abs().amax() if L else 0.0
    tol = 2.0 ** -8 * o.abs() + A * (2.0 ** -11 + 2 * err) + vmax * L * 2.0 ** -25 + 1e-30
    return o, tol

"""Inputs on which every run of 16 keys shows in attention over a packed cache, and a bound
that is tight enough to see one missing at any length the tests use."""
from __future__ import annotations

import torch

RUN = 16  # keys: the smallest tile of any kernel


def key_values(L, hd, generator=None):
    """K and V [L, hd] (fp32, on the CPU): K small, so that all keys weigh alike; V 15 in one dim and 0 in the others, the dim
    changing every RUN keys. So an output's dim is what the runs of that dim weigh, at most L / (RUN * hd) + 1 of them. What
    is left behind the last whole run is 60 times larger, so that a few keys show as a run does."""
    k = torch.randn(L, hd, generator=generator) * 0.25
    v = torch.zeros(L, hd)
    i = torch.arange(L)
    v[i, i // RUN % hd] = 15.0
    v[L - L % RUN:] *= 60.0
    return k, v


def attend(q, k, v, last, scale=None):
    """Attention of rows q [R, hd] over positions 0..last[r] of k, v [L, hd] (float64), and how far a kernel may be from it.
    With e = exp(score - the row's largest), t their sum, A = sum e |v| / t:
      * an output is rounded to bf16: 2^-8 of it;
      * a probability is rounded to fp16, where the largest is 2^7 at least: 2^-11 of it, or half of the smallest
        step, 2^-25, which is 2^-32 of the largest's;
      * the scores are fp32 sums of exact products and one factor, 2^-21 of sum |q k|, and exp2 and its argument
        2^-20: relative errors of a probability, and of t;
      * t is summed in fp32 by at most L / 4 additions in a row (2^-24 each), O by L / 16 products in a row (2^-23: a tensor
        core may cut its sums off)."""
    L = k.shape[0]
    scale = scale or q.shape[1] ** -0.5
    seen = torch.arange(L, device=q.device)[None] <= last[:, None]
    s = ((q @ k.T) * scale).masked_fill_(~seen, float("-inf"))
    e = (s - s.amax(-1, keepdim=True)).exp_()
    t = e.sum(-1, keepdim=True)
    o, A = (e @ v) / t, (e @ v.abs()) / t
    size = ((q.abs() @ k.abs().T) * scale).masked_fill_(~seen, 0.0).amax(-1, keepdim=True)
    rel = 2.0 ** -11 + 2 * (size * 2.0 ** -21 + 2.0 ** -20) + (L // 4 + 64) * 2.0 ** -24 + (L // 16 + 16) * 2.0 ** -23
    lost = (seen.double() @ v.abs()) * 2.0 ** -32 / t
    return o, 2.0 ** -8 * o.abs() + A * rel + lost + 1e-30

"""Rotary positions on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from decode_megakernel_persistent_gb300 import ll
import step_ref
from step_ref import gen, i32

pytestmark = pytest.mark.gpu

SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="bands", factor=32.0, low=1.0, high=4.0, length=8192),
            dict(kind="ramp", factor=16.0, fast=32.0, slow=1.0, length=4096)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_megakernel_persistent_gb300 import build
    build.build()


def check(rope, q, k, lens, n, rot, theta, scaling, interleaved, inverse=False, got=None, mark=9.0):
    """apply() against the formula: angles rounded to fp32 (at most pi 2^-24 off), sin and cos within 2 units of 2^-23, two
    products and a sum: 2^-21 of |a| + |b| is allowed, and the output's rounding."""
    S, T = q.shape[:2]
    if got is None:
        got = tuple(torch.full(t.shape, mark, dtype=t.dtype, device="cuda") for t in (q, k))
        rope.apply(q, k, i32(lens), i32(n) if n is not None else None, q_out=got[0], k_out=got[1], inverse=inverse)
    n = n if n is not None else [T] * S
    pos = torch.tensor([[lens[s] - n[s] + j for j in range(T)] for s in range(S)], device="cuda")
    held = torch.tensor([[0 <= j < n[s] and lens[s] - n[s] + j >= 0 for j in range(T)] for s in range(S)], device="cuda")
    for t, o in zip((q, k), got):
        y, w = step_ref.rotated(t.double(), pos.clamp(min=0), rot, theta, scaling, interleaved, inverse)
        tol = 2.0 ** -21 * w
        tol = tol + step_ref.HALF_STEP[t.dtype] * (y.abs() + tol)
        off = (o.double() - y).abs()
        h = held[..., None, None].expand_as(y)
        assert bool((off <= tol)[h].all()), float((off / tol.clamp(min=1e-30))[h].max())
        if mark is not None:
            assert bool((o == mark)[~h].all())
        assert torch.equal(o[..., rot:][h[..., rot:]], t[..., rot:][h[..., rot:]])
    return got


@pytest.mark.parametrize("hd,rot", [(64, 64), (128, 128), (64, 32), (128, 56), (80, 80), (96, 40), (256, 256), (64, 2), (8, 6), (256, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope(hd, rot, interleaved, scaling, dtype):
    S, T, H, KV = 3, 5, 6, 2
    theta = 500000.0 if hd > 64 else 10000.0
    rope = ll.Rope(hd, theta, rot, interleaved, SCALINGS[scaling])
    q, k = (torch.randn(S, T, h, hd, generator=gen(h), device="cuda").to(dtype) for h in (H, KV))
    check(rope, q, k, [5, 1000, 131072], None, rot, theta, SCALINGS[scaling], interleaved)
    check(rope, q, k, [4, 0, 1 << 30], [3, 0, 5], rot, theta, SCALINGS[scaling], interleaved)


@pytest.mark.parametrize("T,H,KV", [(1, 32, 8), (1, 1, 1), (300, 32, 8), (7, 64, 1), (1000, 3, 3), (2, 200, 100)])
@pytest.mark.parametrize("hd", [64, 128])
def test_counts(T, H, KV, hd):
    rope = ll.Rope(hd)
    q, k = (torch.randn(2, T, h, hd, generator=gen(h), device="cuda").bfloat16() for h in (H, KV))
    check(rope, q, k, [T, T + 77], [T, max(1, T - 1)], hd, 500000.0, None, False)


def test_far_positions_are_exact():
    """One pair at a time, positions up to 2^31: cos and sin to fp32's last places, whatever the angle's size."""
    rope = ll.Rope(64, 10000.0)
    lens = [1, 2, 4097, 1 << 20, (1 << 20) + 1, 1 << 30, (1 << 31) - 1]
    q = torch.zeros(len(lens), 1, 1, 64, device="cuda")
    q[..., :32] = 1.0
    out, _ = rope.apply(q, None, i32(lens), q_out=torch.empty_like(q))
    f, _ = step_ref.frequencies(64, 10000.0, None)
    t = (torch.tensor(lens, dtype=torch.float64)[:, None] - 1) * f
    # (the reference's own angle is off by up to 2^-53 of itself)
    tol = 2.0 ** -21 + t.abs() * 2.0 ** -52
    assert bool(((out[:, 0, 0, :32].double().cpu() - t.cos()).abs() <= tol).all())
    assert bool(((out[:, 0, 0, 32:].double().cpu() - t.sin()).abs() <= tol).all())


@pytest.mark.parametrize("rot", [128, 60])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_strided_and_back(rot, interleaved):
    """Rows of a fused projection turned where they are; turning back gives them again; the inverse is the transpose."""
    S, T, H, KV, hd = 2, 33, 4, 2, 128
    rope = ll.Rope(hd, 500000.0, rot, interleaved)
    rows = torch.randn(S, T, H + 2 * KV, hd, generator=gen(1), device="cuda")
    q, k, v = rows[:, :, :H], rows[:, :, H:H + KV], rows[:, :, H + KV:].clone()
    before = (q.clone(), k.clone())
    lens, n = [40, 5000], [33, 20]
    got = rope.apply(q, k, i32(lens), i32(n))
    assert got[0] is q and got[1] is k
    check(rope, *before, lens, n, rot, 500000.0, None, interleaved, got=got, mark=None)
    assert torch.equal(q[1, 20:], before[0][1, 20:]) and torch.equal(rows[:, :, H + KV:], v)
    turned = q.clone()
    rope.apply(q, k, i32(lens), i32(n), inverse=True)
    assert float((q - before[0]).abs().max()) <= 2.0 ** -19 * 8 and float((k - before[1]).abs().max()) <= 2.0 ** -19 * 8
    # <g, R x> = <R^T g, x>, so a gradient is turned by the inverse
    g = torch.randn(S, T, H, hd, generator=gen(2), device="cuda")
    g[1, 20:] = 0
    back, _ = rope.apply(g, None, i32(lens), i32(n), q_out=torch.zeros_like(g), inverse=True)
    left, right = (g.double() * turned.double()).sum(), (back.double() * before[0].double()).sum()
    assert abs(float(left - right)) <= 2.0 ** -20 * float((g.abs().double() * 8).sum())


def test_scaled_inverse_is_the_transpose():
    scaling = SCALINGS[3]
    rope = ll.Rope(64, 10000.0, scaling=scaling)
    q, k = (torch.randn(1, 9, h, 64, generator=gen(h), device="cuda") for h in (2, 1))
    check(rope, q, k, [700], None, 64, 10000.0, scaling, False, inverse=True)

"""The bound that the packed cache's long-context tests hold attention to, on the CPU: results
with a run of keys, or the share of one of many blocks, left out must lie outside of it."""
import pytest

torch = pytest.importorskip("torch")

import kvq_keys
import kvq_ref


def held(L, hd, bits):
    g = torch.Generator()
    g.manual_seed(L + hd)
    k, v = kvq_keys.key_values(L, hd, g)
    q = torch.randn(2, hd, generator=g).bfloat16().double()
    return q, *(kvq_ref.values(*kvq_ref.quantise(x, bits)) for x in (k, v))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("L", [40, 333, 1000, 4099, 32768, 70001])
def test_missing_keys_are_outside_the_bound(L, hd, bits):
    q, k, v = held(L, hd, bits)
    last = torch.full((2,), L - 1)
    o, tol = kvq_keys.attend(q, k, v, last)
    assert bool(((o.bfloat16().double() - o).abs() <= tol).all())  # (the right result, as it is written, is inside)
    R = kvq_keys.RUN
    runs = {0, R * (L // R // 2), L - L % R - R} | ({L - L % R} if L % R else set())
    splits = [(L * i // 16, L * (i + 1) // 16) for i in (0, 7, 15)]
    for a, b in [(r, min(r + R, L)) for r in runs] + splits:
        if b - a >= L:
            continue
        keep = torch.ones(L, dtype=torch.bool)
        keep[a:b] = False
        short, _ = kvq_keys.attend(q, k[keep], v[keep], torch.full((2,), int(keep.sum()) - 1))
        off = (short.bfloat16().double() - o).abs()
        assert bool((off > tol).any(-1).all()), (a, b, float((off / tol).max()))
        # and by its weight alone, the sum of the weights as it should be
        gone = torch.where(keep[:, None], v, torch.zeros_like(v))
        short, _ = kvq_keys.attend(q, k, gone, last)
        off = (short.bfloat16().double() - o).abs()
        assert bool((off > tol).any(-1).all()), (a, b, float((off / tol).max()))

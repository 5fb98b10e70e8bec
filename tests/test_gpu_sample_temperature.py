"""Sampling at temperatures at the ends of float32's range, where the exponentials' scale is 0 or infinite."""
import numpy as np
import pytest
import torch

import weight_only_bit_split_gb300 as wobs
from test_gpu_decode_ops import BF16, F16, F32, dev, gen, peaked

pytestmark = pytest.mark.gpu
INF = float("inf")


def ordered(row):
    """Token indices by value, largest first, lowest index first among equal ones; those at -infinity and NaN left out."""
    x = np.nan_to_num(row.double().cpu().numpy(), nan=-np.inf, posinf=np.inf, neginf=-np.inf)
    order = np.lexsort((np.arange(len(x)), -x))
    return order[x[order] > -np.inf]


@pytest.mark.parametrize("temperature", [INF, 1e38, 3.4e38, 1e30])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m,n", [(1, 3), (4, 1000), (3, 5003), (2, 128000), (1, 524288)])
def test_a_huge_temperature_draws_evenly(temperature, dtype, m, n):
    """Logits within 50 of each other: their exponentials at T >= 1e30 are 1 in float32.  u lies in the middle of a share."""
    g = gen(51)
    rng = np.random.default_rng(n)
    x = peaked(g, m, n, dtype)
    x[:, n // 3] = -INF
    x[0, n // 2] = float("nan")
    f = lambda v, dt=F32: torch.full((m,), v, dtype=dt, device=dev())  # noqa: E731
    kept = [ordered(x[r]) for r in range(m)]
    for k in (0, max(1, n // 5)):
        at = [int(rng.integers(0, min(len(o), k or n))) for o in kept]
        size = [min(len(o), k or n) for o in kept]
        u = torch.tensor([(a + 0.5) / s for a, s in zip(at, size)], device=dev())
        at = [int(float(v.double()) * s) for v, s in zip(u, size)]       # of the float32 number
        t, p = wobs.wobs_sample(x, u, temperature=f(temperature), top_k=f(k, torch.int32) if k else None, min_p=f(0.5))
        assert t.tolist() == [int(o[a]) for o, a in zip(kept, at)]
        assert np.allclose(p.cpu().numpy(), [1 / s for s in size], rtol=1e-6, atol=0)


def test_an_infinite_temperature_over_float32s_whole_range():
    x = torch.tensor([[3.4e38, -3.4e38, 0.0, -INF], [-3.4e38, 3e38, -INF, float("nan")], [INF, 3e38, INF, -3.4e38], [-INF, -INF, float("nan"), -INF],
                      [-3.4e38, -3.4e38, -3.4e38, -3.4e38]], device=dev())
    hot = torch.full((5,), INF, device=dev())
    want = {0.1: [0, 1, 0, -1, 0], 0.45: [2, 1, 0, -1, 1], 0.55: [2, 0, 2, -1, 2], 0.9: [1, 0, 2, -1, 3]}
    for u, tokens in want.items():
        t, p = wobs.wobs_sample(x, torch.full((5,), u, device=dev()), temperature=hot)
        assert t.tolist() == tokens
        assert np.allclose(p.tolist(), [1 / 3, 0.5, 0.5, 0.0, 0.25], rtol=1e-6)


@pytest.mark.parametrize("temperature", [1e-38, 1e-45, 1e-30])
def test_a_tiny_temperature_draws_among_the_largest(temperature):
    """Whatever lies below the largest value has no mass, however far; u draws among the equal ones."""
    g = gen(52)
    x = randn_rows(g)
    t, p = wobs.wobs_sample(x, torch.tensor([0.1, 0.4, 0.6, 0.99], device=dev()), temperature=torch.full((4,), temperature, device=dev()),
                            min_p=torch.full((4,), 0.01, device=dev()))
    assert t.tolist() == [11, 700, 2000, 4999] and p.tolist() == [0.25] * 4


def randn_rows(g):
    x = torch.randn((4, 5000), generator=g, device=dev()) * 1e9
    x[:, 1::7] = -3.4e38
    x[:, [11, 700, 2000, 4999]] = 2e10
    return x


def test_nan_parameters():
    """A NaN temperature takes the largest logit's token, a NaN top_p or min_p leaves the filter off."""
    x = peaked(gen(53), 5, 3000)
    u = torch.tensor([0.05, 0.3, 0.5, 0.7, 0.95], device=dev())
    nan = torch.full((5,), float("nan"), device=dev())
    plain, chance = wobs.wobs_sample(x, u)
    assert plain.tolist() != x.argmax(-1).tolist()
    for filters in (dict(min_p=nan), dict(top_p=nan), dict(top_p=nan, min_p=nan)):
        t, p = wobs.wobs_sample(x, u, **filters)
        assert torch.equal(t, plain) and torch.equal(p, chance)
    t, p = wobs.wobs_sample(x, u, temperature=nan, min_p=nan)
    assert t.tolist() == x.argmax(-1).tolist() and p.tolist() == [1.0] * 5
    half, _ = wobs.wobs_sample(x, u, min_p=torch.full((5,), 0.5, device=dev()))
    mixed = torch.tensor([0.5, float("nan"), 0.5, float("nan"), -1.0], device=dev())
    t, _ = wobs.wobs_sample(x, u, min_p=mixed)
    assert t.tolist() == [int((half if i in (0, 2) else plain)[i]) for i in range(5)]

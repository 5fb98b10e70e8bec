"""Attention over the 4-bit cache where scores and values span many powers of two."""
import pytest
import torch

import weight_only_bit_split_gb300 as wobs
from test_gpu_decode_ops import BF16, F16, F32, U, dev, gen, held, make_cache, randn

pytestmark = pytest.mark.gpu


def led_cache(g, n, dim, q, lead, value, sink):
    """n tokens of one head whose values have a nonzero mean and scales around ``value``.  Against the query q
    token 5 leads by ``lead`` and has the value scale ``sink``; token 9, 20 below the others, has one of 1000."""
    cache, table, lens = make_cache(g, [n], 64, 1, dim)
    page, slot = table[0].long()[torch.arange(n, device=dev()) // 64], torch.arange(n, device=dev()) % 64
    low, high = (torch.randint(9, 16, (n, dim // 2), generator=g, device=dev(), dtype=torch.uint8) for _ in range(2))
    cache.vq[page, 0, slot] = low | (high << 4)
    cache.vd[page, 0, slot] = (value * (0.5 + torch.rand(n, dim // 32, generator=g, device=dev()))).to(F16)
    cache.kd[page, 0, slot] = (0.02 * cache.kd[page, 0, slot].float()).to(F16)
    code = torch.where(q > 0, 15, 1).to(torch.uint8).view(-1, 2, 16)    # (c - 8) q = 7 |q|
    for token, score, scale in ((5, lead, sink), (9, -20.0, 1000.0)):
        cache.kq[page[token], 0, slot[token]] = (code[:, 0] | (code[:, 1] << 4)).flatten()
        cache.kd[page[token], 0, slot[token]] = score / (7 * float(q.float().abs().sum()) * dim ** -0.5)
        cache.vd[page[token], 0, slot[token]] = scale
    return cache, table, lens


@pytest.mark.parametrize("power", [10, 20, 24, 26, 28, 31, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_so_large_that_nothing_can_be_added_to_them(power, dim):
    """Scores around 2^power, whose float32 spacing is up to 2^17: the output is the leading token's value, as it is where
    float32 scores are subtracted from their maximum."""
    g = gen(32)
    q = randn(g, dim).abs().clamp(0.5, 2.0).to(BF16)
    cache, table, lens = led_cache(g, 300, dim, q, 0.0, 8.0, 8.0)
    cache.kd[table[0, 0], 0, 5] = 2.0                                     # token 5: 14 |q| a dim; the others' scales: 0.02 * 0.3 * 1.05 at most
    q = (q.float() * 2.0 ** power).to(BF16)
    _, v = held(cache, table, 0, 300)
    out = wobs.wobs_attn_kv4(cache, q.expand(1, 1, 4, dim), table, lens, out_dtype=F32)
    assert bool(((out[0, 0].double() - v[5, 0]).abs() <= 2 * U[F16] * v[5, 0].abs()).all())

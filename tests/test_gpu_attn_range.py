"""Attention over the 4-bit cache where the products of a probability and a value's scale span many powers of two:
one token that leads by far, small value scales, a large value that no query looks at."""
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


def attend64(q, cache, table, n, seen):
    """Output, probability-weighted |v|, and the largest product of a probability and a token's largest value scale
    (2^-25 at least), of one query over the first ``seen`` tokens."""
    k, v = (t[:seen, 0] for t in held(cache, table, 0, n))
    t = torch.arange(seen, device=dev())
    scale = cache.vd[table[0].long()[t // 64], 0, t % 64].double().abs().amax(-1).clamp(min=2.0 ** -25)
    s = (k @ q.double()) * q.numel() ** -0.5
    e = torch.exp(s - s.max())
    return e @ v / e.sum(), e @ v.abs() / e.sum(), (e * scale).max() / e.sum()


CASES = [   # tokens, L, group, dim, lead, value, sink
    (32768, 1, 4, 128, 12.0, 0.05, 0.0), (32768, 1, 4, 128, 12.0, 0.005, 2.0 ** -24), (8192, 1, 8, 128, 12.0, 0.0005, 0.01),
    (8192, 3, 5, 128, 12.0, 0.005, 0.0), (32768, 1, 4, 128, 25.0, 0.05, 0.0), (8192, 1, 1, 64, 12.0, 0.005, 0.001),
    (32768, 2, 8, 64, 20.0, 0.02, 2.0 ** -20), (8192, 1, 4, 256, 12.0, 0.005, 0.0), (32768, 2, 16, 256, 18.0, 0.05, 0.0),
    (8192, 1, 4, 128, 0.0, 2.0 ** -18, 2.0 ** -18), (500, 1, 4, 128, 12.0, 2.0 ** -18, 0.0), (32768, 1, 4, 128, 0.0, 8000.0, 8000.0),
    (700, 1, 4, 128, 12.0, 30000.0, 60000.0),
]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("n,L,group,dim,lead,value,sink", CASES)
def test_products_over_many_powers_of_two(dtype, n, L, group, dim, lead, value, sink):
    """Half an ulp of fp16 for a product, as much again for the exponential and the float32 sums.  The largest product
    lies above 2^14, so a subnormal one is off by 2^-25 / 2^14 of the largest, eight times that with its code."""
    g = gen(31)
    q = randn(g, dim, dtype=dtype)
    cache, table, lens = led_cache(g, n, dim, q, lead, value, sink)
    out = wobs.wobs_attn_kv4(cache, q.expand(1, L, group, dim), table, lens, out_dtype=F32)
    for i in range(L):
        seen = n - L + i + 1
        o, a, w = attend64(q, cache, table, n, seen)
        bound = 2 * U[F16] * a + seen * 2.0 ** -36 * w + U[F32] * o.abs()
        err = (out[0, i].double() - o).abs()
        assert bool((err <= bound).all()), f"max error over bound {float((err / bound).max()):.3g}, of the output {float((err / o.abs()).max()):.3g}"


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


@pytest.mark.parametrize("power", [100, 117, 118, 122, 126])
@pytest.mark.parametrize("scale", [None, -0.5, 2.0 ** -20])
def test_queries_at_the_end_of_bf16s_range(power, scale):
    """Queries around 2^power against small keys: the scores are finite, and the largest (smallest, where the scale is
    negative) score's value is the output."""
    g = gen(33)
    q = randn(g, 128).abs().clamp(0.5, 1.9).to(BF16)
    cache, table, lens = led_cache(g, 300, 128, q, 0.0, 8.0, 8.0)
    cache.kd.mul_(2.0 ** -8)
    cache.kd[table[0, 0], 0, 9] = 0.0
    cache.kd[table[0, 0], 0, 5] = (-1 if scale is not None and scale < 0 else 1) * 2.0 ** -12
    q = (q.float() * 2.0 ** power).to(BF16)
    k, v = held(cache, table, 0, 300)
    scores = (k[:, 0] @ q.double()) * (128 ** -0.5 if scale is None else scale)
    assert int(scores.argmax()) == 5 and float(scores.abs().max()) < 3e38
    out = wobs.wobs_attn_kv4(cache, q.expand(1, 1, 4, 128), table, lens, scale=scale, out_dtype=F32)
    assert bool(((out[0, 0].double() - v[5, 0]).abs() <= 2 * U[F16] * v[5, 0].abs()).all())

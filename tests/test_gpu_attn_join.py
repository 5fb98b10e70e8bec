"""Attention over one long sequence of one cache head: more pieces of it than the join holds at a time (400 with one row
tile, 200 with two, on a GPU of 152 SMs)."""
import pytest
import torch

import weight_only_bit_split_gb300 as wobs
from test_gpu_decode_ops import BF16, F16, F32, assert_attention, attend64, dev, gen, held, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tilt", [0.0, 8.0, -8.0])
@pytest.mark.parametrize("n,L,group,dim", [(100003, 1, 4, 128), (90001, 1, 8, 64), (60013, 4, 4, 128), (100003, 3, 5, 64), (70000, 1, 3, 256)])
def test_more_pieces_than_a_batch(dtype, tilt, n, L, group, dim):
    """With a tilt the scores rise or fall by 8 along the sequence, so that every batch of pieces has another maximum."""
    g = gen(81)
    cache, table, lens = make_cache(g, [n], 64, 1, dim)
    q = randn(g, 1, L, group, dim, dtype=dtype)
    if tilt:
        q[..., 32:] = 0                                                  # block 0 makes the scores: 1 s, and s rises by 8
        q[..., :32] = 1.0
        t = torch.arange(n, device=dev())
        page, slot = table[0].long()[t // 64], t % 64
        cache.kq[page, 0, slot, :16] = 0x99                              # every code of block 0 is 1
        cache.kd[page, 0, slot, 0] = (tilt * t.float() / n / (32 * dim ** -0.5)).to(F16)
    out = wobs.wobs_attn_kv4(cache, q, table, lens, out_dtype=F32)
    ks, vs = held(cache, table, 0, n)
    assert_attention(out, attend64(q[0], ks, vs, [n - L + i + 1 for i in range(L)]), F32)
    assert torch.equal(out, wobs.wobs_attn_kv4(cache, q, table, lens, out_dtype=F32))

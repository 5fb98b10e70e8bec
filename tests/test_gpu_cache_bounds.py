"""Lengths that a sequence's block table has no room for: the tokens past its end are left out, the others keep their
positions."""
import pytest
import torch

import weight_only_bit_split_gb300 as wobs
from test_gpu_decode_ops import F32, append_reference, assert_attention, attend64, gen, held, make_cache, randn, same_planes, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,page,entries", [(64, 16, 2), (128, 48, 3)])
@pytest.mark.parametrize("L", [1, 5, 32])
def test_overlong_lengths_leave_out_the_tokens_past_the_end(L, dim, page, entries):
    g = gen(41)
    room = page * entries
    cache, table, _ = make_cache(g, [room] * 6, page, 2, dim)
    given = [room, room + 1, room + 3, room + L, room + 40, 2 ** 31 - 1]
    lens = torch.tensor(given, dtype=torch.int32, device=dev())
    k, v = randn(g, 6, L, 2, dim), randn(g, 6, L, 2, dim)
    planes = [p.clone() for p in (cache.kq, cache.kd, cache.vq, cache.vd)]
    for b, n in enumerate(given):                                        # the tokens in front of the end, at their own places
        inside = L - (n - room)
        if inside > 0:
            now = wobs.Kv4Cache(*planes)
            planes = append_reference(now, k[b:b + 1, :inside], v[b:b + 1, :inside], table[b:b + 1], [room])
    wobs.wobs_kv4_append(cache, k, v, table, lens)
    assert wobs.wobs_error_word() == wobs.DEVICE_CACHE_INDEX
    assert same_planes(cache, planes)
    kr, vr = wobs.wobs_kv4_read(cache, table, lens, L)
    assert wobs.wobs_error_word() == wobs.DEVICE_CACHE_INDEX
    q = randn(g, 6, L, 6, dim, dtype=torch.bfloat16)
    o = wobs.wobs_attn_kv4(cache, q, table, lens, out_dtype=F32)
    assert wobs.wobs_error_word() == wobs.DEVICE_CACHE_INDEX
    for b, n in enumerate(given):
        inside = max(0, L - (n - room))
        ks, vs = held(cache, table, b, room)
        assert torch.equal(kr[b, :inside].double(), ks[room - inside:]) and torch.equal(vr[b, :inside].double(), vs[room - inside:])
        assert not kr[b, inside:].any() and not vr[b, inside:].any()
        seen = [min(room, n - L + i + 1) for i in range(L)]
        for h in range(2):
            assert_attention(o[b:b + 1, :, 3 * h:3 * h + 3], attend64(q[b, :, 3 * h:3 * h + 3], ks[:, h:h + 1], vs[:, h:h + 1], seen), F32)

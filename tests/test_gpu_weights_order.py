"""Outputs of one call as the weights of the next product on the same stream, with no wait between them: the product
sees the new ones."""
import pytest
import torch

import weight_only_bit_split_gb300 as wobs
from test_gpu_decode_ops import BF16, F16, F32, dev, gen, randn

pytestmark = pytest.mark.gpu
ROWS, K = 4096, 256


def products(dtype):
    """A product over weights of ``dtype``, its output the caller's."""
    return {F16: lambda w, x, y: wobs.wobs_gemv_f16(w, x, y), BF16: lambda w, x, y: wobs.wobs_gemv_bf16(w, x, y)}[dtype]


def read_back(g):
    cache = wobs.Kv4Cache.empty(ROWS // 64, 64, 1, K, dev())
    table = torch.randperm(ROWS // 64, generator=g, device=dev()).to(torch.int32)[None]
    lens = torch.tensor([ROWS], dtype=torch.int32, device=dev())
    x = randn(g, 1, ROWS, 1, K)
    k, v = (torch.zeros(1, ROWS, 1, K, dtype=BF16, device=dev()) for _ in range(2))

    def call():
        wobs.wobs_kv4_append(cache, x, x, table, lens)
        wobs.wobs_kv4_read(cache, table, lens, ROWS, dtype=BF16, k=k, v=v)
    return x, call, v.view(ROWS, K)


def dequantised(g):
    x, w, out = randn(g, ROWS, K), randn(g, K), torch.zeros(ROWS, K, dtype=F16, device=dev())
    return x, lambda: wobs.wobs_dequantize_q8_1(wobs.wobs_rmsnorm_q8_1(x, w)[0], F16, out), out


@pytest.mark.parametrize("m", [1, 4])
@pytest.mark.parametrize("make", [read_back, dequantised])
def test_outputs_are_weights_at_once(make, m):
    g = gen(61)
    x, call, weights = make(g)
    product = products(weights.dtype)
    a = randn(g, m, K, dtype=weights.dtype)
    y = torch.zeros(m, ROWS, dtype=F16 if weights.dtype == F16 else F32, device=dev())
    for _ in range(30):
        x.copy_(randn(g, *x.shape))
        for between in range(3):                                         # products and quantisers that run ahead in between
            call()
            for _ in range(between):
                wobs.wobs_quantize_q8_1(x.view(-1, K)[:32])
            product(weights, a, y)
            got = y.clone()
            torch.cuda.synchronize()
            product(weights, a, y)
            assert torch.equal(got, y)
            x.neg_()


def test_the_caches_planes_are_q4_0_weights_at_once():
    g = gen(62)
    cache = wobs.Kv4Cache.empty(ROWS // 64, 64, 1, K, dev())
    table = torch.arange(ROWS // 64, dtype=torch.int32, device=dev())[None]
    lens = torch.tensor([ROWS], dtype=torch.int32, device=dev())
    x = randn(g, 1, ROWS, 1, K)
    xq = wobs.wobs_quantize_q8_1(randn(g, 2, K))
    qs, d = cache.kq.view(ROWS, K // 2), cache.kd.view(ROWS, K // 32)
    y = torch.zeros(2, ROWS, device=dev())
    for _ in range(30):
        x.copy_(randn(g, *x.shape))
        wobs.wobs_kv4_append(cache, x, x, table, lens)
        wobs.wobs_gemv_q4_0_q8_1(qs, d, xq, y)
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, wobs.wobs_gemv_q4_0_q8_1(qs, d, xq, y)[0])
        want_qs, want_d = wobs.wobs_quantize_q4_0(x.view(ROWS, K))
        assert torch.equal(got, wobs.wobs_gemv_q4_0_q8_1(want_qs, want_d, xq)[0])

"""A captured graph's workspace outlives larger calls on its stream."""
import pytest
import torch

import weight_only_bit_split_gb300 as wobs
from test_gpu_decode_ops import BF16, dev, gen, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("step_graph", [True, False])
def test_a_graph_replays_after_its_streams_workspace_grew(step_graph):
    g = gen(71)
    stream = torch.cuda.Stream()
    small, table, lens = make_cache(g, [3000], 16, 1, 64)                # pieces of several CTAs, which meet in the workspace
    large, table2, lens2 = make_cache(g, [3000], 16, 1, 128)
    q, q2 = randn(g, 1, 1, 4, 64, dtype=BF16), randn(g, 1, 4, 4, 128, dtype=BF16)
    want, out = wobs.wobs_attn_kv4(small, q, table, lens), torch.zeros_like(q)
    torch.cuda.synchronize()
    call = lambda: wobs.wobs_attn_kv4(small, q, table, lens, out=out)  # noqa: E731
    if step_graph:
        graph = wobs.StepGraph(call, stream)
    else:
        with torch.cuda.stream(stream):
            call()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
    before = wobs._ws_cache[(0, stream.cuda_stream)]
    size, address = before.numel(), before.data_ptr()
    with torch.cuda.stream(stream):
        wobs.wobs_attn_kv4(large, q2, table2, lens2)
    stream.synchronize()
    assert wobs._ws_cache[(0, stream.cuda_stream)].numel() > size        # the graph still uses the one in front of it
    del before
    with torch.cuda.stream(stream):
        others = [torch.full((size,), 0x5A, dtype=torch.uint8, device=dev()) for _ in range(8)]
    stream.synchronize()
    assert all(t.data_ptr() + t.numel() <= address or address + size <= t.data_ptr() for t in others)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert all(bool((t == 0x5A).all()) for t in others)

"""The cached workspaces (CPU only: streams and device memory are stand-ins)."""
import gc
import types
import weakref

import pytest
import torch

import weight_only_bit_split_gb300 as wobs


@pytest.fixture
def cache(monkeypatch):
    """The workspace cache, empty, with sizes that the test sets (``size[0]``) and memory of the CPU."""
    size, zeros = [0], torch.zeros
    monkeypatch.setattr(wobs, "_ws_cache", {})
    monkeypatch.setattr(wobs, "wobs_workspace_size", lambda *a: size[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(torch, "zeros", lambda n, dtype=None, device=None: zeros(n, dtype=dtype))
    return size


def test_a_replaced_workspace_stays_alive(cache):
    """A captured graph holds a workspace's address, not the tensor: replays must not write into freed memory."""
    kept, sizes = [], []
    for need in (5000, 300_000, 300_001, 700_000, 699_000):
        cache[0] = need
        ws = wobs.workspace(wobs.OP_ATTN_KV4, 1, 8, 64, torch.device("cuda", 0))
        assert ws.numel() >= need and not ws.any()
        sizes.append(ws.numel())
        kept.append(weakref.ref(ws))
        del ws
    gc.collect()
    assert all(r() is not None for r in kept)
    # twice the last one at least, so all together are no more than twice as large as the newest
    assert sum(set(sizes)) <= 2 * sizes[-1] and sizes[3] == sizes[4]

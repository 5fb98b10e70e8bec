"""Limits of the cache's tables (CPU only: every call returns before a launch)."""
import pytest

from test_abi_decode import _append, _attn, _cache, _read


@pytest.mark.parametrize("call", [_append, _read, _attn])
def test_tables_past_31_bits_of_positions_are_refused(call):
    """Positions, and those of the step after the last, are 32-bit numbers."""
    for page, most in ((16, (1 << 27) - 63), (1 << 20, 1 << 11), (1 << 20, (1 << 31) - 1)):
        rc, msg = call(cache=_cache(page_size=page, heads=1, dim=64), ldt=most, most=most)
        assert rc == -3 and "2^31" in msg

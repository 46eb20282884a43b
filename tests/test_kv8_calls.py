"""Calls of the 8-bit KV cache that are refused, without a GPU: flags that mean nothing."""

import pytest

from test_kv8 import B, _attn, _cache  # noqa: F401  (B: the fixture)


@pytest.mark.parametrize("flags", [2, 3, -1, 1 << 30])
def test_unknown_flags_are_refused(B, flags):  # noqa: F811
    assert B.load_library().blt_kv8_attend(_cache(B), _attn(B, flags=flags), None) == B.BLT_ERR_INVALID_ARG
    assert b"flags" in B.load_library().blt_kv8_last_error()

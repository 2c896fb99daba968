"""The cache operations' workspace grows with the list and is never empty."""
import ctypes

import pytest

from online_softmax_attention_gb300 import _abi
from test_cache_refusals import _cache


@pytest.mark.parametrize("pages", [1, 64, 100000])
def test_bytes(pages):
    lib, c = _abi.load(), _cache(n_pages=pages)
    need = [lib.attn_cache_workspace_bytes(ctypes.byref(c), n) for n in (0, 1, 3, 1000, 262144)]
    assert need[0] >= 3 * 4 * pages and need == sorted(need) and all(x % 256 == 0 for x in need)
    for n, x in zip((0, 1, 3, 1000, 262144), need):  # three lists of n + 1, three of the pages, a header
        assert x >= 12 * (n + 1) + 12 * pages

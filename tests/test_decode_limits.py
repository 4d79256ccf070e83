"""Sizes of include/moe_decode.h's calls that no memory holds, on the CPU: they
are refused on the host, and never come out small where numbers are added up or
multiplied."""
import ctypes

import pytest

from padded_permute_combine_gb300 import _lib
from padded_permute_combine_gb300 import build as libbuild

FAKE = 1 << 20  # an aligned non-null address, never dereferenced: host checks fail first
MOST = (1 << 63) - 1
UNSUPPORTED = _lib.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


@pytest.mark.parametrize("requests", [1 << 58, (1 << 58) + 1, 1 << 62, MOST])
def test_select(lib, requests):
    """2^58 x 64 rows are 2^64, which 64 bits hold as none."""
    assert lib.moe_beam_select_workspace_size(requests, 64, 10) == 0
    assert lib.moe_beam_select(FAKE, 1, 10, FAKE, None, requests, 64, 10, 2, -1, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == UNSUPPORTED


@pytest.mark.parametrize("size", [1 << 31, 1 << 62, MOST])
def test_copy(lib, size):
    """A page's pieces are counted, and the count of 2^63 - 1 bytes does not come out negative."""
    some = (_lib.CachePages * 1)(_lib.CachePages(FAKE, MOST, size))
    assert lib.moe_cache_copy(some, 1, 10, FAKE, FAKE, 3, None, None, None) == UNSUPPORTED


@pytest.mark.parametrize("heads,kv", [((1 << 30) + 1, 1), ((1 << 31) - 1, 1), ((1 << 31) - 1, (1 << 31) - 1), ((1 << 30) + 2, (1 << 29) + 1)])
def test_attention_heads(lib, heads, kv):
    """Warps' shares of the heads are counted in 32 bits."""
    assert lib.moe_attention_decode_workspace_size(1, heads, kv, 1) == 0
    cache = ctypes.byref(_lib.KvCache(FAKE, FAKE, 8, 16 * kv, kv, 1, 1, 16, kv, 1))
    rows = ctypes.byref(_lib.Heads(FAKE, heads, 1))
    assert lib.moe_attention_decode(cache, rows, heads, FAKE, 4, 4, FAKE, 1, None, None, 0.1, 0, FAKE, FAKE, FAKE, 1 << 60, None, None) == UNSUPPORTED
    assert lib.moe_attention_decode_workspace_size(1, 1 << 30, 1 << 30, 1) > 0

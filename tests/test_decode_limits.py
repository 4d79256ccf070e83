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

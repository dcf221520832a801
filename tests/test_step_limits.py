"""The largest step tables: sizes whose places or sums would pass 32 bits in the kernels are refused (CPU)."""

import ctypes

import pytest

from quantized_memory_bound_amd import ocq
from test_step_host import _step, _tables


def _workspace(tables, tokens):
    return ocq.lib().ocq_step_tables_workspace_bytes(ctypes.byref(tables), tokens)


@pytest.mark.parametrize("tokens", [(1 << 30) + 1, (1 << 31) - 65536, (1 << 31) - 1])
def test_tokens_whose_places_would_wrap(tokens):
    """A lane of the second launch goes on by up to 64 x 256 x 4 tokens: past 2^31 - 2^16 the next place was below 0, and
    was written to."""
    assert _step(tokens=tokens) == -2 and "2^30" in ocq.last_error()
    assert _workspace(_tables(), tokens) == 0 and _workspace(_tables(), 1 << 30) > 0


@pytest.mark.parametrize("max_pages", [(1 << 30) + 1, (1 << 31) - 16384, (1 << 31) - 1])
def test_pages_whose_places_would_wrap(max_pages):
    """A lane goes on by up to 64 x 256 pages: with more than 2^31 - 2^14 of them it would never have ended."""
    t = _tables(requests=1, max_pages=max_pages, table_stride=max_pages, page_size=1)
    assert _step(t) == -2 and "2^30" in ocq.last_error() and _workspace(t, 5) == 0
    t.max_pages = 1 << 30
    assert _workspace(t, 5) == 64


@pytest.mark.parametrize("requests,max_pages", [(65536, 1 << 15), (4096, 1 << 19), (3, 1 << 30), (2, 1 << 30)])
def test_tables_whose_page_sums_would_wrap(requests, max_pages):
    t = _tables(requests=requests, max_pages=max_pages, table_stride=max_pages, page_size=1)
    assert _step(t) == -2 and "requests * max_pages" in ocq.last_error()
    assert _workspace(t, 5) == 0
    t.max_pages = ((1 << 31) - 1) // requests
    assert _workspace(t, 1 << 20) == (requests + 1) * 32

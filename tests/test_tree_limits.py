"""CPU checks of the tree, cache and page calls at the ends of their ranges: sizes whose sums pass 32 bits,
workspaces that serve smaller calls, tables that overlap.  All of it is decided on the host."""
import ctypes

import pytest

from confidence_driven_speculative_gb300 import _build, binding
from tests.test_tree_abi import EINVAL, EWORKSPACE, pages


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


@pytest.mark.parametrize("B,max_pages,page", [(65536, 65536, 16), (65536, 32768, 1), (16384, 131072, 1), (2, 1 << 30, 1)])
def test_pages_of_more_entries_than_32_bits_count(lib, B, max_pages, page):
    """Ranks of wanted pages are 32-bit sums over the table's entries."""
    assert B * max_pages > 2 ** 31 - 1
    kw = dict(B=B, page_size=page, workspace_bytes=binding.dspark_pages_workspace_size(B, 64))
    assert lib.dspark_update_pages(ctypes.byref(pages(max_pages=max_pages, **kw)), None) == EINVAL
    assert "too large a batch" in binding.last_error()
    kw["workspace_bytes"] = 8  # as many columns as the limit allows: the next check speaks
    assert lib.dspark_update_pages(ctypes.byref(pages(max_pages=(2 ** 31 - 1) // B, **kw)), None) == EWORKSPACE

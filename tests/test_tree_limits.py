"""CPU checks of the tree, cache and page calls at the ends of their ranges: sizes whose sums pass 32 bits,
workspaces that serve smaller calls, tables that overlap.  All of it is decided on the host."""
import ctypes

import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import _build, binding
from oracle import tree as ot
from tests.test_attn_abi import FAKE, fake, valid
from tests.test_tree_abi import EINVAL, EWORKSPACE, cache, pages, tree


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load()


@pytest.mark.parametrize("B,max_pages,page", [(65536, 65536, 16), (65536, 32768, 1), (16384, 131072, 1), (2, 1 << 30, 1)])
def test_pages_of_more_entries_than_32_bits_count(lib, B, max_pages, page):
    """Ranks of wanted pages are 32-bit sums over the table's entries."""
    assert B * max_pages > 2 ** 31 - 1
    kw = dict(B=B, page_size=page, table_out=1 << 45, workspace_bytes=binding.dspark_pages_workspace_size(B, 64))
    assert lib.dspark_update_pages(ctypes.byref(pages(max_pages=max_pages, **kw)), None) == EINVAL
    assert "too large a batch" in binding.last_error()
    kw["workspace_bytes"] = 8  # as many columns as the limit allows: the next check speaks
    assert lib.dspark_update_pages(ctypes.byref(pages(max_pages=(2 ** 31 - 1) // B, **kw)), None) == EWORKSPACE


def test_oracle_nothing_is_kept_of_no_parent():
    """By hand: pages of 16; whatever keep_len says, pages from the first position on."""
    table = np.array([[2, 4, -1, -1, -1]], np.int32)
    out, granted, src, dst, totals = ot.update_pages(table, [-1, 0, 1], [40, 20, 16], [70, 21, 9], 16, 12)
    assert out.tolist() == [[0, 1, 3, 5, 6], [2, 4, -1, -1, -1], [7, -1, -1, -1, -1]]
    assert granted.tolist() == [70, 21, 9] and totals.tolist() == [4, 0]
    assert src.tolist() == dst.tolist() == [-1, -1, -1]


def test_oracle_a_last_page_that_is_missing_is_told():
    """By hand: pages of 16.  Nothing can be written at position 20 if its page is none, except where nobody
    looks at it any more, or writes it."""
    table = np.array([[2, -1, -1, -1], [5, 12, -1, -1]], np.int32)
    out, granted, src, dst, totals = ot.update_pages(
        table, [0, 1, 0, 0, 0], [20, 20, 20, 16, 20], [40, 40, 20, 40, 40], 16, 12, first=[0, 0, 0, 0, 32])
    assert granted.tolist() == [20, 20, 20, 40, 40]
    assert out.tolist() == [[2, -1, 0, -1], [5, -1, 1, -1], [2, -1, -1, -1], [2, 3, 4, -1], [-1, -1, 6, -1]]
    assert totals.tolist() == [5, 0]


HEADS = [(32, 8, 128), (8, 8, 64), (40, 1, 128), (128, 1, 64), (15, 3, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_an_attention_workspace_of_more_rows_serves_fewer(lib, Hq, Hkv, D):
    sizes = [binding.dspark_attn_workspace_size(Hq, Hkv, D, q) for q in range(1, 66)]
    assert sizes == sorted(sizes)
    # the checks that come after the workspace's: a missing cache, missing keys
    a = dict(Hq=Hq, Hkv=Hkv, D=D, k_cache=None, k_rot=None, workspace_bytes=sizes[-1])
    for q_max in range(1, 66):
        for f in (lambda x: lib.dspark_step_attention(x, None), lambda x: lib.dspark_prompt_attention(x, None),
                  lambda x: lib.dspark_step_attention_sinks(x, 4, None),
                  lambda x: lib.dspark_prompt_attention_sinks(x, 4, None),
                  lambda x: lib.dspark_step_attention_tree(x, FAKE, 4, None)):
            assert f(ctypes.byref(valid(q_max=q_max, **a))) == EINVAL, q_max
            assert "is NULL" in binding.last_error() or "outside [1, 64]" in binding.last_error()


def test_chains_and_prompts_do_not_need_what_trees_need(lib):
    """For 32 heads over 8 of 128 and 65 rows a chain's parts take 26 625 024 bytes; 64 rows of a tree take more."""
    a = dict(Hq=32, Hkv=8, D=128, k_cache=None, k_rot=None, workspace_bytes=26625024)
    for q_max in (40, 63, 64, 65):
        for f in (lib.dspark_step_attention, lib.dspark_prompt_attention):
            assert f(ctypes.byref(valid(q_max=q_max, **a)), None) == EINVAL
            assert "is NULL" in binding.last_error()
    assert lib.dspark_step_attention_tree(ctypes.byref(valid(q_max=64, **a)), FAKE, 0, None) == EWORKSPACE
    # and prompts of any length need one size
    small = binding.dspark_attn_workspace_size(32, 8, 128, 8192)
    for q_max in (1, 30, 65, 66, 8192):
        assert lib.dspark_prompt_attention(ctypes.byref(valid(**dict(a, q_max=q_max, workspace_bytes=small))), None) == EINVAL
        assert "is NULL" in binding.last_error()


def test_a_tree_workspace_of_the_largest_batch_serves_smaller_ones(lib):
    """A program sizes its workspace for the most requests, rows and ids that it will see."""
    shapes = [(1, 1, 8), (1, 64, 129280), (1, 74, 129280), (8, 512, 129280), (1024, 4096, 1024), (1025, 4096, 1024),
              (65536, 1 << 24, 1024), (64, 4096, 1 << 24)]
    sizes = {s: binding.dspark_tree_workspace_size(*s) for s in shapes}
    for big in shapes:
        for small in shapes:
            if all(x <= y for x, y in zip(small, big)):
                assert sizes[small] <= sizes[big], (small, big)
    for B, rows, V in shapes:  # what the call asks for is what the size says
        t = tree(B=B, rows=rows, V=V, workspace_bytes=sizes[B, rows, V] - 1)
        assert lib.dspark_verify_tree(ctypes.byref(t), None) == EWORKSPACE
        assert f"needs {sizes[B, rows, V]}" in binding.last_error()


@pytest.mark.parametrize("window", [1, 2, 3, 8, 31, 32, 63, 64, 100])
@pytest.mark.parametrize("sinks", [0, 1, 4, 20, 1 << 30])
@pytest.mark.parametrize("lens", [True, False])
def test_tree_rows_within_a_window(window, sinks, lens):
    """A row sees the ancestors that the same tokens in a chain would see: those inside its window, and sinks."""
    rng = np.random.default_rng(window + sinks)
    n = [64, 0, 64, 17, 40]
    off = np.concatenate([[0], np.cumsum(n)])
    rows = int(off[-1]) + 2
    parent = np.full(rows, 5, np.int32)
    for b, deep in enumerate((1.0, 0.0, 0.9, 1.0, 0.3)):
        for j in range(n[b]):
            parent[off[b] + j] = j - 1 if rng.random() < deep else rng.integers(-1, max(j, 1))
    start = rng.integers(0, 12, 5) if lens else np.zeros(5, int)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    args = (i32(parent), i32(off), i32(start) if lens else None)
    seen, pos, req = binding.tree_rows(*args, window=window, sinks=sinks)
    full = binding.tree_rows(*args)
    assert torch.equal(pos, full[1]) and torch.equal(req, full[2])
    cut = 0
    for b in range(5):
        for j in range(n[b]):
            at, up = j, [j]
            while at > 0 and 0 <= parent[off[b] + at] < at:
                at = int(parent[off[b] + at])
                up.append(at)
            here = start[b] + len(up) - 1
            word = sum(1 << a for d, a in enumerate(up) if d < window or here - d < sinks)
            assert int(seen[off[b] + j]) % (1 << 64) == word, (b, j)
            cut += word != int(full[0][off[b] + j]) % (1 << 64)
    assert window < 64 or cut == 0
    # the last row of the chain of 64 has left the root, at least, and its ancestors up to this place
    assert window > 63 or cut > 0 or start[0] + 63 - window < sinks
    assert (seen[off[-1]:] == 0).all()


def test_tree_rows_refuses_a_negative_window():
    for kw in (dict(window=-1), dict(window=4, sinks=-1)):
        with pytest.raises(ValueError, match="neither is < 0"):
            binding.tree_rows(torch.zeros(3, dtype=torch.int32), torch.tensor([0, 3], dtype=torch.int32), **kw)


def test_tables_that_overlap_are_refused(lib):
    """Rows of table_out are written while other requests read theirs of table_in; 4 and 6 rows of 8 columns."""
    f = lambda at: lib.dspark_update_pages(ctypes.byref(pages(  # noqa: E731
        B=6, table_in=FAKE, table_out=FAKE + at, workspace_bytes=8)), None)
    for at in (-6 * 32 + 4, -32, 0, 32, 4 * 32 - 4):
        assert f(at) == EINVAL, at
        assert "overlaps" in binding.last_error()
    for at in (-6 * 32, 4 * 32):  # side by side: the next check speaks
        assert f(at) == EWORKSPACE, at


def test_commit_path_says_what_is_wrong_with_lengths(lib):
    table, path = fake(4, 8, dtype=torch.int32), fake(4, 9, dtype=torch.int32)
    for bad, what in (([1, 2, 3, 4], "torch tensor"), (np.zeros(4, np.int32), "torch tensor"), (7, "torch tensor"),
                      (fake(4, dtype=torch.int64), "int32"), (fake(5, dtype=torch.int32), "4 elements"),
                      (torch.zeros(4, dtype=torch.int32), "CUDA")):
        with pytest.raises(ValueError, match=what):
            binding.dspark_commit_path(cache(), table, bad, path)


@pytest.mark.parametrize("window", [0, 3])
def test_tree_rows_of_no_requests(window):
    """A batch of padding: nothing is looked up in the lengths, of which there are none."""
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    for rows in ((), (0, 0, 0)):
        for off, lens in ((i32(0), i32()), (i32(0, 0), i32(5)), (i32(0), None)):
            seen, pos, req = binding.tree_rows(i32(*rows), off, lens, window, 2)
            assert (seen == 0).all() and (pos == 0).all() and (req == -1).all() and len(seen) == len(rows)

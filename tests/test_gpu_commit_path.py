"""dspark_commit_path against the oracle: entries are moved, so every bit counts."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import tree as ot
from tests.attn_harness import dev, make_table

pytestmark = pytest.mark.gpu


def make(seed, layers, pages, page, Hkv, D, heads_first=False, pad=0):
    """Two views [layers, pages, page, Hkv, D] with bits of every kind (NaN among them); ``pad``
    elements between the entries that belong to nobody."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        inner = (Hkv, page) if heads_first else (page, Hkv)
        t = torch.randint(-32768, 32768, (layers, pages, *inner, D + pad), generator=gen, device="cuda",
                          dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
        out.append((t.transpose(2, 3) if heads_first else t)[..., :D])
    return out


def whole(t):
    """All of a view's storage, as bits on the host."""
    base = t
    while base._base is not None:
        base = base._base
    return base.contiguous().view(torch.int16).cpu().numpy()


def bits5(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def check(k, v, table, lens, path, stream=None):
    want = [bits5(t) for t in (k, v)]
    outside = [whole(t).copy() for t in (k, v)]
    for w in want:
        for b in range(len(path)):
            ot.commit(w, table[b], 0 if lens is None else int(lens[b]), [int(x) for x in path[b]])
    c = binding.CacheView(k, v)
    args = dev(table), None if lens is None else dev(np.asarray(lens, np.int32)), dev(np.asarray(path, np.int32))
    torch.cuda.synchronize()
    binding.dspark_commit_path(c.cache, *args, stream=stream)
    torch.cuda.synchronize()
    for t, w, o in zip((k, v), want, outside):
        assert np.array_equal(bits5(t), w)
        now = whole(t)
        if now.size != w.size:  # what lies between the entries stays
            assert int((now != o).sum()) <= int((w.reshape(-1) != 0).size)
    return want


def rows_of(paths, q_max):
    return [p + [-1] * (q_max - len(p)) for p in paths]


PATHS = [[0], [0, 1, 2], [0, 2], [0, 1, 3, 4, 8], [0, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11], [3, 4, 5], [0, 5, 9, 16], [],
         list(range(1, 17)), [16], [0, 1, 2, 3, 16]]


@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("heads_first", [False, True])
@pytest.mark.parametrize("layers,Hkv,D", [(1, 1, 64), (3, 2, 128), (2, 8, 128), (2, 3, 8), (1, 5, 200), (2, 1, 512)])
def test_against_the_oracle(cuda_lib, page, heads_first, layers, Hkv, D):
    rng = np.random.default_rng(page)
    lens = rng.integers(0, 50, len(PATHS))
    need = [-(-(int(s) + 17) // page) for s in lens]
    table = make_table(need, sum(need) + 2, max(need), rng)
    k, v = make(1, layers, sum(need) + 2, page, Hkv, D, heads_first)
    check(k, v, table, lens, rows_of(PATHS, 17))


def test_entries_apart(cuda_lib):
    """Strides that leave room between heads: what lies there stays."""
    rng = np.random.default_rng(0)
    need = [3] * len(PATHS)
    table = make_table(need, 40, 3, rng)
    k, v = make(2, 2, 40, 16, 3, 64, pad=8)
    between = [whole(t).reshape(2, 40, 16, 3, 72)[..., 64:].copy() for t in (k, v)]
    check(k, v, table, [9] * len(PATHS), rows_of(PATHS, 17))
    for t, w in zip((k, v), between):
        assert np.array_equal(whole(t).reshape(2, 40, 16, 3, 72)[..., 64:], w)


def test_odd_paths(cuda_lib):
    """The same row twice, rows in front of their places (left), an end in the middle, far rows."""
    paths = [[0, 2, 2, 2], [4, 3, 2, 1, 0], [2, 0, 4, 1], [1, -1, 5, 6], [-3, 4, 5], [0, 1 << 30], [0, 64, 2147483647],
             [5, 5, 5, 5, 5, 5, 7, 6]]
    rng = np.random.default_rng(3)
    table = make_table([6] * len(paths), 60, 6, rng)
    k, v = make(3, 2, 60, 16, 2, 64)
    check(k, v, table, [10, 0, 31, 5, 5, 5, 5, 20], rows_of(paths, 8))


def test_longest_paths(cuda_lib):
    """65 rows that all move by one, and by half, over many pages."""
    paths = [list(range(1, 66)), [min(2 * j, 64 + j) for j in range(65)]]
    table = make_table([140, 140], 300, 140, np.random.default_rng(4))
    for page in (1, 3):
        k, v = make(4, 3, 300, page, 2, 64)
        check(k, v, table, [5, 0], paths)


def test_pages_that_are_none(cuda_lib):
    paths = [[0, 3, 20, 21], [0, 2, 18], [0, 40]]
    table = make_table([4, 4, 2], 12, 4, np.random.default_rng(5))
    table[0, 1] = -1
    table[1, 0] = 12
    k, v = make(5, 2, 12, 16, 2, 64)
    check(k, v, table, [0, 10, 30], rows_of(paths, 4))


def test_no_lengths_means_position_zero(cuda_lib):
    table = make_table([2, 2], 5, 2, np.random.default_rng(6))
    k, v = make(6, 2, 5, 16, 2, 64)
    check(k, v, table, None, rows_of([[0, 4, 9], [1, 3]], 5))


def test_one_tensor_for_keys_and_values(cuda_lib):
    """k and v as the halves of one tensor's entries."""
    kv = make(7, 2, 20, 16, 2, 128)[0]
    k, v = kv[..., :64], kv[..., 64:]
    table = make_table([3] * 4, 20, 3, np.random.default_rng(7))
    check(k, v, table, [3, 9, 20, 0], rows_of([[0, 2, 5], [0, 1, 9], [4], [0, 3]], 12))


def test_cache_past_32_bits(cuda_lib):
    """Entries whose offsets pass 2^31 elements."""
    big = torch.zeros((1, 140000, 64, 2, 128), dtype=torch.bfloat16, device="cuda")
    assert big.numel() > 1 << 31
    table = np.array([[139999, 139000]], np.int32)
    big[0, 139999, :40] = torch.arange(40, device="cuda", dtype=torch.bfloat16)[:, None, None]
    c = binding.CacheView(big, big.clone())
    binding.dspark_commit_path(c.cache, dev(table), dev(np.array([10], np.int32)), dev(np.array([[0, 3, 20, -1]], np.int32)))
    torch.cuda.synchronize()
    assert big[0, 139999, 9:14, 0, 0].tolist() == [9, 10, 13, 30, 13]


def test_streams_and_graphs(cuda_lib):
    rng = np.random.default_rng(8)
    table = make_table([4] * 3, 14, 4, rng)
    k, v = make(8, 4, 14, 16, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(k, v, table, [3, 20, 7], rows_of([[0, 2], [0, 5, 6], [1]], 9), stream=side.cuda_stream)
    c = binding.CacheView(k, v)
    path, lens, tab = dev(np.full((3, 9), -1, np.int32)), dev(np.zeros(3, np.int32)), dev(table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.dspark_commit_path(c.cache, tab, lens, path, stream=side.cuda_stream)
    for new in ([[0, 3, 8], [0], [0, 1, 4]], [[0, 1, 2], [0, 2, 3, 4], []]):
        starts = rng.integers(0, 40, 3).astype(np.int32)
        path.copy_(dev(np.array(rows_of(new, 9), np.int32)))
        lens.copy_(dev(starts))
        want = [bits5(t) for t in (k, v)]
        for w in want:
            for b in range(3):
                ot.commit(w, table[b], int(starts[b]), new[b])
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(bits5(k), want[0]) and np.array_equal(bits5(v), want[1])

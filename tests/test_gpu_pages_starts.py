"""dspark_update_pages where a request has less behind it than its keep_len says: what granted_len then
promises has memory."""
import numpy as np
import pytest

from tests.test_gpu_update_pages import Case

pytestmark = pytest.mark.gpu


def granted_has_memory(c, want):
    """Every position from what is kept to granted_len has a page, but for those that the window left."""
    out, granted = want[:2]
    for b in range(c.B):
        p = b if c.parent is None else c.parent[b]
        keep = int(c.keep[b]) if 0 <= p < len(c.table) else 0
        for pos in range(keep, granted[b]):
            i = pos // c.page
            dropped = c.first is not None and (i + 1) * c.page <= c.first[b] and i * c.page >= c.sinks
            assert dropped or out[b, i] >= 0, (b, pos)


@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5)])
def test_a_request_of_no_parent_starts_from_nothing(cuda_lib, page, window, sinks):
    """keep_len is what the row held before: a request that ended, and one that starts in its place."""
    for seed in range(4):
        c = Case(seed, [90, 33, 64, 1, 128, 200], 12, page, spare=12 * 80 // page + 20, starts=0.4,
                 window=window, sinks=sinks)
        none = c.parent < 0
        assert none.any()
        c.keep[none] = np.random.default_rng(seed).integers(1, 70, none.sum())
        c.want[none] = c.keep[none] + 9
        want = c.check()
        granted_has_memory(c, want)
        assert (want[1] == c.want).all()


def test_no_parent_and_no_table_before(cuda_lib):
    c = Case(1, [], 3, 16, width=6)
    c.keep[:], c.want[:] = [40, 16, 3], [70, 17, 3]
    want = c.check()
    assert (want[0] >= 0).sum(1).tolist() == [5, 2, 1] and want[1].tolist() == [70, 17, 3]


@pytest.mark.parametrize("page", [2, 7, 16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 5)])
@pytest.mark.parametrize("missing", [-1, 1 << 30])
def test_a_last_page_that_is_missing_is_told(cuda_lib, page, window, sinks, missing):
    told = 0
    for seed in range(4):
        c = Case(seed, [90, 33, 64, 1, 128, 200], 14, page, spare=14 * 40 // page + 40, window=window, sinks=sinks)
        for b in np.flatnonzero(c.parent >= 0)[::2]:
            c.table[c.parent[b], c.keep[b] // page] = missing
        want = c.check()
        granted_has_memory(c, want)
        told += ((want[1] < c.want) & (want[1] == c.keep)).sum()
        assert want[4][1] == 0  # no page was missing
    assert told > 0


def test_a_missing_page_that_the_window_left_is_not_missed(cuda_lib):
    c = Case(2, [90, 33], 2, 16, starts=0.0, forks=False, window=1)
    c.keep[:], c.want[:], c.first = [40, 33], [80, 60], np.array([48, 32], np.int32)
    c.table[:, 2] = -1
    want = c.check()
    assert want[1].tolist() == [80, 33]

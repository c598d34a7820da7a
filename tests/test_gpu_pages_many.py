"""dspark_update_pages with more requests than the cluster has threads, and tables near their limit."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.attn_harness import dev
from tests.test_gpu_update_pages import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [16384, 16385, 40000, 65536])
@pytest.mark.parametrize("forks,held", [(True, False), (False, False), (True, True)])
def test_more_requests_than_threads(cuda_lib, B, forks, held):
    """A thread looks after up to four; forks of few into many, or everyone goes on."""
    lens = [1 + i % 11 for i in range(700 if forks else B)]
    want = Case(B, lens, B, 4, spare=B // 2, grow=5, forks=forks, held=held, layers=1, Hkv=1, D=8).check()
    assert want[4][1] > 0 or not forks  # pages ran out
    assert (want[2] >= 0).any() or not forks


def test_a_table_of_nearly_2_to_the_31_entries(cuda_lib):
    """Entries lie past 2^32 bytes; the last requests' are at the end."""
    B, width, page = 2000, 1073000, 1
    assert 2 ** 31 - 2 ** 21 < B * width < 2 ** 31
    num_pages = 9000
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0], table[B - 1, width - 2] = torch.arange(B, device="cuda"), B
    keep, want = np.ones(B, np.int32), np.full(B, 3, np.int32)
    keep[B - 1], want[B - 1] = width - 1, width
    h = binding.PageBuffers(None, B_in=B, B=B, max_pages=width, page_size=page, num_pages=num_pages)
    h.bind(table, dev(keep), dev(want))
    binding.dspark_update_pages(h.pages)
    torch.cuda.synchronize()
    assert h.granted_len.tolist() == want.tolist() and h.totals.tolist() == [num_pages - (B + 1) - 2 * (B - 1) - 1, 0]
    assert int((h.table_out >= 0).sum()) == B + 2 * (B - 1) + 2
    new = h.table_out[:B - 1, 1:3].reshape(-1)  # the lowest free pages, by request
    assert torch.equal(new, torch.arange(B + 1, B + 1 + 2 * (B - 1), dtype=torch.int32, device="cuda"))
    assert h.table_out[B - 1, [0, width - 2, width - 1]].tolist() == [B - 1, B, B + 1 + 2 * (B - 1)]

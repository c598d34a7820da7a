"""dspark_step_attention_tree where the batch has many tiles, so that units hold two blocks of columns, and the
same trees in small batches, where each block is a unit, against the fp64 oracle (bounds: attn_harness.py)."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.attn_harness import dev, wide
from tests.test_gpu_step_attention_tree import Tree

pytestmark = pytest.mark.gpu


class Many(Tree):
    """Trees, and behind them requests of one row each whose tiles fill the CTAs."""

    def __init__(self, seed, ctx, n, Hq, Hkv, D, page, window=0, many=True, **kw):
        long = 2500 if not window else min(2500, window + 300)
        tiles = Hkv * (min(long, window or long) // 128)
        fill = 8 * torch.cuda.get_device_properties(0).multi_processor_count // tiles + 1 if many else 0
        super().__init__(seed, ctx + [long + 3 * i for i in range(fill)], n + [1] * fill, Hq, Hkv, D, page,
                         window=window, **kw)


# rows of a block: 32, 25, 8, 128 (one block holds any tree), 2
GROUPS = [(8, 2), (5, 1), (16, 1), (2, 2), (64, 1)]


@pytest.mark.parametrize("many", [True, False])
@pytest.mark.parametrize("Hq,Hkv", GROUPS)
@pytest.mark.parametrize("D,page", [(128, 16), (64, 1), (128, 48), (64, 128)])
def test_against_the_oracle(cuda_lib, many, Hq, Hkv, D, page):
    Many(1, [700, 0, 64, 1300, 127], [64, 33, 0, 50, 9], Hq, Hkv, D, page, many=many, heads_first=page == 48).check()


@pytest.mark.parametrize("many", [True, False])
@pytest.mark.parametrize("window,sinks", [(200, 0), (300, 4), (400, 150)])
def test_window_and_sinks(cuda_lib, many, window, sinks):
    Many(2, [700, 0, 640, 1300, 127], [64, 33, 64, 50, 9], 8, 2, 128, 16, window=window, sinks=sinks, many=many).check()


@pytest.mark.parametrize("many", [True, False])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("ctx", [100, 300])
def test_a_draft_that_blew_up_reaches_its_descendants_only(cuda_lib, many, value, ctx):
    c = Many(3, [ctx, 30], [60, 40], 8, 2, 128, 16, many=many)
    clean = c.call()
    words = c.words.cpu().numpy().view(np.uint64)
    j = 5
    c.vc[int(c.table[0, (ctx + j) // 16]), (ctx + j) % 16, 1, 5] = value
    got = c.call()
    hit = np.zeros_like(got, bool)
    below = [i for i in range(60) if int(words[i]) >> j & 1]
    assert j in below and len(below) < 60 and max(below) >= 32
    hit[below, 4:8, 5] = True
    assert np.array_equal(got[~hit], clean[~hit])
    assert np.isnan(got[hit]).all() if np.isnan(value) else (got[hit] == value).all()


@pytest.mark.parametrize("many", [True, False])
def test_masked_keys_may_hold_anything(cuda_lib, many):
    c = Many(4, [400, 37, 1000], [50, 33, 64], 8, 2, 128, 16, window=250, sinks=5, many=many)
    kc, vc = wide(c.kc), wide(c.vc)
    used = np.zeros(kc.shape[:2], bool)
    for b in range(c.B):
        for p in range(c.ctx[b] + c.n[b]):
            if p > c.ctx[b] - c.window or p < 5:
                used[c.table[b, p // 16], p % 16] = True
    for t in (c.kc, c.vc):
        bad = torch.where(torch.rand(t.shape, device="cuda") < 0.5, float("nan"), float("inf"))
        t.copy_(torch.where(dev(used)[:, :, None, None], t.float(), bad).to(torch.bfloat16))
    c.check(kc=np.where(used[:, :, None, None], kc, 0.0), vc=np.where(used[:, :, None, None], vc, 0.0))


@pytest.mark.parametrize("many", [True, False])
@pytest.mark.parametrize("page", [1, 16])
def test_bad_pages_are_masked(cuda_lib, many, page):
    c = Many(5, [300, 20, 5, 500], [40, 2, 33, 60], 8, 2, 128, page, many=many)
    c.table[0, 100 // page: 200 // page + 1] = -1
    c.table[1, :] = c.num_pages
    c.table[3, 0] = 1 << 30
    c.table[3, 510 // page] = -7
    c.bind()
    got = c.check()
    assert np.all(got[c.row_off[1]:c.row_off[2]] == 0.0)


def test_sharp_softmax_and_far_scores(cuda_lib):
    Many(6, [900, 60], [40, 64], 8, 2, 128, 16, q_std=24.0).check()


def test_same_bits_every_time(cuda_lib):
    for many in (True, False):
        c = Many(7, [4000, 17, 900], [60, 1, 45], 32, 8, 128, 16, many=many)
        first = c.call()
        for _ in range(5):
            assert np.array_equal(c.call(), first)


@pytest.mark.parametrize("D,page", [(128, 16), (64, 1)])
def test_a_wait_that_runs_out(cuda_lib, D, page):
    c = Many(8, [4000, 9, 700], [64, 33, 50], 8, 2, D, page)
    want = c.call()
    try:
        binding.dspark_set_wait_timeout_ns(100)
        binding.dspark_step_attention_tree(c.h.attn, c.words, 0)
        torch.cuda.synchronize()  # the launch returned
        status = c.h.device_status()
    finally:
        binding.dspark_set_wait_timeout_ns(0)
    assert status == 1
    binding.dspark_workspace_init(c.h.workspace.data_ptr(), c.h.ws_bytes)
    assert np.array_equal(c.call(), want)

"""Calls on trees, sinks and pages that the other files do not make: a wait that runs out, new host
threads, the largest batches, far pages, two of them side by side."""
import threading

import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.attn_harness import dev, wide
from tests.test_gpu_attention_hosts import in_a_thread
from tests.test_gpu_attention_sinks import Prompt, Step, check_prompt
from tests.test_gpu_commit_path import bits5, make
from tests.test_gpu_step_attention_tree import Tree
from tests import test_gpu_update_pages as pages
from tests import test_gpu_verify_tree as verify

pytestmark = pytest.mark.gpu

STATUS_WAIT = 1


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind,shape", [
    ("tree", dict(ctx=[700], n=[3])),                          # a tile a CTA
    ("tree", dict(ctx=[9000, 4000, 4], n=[64, 17, 2])),        # cut units, one and two blocks
    ("tree", dict(ctx=[11 * i % 500 for i in range(300)], n=[1 + i % 9 for i in range(300)])),
    ("sinks", dict(ctx=[9000, 4000, 4], n=[9, 17, 2])),
    ("prompt", [3000, 31, 600]),
])
def test_a_wait_that_runs_out(cuda_lib, kind, shape, D, page):
    if kind == "tree":
        c = Tree(1, Hq=8, Hkv=2, D=D, page=page, **shape)
        call = lambda: binding.dspark_step_attention_tree(c.h.attn, c.words, 0)  # noqa: E731
    elif kind == "sinks":
        c = Step(1, 4, Hq=8, Hkv=2, D=D, page=page, window=600, **shape)
        call = lambda: binding.dspark_step_attention_sinks(c.h.attn, 4)  # noqa: E731
    else:
        c = Prompt(1, 4, shape, Hq=8, Hkv=2, D=D, window=200)
        call = lambda: binding.dspark_prompt_attention_sinks(c.h.attn, 4)  # noqa: E731
    want = c.call()
    try:
        binding.dspark_set_wait_timeout_ns(100)
        call()
        torch.cuda.synchronize()  # the launch returned
        status = c.h.device_status()
    finally:
        binding.dspark_set_wait_timeout_ns(0)
    assert status == STATUS_WAIT
    binding.dspark_workspace_init(c.h.workspace.data_ptr(), c.h.ws_bytes)
    assert np.array_equal(c.call(), want)


def test_the_first_cuda_call_of_a_thread(cuda_lib):
    stream = torch.cuda.Stream()
    tree = Tree(2, ctx=[90, 700], n=[30, 1], Hq=8, Hkv=2, D=128, page=16)
    sinks = Step(2, 4, ctx=[90, 700], n=[3, 1], Hq=8, Hkv=2, D=64, page=1, window=50)
    prompt = Prompt(2, 4, [70, 300], Hq=4, Hkv=2, D=128, window=100)
    for c, call in ((tree, lambda: binding.dspark_step_attention_tree(tree.h.attn, tree.words, 0, stream.cuda_stream)),
                    (sinks, lambda: binding.dspark_step_attention_sinks(sinks.h.attn, 4, stream.cuda_stream)),
                    (prompt, lambda: binding.dspark_prompt_attention_sinks(prompt.h.attn, 4, stream.cuda_stream))):
        want = c.call()
        c.h.out.fill_(7.0)
        torch.cuda.synchronize()
        in_a_thread(call)
        torch.cuda.synchronize()
        assert np.array_equal(wide(c.h.out), want)
    v, p = verify.Case(2, [17, 3], 32000), pages.Case(2, [90, 33, 64], 12, 16, spare=60)
    hv, hp = v.handle(), p.handle()
    torch.cuda.synchronize()
    in_a_thread(lambda: binding.dspark_verify_tree(hv.tree, stream.cuda_stream))
    v.check(hv, call=False)
    k, w = make(2, 2, 6, 16, 2, 64)
    table, path, lens = dev(np.array([[3, 1]], np.int32)), dev(np.array([[0, 5, 9]], np.int32)), dev(np.array([4], np.int32))
    before = bits5(k)
    c = binding.CacheView(k, w)
    torch.cuda.synchronize()
    in_a_thread(lambda: binding.dspark_commit_path(c.cache, table, lens, path, stream=stream.cuda_stream))
    torch.cuda.synchronize()
    assert np.array_equal(bits5(k)[:, 3, 5], before[:, 3, 9]) and np.array_equal(bits5(k)[:, 3, 6], before[:, 3, 13])
    old = [bits5(t) for t in p.caches]
    in_a_thread(lambda: binding.dspark_update_pages(hp.pages, stream.cuda_stream))
    torch.cuda.synchronize()
    assert np.array_equal(hp.table_out.cpu().numpy(), p.want_all()[0]) and len(old) == 2


def test_trees_from_two_threads_with_shapes_of_their_own(cuda_lib):
    """Different amounts of shared memory and workspaces of their own, side by side."""
    cases = [Tree(3, ctx=[300, 40, 9000], n=[10, 3, 64], Hq=8, Hkv=1, D=128, page=16),
             Tree(4, ctx=[500, 90], n=[16, 9], Hq=8, Hkv=2, D=64, page=7)]
    want = [c.call() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.h.out.fill_(7.0)
    torch.cuda.synchronize()
    errors, ready = [], threading.Barrier(len(cases))

    def work(c, stream):
        try:
            ready.wait()
            for _ in range(1000):
                binding.dspark_step_attention_tree(c.h.attn, c.words, 0, stream.cuda_stream)
        except Exception as e:  # noqa: BLE001 (shown below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c, w in zip(cases, want):
        assert c.h.device_status() == 0
        assert np.array_equal(wide(c.h.out), w)


def test_one_workspace_serves_trees_and_chains_in_turn(cuda_lib):
    """dspark_step_attention and its variants share a workspace that is zeroed once."""
    t = Tree(5, ctx=[9000, 40, 3000], n=[17, 3, 9], Hq=8, Hkv=2, D=128, page=16)
    s = Step(5, 4, ctx=[9000, 40, 3000], n=[17, 3, 9], Hq=8, Hkv=2, D=128, page=16, window=2000)
    want = t.call(), s.call()
    size = max(t.h.ws_bytes, s.h.ws_bytes)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for c in (t, s):
        c.h.attn.workspace, c.h.attn.workspace_bytes = ws.data_ptr(), size
    for _ in range(3):
        for c, w in ((t, want[0]), (s, want[1])):
            assert np.array_equal(c.call(), w)
            binding.dspark_step_attention(c.h.attn)
    torch.cuda.synchronize()


@pytest.mark.parametrize("B", [129, 2000])
def test_many_trees(cuda_lib, B):
    Tree(6, ctx=[(37 * i) % 150 for i in range(B)], n=[i % 4 for i in range(B)], Hq=2, Hkv=1, D=64, page=16).check()


def test_the_largest_batch(cuda_lib):
    """65536 requests, most of them without a row."""
    B = 65536
    n = [0] * B
    ctx = [0] * B
    for b in (0, 1, 777, 40000, 65535):
        n[b], ctx[b] = 3, 20
    Tree(7, ctx=ctx, n=n, Hq=2, Hkv=1, D=64, page=32).check()
    verify.Case(7, n, 64).check()


def test_far_pages(cuda_lib):
    """Entries whose offsets in the caches pass 2^31 elements."""
    c = Tree(8, ctx=[200, 70], n=[40, 5], Hq=4, Hkv=2, D=128, page=64, spare=140000)
    assert c.kc.numel() > 1 << 31 and c.table.max() > 100000
    words = c.words.cpu().numpy().view(np.uint64)
    got = c.call()
    from oracle import attention as oa
    q, pos = wide(c.q), c.tree_pos.cpu().numpy()
    from tests.attn_harness import assert_close
    for b in range(2):
        r0, r1 = c.row_off[b], c.row_off[b + 1]
        m = c.ctx[b] + c.n[b]
        pages_b = dev(c.table[b][: -(-m // 64)]).long()
        k, v = (wide(t[pages_b]).reshape(-1, 2, 128)[:m] for t in (c.kc, c.vc))
        seen = oa.seen_tree(c.ctx[b], words[r0:r1], pos[r0:r1], m)
        o, spread, ds = oa.attend_seen(q[r0:r1], k, v, seen, c.scale)
        assert_close(got[r0:r1], o, spread, ds, m, b)


@pytest.mark.parametrize("G", [3, 5, 6, 20, 40, 64, 100, 127, 128])
def test_groups_that_do_not_divide_a_block(cuda_lib, G):
    """Rows of a block that are no whole number of vectors; blocks of one row."""
    Tree(9, ctx=[150, 0, 300], n=[7, 1, 13], Hq=2 * G, Hkv=2, D=64, page=16, window=100, sinks=3).check()


def test_queries_of_padding_rows_may_hold_anything(cuda_lib):
    c = Tree(10, ctx=[300, 40], n=[5, 33], Hq=8, Hkv=2, D=128, page=16, extra_rows=40)
    clean = c.call()
    c.q[38:] = float("nan")
    assert np.array_equal(c.call(), clean)
    c.q[38:] = float("inf")
    assert np.array_equal(c.call(), clean)


def test_a_row_that_blew_up_stays_alone(cuda_lib):
    """NaN in one row's queries: the others are what they were."""
    c = Tree(11, ctx=[300, 40], n=[60, 33], Hq=8, Hkv=2, D=128, page=16)
    clean = c.call()
    c.q[7, 3] = float("nan")
    got = c.call()
    hit = np.zeros_like(got, bool)
    hit[7, 3] = True
    assert np.array_equal(got[~hit], clean[~hit]) and np.isnan(got[hit]).all()


def test_large_finite_values(cuda_lib):
    """Values near bfloat16's largest: sums stay finite where the values' own weighted mean does."""
    c = Tree(12, ctx=[900, 60], n=[30, 64], Hq=8, Hkv=2, D=128, page=16)
    c.vc.copy_((c.vc.float() * 1e37).to(torch.bfloat16))
    got = c.check()
    assert np.isfinite(got[: c.row_off[-1]]).all()


@pytest.mark.parametrize("far", [200.0, 1e4])
def test_scores_far_from_zero(cuda_lib, far):
    """All scores lie far from 0 and close together."""
    c = Tree(13, ctx=[700, 60], n=[30, 10], Hq=4, Hkv=2, D=128, page=16, q_std=0.5)
    c.kc[..., 0] = 8.0
    c.q[..., 0] = far
    c.check()


def test_prompt_sinks_bounds_of_the_window(cuda_lib):
    """Windows and sinks past 32 bits' middle, and prompts shorter than either."""
    for window, sinks in (((1 << 31) - 1, 5), (5, (1 << 31) - 1), ((1 << 31) - 1, (1 << 31) - 1)):
        check_prompt(Prompt(14, sinks, [130, 3, 300], Hq=4, Hkv=2, D=64, window=window))
        Step(14, sinks, ctx=[130, 0, 300], n=[3, 2, 9], Hq=4, Hkv=2, D=64, page=16, window=window).check()
        Tree(14, ctx=[130, 0, 300], n=[3, 2, 9], Hq=4, Hkv=2, D=64, page=16, window=window, sinks=sinks).check()

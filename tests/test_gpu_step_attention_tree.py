"""dspark_step_attention_tree and dspark_rope_append_tree against the fp64 oracle (bounds:
attn_harness.py)."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests.attn_harness import assert_close, dev, wide
from tests.test_gpu_step_attention import Case

pytestmark = pytest.mark.gpu


def random_tree(rng, n, deep=0.5):
    return [-1] + [int(j - 1 if rng.random() < deep else rng.integers(0, j)) for j in range(1, n)]


class Tree(Case):
    """A batch of trees.  ``words``: what the rows see; by default themselves and their ancestors."""

    def __init__(self, seed, ctx, n, Hq, Hkv, D, page, window=0, sinks=0, words=None, deep=0.5, **kw):
        super().__init__(seed, ctx, n, Hq, Hkv, D, page, window=window, **kw)
        rng = np.random.default_rng(seed + 1)
        self.sinks = sinks
        parent = np.array([p for m in n for p in (random_tree(rng, m, deep) if m else [])]
                          + [0] * (self.rows - sum(n)), np.int32)
        self.parent = dev(parent)
        seen, pos, _ = binding.tree_rows(self.parent, dev(self.row_off), dev(np.array(ctx, np.int32)))
        self.words = seen if words is None else dev(np.array(words, np.uint64).view(np.int64))
        self.tree_pos = pos
        self.bind()

    def bind(self, seq_lens=True):
        super().bind(seq_lens)
        if hasattr(self, "tree_pos"):
            self.h.attn.packed_pos = self.tree_pos.data_ptr()

    def call(self, stream=None):
        self.h.out.fill_(7.0)
        binding.dspark_step_attention_tree(self.h.attn, self.words, self.sinks, stream)
        torch.cuda.synchronize()
        assert self.h.device_status() == 0
        return wide(self.h.out)

    def check(self, got=None, kc=None, vc=None):
        got = self.call() if got is None else got
        q = wide(self.q)
        kc, vc = (wide(self.kc) if kc is None else kc), (wide(self.vc) if vc is None else vc)
        words, pos = self.words.cpu().numpy().view(np.uint64), self.tree_pos.cpu().numpy()
        for b in range(self.B):
            r0, r1 = self.row_off[b], self.row_off[b + 1]
            m = self.ctx[b] + self.n[b]
            k, valid = oa.gather(kc, self.table[b], m)
            v, _ = oa.gather(vc, self.table[b], m)
            seen = oa.seen_tree(self.ctx[b], words[r0:r1], pos[r0:r1], m, self.window, self.sinks, valid)
            o, spread, ds = oa.attend_seen(q[r0:r1], k, v, seen, self.scale)
            assert_close(got[r0:r1], o, spread, ds, m, b)
        assert np.all(got[self.row_off[-1]:] == 7.0)  # padding rows stay as they were
        return got


SHAPES = [
    # a root alone: the first token of all, in a tile, at its end
    dict(ctx=[0], n=[1], Hq=1, Hkv=1, D=128, page=16),
    dict(ctx=[127], n=[1], Hq=8, Hkv=2, D=64, page=32),
    dict(ctx=[1999], n=[1], Hq=32, Hkv=8, D=128, page=16),
    # trees in one tile, over a tile's border, from its first key on; requests without rows
    dict(ctx=[5, 120, 0, 300, 255, 128], n=[3, 17, 0, 64, 1, 33], Hq=16, Hkv=4, D=128, page=16),
    dict(ctx=[100, 64, 0], n=[64, 64, 64], Hq=4, Hkv=4, D=64, page=64),
    # odd groups, more rows than a block of columns takes
    dict(ctx=[700, 1, 64], n=[17, 40, 2], Hq=15, Hkv=3, D=128, page=64),
    dict(ctx=[90, 511], n=[64, 13], Hq=7, Hkv=1, D=64, page=256),
    dict(ctx=[400, 30], n=[60, 16], Hq=16, Hkv=1, D=128, page=16),
    dict(ctx=[140], n=[5], Hq=128, Hkv=1, D=64, page=16),
    # pages of every kind
    dict(ctx=[50, 333], n=[25, 2], Hq=8, Hkv=2, D=128, page=1),
    dict(ctx=[50, 333], n=[25, 2], Hq=8, Hkv=2, D=128, page=7),
    dict(ctx=[200, 333], n=[25, 2], Hq=8, Hkv=2, D=128, page=48),
    # more requests than CTAs
    dict(ctx=[3 * i % 197 for i in range(200)], n=[1 + i % 9 for i in range(200)], Hq=2, Hkv=1, D=64, page=16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(
    str(x) for x in (s["ctx"][0], s["n"][0], s["Hq"], s["Hkv"], s["D"], s["page"])))
@pytest.mark.parametrize("heads_first", [False, True])
def test_against_the_oracle(cuda_lib, shape, heads_first):
    Tree(1, heads_first=heads_first, **shape).check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (129, 130), (300, 7), (5000, 9)])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_window_and_sinks(cuda_lib, window, sinks, page):
    Tree(2, ctx=[0, 127, 640, 1000, 1500], n=[3, 9, 64, 1, 30], Hq=10, Hkv=2, D=128, page=page,
         window=window, sinks=sinks).check()


@pytest.mark.parametrize("D", [64, 128])
def test_any_set_of_rows(cuda_lib, D):
    """Words that are no tree: nothing, everything (rows that are not there among it), later rows."""
    rng = np.random.default_rng(3)
    n = [64, 5, 40]
    rows = sum(n) + 3
    words = rng.integers(0, 1 << 64, rows, dtype=np.uint64)
    words[:3] = [0, (1 << 64) - 1, 1 << 63]
    words[64] = 0
    words[70] = (1 << 64) - 1
    got = Tree(3, ctx=[0, 0, 90], n=n, Hq=6, Hkv=2, D=D, page=16, words=words).check()
    assert np.all(got[0] == 0.0) and np.all(got[64] == 0.0)  # rows that see nothing


def test_a_chain_is_the_step_attention(cuda_lib):
    """Where the tree is a chain, both calls are held to one result."""
    kw = dict(ctx=[300, 40, 700], n=[17, 9, 1], Hq=8, Hkv=2, D=128, page=16)
    a, b = Case(4, **kw), Tree(4, deep=1.0, **kw)
    assert torch.equal(a.q, b.q) and torch.equal(a.kc, b.kc)
    a.check(got=b.call())


def test_no_seq_lens_means_position_zero(cuda_lib):
    c = Tree(5, ctx=[0, 0], n=[20, 2], Hq=4, Hkv=2, D=128, page=16)
    c.bind(seq_lens=False)
    c.check()


def test_sharp_softmax(cuda_lib):
    Tree(6, ctx=[900, 60], n=[30, 64], Hq=8, Hkv=2, D=128, page=16, q_std=24.0).check()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("ctx", [100, 120])
def test_a_draft_that_blew_up_reaches_its_descendants_only(cuda_lib, value, ctx):
    c = Tree(7, ctx=[ctx, 30], n=[40, 3], Hq=8, Hkv=2, D=128, page=16)
    clean = c.call()
    words = c.words.cpu().numpy().view(np.uint64)
    j = 5
    c.vc[int(c.table[0, (ctx + j) // 16]), (ctx + j) % 16, 1, 5] = value
    got = c.call()
    hit = np.zeros_like(got, bool)
    below = [i for i in range(40) if int(words[i]) >> j & 1]
    assert j in below and len(below) < 40
    hit[below, 4:8, 5] = True
    assert np.array_equal(got[~hit], clean[~hit])
    assert np.isnan(got[hit]).all() if np.isnan(value) else (got[hit] == value).all()


def test_masked_keys_may_hold_anything(cuda_lib):
    """NaN and infinities behind the last row, in pages of nobody, between the sinks and the window."""
    for window, sinks in ((0, 0), (40, 0), (40, 5)):
        c = Tree(8, ctx=[400, 37], n=[9, 3], Hq=8, Hkv=2, D=128, page=16, window=window, sinks=sinks)
        kc, vc = wide(c.kc), wide(c.vc)
        used = np.zeros(kc.shape[:2], bool)
        for b in range(c.B):
            for p in range(c.ctx[b] + c.n[b]):
                if not window or p > c.ctx[b] - window or p < sinks:
                    used[c.table[b, p // 16], p % 16] = True
        for t in (c.kc, c.vc):
            bad = torch.where(torch.rand(t.shape, device="cuda") < 0.5, float("nan"), float("inf"))
            t.copy_(torch.where(dev(used)[:, :, None, None], t.float(), bad).to(torch.bfloat16))
        c.check(kc=np.where(used[:, :, None, None], kc, 0.0), vc=np.where(used[:, :, None, None], vc, 0.0))


@pytest.mark.parametrize("page", [1, 16, 64])
def test_bad_pages_are_masked_and_can_leave_rows_empty(cuda_lib, page):
    c = Tree(9, ctx=[300, 20, 5, 500], n=[4, 2, 3, 60], Hq=8, Hkv=2, D=128, page=page)
    c.table[0, 100 // page: 200 // page + 1] = -1
    c.table[1, :] = c.num_pages
    c.table[3, 0] = 1 << 30
    c.table[3, 510 // page] = -7  # a page of the tree itself
    c.bind()
    got = c.check()
    assert np.all(got[c.row_off[1]:c.row_off[2]] == 0.0)


def test_positions_past_the_table_are_masked(cuda_lib):
    c = Tree(10, ctx=[60, 31], n=[30, 2], Hq=4, Hkv=2, D=128, page=16)
    c.table = np.ascontiguousarray(c.table[:, :5])  # 80 positions of 90
    c.max_pages = c.h.attn.max_pages = 5
    c.bind()
    c.check()


def test_same_bits_every_time_and_on_any_stream(cuda_lib):
    c = Tree(11, ctx=[4000, 17, 900], n=[60, 1, 25], Hq=32, Hkv=8, D=128, page=16)
    first = c.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(6):
        assert np.array_equal(c.call(side.cuda_stream if k % 2 else None), first)


def test_graph_replays_follow_the_batch(cuda_lib):
    """One captured call serves other trees, lengths and pages: they are read on the device."""
    kw = dict(Hq=8, Hkv=2, D=128, page=16, q_max=48, window=200, sinks=4)
    a = Tree(12, ctx=[300, 40, 700], n=[5, 48, 1], extra_rows=20, **kw)
    b = Tree(13, ctx=[90, 600, 7], n=[30, 1, 20], extra_rows=23, **kw)
    assert a.rows == b.rows
    want = b.call()
    off, lens, table = dev(a.row_off), dev(np.array(a.ctx, np.int32)), torch.zeros(
        (3, max(a.max_pages, b.max_pages)), dtype=torch.int32, device="cuda")
    words, pos, kc = a.words.clone(), a.tree_pos.clone(), max(a.num_pages, b.num_pages)
    cache = torch.zeros((2, kc, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = a.q.clone()
    h = binding.AttnBuffers(B=3, rows=a.rows, q_max=48, Hq=8, Hkv=2, D=128, page_size=16, num_pages=kc,
                            max_pages=table.shape[1], window=200)
    h.bind(q_rot=q, k_cache=cache[0], v_cache=cache[1], row_off=off, packed_pos=pos, seq_lens=lens, block_table=table)

    def load(c):
        table.fill_(-1)
        table[:, :c.max_pages] = dev(c.table)
        for t, x in ((off, dev(c.row_off)), (lens, dev(np.array(c.ctx, np.int32))), (words, c.words),
                     (pos, c.tree_pos), (q, c.q)):
            t.copy_(x)
        cache[0, :c.num_pages], cache[1, :c.num_pages] = c.kc, c.vc

    load(a)
    binding.dspark_step_attention_tree(h.attn, words, 4)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        binding.dspark_step_attention_tree(h.attn, words, 4, side.cuda_stream)
    for c, w in ((a, a.call()), (b, want)):
        load(c)
        h.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(wide(h.out)[:c.row_off[-1]], w[:c.row_off[-1]])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("page,rows", [(1, 40), (16, 40), (16, 3000)])
def test_append(cuda_lib, interleaved, page, rows):
    """Siblings turn by one position and lie at places of their own."""
    rng = np.random.default_rng(14)
    B, Hq, Hkv, D = 3, 4, 2, 128
    n, ctx = [17, 1, 9], [30, 0, 63]
    off = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    parent = np.array([p for m in n for p in random_tree(rng, m)] + [0] * (rows - sum(n)), np.int32)
    _, pos, req = binding.tree_rows(dev(parent), dev(off), dev(np.array(ctx, np.int32)))
    max_pages = -(-(max(ctx) + 17) // page)
    num_pages = B * max_pages
    table = rng.permutation(num_pages).reshape(B, max_pages).astype(np.int32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn((rows, (Hq + 2 * Hkv) * D), generator=gen, device="cuda").to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    kc, vc = (torch.full((num_pages, page, Hkv, D), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    h = binding.AttnBuffers(B=B, rows=rows, q_max=17, Hq=Hq, Hkv=Hkv, D=D, page_size=page, num_pages=num_pages,
                            max_pages=max_pages, rot_dim=D, interleaved=interleaved)
    common = dict(q=q, k=k, v=v, row_off=dev(off), row_req=req, packed_pos=pos,
                  seq_lens=dev(np.array(ctx, np.int32)), rope_freq=binding.rope_freq(D))
    h.bind(k_cache=kc, v_cache=vc, block_table=dev(table), **common)
    binding.dspark_rope_append_tree(h.attn)
    # the rotation is dspark_rope_append's, to the bit
    h2 = binding.AttnBuffers(B=B, rows=rows, q_max=17, Hq=Hq, Hkv=Hkv, D=D, page_size=page, num_pages=num_pages,
                             max_pages=max_pages, rot_dim=D, interleaved=interleaved, k_rot=True)
    h2.bind(k_cache=torch.zeros_like(kc), v_cache=torch.zeros_like(vc), block_table=dev(table), **common)
    binding.dspark_rope_append(h2.attn)
    torch.cuda.synchronize()
    assert torch.equal(h.q_rot[:off[-1]], h2.q_rot[:off[-1]])
    want_k, want_v = torch.full_like(kc, 5.0), torch.full_like(vc, 5.0)
    for b in range(B):
        for j in range(n[b]):
            p = ctx[b] + j
            want_k[int(table[b, p // page]), p % page] = h2.k_rot[off[b] + j]
            want_v[int(table[b, p // page]), p % page] = v[off[b] + j]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)

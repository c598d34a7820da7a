"""dspark_step_attention against the fp64 oracle (bounds: attn_harness.py)."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests.attn_harness import assert_close, bits, dev, make_cache, make_table, packed, wide

pytestmark = pytest.mark.gpu


class Case:
    """A batch on the device: ctx cached positions, n rows per request."""

    def __init__(self, seed, ctx, n, Hq, Hkv, D, page, window=0, heads_first=False, q_max=None,
                 q_std=2.0, extra_rows=3, seq_lens=True, scale=None, spare=2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.ctx, self.n, self.window = ctx, n, window
        self.B, self.rows = len(n), sum(n) + extra_rows
        self.row_off, self.row_req, self.pos = packed(ctx, n, self.rows)
        need = [-(-(c + m) // page) for c, m in zip(ctx, n)]
        self.num_pages, self.max_pages = sum(need) + spare, max(max(need), 1)
        self.table = make_table(need, self.num_pages, self.max_pages, rng)
        self.kc = make_cache(self.num_pages, page, Hkv, D, heads_first, gen)
        self.vc = make_cache(self.num_pages, page, Hkv, D, heads_first, gen)
        self.q = (q_std * torch.randn((self.rows, Hq, D), generator=gen, device="cuda")).to(torch.bfloat16)
        self.page, self.Hq, self.Hkv, self.D = page, Hq, Hkv, D
        self.q_max = q_max or max(max(n), 1)
        self.scale = D ** -0.5 if scale is None else scale
        self.h = binding.AttnBuffers(B=self.B, rows=self.rows, q_max=self.q_max, Hq=Hq, Hkv=Hkv,
                                     D=D, page_size=page, num_pages=self.num_pages,
                                     max_pages=self.max_pages, window=window, scale=self.scale)
        self.bind(seq_lens)

    def bind(self, seq_lens=True):
        self.h.bind(q_rot=self.q, k_cache=self.kc, v_cache=self.vc, row_off=dev(self.row_off),
                    seq_lens=dev(np.array(self.ctx, np.int32)) if seq_lens else None,
                    block_table=dev(self.table))

    def call(self, stream=None):
        self.h.out.fill_(7.0)
        binding.dspark_step_attention(self.h.attn, stream)
        torch.cuda.synchronize()
        assert self.h.device_status() == 0
        return wide(self.h.out)

    def check(self, got=None, kc=None, vc=None):
        """``kc``, ``vc``: the cache values to expect, where they are not the cache's own."""
        got = self.call() if got is None else got
        q = wide(self.q)
        kc, vc = (wide(self.kc) if kc is None else kc), (wide(self.vc) if vc is None else vc)
        for b in range(self.B):
            r0, r1 = self.row_off[b], self.row_off[b + 1]
            m = self.ctx[b] + self.n[b]
            k, valid = oa.gather(kc, self.table[b], m)
            v, _ = oa.gather(vc, self.table[b], m)
            o, spread, ds = oa.attend(q[r0:r1], k, v, self.ctx[b], self.scale, self.window, valid)
            assert_close(got[r0:r1], o, spread, ds, m, b)
        assert np.all(got[self.row_off[-1]:] == 7.0)  # padding rows stay as they were
        return got


SHAPES = [
    # one token of one request: the first of all, in a tile, at its end, over several
    dict(ctx=[0], n=[1], Hq=1, Hkv=1, D=128, page=16),
    dict(ctx=[126], n=[1], Hq=4, Hkv=1, D=128, page=64),
    dict(ctx=[127], n=[1], Hq=8, Hkv=2, D=64, page=32),
    dict(ctx=[128], n=[1], Hq=8, Hkv=8, D=128, page=128),
    dict(ctx=[1999], n=[1], Hq=32, Hkv=8, D=128, page=16),
    # a step's rows: requests without rows, rows over a tile's border, odd groups
    dict(ctx=[5, 120, 0, 300, 255], n=[3, 17, 0, 9, 1], Hq=16, Hkv=4, D=128, page=16),
    dict(ctx=[700, 1, 64], n=[17, 17, 2], Hq=15, Hkv=3, D=128, page=64),
    dict(ctx=[90, 511], n=[4, 13], Hq=7, Hkv=1, D=64, page=256),
    # pages of every kind: single slots, odd ones, larger than a tile, no power of two
    dict(ctx=[50, 333], n=[5, 2], Hq=8, Hkv=2, D=128, page=1),
    dict(ctx=[50, 333], n=[5, 2], Hq=8, Hkv=2, D=128, page=7),
    dict(ctx=[50, 333], n=[5, 2], Hq=8, Hkv=2, D=64, page=4),
    dict(ctx=[200, 333], n=[5, 2], Hq=8, Hkv=2, D=128, page=8),
    dict(ctx=[200, 333], n=[5, 2], Hq=8, Hkv=2, D=128, page=48),
    dict(ctx=[200, 733], n=[5, 2], Hq=8, Hkv=2, D=128, page=384),
    # many rows and heads of one cached head
    dict(ctx=[400, 30], n=[17, 16], Hq=16, Hkv=1, D=128, page=16),
    dict(ctx=[140], n=[65], Hq=16, Hkv=2, D=128, page=16),
    dict(ctx=[140], n=[65], Hq=7, Hkv=1, D=64, page=16),
    # more requests than CTAs, one tile each
    dict(ctx=[3 * i % 97 for i in range(200)], n=[1 + i % 4 for i in range(200)], Hq=2, Hkv=1, D=64,
         page=16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(
    str(x) for x in (s["ctx"][0], s["n"][0], s["Hq"], s["Hkv"], s["D"], s["page"])))
@pytest.mark.parametrize("heads_first", [False, True])
def test_against_the_oracle(cuda_lib, shape, heads_first):
    Case(1, heads_first=heads_first, **shape).check()


@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 5000])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_window(cuda_lib, window, page):
    Case(2, ctx=[0, 127, 640, 1000], n=[3, 9, 17, 1], Hq=10, Hkv=2, D=128, page=page,
         window=window).check()


@pytest.mark.parametrize("D", [64, 128])
def test_no_seq_lens_means_position_zero(cuda_lib, D):
    Case(3, ctx=[0, 0], n=[5, 2], Hq=4, Hkv=2, D=D, page=16, seq_lens=False).check()


def test_sharp_softmax_and_a_maximum_that_comes_late(cuda_lib):
    """Scores of standard deviation 24: nearly one key per row; and keys whose length grows with
    the position, so that every tile brings a new maximum."""
    Case(4, ctx=[900, 60], n=[9, 2], Hq=8, Hkv=2, D=128, page=16, q_std=24.0).check()
    c = Case(5, ctx=[1500], n=[7], Hq=8, Hkv=2, D=128, page=16)
    t = torch.arange(c.num_pages * 16, device="cuda")
    grow = torch.zeros(c.num_pages * 16, device="cuda")
    for i, page in enumerate(c.table[0]):
        grow[int(page) * 16: int(page) * 16 + 16] = (t[i * 16: i * 16 + 16] / 200.0)
    c.kc.copy_((c.kc.float() * grow.view(c.num_pages, 16, 1, 1)).to(torch.bfloat16))
    c.check()


def test_masked_keys_may_hold_anything(cuda_lib):
    """NaN and infinities behind the last position, in pages of nobody, before the window, and in
    keys and values of later rows: they reach the rows that see them and no others."""
    for window in (0, 40):
        c = Case(6, ctx=[200, 37], n=[9, 3], Hq=8, Hkv=2, D=128, page=16, window=window)
        kc, vc = wide(c.kc), wide(c.vc)
        used = np.zeros(kc.shape[:2], bool)
        for b in range(c.B):
            for p in range(c.ctx[b] + c.n[b]):
                if not window or p > c.ctx[b] - window:
                    used[c.table[b, p // 16], p % 16] = True
        for t in (c.kc, c.vc):
            bad = torch.where(torch.rand(t.shape, device="cuda") < 0.5, float("nan"), float("inf"))
            t.copy_(torch.where(dev(used)[:, :, None, None], t.float(), bad).to(torch.bfloat16))
        c.check(kc=np.where(used[:, :, None, None], kc, 0.0), vc=np.where(used[:, :, None, None], vc, 0.0))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("window", [0, 30])
def test_a_draft_that_blew_up_reaches_later_rows_only(cuda_lib, value, window):
    c = Case(7, ctx=[100], n=[8], Hq=8, Hkv=2, D=128, page=16, window=window)
    clean = c.call()
    p = 103  # row 3's own key: seen by rows 3.., not by rows 0..2
    c.vc[int(c.table[0, p // 16]), p % 16, 1, 5] = value
    got = c.call()
    hit = np.zeros_like(got, bool)
    hit[3:8, 4:8, 5] = True
    assert np.array_equal(got[~hit], clean[~hit])
    if np.isnan(value):
        assert np.isnan(got[hit]).all()
    else:
        assert (got[hit] == value).all()
    # and one at the window's far edge: seen by the rows that still reach back to it
    if window:
        c = Case(7, ctx=[100], n=[8], Hq=8, Hkv=2, D=128, page=16, window=window)
        p = 100 - window + 1 + 2  # rows 0, 1, 2
        c.vc[int(c.table[0, p // 16]), p % 16, 0, 9] = value
        got = c.call()
        hit = np.zeros_like(got, bool)
        hit[0:3, 0:4, 9] = True
        assert np.array_equal(got[~hit], clean[~hit])
        assert np.isnan(got[hit]).all() if np.isnan(value) else (got[hit] == value).all()


@pytest.mark.parametrize("page", [1, 16, 64])
def test_bad_pages_are_masked_and_can_leave_rows_empty(cuda_lib, page):
    c = Case(8, ctx=[300, 20, 5, 500], n=[4, 2, 3, 17], Hq=8, Hkv=2, D=128, page=page)
    c.table[0, 100 // page: 200 // page + 1] = -1           # a hole
    c.table[1, :] = c.num_pages                              # nothing at all
    c.table[3, 0] = 1 << 30
    c.bind()
    got = c.check()
    r0, r1 = c.row_off[1], c.row_off[2]
    assert np.all(got[r0:r1] == 0.0)


def test_positions_past_the_table_are_masked(cuda_lib):
    """seq_lens beyond max_pages pages: the keys that have a page count, nothing is read past it."""
    c = Case(9, ctx=[60, 31], n=[3, 2], Hq=4, Hkv=2, D=128, page=16)
    c.ctx = [64 + 500, 31]
    c.bind()
    c.check()


def test_same_bits_every_time_and_on_any_stream(cuda_lib):
    c = Case(10, ctx=[4000, 17, 900], n=[17, 1, 5], Hq=32, Hkv=8, D=128, page=16)
    first = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(6):
        assert np.array_equal(c.call(side.cuda_stream if k % 2 else None), first)


def test_graph_replays_follow_the_batch(cuda_lib):
    """One captured call serves other lengths, offsets and pages: they are read on the device."""
    a = Case(11, ctx=[300, 40, 700], n=[5, 9, 1], Hq=8, Hkv=2, D=128, page=16)
    b = Case(12, ctx=[10, 650, 0], n=[9, 2, 4], Hq=8, Hkv=2, D=128, page=16)
    rows = max(a.rows, b.rows)
    num_pages, max_pages = max(a.num_pages, b.num_pages), max(a.max_pages, b.max_pages)
    h = binding.AttnBuffers(B=3, rows=rows, q_max=9, Hq=8, Hkv=2, D=128, page_size=16,
                            num_pages=num_pages, max_pages=max_pages)
    q = torch.zeros((rows, 8, 128), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((num_pages, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    off, lens = dev(np.zeros(4, np.int32)), dev(np.zeros(3, np.int32))
    table = torch.zeros((3, max_pages), dtype=torch.int32, device="cuda")
    h.bind(q_rot=q, k_cache=kc, v_cache=vc, row_off=off, seq_lens=lens, block_table=table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    binding.dspark_step_attention(h.attn, side.cuda_stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.dspark_step_attention(h.attn, side.cuda_stream)
    for c in (a, b, a):
        q[: c.rows] = c.q
        kc[: c.num_pages], vc[: c.num_pages] = c.kc, c.vc
        off.copy_(dev(c.row_off))
        lens.copy_(dev(np.array(c.ctx, np.int32)))
        table.zero_()
        table[:, : c.max_pages] = dev(c.table)
        g.replay()
        torch.cuda.synchronize()
        assert h.device_status() == 0
        used = c.row_off[-1]
        assert np.array_equal(wide(h.out)[:used], c.call()[:used])


def test_a_cache_past_two_to_the_31_elements(cuda_lib):
    Hkv, D, page = 8, 128, 64
    num_pages = ((1 << 31) + (1 << 21)) // (Hkv * D * page)
    c = Case(13, ctx=[1], n=[1], Hq=8, Hkv=Hkv, D=D, page=page, spare=num_pages - 1)
    c.ctx, c.n = [250], [1]
    c.table = np.array([[num_pages - 1, 3, num_pages - 2, num_pages - 3]], np.int32)
    c.max_pages = 4
    c.h.attn.max_pages = 4
    c.bind()
    got = c.call()
    k = torch.cat([c.kc[int(p)] for p in c.table[0]])[:251]
    v = torch.cat([c.vc[int(p)] for p in c.table[0]])[:251]
    o, spread, ds = oa.attend(wide(c.q)[:1], wide(k), wide(v), 250, c.scale)
    assert_close(got[:1], o, spread, ds, 251)


def test_append_then_attend_is_the_attention_of_the_whole_sequence(cuda_lib):
    """Three steps of rows appended and attended, against the oracle on the whole sequence."""
    gen = torch.Generator(device="cuda").manual_seed(14)
    rng = np.random.default_rng(14)
    B, Hq, Hkv, D, page = 3, 8, 2, 128, 16
    max_pages, num_pages = 8, 30
    table = make_table([max_pages] * B, num_pages, max_pages, rng)
    kc = make_cache(num_pages, page, Hkv, D, False, gen, 0.0)
    vc = make_cache(num_pages, page, Hkv, D, False, gen, 0.0)
    ctx = [0, 0, 0]
    keys = [np.zeros((0, Hkv, D))] * B
    vals = [np.zeros((0, Hkv, D))] * B
    for n in ([40, 7, 1], [5, 0, 1], [17, 9, 3]):
        n = [min(x, 65) for x in n]
        rows = sum(n) + 2
        row_off, row_req, pos = packed(ctx, n, rows)
        q, k, v = (torch.randn((rows, h, D), generator=gen, device="cuda").to(torch.bfloat16)
                   for h in (Hq, Hkv, Hkv))
        h = binding.AttnBuffers(B=B, rows=rows, q_max=max(n), Hq=Hq, Hkv=Hkv, D=D, page_size=page,
                                num_pages=num_pages, max_pages=max_pages, rot_dim=D, k_rot=True)
        h.bind(q=q, k=k, v=v, k_cache=kc, v_cache=vc, row_off=dev(row_off), row_req=dev(row_req),
               packed_pos=dev(pos), seq_lens=dev(np.array(ctx, np.int32)), block_table=dev(table),
               rope_freq=binding.rope_freq(D, 1e6))
        binding.dspark_rope_append(h.attn)
        binding.dspark_step_attention(h.attn)
        torch.cuda.synchronize()
        got = wide(h.out)
        for b in range(B):
            r0, r1 = row_off[b], row_off[b + 1]
            keys[b] = np.concatenate([keys[b], wide(h.k_rot)[r0:r1]])
            vals[b] = np.concatenate([vals[b], wide(v)[r0:r1]])
            o, spread, ds = oa.attend(wide(h.q_rot)[r0:r1], keys[b], vals[b], ctx[b], D ** -0.5)
            assert_close(got[r0:r1], o, spread, ds, ctx[b] + n[b])
        ctx = [c + m for c, m in zip(ctx, n)]
    assert bits(kc).any()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 6, 8, 10, 12, 14, 16, 18, 20, 23])
@pytest.mark.parametrize("D", [64, 128])
def test_every_width_of_a_block(cuda_lib, rows, D):
    """8 to 184 columns of one cached head: each way of holding S, P and the queries once or twice,
    and the division into blocks."""
    Case(15, ctx=[333, 1000 - rows, 5], n=[rows, rows, max(rows - 3, 1)], Hq=8, Hkv=1, D=D, page=16).check()


def test_one_cached_head_for_128_query_heads(cuda_lib):
    Case(16, ctx=[150, 40], n=[3, 2], Hq=128, Hkv=1, D=128, page=16).check()


@pytest.mark.parametrize("page", [1, 16])
def test_many_requests_of_very_different_lengths(cuda_lib, page):
    """More requests than one warp looks at, a few of them long: units cut over many CTAs between
    short ones."""
    ctx = [(7 * i) % 40 for i in range(300)]
    ctx[3], ctx[150], ctx[299] = 3000, 1700, 2222
    Case(17, ctx=ctx, n=[1 + i % 3 for i in range(300)], Hq=4, Hkv=2, D=64, page=page).check()


@pytest.mark.parametrize("page", [1, 3, 16])
@pytest.mark.parametrize("heads_first", [False, True])
def test_keys_and_values_in_one_tensor(cuda_lib, page, heads_first):
    """The caches are two views of one [pages, 2, ...] tensor: pages further apart than they are
    long."""
    c = Case(18, ctx=[140, 9], n=[4, 2], Hq=8, Hkv=2, D=128, page=page)
    shape = (c.num_pages, 2, 2, page, 128) if heads_first else (c.num_pages, 2, page, 2, 128)
    both = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = (both[:, i].transpose(1, 2) if heads_first else both[:, i] for i in (0, 1))
    k.copy_(c.kc)
    v.copy_(c.vc)
    c.kc, c.vc = k, v
    c.bind()
    c.check()

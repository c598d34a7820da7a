"""dspark_step_attention_sinks and dspark_prompt_attention_sinks against the fp64 oracle (bounds:
attn_harness.py)."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests import test_gpu_prompt_attention as prompt
from tests.attn_harness import assert_close, dev, wide
from tests.test_gpu_step_attention import Case

pytestmark = pytest.mark.gpu


class Step(Case):
    def __init__(self, seed, sinks, **kw):
        super().__init__(seed, **kw)
        self.sinks = sinks

    def call(self, stream=None):
        self.h.out.fill_(7.0)
        binding.dspark_step_attention_sinks(self.h.attn, self.sinks, stream)
        torch.cuda.synchronize()
        assert self.h.device_status() == 0
        return wide(self.h.out)

    def check(self, got=None, kc=None, vc=None):
        got = self.call() if got is None else got
        q = wide(self.q)
        kc, vc = (wide(self.kc) if kc is None else kc), (wide(self.vc) if vc is None else vc)
        for b in range(self.B):
            r0, r1 = self.row_off[b], self.row_off[b + 1]
            m = self.ctx[b] + self.n[b]
            k, valid = oa.gather(kc, self.table[b], m)
            v, _ = oa.gather(vc, self.table[b], m)
            seen = oa.seen_step(self.ctx[b], self.n[b], m, self.window, self.sinks, valid)
            o, spread, ds = oa.attend_seen(q[r0:r1], k, v, seen, self.scale)
            assert_close(got[r0:r1], o, spread, ds, m, b)
        assert np.all(got[self.row_off[-1]:] == 7.0)
        return got


@pytest.mark.parametrize("sinks", [1, 4, 16, 127, 128, 129, 300, 5000])
@pytest.mark.parametrize("window", [1, 16, 100, 129, 384, 5000])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_step(cuda_lib, sinks, window, page):
    Step(1, sinks, ctx=[0, 127, 640, 1000, 3, 1407], n=[3, 9, 17, 1, 0, 5], Hq=10, Hkv=2, D=128, page=page,
         window=window, heads_first=page == 64).check()


@pytest.mark.parametrize("shape", [
    dict(ctx=[2000], n=[1], Hq=32, Hkv=8, D=128, page=16),
    dict(ctx=[1999, 7], n=[65, 65], Hq=7, Hkv=1, D=64, page=48),
    dict(ctx=[900], n=[17], Hq=128, Hkv=1, D=64, page=128),
    dict(ctx=[3 * i % 997 for i in range(200)], n=[1 + i % 4 for i in range(200)], Hq=2, Hkv=1, D=64, page=16),
], ids=lambda s: str(s["ctx"][0]) + "-" + str(s["Hq"]))
def test_step_shapes(cuda_lib, shape):
    Step(2, 4, window=150, **shape).check()


@pytest.mark.parametrize("page", [1, 8, 24, 64])
@pytest.mark.parametrize("sinks", [3, 30, 65])
def test_step_every_place_of_the_window_in_its_first_tile(cuda_lib, sinks, page):
    # 64 requests whose windows begin at every second key of a tile: the sinks fit in front of some of them
    Step(12, sinks, ctx=[500 + 131 * i for i in range(64)], n=[1 + i % 5 for i in range(64)], Hq=4, Hkv=2, D=128,
         page=page, window=200 + sinks).check()


@pytest.mark.parametrize("sinks", [2**31 - 1, 2**31 - 9])
@pytest.mark.parametrize("page", [1, 16])
def test_step_sinks_without_end(cuda_lib, sinks, page):
    # windows that begin around the end of a tile
    Step(13, sinks, ctx=[99 + w for w in range(24, 34)] + [355], n=[1, 3] * 5 + [2], Hq=4, Hkv=2, D=128, page=page,
         window=100).check()


def test_step_without_sinks_or_window_is_the_plain_call(cuda_lib):
    kw = dict(ctx=[300, 40, 700], n=[17, 9, 1], Hq=8, Hkv=2, D=128, page=16)
    for window, sinks in ((0, 0), (0, 9), (100, 0)):
        a, b = Case(3, window=window, **kw), Step(3, sinks, window=window, **kw)
        assert np.array_equal(b.call(), a.call())


@pytest.mark.parametrize("page", [1, 16, 64])
def test_step_pages_between_the_sinks_and_the_window_are_not_needed(cuda_lib, page):
    """Dropped pages: table entries that are none, and others' pages full of NaN, give what the whole
    table gives."""
    c = Step(4, 20, ctx=[1500, 800], n=[9, 17], Hq=8, Hkv=2, D=128, page=page, window=130)
    want = c.check()
    spoiled = set()
    for b in range(2):
        for i in range(c.max_pages):
            if i * page >= 20 and (i + 1) * page <= c.ctx[b] - 130 + 1:
                spoiled.add(int(c.table[b, i]))
                c.table[b, i] = [-1, 1 << 30, c.table[b, i]][i % 3]
    at = torch.tensor(sorted(spoiled), device="cuda")
    c.kc[at], c.vc[at] = float("nan"), float("inf")
    c.bind()
    assert np.array_equal(c.call(), want)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("pos", [2, 19, 1371, 1376])
def test_step_a_value_that_is_not_finite_reaches_the_rows_that_see_it(cuda_lib, value, pos):
    c = Step(5, 20, ctx=[1500], n=[9], Hq=8, Hkv=2, D=128, page=16, window=130)
    clean = c.call()
    c.vc[int(c.table[0, pos // 16]), pos % 16, 1, 5] = value
    got = c.call()
    hit = np.zeros_like(got, bool)
    hit[[j for j in range(9) if pos < 20 or pos > 1500 + j - 130], 4:8, 5] = True
    assert hit.any()
    assert np.array_equal(got[~hit], clean[~hit])
    assert np.isnan(got[hit]).all() if np.isnan(value) else (got[hit] == value).all()


def test_step_bad_sink_pages_and_rows_that_see_nothing(cuda_lib):
    c = Step(6, 20, ctx=[1500, 40], n=[4, 2], Hq=8, Hkv=2, D=128, page=16, window=33)
    c.table[0, 0] = -1
    c.table[1, :] = -1
    c.bind()
    got = c.check()
    assert np.all(got[4:6] == 0.0)


def test_step_same_bits_and_graphs(cuda_lib):
    c = Step(7, 4, ctx=[4000, 17, 900], n=[17, 1, 5], Hq=32, Hkv=8, D=128, page=16, window=700)
    first = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.dspark_step_attention_sinks(c.h.attn, 4, side.cuda_stream)
    for k in range(4):
        c.h.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(wide(c.h.out), first)
        assert np.array_equal(c.call(side.cuda_stream), first)


class Prompt(prompt.Case):
    def __init__(self, seed, sinks, n, **kw):
        super().__init__(seed, n, **kw)
        self.sinks = sinks

    def call(self, stream=None):
        self.h.out.fill_(7.0)
        binding.dspark_prompt_attention_sinks(self.h.attn, self.sinks, stream)
        torch.cuda.synchronize()
        assert self.h.device_status() == 0
        return wide(self.h.out)


def check_prompt(c, got=None, k=None, v=None, rows=None):
    got = c.call() if got is None else got
    q = wide(c.q)
    k, v = (wide(c.k) if k is None else k), (wide(c.v) if v is None else v)
    for b in range(len(c.n)):
        r0, m = c.row_off[b], c.n[b]
        some = np.arange(m) if m <= 300 or rows is None else np.unique(np.linspace(0, m - 1, rows).astype(int))
        seen = oa.seen_step(0, m, m, c.window, c.sinks)[some]
        o, spread, ds = oa.attend_seen(q[r0 + some], k[r0:r0 + m], v[r0:r0 + m], seen, c.scale)
        assert_close(got[r0 + some], o, spread, ds, m, b)
    assert np.all(got[c.row_off[-1]:] == 7.0)
    return got


@pytest.mark.parametrize("sinks", [1, 4, 127, 128, 129, 200, 5000])
@pytest.mark.parametrize("window", [1, 16, 100, 128, 129, 300, 384])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt(cuda_lib, sinks, window, D):
    check_prompt(Prompt(1, sinks, [1, 5, 130, 777, 0, 256], Hq=4, Hkv=2, D=D, window=window), rows=60)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_long(cuda_lib, D):
    check_prompt(Prompt(2, 4, [3000, 1500, 77], Hq=10, Hkv=2, D=D, window=500), rows=40)


def test_prompt_without_sinks_or_window_is_the_plain_call(cuda_lib):
    for window, sinks in ((0, 0), (0, 9), (100, 0)):
        a = prompt.Case(3, [300, 40, 700], Hq=4, Hkv=2, D=128, window=window)
        b = Prompt(3, sinks, [300, 40, 700], Hq=4, Hkv=2, D=128, window=window)
        assert np.array_equal(b.call(), a.call())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("pos", [0, 3, 4, 130, 500, 899])
@pytest.mark.parametrize("window", [90, 257])
def test_prompt_a_value_that_is_not_finite_reaches_the_rows_that_see_it(cuda_lib, value, pos, window):
    c = Prompt(4, 4, [900, 20], Hq=4, Hkv=2, D=128, window=window)
    clean = c.call()
    c.v[pos, 1, 5] = value
    got = c.call()
    hit = np.zeros_like(got, bool)
    hit[[i for i in range(900) if i >= pos and (i < pos + window or pos < 4)], 2:4, 5] = True
    assert np.array_equal(got[~hit], clean[~hit])
    assert np.isnan(got[hit]).all() if np.isnan(value) else (got[hit] == value).all()


def test_prompt_keys_of_others_may_hold_anything(cuda_lib):
    """Keys and values of the second prompt are NaN: the first one, in front, does not see them."""
    c = Prompt(5, 4, [300, 200], Hq=4, Hkv=2, D=128, window=64)
    clean = c.call()
    c.k[300:], c.v[300:] = float("nan"), float("inf")
    assert np.array_equal(c.call()[:300], clean[:300])


def test_prompt_same_bits_and_graphs(cuda_lib):
    c = Prompt(6, 4, [31 * i % 600 for i in range(40)], Hq=8, Hkv=2, D=128, window=100)
    first = check_prompt(c, rows=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.dspark_prompt_attention_sinks(c.h.attn, 4, side.cuda_stream)
    for k in range(4):
        c.h.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(wide(c.h.out), first)

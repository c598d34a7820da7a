"""dspark_prompt_attention against the fp64 oracle (bounds: attn_harness.py)."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests.attn_harness import assert_close, dev, offsets, wide

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, seed, n, Hq, Hkv, D, window=0, q_std=2.0, extra_rows=5, q_max=None,
                 fused_v=True):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.window, self.scale = n, window, D ** -0.5
        self.rows = sum(n) + extra_rows
        self.row_off = offsets(n)
        rnd = lambda h, s=1.0: (s * torch.randn((self.rows, h, D), generator=gen, device="cuda")).to(torch.bfloat16)
        self.q, self.k = rnd(Hq, q_std), rnd(Hkv)
        wide_v = rnd(Hkv + 3) if fused_v else rnd(Hkv)
        self.v = wide_v[:, 2: 2 + Hkv] if fused_v else wide_v  # rows further apart than Hkv heads
        self.h = binding.AttnBuffers(B=len(n), rows=self.rows, q_max=q_max or max(max(n), 1), Hq=Hq,
                                     Hkv=Hkv, D=D, window=window, prompt=True)
        self.bind()

    def bind(self):
        self.h.bind(q_rot=self.q, k_rot=self.k, v=self.v, row_off=dev(self.row_off))

    def call(self, stream=None):
        self.h.out.fill_(7.0)
        binding.dspark_prompt_attention(self.h.attn, stream)
        torch.cuda.synchronize()
        assert self.h.device_status() == 0
        return wide(self.h.out)

    def check(self, got=None, pick=None):
        """``pick``: the rows of a request to compare (all, where None)."""
        got = self.call() if got is None else got
        q, k, v = wide(self.q), wide(self.k), wide(self.v)
        for b in range(len(self.n)):
            r0, r1 = self.row_off[b], self.row_off[b + 1]
            for i in range(r1 - r0) if pick is None else pick(r1 - r0):
                o, spread, ds = oa.attend(q[r0 + i: r0 + i + 1], k[r0: r0 + i + 1],
                                          v[r0: r0 + i + 1], i, self.scale, self.window)
                assert_close(got[r0 + i: r0 + i + 1], o, spread, ds, i + 1, (b, i))
        assert np.all(got[self.row_off[-1]:] == 7.0)
        return got


def edges(n):
    """The rows next to the borders of 64, 128 and 256, the ends, and a few between."""
    near = {0, 1, n - 2, n - 1} | {m + d for m in range(0, n + 1, 64) for d in (-1, 0, 1)}
    return sorted(i for i in near | {n // 3, n // 2} if 0 <= i < n)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 127, 128, 129, 255, 256, 257, 400])
def test_one_prompt(cuda_lib, n, D):
    Case(1, [n], Hq=4, Hkv=2, D=D).check(pick=edges)


@pytest.mark.parametrize("shape", [
    dict(n=[3, 0, 130, 1, 0, 77, 256], Hq=8, Hkv=2, D=128),       # empty ones among them
    dict(n=[300, 40, 513], Hq=5, Hkv=1, D=128),                   # an odd group
    dict(n=[64, 65, 66], Hq=6, Hkv=6, D=64),                      # no groups
    dict(n=[1] * 40, Hq=4, Hkv=1, D=64),
    dict(n=[700, 9], Hq=14, Hkv=2, D=64),
], ids=lambda s: f"B{len(s['n'])}-{s['Hq']}-{s['Hkv']}-{s['D']}")
def test_packed_prompts(cuda_lib, shape):
    Case(2, **shape).check(pick=edges)


@pytest.mark.parametrize("window", [1, 2, 64, 127, 128, 129, 300, 5000])
@pytest.mark.parametrize("D", [64, 128])
def test_window(cuda_lib, window, D):
    Case(3, [520, 33, 257], Hq=4, Hkv=2, D=D, window=window).check(pick=edges)


def test_long_prompt(cuda_lib):
    Case(4, [4500, 1025], Hq=8, Hkv=2, D=128).check(pick=lambda n: [0, 1, n // 7, n // 2, n - 129, n - 128, n - 1])


def test_sharp_softmax_and_a_maximum_that_comes_late(cuda_lib):
    Case(5, [400], Hq=4, Hkv=2, D=128, q_std=24.0).check(pick=edges)
    c = Case(6, [900], Hq=4, Hkv=2, D=128)
    grow = torch.arange(c.rows, device="cuda")[:, None, None] / 120.0
    c.k.copy_((c.k.float() * grow).to(torch.bfloat16))
    c.check(pick=edges)


def test_neighbours_and_later_rows_may_hold_anything(cuda_lib):
    """A prompt of NaN and infinities next to others, and a row that blew up inside one: it
    reaches its own and later rows of its own prompt."""
    c = Case(7, [100, 200, 150], Hq=4, Hkv=2, D=128)
    clean = c.call()
    for t in (c.k, c.v):
        t[100:300] = float("nan")
        t[450:] = float("inf")  # the padding rows
    got = c.call()
    assert np.array_equal(got[:100], clean[:100]) and np.array_equal(got[300:450], clean[300:450])
    assert np.isnan(got[100:300]).all()
    for value in (float("nan"), float("inf")):
        c = Case(7, [100, 200, 150], Hq=4, Hkv=2, D=128)
        c.v[100 + 130, 1, 5] = value
        got = c.call()
        hit = np.zeros_like(got, bool)
        hit[230:300, 2:4, 5] = True
        assert np.array_equal(got[~hit], clean[~hit])
        assert np.isnan(got[hit]).all() if np.isnan(value) else np.isinf(got[hit]).all()


def test_a_value_that_blew_up_leaves_the_window(cuda_lib):
    c = Case(8, [600], Hq=2, Hkv=1, D=128, window=100)
    clean = c.call()
    c.v[250, 0, 7] = float("nan")
    got = c.call()
    hit = np.zeros_like(got, bool)
    hit[250:350, :, 7] = True
    assert np.array_equal(got[~hit], clean[~hit]) and np.isnan(got[hit]).all()


def test_rows_past_q_max_are_not_computed(cuda_lib):
    c = Case(9, [300, 40], Hq=4, Hkv=2, D=128, q_max=130)
    got = c.call()
    assert np.all(got[130:300] == 7.0)
    full = Case(9, [300, 40], Hq=4, Hkv=2, D=128).call()
    assert np.array_equal(got[:130], full[:130]) and np.array_equal(got[300:340], full[300:340])


def test_same_bits_every_time_on_any_stream_and_in_a_graph(cuda_lib):
    c = Case(10, [700, 33, 1400], Hq=10, Hkv=2, D=128)
    first = c.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for k in range(4):
        assert np.array_equal(c.call(side.cuda_stream if k % 2 else None), first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        binding.dspark_prompt_attention(c.h.attn, side.cuda_stream)
    for _ in range(2):
        c.h.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(wide(c.h.out), first)


@pytest.mark.parametrize("D", [64, 128])
def test_an_output_on_a_16_byte_border(cuda_lib, D):
    c = Case(11, [300, 31], Hq=4, Hkv=2, D=D)
    want = c.call()
    room = torch.full((c.rows * 4 * D + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    c.h.attn.out = room.data_ptr() + 16
    binding.dspark_prompt_attention(c.h.attn)
    torch.cuda.synchronize()
    assert c.h.device_status() == 0
    got = wide(room)
    assert np.all(got[:8] == 7.0) and np.array_equal(got[8:].reshape(want.shape), want)


@pytest.mark.parametrize("grow", [200.0, 900.0])
def test_scores_far_past_the_first_tiles(cuda_lib, grow):
    """Later keys are longer by far: scores rise past the first tile's by more than the weights'
    slack, and by more than fp32's exponent holds."""
    c = Case(12, [700], Hq=4, Hkv=2, D=128)
    at = torch.arange(c.rows, device="cuda")[:, None, None]
    c.k.copy_((c.k.float() * (1.0 + grow / 30.0 * (at // 128))).to(torch.bfloat16))
    c.check(pick=edges)

"""The attention calls at the ends of the number range: scores far from zero, large values.

In the first tests the rows and keys lie along one entry of the head, with powers of two or
few bits, so every score is exact in fp32 and a softmax over them is uniform
over the keys that tie for the maximum: the weights are exactly 1 and 0, and
what is left is the output's own rounding and the fp32 sums (the harness's
bound with ds = 0).
"""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests.attn_harness import assert_close, dev, make_table, offsets, wide

pytestmark = pytest.mark.gpu

KEYS = 300  # positions: three tiles, the last one ragged


def along(x, heads, D):
    """[n, heads, D] bfloat16 with ``x`` [n] in entry 3 and zeros elsewhere."""
    t = torch.zeros((len(x), heads, D), dtype=torch.float64)
    t[:, :, 3] = torch.as_tensor(x, dtype=torch.float64)[:, None]
    return t.to(torch.bfloat16).cuda()


def step_outputs(q, keys, v, scale, page=16, B=160):
    """Rows of q at the last positions of B requests that share the given keys and values: enough
    that some units lie whole in a CTA and others are cut.  All requests give the same."""
    n, Hq, D = q.shape
    m, Hkv = v.shape[:2]
    pages = -(-m // page)
    table = make_table([pages], pages + 1, pages, np.random.default_rng(0))
    cache = []
    for t in (keys, v):
        c = torch.zeros((pages + 1, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
        at = dev(table[0]).long()[torch.arange(m, device="cuda") // page]
        c[at, torch.arange(m, device="cuda") % page] = t
        cache.append(c)
    h = binding.AttnBuffers(B=B, rows=B * n, q_max=n, Hq=Hq, Hkv=Hkv, D=D, page_size=page,
                            num_pages=pages + 1, max_pages=pages, scale=scale)
    h.bind(q_rot=q.repeat(B, 1, 1), k_cache=cache[0], v_cache=cache[1], row_off=dev(offsets([n] * B)),
           seq_lens=dev(np.full(B, m - n, np.int32)), block_table=dev(np.repeat(table, B, 0)))
    binding.dspark_step_attention(h.attn)
    torch.cuda.synchronize()
    assert h.device_status() == 0
    return wide(h.out).reshape(B, n, Hq, D)


def prompt_outputs(q, keys, v, scale):
    """The last rows of a prompt whose every row has the query of q's first row (a batch of one)."""
    n, Hq, D = q.shape
    m, Hkv = v.shape[:2]
    h = binding.AttnBuffers(B=1, rows=m, q_max=m, Hq=Hq, Hkv=Hkv, D=D, scale=scale, prompt=True)
    h.bind(q_rot=q[:1].expand(m, Hq, D).contiguous(), k_rot=keys, v=v, row_off=dev(offsets([m])))
    binding.dspark_prompt_attention(h.attn)
    torch.cuda.synchronize()
    assert h.device_status() == 0
    return wide(h.out)[None, m - n:]


CALLS = {"step": step_outputs, "prompt": prompt_outputs}


def check_ties(call, D, q, k, v=None, n=3, Hq=4, Hkv=2):
    """Softmax over exact scores that tie or lie further apart than any exponent."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    if v is None:
        v = torch.randn((KEYS, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
    got = CALLS[call](along([q] * n, Hq, D), along(k, Hkv, D), v, 1.0)
    s = wide(along([q], 1, D))[0, 0, 3] * wide(along(k, 1, D))[:, 0, 3]
    vw = wide(v)
    for j in range(n):
        seen = np.arange(KEYS) <= KEYS - n + j
        top = s[seen].max()
        rest = s[seen & (s < top)]
        assert len(rest) == 0 or top - rest.max() > 300  # the others weigh nothing
        tied = seen & (s == top)
        o = vw[tied].mean(0)[np.arange(Hq) // (Hq // Hkv)]
        spread = np.abs(vw[tied]).mean(0)[np.arange(Hq) // (Hq // Hkv)]
        assert_close(got[:, j], o, spread, np.zeros(Hq), KEYS, (call, j))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("power", [24, 28, 30, 31, 40, 90, 120])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_from_zero(cuda_lib, call, D, power, sign):
    """Scores near +-2^power: three levels a 64th of that apart, or all of them tied.  The last
    rows' maximum comes early, late, and in every tile."""
    q = 2.0 ** (power // 2)
    unit = sign * 2.0 ** (power - power // 2 - 6)
    j = np.arange(KEYS)
    check_ties(call, D, q, np.full(KEYS, 73 * unit))
    level = 73 + 2 * (j % 3)
    check_ties(call, D, q, level * unit)
    early, late = np.full(KEYS, 73.0), np.full(KEYS, 73.0)
    early[5] += 4 * sign
    late[270] += 4 * sign
    check_ties(call, D, q, early * unit)
    check_ties(call, D, q, late * unit)
    check_ties(call, D, q, (73 + sign * (j // 64)) * unit)  # each tile passes the one before


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("rise", [4.0, 10.0, 11.5, 20.0, 21.5, 60.0])
@pytest.mark.parametrize("power", [100, 115])
def test_large_finite_values_under_a_late_maximum(cuda_lib, call, D, rise, power):
    """Values near 2^power whose averages are as large.  From the second tile on the scores lie
    ``rise`` above the first tile's."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    v = (2.0 ** power * torch.randn((KEYS, 2, D), generator=gen, device="cuda")).to(torch.bfloat16)
    k = np.where(np.arange(KEYS) < 128, 0.0, rise)
    n, Hq = 3, 4
    q, keys = along([1.0] * n, Hq, D), along(k, 2, D)
    got = CALLS[call](q, keys, v, 1.0)
    o, spread, ds = oa.attend(wide(q), wide(keys), wide(v), KEYS - n, 1.0)
    for out in got:
        assert_close(out, o, spread, ds, KEYS, (call, rise))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("power", [12, 16, 20])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_close_together_far_from_zero(cuda_lib, call, D, power, sign):
    """Scores +-2^power + u with u of an eighth's steps in [-4, 4): exact in fp32, and a softmax of them
    is a softmax of the u (ds is theirs)."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, Hq, Hkv = 3, 4, 2
    u = torch.randint(-32, 32, (KEYS,), generator=gen, device="cuda") / 8.0
    q = along([2.0 ** (power // 2)] * n, Hq, D)
    k = along([sign * 2.0 ** (power - power // 2)] * KEYS, Hkv, D)
    q[:, :, 5], k[:, :, 5] = 1.0, u[:, None].to(torch.bfloat16)
    v = torch.randn((KEYS, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
    got = CALLS[call](q, k, v, 1.0)
    only_u = torch.zeros_like(q)
    only_u[:, :, 5] = 1.0
    o, spread, ds = oa.attend(wide(only_u), wide(k), wide(v), KEYS - n, 1.0)
    for out in got:
        assert_close(out, o, spread, ds, KEYS, (call, power))

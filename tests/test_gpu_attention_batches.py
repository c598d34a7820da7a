"""The attention calls on batches at the ends of their range: more requests than the kernels give a
thread one of, empty requests among them; packed rows past 2^31 elements; the widest groups, the
longest pages, one cached head over many CTAs."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests import test_gpu_prompt_attention as prompt
from tests import test_gpu_step_attention as step
from tests.attn_harness import assert_close, dev, offsets, wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [641, 700, 3000])
@pytest.mark.parametrize("page", [1, 16])
def test_step_of_many_requests(cuda_lib, B, page):
    """Two and five requests a thread when the cut is found."""
    n = [0 if i % 5 == 2 or 100 < i < 130 else 1 + i % 2 for i in range(B)]
    ctx = [(7 * i) % 40 for i in range(B)]
    ctx[3], ctx[B // 2], ctx[B - 1] = 2000, 700, 1300
    step.Case(1, ctx=ctx, n=n, Hq=2, Hkv=1, D=64, page=page).check()


@pytest.mark.parametrize("B", [129, 1000])
def test_prompts_of_many_requests(cuda_lib, B):
    """Two and eight prompts a thread when the units are counted."""
    n = [0 if i % 4 == 1 or 60 < i < 90 else 1 + (5 * i) % 37 for i in range(B)]
    n[5], n[B - 2] = 300, 520
    prompt.Case(2, n, Hq=2, Hkv=1, D=64).check(pick=lambda m: [0, m // 2, m - 1] if m else [])


def test_only_empty_requests(cuda_lib):
    c = step.Case(3, ctx=[0] * 200, n=[0] * 200, Hq=2, Hkv=1, D=64, page=16)
    assert np.all(c.call() == 7.0)
    c = prompt.Case(3, [0] * 200, Hq=2, Hkv=1, D=64)
    assert np.all(c.call() == 7.0)


ROWS, HEADS = (1 << 31) // (128 * 128) + 40, 128  # 2^31 elements and some rows more


def far_rows(rows, heads, seed):
    """[rows, heads, 128] of which only the last 200 rows hold anything."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.zeros((rows, heads, 128), dtype=torch.bfloat16, device="cuda")
    t[-200:] = torch.randn((200, heads, 128), generator=gen, device="cuda").to(torch.bfloat16)
    return t


def test_prompt_rows_past_two_to_the_31_elements(cuda_lib):
    n = [70, 90]
    r0 = ROWS - sum(n) - 3
    h = binding.AttnBuffers(B=2, rows=ROWS, q_max=90, Hq=HEADS, Hkv=HEADS, D=128, prompt=True)
    q, k, v = (far_rows(ROWS, HEADS, s) for s in (1, 2, 3))
    h.bind(q_rot=q, k_rot=k, v=v, row_off=dev(offsets(n) + np.int32(r0)))
    binding.dspark_prompt_attention(h.attn)
    torch.cuda.synchronize()
    assert h.device_status() == 0
    assert int(h.out[:r0].count_nonzero()) == 0 and int(h.out[r0 + sum(n):].count_nonzero()) == 0
    at = r0
    for m in n:
        for heads in (slice(0, 2), slice(HEADS - 2, HEADS)):
            qw, kw, vw = (wide(t[at: at + m, heads].contiguous()) for t in (q, k, v))
            o, spread, ds = oa.attend(qw, kw, vw, 0, 128 ** -0.5)
            assert_close(wide(h.out[at: at + m, heads].contiguous()), o, spread, ds, m)
        at += m


def test_step_and_append_rows_past_two_to_the_31_elements(cuda_lib):
    """The rows' queries, rotated queries and outputs; keys and values come along from the same
    rows."""
    n, ctx, page, Hkv = [5, 9], [0, 0], 16, 2
    r0 = ROWS - sum(n) - 3
    rows = np.full(ROWS, -1, np.int32)
    pos = np.zeros(ROWS, np.int32)
    rows[r0: r0 + 14], pos[r0: r0 + 14] = [0] * 5 + [1] * 9, list(range(5)) + list(range(9))
    q, k, v = far_rows(ROWS, HEADS, 4), far_rows(ROWS, Hkv, 5), far_rows(ROWS, Hkv, 6)
    kc, vc = (torch.zeros((2, page, Hkv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    h = binding.AttnBuffers(B=2, rows=ROWS, q_max=9, Hq=HEADS, Hkv=Hkv, D=128, page_size=page, num_pages=2,
                            max_pages=1, rot_dim=0)
    h.bind(q=q, k=k, v=v, k_cache=kc, v_cache=vc, row_off=dev(offsets(n) + np.int32(r0)), row_req=dev(rows),
           packed_pos=dev(pos), seq_lens=dev(np.array(ctx, np.int32)), block_table=dev(np.array([[1], [0]], np.int32)))
    binding.dspark_rope_append(h.attn)
    binding.dspark_step_attention(h.attn)
    torch.cuda.synchronize()
    assert h.device_status() == 0
    assert torch.equal(h.q_rot[r0: r0 + 14], q[r0: r0 + 14]) and int(h.q_rot[:r0].count_nonzero()) == 0
    assert int(h.out[:r0].count_nonzero()) == 0 and int(h.out[r0 + 14:].count_nonzero()) == 0
    at = r0
    for m in n:
        qw, kw, vw = (wide(t[at: at + m]) for t in (q, k, v))
        o, spread, ds = oa.attend(qw, kw, vw, 0, 128 ** -0.5)
        assert_close(wide(h.out[at: at + m]), o, spread, ds, m)
        at += m


@pytest.mark.parametrize("D", [64, 128])
def test_the_widest_groups(cuda_lib, D):
    step.Case(7, ctx=[200], n=[65], Hq=128, Hkv=1, D=D, page=16).check()
    prompt.Case(7, [150, 33], Hq=256, Hkv=1, D=D).check(pick=lambda m: [0, m // 2, m - 1])
    prompt.Case(7, [150, 33], Hq=256, Hkv=256, D=D).check(pick=lambda m: [0, m // 2, m - 1])


@pytest.mark.parametrize("page", [24, 40, 1000, 65536])
def test_pages_of_other_sizes(cuda_lib, page):
    step.Case(8, ctx=[2500, 39], n=[5, 2], Hq=8, Hkv=2, D=128, page=page, spare=1).check()


@pytest.mark.parametrize("n", [1, 17])
def test_one_cached_head_over_all_ctas(cuda_lib, n):
    """Parts of one unit on more than 100 CTAs."""
    step.Case(9, ctx=[30000], n=[n], Hq=8, Hkv=1, D=128, page=64).check()

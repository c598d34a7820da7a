"""dspark_rope_append against the fp64 oracle.

A rotated element is x cos - y sin in fp32, rounded once to bfloat16: the
sine and cosine are off by at most 2^-23 (the angle's 2^-25 of a half turn, and two
ulp of the function), the two products and their sum by 2^-23 more, so
|got - want| <= 2^-8 |want| + 2^-21 (|x| + |y|).  Copies (values, unrotated
entries) are exact, and so is everything that must stay untouched.
"""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa
from tests.attn_harness import bits, dev, make_cache, make_table, packed, wide

pytestmark = pytest.mark.gpu


def run_case(seed, ctx, n, rows, Hq, Hkv, D, page, rot, theta, interleaved, heads_first, k_rot,
             bad_pages=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(n)
    row_off, row_req, pos = packed(ctx, n, rows)
    need = [-(-(c + m) // page) for c, m in zip(ctx, n)]
    max_pages = max(max(need), 1)
    num_pages = sum(need) + 2
    table = make_table(need, num_pages, max_pages, rng)
    if bad_pages:  # one request's pages are no memory
        table[0, :] = np.where(np.arange(max_pages) % 2 == 0, -1, num_pages)
    qkv = torch.randn((rows, (Hq + 2 * Hkv) * D), generator=gen, device="cuda").to(torch.bfloat16)
    q = qkv[:, : Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D: (Hq + Hkv) * D].unflatten(1, (Hkv, D))
    v = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    kc = make_cache(num_pages, page, Hkv, D, heads_first, gen)
    vc = make_cache(num_pages, page, Hkv, D, heads_first, gen)
    kc0, vc0 = wide(kc), wide(vc)
    h = binding.AttnBuffers(B=B, rows=rows, q_max=max(max(n), 1), Hq=Hq, Hkv=Hkv, D=D,
                            page_size=page, num_pages=num_pages, max_pages=max_pages, rot_dim=rot,
                            interleaved=interleaved, k_rot=k_rot)
    h.q_rot.fill_(7.0)
    if k_rot:
        h.k_rot.fill_(7.0)
    h.bind(q=q, k=k, v=v, k_cache=kc, v_cache=vc, row_off=dev(row_off), row_req=dev(row_req),
           packed_pos=dev(pos), block_table=dev(table),
           rope_freq=binding.rope_freq(rot, theta) if rot else None)
    binding.dspark_rope_append(h.attn)
    torch.cuda.synchronize()

    inv = theta ** (-2.0 * np.arange(rot // 2) / rot) if rot else np.zeros(0)
    used = row_req >= 0
    want = {}
    for name, x, got in (("q", q, h.q_rot), ("k", k, h.k_rot)):
        xw = wide(x)
        y = oa.rope(xw, pos, inv, interleaved)
        y0 = oa.rope(np.abs(xw), np.zeros(rows), inv, interleaved)
        pair = np.array(y0)  # |x| + |y| of each rotated pair
        half = rot // 2
        i0, i1 = ((slice(0, rot, 2), slice(1, rot, 2)) if interleaved
                  else (slice(0, half), slice(half, rot)))
        pair[..., i0] = pair[..., i1] = y0[..., i0] + y0[..., i1]
        pair[..., rot:] = 0
        tol = np.where(np.arange(D) < rot, 2.0 ** -8 * np.abs(y) + 2.0 ** -21 * pair, 0.0)
        want[name] = (y, tol)
        if got is not None:
            g = wide(got)
            assert np.all(np.abs(g - y)[used] <= tol[used]), name
            assert np.all(g[~used] == 7.0)
    vw = wide(v)
    for name, got, before, rows_, tol in (("k", kc, kc0, *want["k"]),
                                          ("v", vc, vc0, vw, np.zeros_like(vw))):
        c, t = np.array(before), np.zeros_like(before)
        oa.append(c, rows_, row_req, pos, table)
        oa.append(t, tol, row_req, pos, table)
        assert np.all(np.abs(wide(got) - c) <= t), name
    return h


@pytest.mark.parametrize("case", [
    # one row; one head; full rotation
    dict(ctx=[0], n=[1], rows=1, Hq=1, Hkv=1, D=64, page=16, rot=64),
    # a step's rows with padding, an empty request, ragged lengths, token-level pages
    dict(ctx=[5, 0, 130, 77], n=[3, 1, 0, 9], rows=40, Hq=8, Hkv=2, D=128, page=1, rot=128),
    # odd pages, head counts that are no power of two, partial rotation
    dict(ctx=[1000, 3], n=[17, 16], rows=34, Hq=15, Hkv=3, D=128, page=7, rot=32),
    dict(ctx=[31, 32, 33], n=[2, 2, 2], rows=7, Hq=40, Hkv=8, D=64, page=32, rot=48),
    # more head slots than a thread keeps in flight
    dict(ctx=[9, 64], n=[4, 5], rows=9, Hq=128, Hkv=64, D=128, page=64, rot=128),
    # no rotation: a plain append
    dict(ctx=[12, 1], n=[5, 6], rows=12, Hq=4, Hkv=4, D=128, page=16, rot=0),
    # a prompt over several pages
    dict(ctx=[0, 0], n=[300, 77], rows=380, Hq=6, Hkv=2, D=128, page=48, rot=128),
])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads_first", [False, True])
def test_against_the_oracle(cuda_lib, case, interleaved, heads_first):
    run_case(1, theta=1.0e4, interleaved=interleaved, heads_first=heads_first,
             k_rot=heads_first, **case)


def test_far_positions_keep_their_angle(cuda_lib):
    """Positions near 2^20 with a slow and a fast frequency."""
    run_case(2, ctx=[(1 << 20) - 9, 1 << 19], n=[8, 3], rows=11, Hq=2, Hkv=1, D=128, page=128,
             rot=128, theta=5.0e6, interleaved=False, heads_first=False, k_rot=True)


def test_bad_pages_store_nothing(cuda_lib):
    run_case(3, ctx=[40, 7], n=[6, 4], rows=10, Hq=4, Hkv=2, D=128, page=16, rot=128, theta=1e4,
             interleaved=False, heads_first=False, k_rot=True, bad_pages=True)


def test_queries_in_place_and_keys_alone(cuda_lib):
    """q_rot may be q; q = NULL handles the keys only and k = v = NULL the queries only, with the
    bits of the joint call."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows, Hq, Hkv, D, page = 5, 4, 2, 128, 16
    q = torch.randn((rows, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    k = torch.randn((rows, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.randn((rows, Hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
    row_off, row_req, pos = packed([30], [5], rows)
    table = dev(np.array([[2, 0, 1]], np.int32))
    freq = binding.rope_freq(D, 1e4)

    def make(**kw):
        h = binding.AttnBuffers(B=1, rows=rows, q_max=5, Hq=Hq, Hkv=Hkv, D=D, page_size=page,
                                num_pages=3, max_pages=3, rot_dim=D)
        kc = make_cache(3, page, Hkv, D, False, gen, 0.0)
        vc = make_cache(3, page, Hkv, D, False, gen, 0.0)
        h.bind(row_req=dev(row_req), packed_pos=dev(pos), block_table=table, rope_freq=freq,
               k_cache=kc, v_cache=vc, **kw)
        binding.dspark_rope_append(h.attn)
        torch.cuda.synchronize()
        return bits(h.q_rot), bits(kc), bits(vc)

    both = make(q=q, k=k, v=v)
    only_k = make(k=k, v=v)
    only_q = make(q=q)
    inplace = q.clone()
    same = make(q=inplace, q_rot=inplace, k=k, v=v)
    assert np.array_equal(only_k[1], both[1]) and np.array_equal(only_k[2], both[2])
    assert not only_k[0].any() and not only_q[1].any() and not only_q[2].any()
    assert np.array_equal(only_q[0], both[0])
    for a, b in zip(same, both):
        assert np.array_equal(a, b)


def test_a_cache_past_two_to_the_31_elements(cuda_lib):
    """The last page of a cache of 2^31 + 2^20 elements takes its rows."""
    Hkv, D, page = 8, 128, 64
    num_pages = ((1 << 31) + (1 << 20)) // (Hkv * D * page)
    kc = torch.zeros((num_pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.randn((2, Hkv, D), device="cuda").to(torch.bfloat16)
    v = torch.randn((2, Hkv, D), device="cuda").to(torch.bfloat16)
    row_off, row_req, pos = packed([page - 2], [2], 2)
    h = binding.AttnBuffers(B=1, rows=2, q_max=2, Hq=8, Hkv=Hkv, D=D, page_size=page,
                            num_pages=num_pages, max_pages=1, rot_dim=0)
    h.bind(k=k, v=v, k_cache=kc, v_cache=vc, row_req=dev(row_req), packed_pos=dev(pos),
           block_table=dev(np.array([[num_pages - 1]], np.int32)))
    binding.dspark_rope_append(h.attn)
    torch.cuda.synchronize()
    assert torch.equal(kc[-1, -2:], k) and torch.equal(vc[-1, -2:], v)
    assert int(kc[:-1].count_nonzero()) == 0 and int(vc[:-1].count_nonzero()) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows", [2127, 2129, 4400, 8512, 8514])
def test_long_lists_of_row_slots(cuda_lib, rows, interleaved, D):
    """Lists that CTAs walk and lists with a CTA for each slot, a few rows in front of padding or
    every slot in use (the last one too)."""
    n = [(5 * i) % 8 for i in range(250)]
    if rows != 4400:
        n.append(rows - sum(n))
    run_case(6, ctx=[(11 * i) % 90 for i in range(len(n))], n=n, rows=rows, Hq=2, Hkv=1, D=D, page=16,
             rot=D, theta=1.0e4, interleaved=interleaved, heads_first=False, k_rot=True)

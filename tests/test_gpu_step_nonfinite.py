"""dspark_step_attention: values that are not finite at keys which some rows of a block see and
others do not.  They must reach the rows that see them and no others, in every unit that a CTA
walks, in units cut over several CTAs, in gathered and boxed pages and for both head sizes.

The result is compared with the same call on finite values: a replaced value changes the entries
of the rows that see it, and no bit elsewhere (its weight in the other rows is 0 either way)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_step_attention import Case

pytestmark = pytest.mark.gpu


def poison(c, picks, values):
    """Puts values[i] at (request, position, cached head, entry) = picks[i] of the values."""
    b, p, h, d = (np.array(x) for x in zip(*picks))
    page = torch.as_tensor(c.table[b, p // c.page].astype(np.int64)).cuda()
    at = [torch.as_tensor(x.astype(np.int64)).cuda() for x in (p % c.page, h, d)]
    c.vc[page, at[0], at[1], at[2]] = torch.as_tensor(values, dtype=torch.float32).cuda().to(torch.bfloat16)


def expect(c, clean, picks, values):
    """``clean`` with what the poisoned values make of it."""
    want = clean.copy()
    G = c.Hq // c.Hkv
    with np.errstate(invalid="ignore"):
        for (b, p, h, d), x in zip(picks, values):
            r0 = c.row_off[b]
            pos = c.ctx[b] + np.arange(c.n[b])
            rows = r0 + np.nonzero((p <= pos) & ((c.window == 0) | (p > pos - c.window)))[0]
            want[rows, h * G: (h + 1) * G, d] += x
    return want


def check(c, per_request, seed):
    """One pass on finite values, one with ``per_request`` keys of each request spoilt."""
    rng = np.random.default_rng(seed)
    clean = c.call()
    picks, values = [], []
    for b in range(c.B):
        if c.n[b] < 2:
            continue
        for _ in range(per_request):
            # a draft's own key, or the far edge of the window
            j = int(rng.integers(1, c.n[b]))
            p = c.ctx[b] + j
            if c.window and p - c.window >= 0 and rng.random() < 0.5:
                p -= c.window
            picks.append((b, p, int(rng.integers(c.Hkv)), int(rng.integers(c.D))))
            values.append(float(rng.choice([np.nan, np.inf, -np.inf])))
    poison(c, picks, values)
    want = expect(c, clean, picks, values)
    got = c.call()
    assert np.isnan(want).any() and np.isinf(want).any()
    assert np.array_equal(got, want, equal_nan=True), np.argwhere(~((got == want) | (np.isnan(got) & np.isnan(want))))[:5]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [0, 90])
def test_many_units_a_cta(cuda_lib, D, page, window):
    """1600 units of one to three tiles: ten or so on every CTA, half of them with spoilt values."""
    rng = np.random.default_rng(1)
    ctx = [int(x) for x in rng.integers(0, 300, 400)]
    n = [int(x) for x in rng.integers(0, 10, 400)]
    c = Case(1, ctx=ctx, n=n, Hq=8, Hkv=4, D=D, page=page, window=window)
    for turn in range(3):
        check(c, per_request=1, seed=turn)
        c = Case(2 + turn, ctx=ctx, n=n, Hq=8, Hkv=4, D=D, page=page, window=window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("window", [0, 700, 3000])
def test_cut_units(cuda_lib, D, page, window):
    """A few long requests: every unit is cut over many CTAs and joined."""
    check(Case(5, ctx=[5000, 2100, 3333], n=[9, 17, 2], Hq=8, Hkv=2, D=D, page=page, window=window),
          per_request=3, seed=6)


@pytest.mark.parametrize("D", [64, 128])
def test_blocks_of_rows(cuda_lib, D):
    """65 rows of 8 heads: several blocks, and keys that whole blocks see in full or not at all."""
    check(Case(7, ctx=[100, 900], n=[65, 40], Hq=8, Hkv=1, D=D, page=16), per_request=12, seed=8)

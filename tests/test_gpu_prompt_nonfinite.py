"""dspark_prompt_attention: values that are not finite.  They must reach the rows that see them and
no others, wherever the key lies between the two blocks of a unit, for windows that cut one block's
tile, the other's or both, and in every unit that a CTA walks.

The result is compared with the same call on finite values: a replaced value changes the entries
of the rows that see it, and no bit elsewhere (its weight in the other rows is 0 either way)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu


def check(c, picks, values):
    """picks: (prompt, row of it, cached head, entry)."""
    clean = c.call()
    want = clean.copy()
    G = c.q.shape[1] // c.k.shape[1]
    with np.errstate(invalid="ignore"):
        for (b, p, h, d), x in zip(picks, values):
            r0 = c.row_off[b]
            end = min(c.n[b], p + c.window) if c.window else c.n[b]
            want[r0 + p: r0 + end, h * G: (h + 1) * G, d] += x
    at = [torch.tensor(x).cuda() for x in zip(*[(int(c.row_off[b]) + p, h, d) for b, p, h, d in picks])]
    c.v[at[0], at[1], at[2]] = torch.tensor(values).cuda().to(torch.bfloat16)
    got = c.call()
    assert np.isnan(want).any() and np.isinf(want).any()
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert same.all(), np.argwhere(~same)[:5].tolist()


def spoil(rng, n, Hkv, D, count):
    """``count`` keys of each prompt longer than a row, at different entries."""
    picks, values = [], []
    for b, m in enumerate(n):
        if m < 2:
            continue
        entries = rng.permutation(Hkv * D)[:count]
        for e in entries:
            picks.append((b, int(rng.integers(m)), int(e) // D, int(e) % D))
            values.append(float(rng.choice([np.nan, np.inf, -np.inf])))
    return picks, values


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 2, 60, 100, 127, 128, 129, 200, 255, 256, 300, 500])
def test_keys_all_over_a_unit(cuda_lib, D, window):
    """Every eighth key of prompts of several units, each in an entry of its own."""
    n = [700, 300, 512]
    picks, values = [], []
    rng = np.random.default_rng(window)
    for b, m in enumerate(n):
        for i, p in enumerate(range(b, m, 8)):
            picks.append((b, p, i // D, i % D))
            values.append(float(rng.choice([np.nan, np.inf, -np.inf])))
    check(Case(1, n, Hq=4, Hkv=2, D=D, window=window), picks, values)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 2, 130, 200, 400])
def test_many_units_a_cta(cuda_lib, D, window):
    """More than 2000 units: a dozen on every CTA, and marks of older units all around."""
    rng = np.random.default_rng(2)
    n = [int(x) for x in rng.integers(1, 700, 64)]
    c = Case(2, n, Hq=16, Hkv=4, D=D, window=window)
    check(c, *spoil(rng, n, 4, D, count=3))

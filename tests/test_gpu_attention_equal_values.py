"""Values that are the same at all keys come out as they are: o is the value times the sum of the
rounded weights, and l is that sum too.  What is left is the fp32 sums' rounding, at most n 2^-23 of
the value for n keys, below the half step of 2^-9 that would change the rounded output."""
import numpy as np
import pytest

from tests import test_gpu_prompt_attention as prompt
from tests import test_gpu_step_attention as step
from tests.attn_harness import wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 50, 200])
def test_prompt(cuda_lib, D, window):
    n = [700, 1, 40, 129]
    c = prompt.Case(1, n, Hq=10, Hkv=2, D=D, window=window, q_std=3.0)
    c.v.copy_(c.v[7].clone().expand_as(c.v))
    got = c.call()[: sum(n)]
    assert np.array_equal(got, np.broadcast_to(np.repeat(wide(c.v)[7], 5, axis=0), got.shape))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("window", [0, 1, 200])
def test_step(cuda_lib, D, page, window):
    n = [5, 9, 2, 1]
    c = step.Case(2, ctx=[0, 1300, 127, 40], n=n, Hq=10, Hkv=2, D=D, page=page, window=window, q_std=3.0)
    c.vc.copy_(c.vc[0, 0].clone().expand_as(c.vc))
    got = c.call()[: sum(n)]
    assert np.array_equal(got, np.broadcast_to(np.repeat(wide(c.vc)[0, 0], 5, axis=0), got.shape))

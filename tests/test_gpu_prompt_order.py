"""dspark_prompt_attention on many short prompts with a window, over and over: units without a second
block stand between units with one, so that the two blocks' warps are in different units of a CTA.
Every pass gives the first one's bits, and those are the oracle's within its bounds; the values'
tiles are scanned while others are still on their way."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.test_gpu_prompt_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 100, 129, 250])
@pytest.mark.parametrize("longest", [200, 300])
def test_short_prompts_with_a_window(cuda_lib, window, D, longest):
    rng = np.random.default_rng(window)
    n = [int(x) for x in np.where(rng.random(40) < 0.3, 0, rng.integers(1, longest + 1, 40))]
    c = Case(1, n, Hq=12, Hkv=3, D=D, window=window)
    first = c.check(pick=lambda m: sorted({0, m // 2, m - 1} | ({127, 128} if m > 129 else set())) if m else [])
    outs = []
    for _ in range(300):
        out = torch.full_like(c.h.out, 7.0)
        c.h.attn.out = out.data_ptr()
        binding.dspark_prompt_attention(c.h.attn)
        outs.append(out)
    torch.cuda.synchronize()
    assert c.h.device_status() == 0
    want = torch.as_tensor(first).cuda()
    assert all(torch.equal(out.double(), want) for out in outs)

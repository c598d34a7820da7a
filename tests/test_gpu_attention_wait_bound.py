"""A bounded device wait of the attention calls that runs out.

The first wait of every CTA gives up after the bound that dspark_set_wait_timeout_ns sets, however
short it is.  Here that is 100 ns, less than any copy takes: the launch must still return, report
the status, and after dspark_workspace_init and the default bound restored, the next call must give
what the call before gave.
"""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests import test_gpu_prompt_attention as prompt
from tests import test_gpu_step_attention as step
from tests.attn_harness import wide

pytestmark = pytest.mark.gpu

STATUS_WAIT = 1


def check(c, call):
    want = c.call()
    default = binding.dspark_wait_timeout_ns()
    assert default == 2_000_000_000
    try:
        binding.dspark_set_wait_timeout_ns(100)
        call(c.h.attn)
        torch.cuda.synchronize()  # the launch returned
        status = c.h.device_status()
    finally:
        binding.dspark_set_wait_timeout_ns(0)  # 0 restores the default
    assert status == STATUS_WAIT
    binding.dspark_workspace_init(c.h.workspace.data_ptr(), c.h.ws_bytes)
    assert c.h.device_status() == 0
    assert np.array_equal(c.call(), want)


@pytest.mark.parametrize("page", [16, 1])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", [
    dict(ctx=[700], n=[3], Hq=8, Hkv=2),                                # a tile a CTA
    dict(ctx=[20000, 9000, 4], n=[9, 17, 2], Hq=8, Hkv=2),              # cut units of many tiles
    dict(ctx=[11 * i % 500 for i in range(300)], n=[1 + i % 9 for i in range(300)], Hq=8, Hkv=4),
])
def test_step(cuda_lib, shape, D, page):
    check(step.Case(1, D=D, page=page, **shape), binding.dspark_step_attention)


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [[50], [3000], [31 * i % 600 for i in range(40)]])
def test_prompt(cuda_lib, n, D, window):
    check(prompt.Case(2, n, Hq=8, Hkv=2, D=D, window=window), binding.dspark_prompt_attention)

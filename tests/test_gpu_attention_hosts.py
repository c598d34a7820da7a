"""The attention calls from host threads that have not used CUDA before."""
import threading

import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.attn_harness import wide
from tests import test_gpu_prompt_attention as prompt
from tests.test_gpu_step_attention import Case

pytestmark = pytest.mark.gpu


def in_a_thread(work):
    """Runs ``work`` in a host thread of its own; an exception in it is raised here."""
    errors = []

    def body():
        try:
            work()
        except Exception as e:  # noqa: BLE001 (raised below)
            errors.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    if errors:
        raise errors[0]


def test_the_first_cuda_call_of_a_thread(cuda_lib):
    """No context is current in a new thread before its first runtime call."""
    stream = torch.cuda.Stream()
    for c, call in ((Case(3, ctx=[90, 700], n=[3, 1], Hq=8, Hkv=2, D=128, page=16), binding.dspark_step_attention),
                    (Case(3, ctx=[90, 700], n=[3, 1], Hq=8, Hkv=2, D=64, page=1), binding.dspark_step_attention),
                    (prompt.Case(3, [70, 300], Hq=4, Hkv=2, D=128), binding.dspark_prompt_attention)):
        want = c.call()
        c.h.out.fill_(7.0)
        torch.cuda.synchronize()
        in_a_thread(lambda: call(c.h.attn, stream.cuda_stream))
        torch.cuda.synchronize()
        assert np.array_equal(wide(c.h.out), want)

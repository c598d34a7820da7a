"""The attention calls from host threads that have not used CUDA before, and dspark_step_attention
in different shapes side by side: shapes that ask for different amounts of shared memory, from
several host threads and within one captured graph."""
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


def two_shapes():
    """80 and 128 columns of 128 entries: more and fewer bytes of shared memory."""
    return (Case(1, ctx=[300, 40], n=[10, 3], Hq=8, Hkv=1, D=128, page=16),
            Case(2, ctx=[500, 90], n=[16, 9], Hq=8, Hkv=1, D=128, page=16))


def test_two_threads_with_shapes_of_their_own(cuda_lib):
    cases = two_shapes()
    want = [c.call() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.h.out.fill_(7.0)
    torch.cuda.synchronize()
    errors, ready = [], threading.Barrier(len(cases))

    def work(c, stream):
        try:
            ready.wait()
            for _ in range(3000):
                binding.dspark_step_attention(c.h.attn, stream.cuda_stream)
        except Exception as e:  # noqa: BLE001 (shown below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c, w in zip(cases, want):
        assert c.h.device_status() == 0
        assert np.array_equal(wide(c.h.out), w)


@pytest.mark.parametrize("order", [(0, 1), (1, 0), (0, 1, 0)])
def test_two_shapes_in_one_graph(cuda_lib, order):
    cases = two_shapes()
    want = [c.call() for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for i in order:
            binding.dspark_step_attention(cases[i].h.attn, side.cuda_stream)
    for _ in range(2):
        for c in cases:
            c.h.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert np.array_equal(wide(c.h.out), w)

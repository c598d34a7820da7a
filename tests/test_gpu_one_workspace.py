"""One workspace of the largest batch serves the smaller ones: sized as a program sizes it, once."""
import numpy as np
import pytest
import torch

from confidence_driven_speculative_gb300 import binding
from tests.test_gpu_attention_sinks import Prompt, Step
from tests.test_gpu_step_attention_tree import Tree
from tests import test_gpu_verify_tree as verify

pytestmark = pytest.mark.gpu


def workspace(size):
    ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
    ws[size:] = 0xa5  # nothing is written behind it
    binding.dspark_workspace_init(ws.data_ptr(), size)
    return ws


def test_attention_calls_on_a_workspace_of_65_rows(cuda_lib):
    heads = dict(Hq=32, Hkv=8, D=128)
    size = binding.dspark_attn_workspace_size(32, 8, 128, 65)
    ws = workspace(size)
    long = dict(ctx=[3000, 40, 700, 1], page=16, **heads)
    cases = [Step(1, 4, n=[64, 3, 33, 9], window=900, **long), Tree(2, n=[64, 1, 33, 17], **long),
             Step(3, 4, n=[40, 3, 2, 9], window=900, **long), Tree(4, n=[9, 1, 2, 3], **long),
             Prompt(5, 4, [300, 31], window=100, **heads)]
    want = [c.call() for c in cases]
    for c in cases:
        c.h.attn.workspace, c.h.attn.workspace_bytes = ws.data_ptr(), size
    for _ in range(2):
        for c, w in zip(cases, want):
            assert np.array_equal(c.call(), w)
    assert binding.dspark_read_device_status(ws.data_ptr()) == 0
    assert (ws[size:] == 0xa5).all()


@pytest.mark.parametrize("largest", [(1024, 4096, 1024), (1025, 70000, 1024), (64, 4096, 129280)])
def test_tree_verifies_on_a_workspace_of_the_largest_batch(cuda_lib, largest):
    """Few rows read at once and many walked, in turn: keys and counters are back at zero after each."""
    size = binding.dspark_tree_workspace_size(*largest)
    ws = workspace(size)
    cases = [verify.Case(30 + i, n, V, dtype) for i, (n, V, dtype) in enumerate((
        ([30], 4096, torch.bfloat16), ([3, 5, 0, 64, 9], 1024, torch.float32), ([1] * 1020, 64, torch.bfloat16),
        ([20] * 60, 1024, torch.bfloat16), ([2] * 600, 64, torch.float32), ([64, 1], 512, torch.bfloat16),
        ([1] * 1200, 64, torch.bfloat16)))]
    handles = [c.handle() for c in cases]
    for _ in range(2):
        for c, h in zip(cases, handles):
            h.tree.workspace, h.tree.workspace_bytes = ws.data_ptr(), size
            c.commit = h._keep["seq_lens_commit"]
            c.check(h)
    assert (ws[size:] == 0xa5).all() and (ws[:size] == 0).all()


def test_short_prompts_on_a_workspace_of_long_ones(cuda_lib):
    size = binding.dspark_attn_workspace_size(8, 2, 128, 8192)
    ws = workspace(size)
    for n in ([30, 5, 17], [64], [65, 1], [66, 300]):
        c = Prompt(6, 4, n, Hq=8, Hkv=2, D=128, window=20)
        want = c.call()
        c.h.attn.workspace, c.h.attn.workspace_bytes = ws.data_ptr(), size
        for _ in range(2):
            assert np.array_equal(c.call(), want)
    assert (ws[size:] == 0xa5).all()

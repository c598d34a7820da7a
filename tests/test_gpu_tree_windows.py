"""Trees deeper than a layer's window is long: a chain given as a tree is the chain (bounds: attn_harness.py)."""
import numpy as np
import pytest

from confidence_driven_speculative_gb300 import binding
from tests.attn_harness import dev
from tests.test_gpu_attention_sinks import Step
from tests.test_gpu_step_attention_tree import Tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (16, 0), (16, 4), (2, 70), (63, 1)])
@pytest.mark.parametrize("page", [1, 16])
def test_a_chain_in_a_window_shorter_than_it(cuda_lib, window, sinks, page):
    kw = dict(ctx=[300, 0, 40, 65, 1], n=[64, 64, 30, 9, 1], Hq=8, Hkv=2, D=128, page=page, window=window)
    a, t = Step(4, sinks, **kw), Tree(4, sinks=sinks, deep=1.0, **kw)
    assert (a.q == t.q).all() and (a.kc == t.kc).all()
    t.words, pos, _ = binding.tree_rows(t.parent, dev(t.row_off), dev(np.array(kw["ctx"], np.int32)), window, sinks)
    assert (pos == t.tree_pos).all()
    got = t.call()
    a.check(got=got)   # the chain's rows, by the step's visibility
    t.check(got=got)   # and the tree's, by the bits

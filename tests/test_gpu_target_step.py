"""The attention calls together with the verify step (examples/target_step.py): prompts in, then
speculative steps over the paged cache."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import attention as oa
from tests.attn_harness import assert_close, wide

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "target_step.py")


def load_example():
    spec = importlib.util.spec_from_file_location("target_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def check_last_step(r):
    """The last step's attention output against the oracle on the cache as it lies."""
    q, out = wide(r["q_rot"]), wide(r["out"])
    kc, vc = wide(r["cache"][0]), wide(r["cache"][1])
    table, off, start = (r[k].cpu().numpy() for k in ("table", "row_off", "start"))
    for b in range(len(start)):
        r0, r1 = off[b], off[b + 1]
        m = int(start[b]) + r1 - r0
        k, _ = oa.gather(kc, table[b], m)
        v, _ = oa.gather(vc, table[b], m)
        o, spread, ds = oa.attend(q[r0:r1], k, v, int(start[b]), r["scale"])
        assert_close(out[r0:r1], o, spread, ds, m, b)


@pytest.mark.parametrize("page", [1, 16])
def test_prompts_then_steps(cuda_lib, page):
    r = load_example().run(page=page, seed=page)
    check_last_step(r)
    lengths = np.stack([x.cpu().numpy() for x in r["lengths"]])
    grown = np.diff(lengths, axis=0)
    assert np.all(grown >= 1) and np.all(grown <= 9)
    assert np.array_equal(grown[-1], r["emitted"].cpu().numpy())

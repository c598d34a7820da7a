"""dspark_commit_path of many requests and layers, two layers to a CTA, against the oracle."""
import numpy as np
import pytest

from tests.attn_harness import make_table
from tests.test_gpu_commit_path import check, make, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,layers", [(300, 8), (900, 3), (520, 5), (2600, 1), (1300, 2)])
@pytest.mark.parametrize("page,Hkv,D", [(4, 2, 8), (16, 1, 64)])
def test_many_requests_and_layers(cuda_lib, B, layers, page, Hkv, D):
    """An odd number of layers leaves the last CTAs of two with one."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 9, B)
    paths = []
    for _ in range(B):
        n = int(rng.integers(0, 12))
        paths.append(sorted(rng.choice(12, n, replace=False).tolist()))
    need = [-(-(int(s) + 12) // page) for s in lens]
    table = make_table(need, sum(need), max(need), rng)
    k, v = make(1, layers, sum(need), page, Hkv, D, heads_first=layers % 2 == 1)
    check(k, v, table, lens, rows_of(paths, 12))

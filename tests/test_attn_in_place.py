"""CPU checks: dspark_rope_append refuses to rotate rows in place that are not contiguous.  (That it takes
contiguous ones is a GPU test's: the call would go on to the launch.)"""
import pytest

from confidence_driven_speculative_gb300 import binding
from tests.test_attn_abi import FAKE, lib, status, valid  # noqa: F401 (lib is a fixture)


@pytest.mark.parametrize("which,heads", [("q", 8), ("k", 2)])
def test_in_place_wants_contiguous_rows(lib, which, heads):  # noqa: F811
    other = "k" if which == "q" else "q"
    for stride in (12 * 128, heads * 128 + 8):
        a = valid(**{which: FAKE << 4, which + "_rot": FAKE << 4, which + "_stride": stride,
                     other + "_rot": FAKE << 5})
        assert status(lib, "dspark_rope_append", a) == binding.DSPARK_EINVAL
        assert f"{which}_rot is {which}" in binding.last_error()

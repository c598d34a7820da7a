"""Pins of the attention oracle (CPU), and the frequencies of the binding."""
import math

import numpy as np
import pytest

from confidence_driven_speculative_gb300 import binding
from oracle import attention as oa


def test_rope_is_a_rotation_and_depends_on_the_distance_only():
    rng = np.random.default_rng(0)
    inv = 10000.0 ** (-np.arange(8) / 8.0)
    for inter in (False, True):
        q, k = rng.normal(size=(2, 1, 1, 20))
        dot = lambda i, j: float((oa.rope(q, [i], inv, inter) * oa.rope(k, [j], inv, inter)).sum())
        assert dot(7, 3) == pytest.approx(dot(104, 100), abs=1e-12)
        assert dot(5, 5) == pytest.approx(float((q * k).sum()), abs=1e-12)
        y = oa.rope(q, [9], inv, inter)
        assert np.linalg.norm(y) == pytest.approx(np.linalg.norm(q))
        assert np.array_equal(y[..., 16:], q[..., 16:])  # past the rotated part


def test_rope_by_hand():
    x = np.array([[[1.0, 0.0, 0.0, 2.0]]])
    y = oa.rope(x, [1], [math.pi / 2, 0.0], False)       # pairs (0, 2), (1, 3)
    np.testing.assert_allclose(y[0, 0], [0.0, 0.0, 1.0, 2.0], atol=1e-15)
    y = oa.rope(x, [1], [math.pi / 2, math.pi], True)    # pairs (0, 1), (2, 3)
    np.testing.assert_allclose(y[0, 0], [0.0, 1.0, 0.0, -2.0], atol=1e-15)


def test_attend_by_hand():
    k = np.zeros((3, 1, 2))
    k[:, 0, 0] = [0.0, math.log(2.0), math.log(4.0)]
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[-1.0, 3.0]]])
    q = np.tile(np.array([1.0, 0.0]), (3, 2, 1))
    o, spread, ds = oa.attend(q, k, v, 0, 1.0)
    np.testing.assert_allclose(o[0, 0], [1, 0])
    np.testing.assert_allclose(o[1, 1], [1 / 3, 2 / 3])
    np.testing.assert_allclose(o[2, 0], [(1 - 4) / 7, (2 + 12) / 7])
    np.testing.assert_allclose(spread[2, 0], [5 / 7, 2])
    assert ds[2, 0] == pytest.approx(math.log(4.0))
    o, _, _ = oa.attend(q, k, v, 0, 1.0, window=1)       # a row sees itself only
    np.testing.assert_allclose(o[:, 0], v[:, 0])
    o, _, _ = oa.attend(q, k, v, 0, 1.0, valid=np.array([False, True, True]))
    assert np.all(o[0] == 0) and np.allclose(o[1, 0], v[1, 0])


def test_append_and_gather_are_inverse():
    rng = np.random.default_rng(1)
    cache = np.zeros((5, 3, 2, 4))
    table = np.array([[4, 0, -1], [2, 9, 1]], np.int32)
    rows = rng.normal(size=(7, 2, 4))
    req = np.array([0, 0, 0, 1, 1, -1, 1])
    pos = np.array([0, 5, 6, 2, 4, 0, 8])
    oa.append(cache, rows, req, pos, table)
    got, valid = oa.gather(cache, table[0], 10)
    assert valid.tolist() == [True] * 6 + [False] * 4    # page -1, then past the table
    assert np.array_equal(got[0], rows[0]) and np.array_equal(got[5], rows[1])
    got, valid = oa.gather(cache, table[1], 9)
    assert valid.tolist() == [True] * 3 + [False] * 3 + [True] * 3
    assert np.array_equal(got[2], rows[3]) and np.array_equal(got[8], rows[6])
    assert np.count_nonzero(cache) == 4 * 8


def test_bf16_rounding():
    assert oa.round_bf16(1.0 + 2.0 ** -8) == 1.0          # half a step: to even
    assert oa.round_bf16(1.0 + 3 * 2.0 ** -8) == 1.0 + 2.0 ** -6
    assert oa.widen(np.array([0x3F80, 0xC040], np.uint16)).tolist() == [1.0, -3.0]


@pytest.mark.parametrize("theta,rot", [(1e4, 128), (5e6, 64), (1.0, 16)])
def test_frequencies_are_turns_per_position(theta, rot):
    f = binding.rope_freq(rot, theta, device="cpu").numpy().view(np.uint64)
    for i in range(rot // 2):
        want = theta ** (-2.0 * i / rot)
        assert int(f[i]) / 2.0 ** 64 * 2 * math.pi == pytest.approx(want, rel=1e-15)
    # the phase at a far position, by exact integers, against the angle in 64 bits
    p = (1 << 20) + 3
    phase = (int(f[1]) * p) % (1 << 64) / 2.0 ** 64
    turns = p * theta ** (-2.0 / rot) / (2 * math.pi)
    assert abs((phase - turns + 0.5) % 1.0 - 0.5) < 1e-9
    with pytest.raises(ValueError, match="entries"):
        binding.rope_freq(rot, inv_freq=[1.0], device="cpu")

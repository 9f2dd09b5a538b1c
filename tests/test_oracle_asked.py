"""The whole numbers that stand for a kv head's queries: of exact sums, ties to even."""
import numpy as np
import pytest

from oracle import layer_ops as ref


def asked(*heads):
    u, d = ref.asked(np.array(heads, np.float64))
    return u.tolist(), d.tolist()


@pytest.mark.parametrize("tiny", [2.0 ** -20, 2.0 ** -26, 2.0 ** -60, 2.0 ** -133])
def test_a_head_far_below_the_others_counts(tiny):
    assert asked([127, 62.5, -0.5], [0, tiny, -tiny]) == ([127, 63, 0], [0, 0, 1])
    assert asked([127, 62.5, -0.5], [0, 0, 0]) == ([127, 62, 0], [0, 0, 0])
    assert asked([127, 62.5, 61.5], [tiny, 0, 0]) == ([64, 31, 31], [0, 0, 0])      # past 127 of a unit
    assert asked([127, 1], [-tiny, tiny]) == ([127, 1], [0, 0])


def test_the_largest_sums():
    big = 2.0 ** 128 - 2.0 ** 104
    parts = [2.0 ** 128 - 2.0 ** 120, 2.0 ** 120 - 2.0 ** 112, 2.0 ** 112 - 2.0 ** 104]
    assert sum(parts) == big
    heads = [[p, p / 2] for p in parts]
    assert asked(*heads) == ([64, 32], [0, 0])
    assert asked(*heads, [1.0, 0]) == ([0, 0], [0, 0]) == asked(*heads, [-1.0, 0])
    assert asked([np.inf, 1]) == asked([np.nan, 1]) == ([0, 0], [0, 0])
    assert asked([2.0 ** -101, 2.0 ** -100]) == ([0, 1], [0, 0]) and asked([2.0 ** -101 * 1.5, 0]) == ([1, 0], [0, 0])


def test_sums_without_a_rounding_are_as_before():
    q = np.round(np.random.default_rng(1).standard_normal((8, 64)) * 64) / 64
    u, d = ref.asked(q)
    up, down = np.maximum(q, 0).sum(0), np.maximum(-q, 0).sum(0)
    f = ref.unit(max(up.max(), down.max()))
    assert np.array_equal(u, np.rint(up / 2.0 ** f)) and np.array_equal(d, np.rint(down / 2.0 ** f))

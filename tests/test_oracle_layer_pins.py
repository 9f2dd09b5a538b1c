"""The fp64 definitions of the operators around the cache's attention, pinned to closed forms and to each other."""
import numpy as np

from oracle import kv4, layer_ops as ref


def test_norm_of_equal_values_is_their_sign():
    y = ref.add_rmsnorm(np.array([[3.0, -3.0, 3.0, 3.0]]), np.array([1.0, 2.0, 0.5, 0.0]), 0.0)
    assert np.allclose(y, [[1.0, -2.0, 0.5, 0.0]])
    assert np.allclose(ref.block_scales(y, 2), [[2.0 / 448, 0.5 / 448]])


def test_rotation_keeps_lengths_and_adds_up():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 64))
    for pairs in (False, True):
        a = ref.rotate(x, [5, 9], 64, pairs)
        assert np.allclose((a ** 2).sum(-1), (x ** 2).sum(-1))
        b = ref.rotate(a, [7, 1], 64, pairs)
        assert np.allclose(b, ref.rotate(x, [12, 10], 64, pairs))
        # a quarter turn of the first pair
        y = ref.rotate(x, [np.pi / 2] * 2, 32, pairs)
        assert np.allclose(y[..., 0], -x[..., 1 if pairs else 16]) and np.array_equal(y[..., 32:], x[..., 32:])


def test_bounds_hold_and_are_tight():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((16, 2, 64)) * np.array([1.0, 300.0])[None, :, None]
    hi, lo, e = ref.page_bounds(k)
    s = 2.0 ** e[:, None]
    assert (hi * s >= k.max(0)).all() and (lo * s <= k.min(0)).all()
    assert (hi * s - k.max(0) < s).all() and (k.min(0) - lo * s < s).all()
    assert np.abs(np.concatenate([hi, lo])).max() <= 127
    # half the unit would not do
    assert (np.abs(k).max((0, 2)) > 127 * s[:, 0] / 2).all()
    k[3, 1, 5] = np.nan
    assert ref.page_bounds(k)[2][1] == ref.UNBOUNDED
    assert not ref.page_bounds(np.zeros((3, 1, 64)))[2].any()


def test_score_is_above_the_products():
    """With whole-number queries of the unit's range nothing is rounded, and the score bounds sum_h q_h . k."""
    rng = np.random.default_rng(2)
    q = rng.integers(-30, 31, (4, 64)).astype(float)
    q[0, 0] = 100
    u, d = ref.asked(q)
    f = ref.unit(max(np.maximum(q, 0).sum(0).max(), np.maximum(-q, 0).sum(0).max()))
    k = rng.standard_normal((16, 1, 64)) * 3
    hi, lo, e = ref.page_bounds(k)
    bound = (u * hi[0] - d * lo[0]).sum() * 2.0 ** (e[0] + f)
    assert bound >= (q.sum(0) @ k[:, 0].T).max() - 64 * 4 * 2.0 ** f


def test_pick_takes_the_ends_the_best_and_the_lower_of_equals():
    rec = [(np.full(4, v), np.zeros(4, int), 0) for v in (1, 5, 2, 5, 5, 0, 1)]
    q = np.ones((2, 4))
    assert ref.pick(q, 6 * 16 + 3, rec, 16, 4, 1, 1) == [0, 1, 3, 6]
    assert ref.pick(q, 6 * 16 + 3, rec, 16, 4, 0, 2) == [1, 3, 5, 6]
    assert ref.pick(q, 2 * 16, rec, 16, 4, 1, 1) == [0, 1, 2, -1]
    assert ref.pick(q, -1, rec, 16, 2, 1, 1) == [-1, -1]
    rec[5] = (np.zeros(4, int), np.zeros(4, int), ref.UNBOUNDED)
    rec[1] = None
    assert ref.pick(q, 6 * 16, rec, 16, 4, 1, 1) == [0, 3, 5, 6]
    assert ref.pick(-q, 6 * 16, [(x[0], x[0] - 1, x[2]) if x else None for x in rec], 16, 3, 1, 1) == [0, 5, 6]


def test_all_pages_picked_is_dense_attention():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64))
    q = rng.standard_normal((1, 6, 64))
    want = kv4.attention(q, k, v, 0, 0.1)
    got = ref.attention_picked(q[0], k, v, 39, np.array([[0, 1, 2, -1]] * 2), 16, 0.1)
    for w, g in zip(want, got):
        assert np.allclose(w[0], g)

"""The 4-bit cache's oracle against closed forms and invariants (CPU)."""
import numpy as np
import pytest

from oracle import kv4 as ref


def test_grids():
    assert ref.E2M1.tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6]
    assert ref.E4M3[0] == 0 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[126] == 448 and (np.diff(ref.E4M3) > 0).all()


def test_representable_values_come_back():
    for s in (2.0 ** -9, 0.375, 1.0, 448.0):
        x = np.concatenate([ref.E2M1, -ref.E2M1]) * s
        code, sb = ref.quantise(x[None])
        assert np.array_equal(ref.values(code, sb)[0], x)


def test_rounding_ties_go_to_the_even_code():
    x = np.zeros((1, 16))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    code, sb = ref.quantise(x)
    assert ref.values(code, sb)[0, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]


def test_error_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((500, 64)) * np.exp(rng.uniform(-3, 6, (500, 1)))
    code, sb = ref.quantise(x)
    got = ref.values(code, sb)
    s = np.repeat(ref.E4M3[sb], 16, -1)
    # a scale off by 2^-4 can put the block's largest above 6 s: it saturates, by up to 6/16 s
    step = np.where(np.abs(x) / s < 2, 0.5, np.where(np.abs(x) / s < 4, 1.0, 2.0))
    assert (np.abs(got - x) <= step / 2 * s * (1 + 1e-12)).all()


def test_small_nan_and_large_blocks():
    x = np.zeros((4, 16))
    x[0] = 2.0 ** -9 * 2.9            # top / 6 rounds to scale 0
    x[1, 3] = np.nan
    x[2, 5] = np.inf
    x[3, 0] = 1e5
    code, sb = ref.quantise(x)
    v = ref.values(code, sb)
    assert (v[0] == 0).all() and np.isnan(v[1]).all() and v[2, 5] == 2688 and v[3, 0] == 2688


def test_layout_round_trip_and_page_borders():
    rng = np.random.default_rng(1)
    P, H, D, n = 16, 2, 64, 41
    pool = np.zeros((5, H, P // 16, 18 * D), np.uint8)
    table = np.array([3, 0, 4, -1])
    kv = rng.standard_normal((n, 2, H, D))
    for t in range(n):
        ref.store(pool, table, t, kv[t, 0], kv[t, 1], P)
    k, v = ref.load(pool, table, n, P)
    assert np.array_equal(k, ref.values(*ref.quantise(kv[:, 0]))) and np.array_equal(v, ref.values(*ref.quantise(kv[:, 1])))
    assert not pool[1].any() and not pool[2].any()


@pytest.mark.parametrize("window", [0, 1, 5])
def test_attention_by_hand(window):
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse, _, _ = ref.attention(q, k, v, window, 0.3)
    for i in range(3):
        for h in range(4):
            js = [j for j in range(9) if j <= 6 + i and (not window or j > 6 + i - window)]
            w = np.array([np.exp(0.3 * sum(q[i, h, d] * k[j, h // 2, d] for d in range(8))) for j in js])
            assert np.allclose(o[i, h], sum(x * v[j, h // 2] for x, j in zip(w, js)) / w.sum())
            assert np.isclose(lse[i, h], np.log(w.sum()))


def test_rows_before_the_cache_are_empty():
    o, lse, _, _ = ref.attention(np.ones((3, 1, 8)), np.ones((1, 1, 8)), np.ones((1, 1, 8)))
    assert (o[:2] == 0).all() and (lse[:2] == -np.inf).all() and (o[2] == 1).all()


def test_pages_keep_counts():
    rng = np.random.default_rng(3)
    p = ref.Pages(40, 8, 6, 16)
    data = [np.arange(40)[:, None].repeat(2, 1)]
    for step in range(200):
        op = rng.integers(4)
        if op == 0:
            p.alloc([int(rng.integers(-min(9, p.lens[b]), 20)) if p.lens[b] < 70 else 0 for b in range(8)])
        elif op == 1:
            src = [b for b in range(8) if p.lens[b]]
            dst = [b for b in range(8) if not p.lens[b]]
            if src and dst:
                p.fork([src[0]] * len(dst[:2]), dst[:2], data)
        elif op == 2:
            p.free([int(rng.integers(8))])
        else:
            live = p.compact(data)
            assert all(p.refs[:live]) and not any(p.refs[live:])
        count = [0] * 40
        for b in range(8):
            for j, page in enumerate(p.table[b]):
                assert (page >= 0) == (j < p.held(b))
                if page >= 0:
                    count[page] += 1
        assert count == p.refs

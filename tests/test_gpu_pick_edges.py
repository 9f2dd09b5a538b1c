"""Picks where sums of queries need more bits than fp32 has, where page numbers are out of range, and in rows of many places."""
import numpy as np
import pytest
import torch

from test_gpu_kv4_layer import BF, DEV, FP, _lib, cu_of, dev, i32, kda, new_err, pick, picks_of, random_bounds  # noqa: F401

pytestmark = pytest.mark.gpu


def spans(T, H, G, D, dtype, seed):
    """Queries whose sums lie on a tie, or on the border of a unit, but for a head far below the others."""
    rng = np.random.default_rng(seed)
    q = np.zeros((T, H, G, D))
    sign = rng.choice([-1, 1], (T, H, D))
    whole = rng.integers(0, 126, (T, H, D)) + 0.5
    part = np.floor(whole * rng.random((T, H, D)))
    at = np.argsort(rng.random((T, H, G, D)), 2)                 # an order of the heads, channel by channel
    low = -24 if dtype is FP else -60
    tiny = 2.0 ** rng.integers(low, -16, (T, H, D)) * (rng.random((T, H, D)) < 0.7)
    rows = [part, whole - part, tiny] if G > 2 else [whole, tiny]
    whole[..., 0], part[..., 0] = 127, 63                        # the unit's border: 127, or 127 and little more
    if G > 2:
        rows[1][..., 0] = 64
    tiny[..., 0] *= rng.random((T, H)) < 0.3
    for i, r in enumerate(rows):
        np.put_along_axis(q, at[:, :, i:i + 1], (r * sign)[:, :, None], 2)
    scale = 2.0 ** rng.integers(-3, 4, (T, H, 1, 1)) if dtype is BF else 1.0
    out = torch.from_numpy((q * scale).reshape(T, H * G, D)).to(dtype)
    assert torch.equal(out.double(), torch.from_numpy((q * scale).reshape(T, H * G, D)))
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("news,H,G,D", [([1] * 12, 2, 2, 64), ([1] * 7, 3, 5, 128), ([1] * 3, 9, 12, 64), ([5, 1, 11], 2, 2, 64), ([9, 3], 2, 5, 128), ([4, 8], 1, 19, 128)])
def test_sums_of_more_bits_than_fp32(news, H, G, D, dtype):
    lens = [5000 + 37 * b for b in range(len(news))]
    rec, table = random_bounds(lens, H, D, 16, 31)
    rec[..., 2 * D] = 0
    q = spans(sum(news), H, G, D, dtype, 32)
    got, err = pick(q, news, lens, rec, table, 16, 90, 1, 2)
    assert err == 0 and np.array_equal(got, picks_of(q, news, lens, rec, table, 16, 90, 1, 2))


@pytest.mark.parametrize("news", [[1] * 4, [2, 2]])
def test_sums_at_the_end_of_fp32(news):
    """A head's magnitudes add up to the largest fp32, to a little more, or with a rounding on the way."""
    lens = [640] * len(news)
    rec, table = random_bounds(lens, 1, 64, 16, 33)
    q = np.zeros((4, 5, 64))
    parts = [2.0 ** 128 - 2.0 ** 120, 2.0 ** 120 - 2.0 ** 112, 2.0 ** 112 - 2.0 ** 104]
    rng = np.random.default_rng(34)
    q[:, :3, 1:] = 2.0 ** rng.integers(119, 127, (4, 3, 63)) * rng.choice([-1, 1], (4, 3, 63))
    for t in range(4):
        q[t, :3, 0] = parts
    q[1, 3, 0], q[2, 3, 0], q[3, 3, 0], q[3, 2, 0] = 2.0 ** 90, -2.0 ** 90, 2.0 ** 90, 2.0 ** 111
    q = torch.from_numpy(q).to(BF)
    got, err = pick(q, news, lens, rec, table, 16, 9, 1, 2)
    want = picks_of(q, news, lens, rec, table, 16, 9, 1, 2)
    assert err == 0 and np.array_equal(got, want)
    assert want[1, 0].tolist() == want[2, 0].tolist() == list(range(7)) + [38, 39] != want[0, 0].tolist()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("news,G,D", [([1, 1], 5000, 64), ([2, 1], 5000, 128), ([1] * 6, 70, 128)])
def test_many_heads_of_every_size(news, G, D, dtype):
    """Sums of thousands of values that lie far apart."""
    lens = [3000 + b for b in range(len(news))]
    rec, table = random_bounds(lens, 1, D, 16, 38)
    g = torch.Generator().manual_seed(39)
    q = torch.randn(sum(news), G, D, generator=g) * torch.exp2(torch.randint(-12, 3, (sum(news), G, D), generator=g).float())
    q = q.to(dtype)
    got, err = pick(q, news, lens, rec, table, 16, 60, 1, 2)
    assert err == 0 and np.array_equal(got, picks_of(q, news, lens, rec, table, 16, 60, 1, 2))


@pytest.mark.parametrize("news", [[1, 1], [2, 3]])
@pytest.mark.parametrize("page", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
def test_every_page_out_of_range_is_told(news, page):
    lens = [640, 640]
    rec, table = random_bounds(lens, 2, 64, 16, 35)
    table[0, 7] = page
    q = torch.randn(sum(news), 4, 64, generator=torch.Generator().manual_seed(36)).to(BF)
    got, err = pick(q, news, lens, rec, table, 16, 8, 1, 1)
    assert err == 32 and np.array_equal(got, picks_of(q, news, lens, rec, table, 16, 8, 1, 1))


@pytest.mark.parametrize("count", [2 ** 31 - 1, 2 ** 31 - 100])
def test_as_many_places_as_an_int_counts(count):
    """A row of 8.6 GB whose token takes all of its pages: places in it are counted past 2^31 - 1 by no thread."""
    rec, table = random_bounds([500], 1, 64, 16, 37)
    picked = torch.full((1, 1, count), 5, dtype=torch.int32, device=DEV)
    got = kda().kda_kv4_pick(torch.ones(1, 1, 64, dtype=BF, device=DEV), i32([0, 1]), 1, i32([500]), dev(table), dev(rec), 16, count, picked=picked)
    assert got is picked and picked[0, 0, :32].tolist() == list(range(32)) and int(picked[0, 0, 32:].max()) == -1
    assert int(picked[0, 0, 32:].min()) == -1
    del picked, got
    torch.cuda.empty_cache()

"""The paged 4-bit cache's attention at its edges."""
import numpy as np
import pytest
import torch

from kv4_testutil import HALF_STEP, cu_of, make_cache, packed_q
from oracle import kv4 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()


def kda():
    import kda_state_gb300
    return kda_state_gb300


@pytest.fixture(scope="module")
def ws():
    return kda().make_kv4_workspace()


def dev(x, dtype=None):
    return torch.as_tensor(x, dtype=dtype).to(DEV)


def attend(pool, table, news, lens, q, ws, window=0, scale=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = kda().kda_kv4_attention(q.to(DEV), cu_of(news).to(DEV), max(news), dev(lens, torch.int32), dev(table), dev(pool),
                                     scale=scale, window=window, workspace=ws, dev_err=err, **kw)
    torch.cuda.synchronize()
    return o, lse, int(err)


def definition(q, k, v, there, window, scale):
    """o, lse of rows q [n, Hq, D] over k, v [len, H, D] in fp64, of whose positions only those `there` exist; with the
    bounds on their errors that kv4_testutil.expected derives, before the rounding of o."""
    n, Hq, D = q.shape
    L, G = k.shape[0], Hq // k.shape[1]
    q, at = q.double().numpy(), np.arange(L)
    last = L - n + np.arange(n)[:, None]
    seen = (at <= last) & there & ((at > last - window) if window else True)
    # [Hkv, n G, D] queries, [Hkv, L, D] keys and values: batched products
    q = q.reshape(n, -1, G, D).transpose(1, 0, 2, 3).reshape(-1, n * G, D)
    k, v = k.transpose(1, 0, 2), v.transpose(1, 0, 2)
    rows = lambda x: x.reshape(k.shape[0], n, G, -1).transpose(1, 0, 2, 3).reshape(n, Hq, -1)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.where(seen[:, None], rows(q @ k.transpose(0, 2, 1)) * scale, -np.inf)
        big = np.where(seen[:, None], rows(np.abs(q) @ np.abs(k).transpose(0, 2, 1)) * abs(scale), 0).max(-1)
        m = np.max(s, -1, keepdims=True)
        p = np.exp(s - np.where(np.isneginf(m), 0, m))
        total = p.sum(-1)
        lse = m[..., 0] + np.log(total)
        # a NaN value reaches the rows that see it, whatever its weight
        bad = np.repeat((seen.astype(float) @ np.isnan(v).astype(float)).transpose(1, 0, 2) > 0, G, 1)
        weights = p.reshape(n, -1, G, L).transpose(1, 0, 2, 3).reshape(-1, n * G, L)
        mean = lambda x: rows(weights @ np.nan_to_num(x)) / np.where(total == 0, 1, total)[..., None]
        o, a = np.where(bad, np.nan, mean(v)), mean(np.abs(v))
    es = 2 * D * 2.0 ** -23 * big + 2.0 ** -20
    bo = a * (2.0 ** -11 + 4 * es[..., None]) + 2.0 ** -30 * max(1, L) * np.nanmax(np.abs(v), initial=0)
    return o, lse, bo, es + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def close(o, lse, want, dtype):
    wo, wl, bo, bl = want
    go, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(go), np.isnan(wo)) and np.array_equal(np.isnan(gl), np.isnan(wl))
    assert np.array_equal(np.isneginf(gl), np.isneginf(wl))
    ok, okl = ~np.isnan(wo), np.isfinite(wl)
    assert (np.abs(go - wo)[ok] <= (bo + HALF_STEP[dtype] * np.abs(wo) * 1.01 + 2.0 ** -24)[ok]).all()
    assert (np.abs(gl[okl] - wl[okl]) <= bl[okl]).all()


# ---------------------------------------------------------------------------
# pages that cannot be read
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("page", [-1, -2, -3, -2 ** 31, None, 2 ** 31 - 1])
@pytest.mark.parametrize("news", [[1, 1], [3, 5], [90, 70]])
def test_entries_that_name_no_page(ws, news, page):
    """Tokens of a page out of range are left out and flagged, whatever number the entry holds."""
    lens, D, P, H, Hq = [100, 130], 128, 16, 1, 4
    pool, table = make_cache(lens, H, D, P, 60)
    q = packed_q(news, Hq, D, BF, 61)
    t = table.copy()
    t[1, 2] = len(pool) if page is None else page
    for window in (0, 40):
        if window and news[0] < 9:
            continue                       # single tokens then see nothing of that page
        o, lse, err = attend(pool, t, news, lens, q, ws, window)
        assert err == 32
        at = 0
        for b, n in enumerate(news):
            there = np.ones(lens[b], bool)
            there[2 * P:3 * P] = b != 1
            close(o[at:at + n], lse[at:at + n],
                  definition(q[at:at + n], *ref.load(pool, table[b], lens[b], P), there, window, D ** -0.5), BF)
            at += n


# ---------------------------------------------------------------------------
# windows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("news,lens,Hq,Hkv", [([8, 2], [2, 9], 1, 1), ([5, 4], [1, 60], 6, 2), ([40, 17], [20, 300], 8, 1),
                                              ([700, 599], [30, 599], 64, 8)])
def test_windows_longer_than_the_cache(ws, news, lens, Hq, Hkv):
    """A window no row can fill is no window, also for requests with rows before their first token."""
    D, P = 64, 16
    pool, table = make_cache(lens, Hkv, D, P, 62)
    q = packed_q(news, Hq, D, BF, 63)
    want = attend(pool, table, news, lens, q, ws)
    rows = lambda b, x: definition(x, *ref.load(pool, table[b], lens[b], P), np.ones(lens[b], bool), 0, D ** -0.5)
    n, last = news[0], q[-min(3, news[1]):]
    close(want[0][:n], want[1][:n], rows(0, q[:n]), BF)
    close(want[0][-len(last):], want[1][-len(last):], rows(1, last), BF)
    for window in (max(lens), table.shape[1] * P, table.shape[1] * P + 1, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1):
        o, lse, err = attend(pool, table, news, lens, q, ws, window)
        assert err == 0 and torch.equal(lse, want[1]) and torch.equal(o, want[0])


# ---------------------------------------------------------------------------
# scores of every size
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("news,lens", [([1, 1, 1], [300, 40, 9000]), ([3, 4, 2], [300, 40, 9000]), ([90, 40, 64], [300, 40, 3000]),
                                       ([700, 1, 599], [1500, 77, 2000])])
def test_scores_of_every_size(ws, news, lens, D):
    """Scores far apart, from 2^20 to 2^122 and below zero: the largest, tied ones, share the row.

    Keys are one value in all channels, so that scores are exact; ties have equal weights, all else
    none, and the sums are exact too.  What is left is the quotient (2^-20) and o's rounding; lse is
    a product of four roundings (2^-22 of it)."""
    P, H, Hq = 64, 8 if news[0] == 700 else 1, 64 if news[0] == 700 else 4
    rng = np.random.default_rng(70)
    pool, table = make_cache([0] * 3, H, D, P, 71)
    need = [-(-n // P) for n in lens]
    pool = np.full((sum(need), H, P // 16, 18 * D), 255, np.uint8)
    table = np.full((3, max(need) + 1), -1, np.int32)
    pages = rng.permutation(sum(need))
    level, value = [], []
    for b, n in enumerate(lens):
        table[b, :need[b]] = pages[sum(need[:b]):sum(need[:b + 1])]
        level.append(rng.choice([1.0, 1.5, 2.0], n))
        value.append(rng.choice([-6.0, -4, -3, -2, -1.5, -1, 0.5, 1, 1.5, 2, 3, 4, 6], (n, D)))
        value[b][:, ::16] = 6.0            # a scale of 1 for each block
        for pos in range(n):
            ref.store(pool, table[b], pos, np.full((H, D), level[b][pos]), np.repeat(value[b][pos:pos + 1], H, 0), P)
        k, v = ref.load(pool, table[b], n, P)                  # as they are stored
        level[b], value[b] = k[:, 0, 0], v[:, 0]
    for power in (20, 24, 27, 28, 31, 40, 64, 100, 114):
        for sign in (1.0, -1.0):
            q = torch.full((sum(news), Hq, D), 2.0 ** power).to(BF)
            o, lse, err = attend(pool, table, news, lens, q, ws, scale=sign)
            assert err == 0
            at = 0
            for b, n in enumerate(news):
                for i in sorted({0, 1, n // 2, n - 2, n - 1} & set(range(n))):
                    last = lens[b] - n + i
                    x = level[b][:last + 1] * sign
                    wo = value[b][:last + 1][x == x.max()].mean(0)
                    wl = x.max() * D * 2.0 ** power + np.log((x == x.max()).sum())
                    go, gl = o[at + i].double().cpu().numpy(), lse[at + i].double().cpu().numpy()
                    assert (np.abs(go - wo) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(wo) + 2.0 ** -20 * 6).all(), (power, sign, b, i)
                    assert (np.abs(gl - wl) <= 2.0 ** -22 * np.abs(wl)).all(), (power, sign, b, i)
                at += n


@pytest.mark.parametrize("news,lens", [([1, 1], [300, 9000]), ([3, 5], [40, 9000]), ([90, 64], [300, 3000])])
def test_scores_near_zero(ws, news, lens):
    """Queries so small that all of a row's tokens weigh the same."""
    D, P, H, Hq = 64, 64, 1, 4
    pool, table = make_cache(lens, H, D, P, 74)
    for power in (-126, -110, -104, -102, -101, -100, -99, -98, -97, -96, -90, -60):
        q = packed_q(news, Hq, D, BF, 75) * 2.0 ** power
        o, lse, err = attend(pool, table, news, lens, q, ws, scale=1.0)
        assert err == 0
        at = 0
        for b, n in enumerate(news):
            close(o[at:at + n], lse[at:at + n],
                  definition(q[at:at + n], *ref.load(pool, table[b], lens[b], P), np.ones(lens[b], bool), 0, 1.0), BF)
            at += n


@pytest.mark.parametrize("news", [[1, 1, 1], [4, 5, 2], [90, 30, 64]])
def test_infinite_queries(ws, news):
    """A query with an infinity has NaN results, of one sign or both, unless its row sees nothing."""
    D, P, H, Hq = 128, 16, 2, 4
    lens = [300, max(news[1] - 2, 0), 200]                      # the second request's first rows see nothing
    pool, table = make_cache(lens, H, D, P, 72)
    for b, n in enumerate(lens):
        for pos in range(n):
            ref.store(pool, table[b], pos, np.full((H, D), -1.0 - pos % 3), np.ones((H, D)), P)
    q = packed_q(news, Hq, D, BF, 73)
    q[0, 1, 7] = float("inf")                                   # all of its scores are -inf
    q[news[0], 0, 3] = float("inf")                             # a row that sees nothing
    q[sum(news[:2]), 2, 9] = -float("inf")                      # all of its scores are +inf
    q[-1, 3, 0] = float("nan")
    for window in (0, 30):
        o, lse, err = attend(pool, table, news, lens, q, ws, window)
        assert err == 0
        nan = torch.zeros(sum(news), Hq, dtype=torch.bool)
        nan[0, 1] = nan[sum(news[:2]), 2] = nan[-1, 3] = True
        assert torch.equal(lse.isnan().cpu(), nan) and torch.equal(o.isnan().cpu(), nan[..., None].expand(-1, -1, D))
        assert not o[news[0], 0].any() and lse[news[0], 0] == -float("inf")


# ---------------------------------------------------------------------------
# pages that cannot be read, and NaN, in requests that are cut and in wide parts
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("news,lens,Hq,Hkv,D,dtype", [
    ([1, 1], [2500, 1300], 8, 1, 128, BF),                    # few rows, joined over blocks
    ([9, 3], [2500, 1300], 2, 2, 64, FP),
    ([70, 40], [2500, 1300], 4, 2, 128, BF),                  # tiles of 128 rows, cut along the tokens and joined
    ([90, 33], [1900, 1300], 2, 1, 64, FP),
    ([700, 599], [1500, 700], 64, 8, 128, BF),                # tiles of 256 rows
    ([700, 599], [1500, 700], 64, 8, 64, FP)])
def test_missing_pages_and_nan_among_many(ws, news, lens, Hq, Hkv, D, dtype, window):
    """Pages out of range in the middle of a request, and NaN keys and values in single heads, against the definition of
    every row."""
    P = 64
    pool, table = make_cache(lens, Hkv, D, P, 76)
    one, nan = np.full((Hkv, D), 0.5), np.full((Hkv, D), 0.5)
    nan[0, 17] = np.nan
    early, late = lens[0] - news[0] - 200 if news[0] < 400 else 300, lens[0] - max(2, news[0] // 2)
    ref.store(pool, table[0], early, one, nan, P)             # a value that many rows see
    ref.store(pool, table[0], late, one, nan, P)              # one that the last rows see
    ref.store(pool, table[1], lens[1] - 2, nan, one, P)       # a key near the end
    q = packed_q(news, Hq, D, dtype, 77)
    t = table.copy()
    gone = [[1, 2, lens[0] // P // 2, lens[0] // P - 1], [0, lens[1] // P - 3]]
    for b, pages in enumerate(gone):
        t[b, pages] = [-1, len(pool), -2, 2 ** 31 - 1][:len(pages)]
    o, lse, err = attend(pool, t, news, lens, q, ws, window)
    assert err == 32
    o2, lse2, _ = attend(pool, t, news, lens, q, ws, window)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16)) and torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    at = 0
    for b, n in enumerate(news):
        there = np.ones(lens[b], bool)
        for page in gone[b]:
            there[page * P:(page + 1) * P] = False
        k, v = ref.load(pool, table[b], lens[b], P)
        for i in range(0, n, 100):                            # (100 rows at a time: the definition holds all scores)
            z = min(n, i + 100)
            upto = lens[b] - n + z
            close(o[at + i:at + z], lse[at + i:at + z], definition(q[at + i:at + z], k[:upto], v[:upto], there[:upto], window,
                                                                   D ** -0.5), dtype)
        at += n


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("D,dtype", [(128, BF), (64, FP)])
def test_every_row_of_wide_parts(ws, D, dtype, window):
    news, lens, Hq, Hkv, P = [700, 1, 599], [900, 77, 599], 64, 8, 32
    pool, table = make_cache(lens, Hkv, D, P, 78)
    q = packed_q(news, Hq, D, dtype, 79, 2.0)
    o, lse, err = attend(pool, table, news, lens, q, ws, window)
    assert err == 0
    at = 0
    for b, n in enumerate(news):
        k, v = ref.load(pool, table[b], lens[b], P)
        for i in range(0, n, 100):
            z = min(n, i + 100)
            upto = lens[b] - n + z
            close(o[at + i:at + z], lse[at + i:at + z], definition(q[at + i:at + z], k[:upto], v[:upto], np.ones(upto, bool), window,
                                                                   D ** -0.5), dtype)
        at += n


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 64, 2)])
def test_append_writes_its_bytes_and_no_others(dtype, D, P, H):
    """Every byte of the pool is the oracle's, but for the codes of the blocks that hold a NaN (their scale says it)."""
    news, starts = [3, 20, 1], [0, 30, P - 1]
    lens = [a + n for a, n in zip(starts, news)]
    rng = np.random.default_rng(80)
    need = [-(-n // P) for n in lens]
    pool = rng.integers(0, 256, (sum(need) + 3, H, P // 16, 18 * D), dtype=np.uint8)
    table = np.full((3, max(need)), -1, np.int32)
    order = rng.permutation(len(pool))
    for b, n in enumerate(need):
        table[b, :n] = order[sum(need[:b]):sum(need[:b]) + n]
    x = (torch.randn(sum(news), 2, H, D, generator=torch.Generator().manual_seed(81)) * 3).to(dtype)
    x[4, 0, 1, 20] = x[9, 1, 0, 3] = float("nan")
    want, free = pool.copy(), np.zeros(pool.shape, bool)
    t = 0
    for b, n in enumerate(news):
        for i in range(n):
            k, v = x[t].double().numpy()
            ref.store(want, table[b], starts[b] + i, k, v, P)
            page, tile, tok = ref.place(table[b], starts[b] + i, P)
            for y, base in ((k, 0), (v, 9 * D)):
                for h, c in zip(*np.nonzero(np.isnan(y))):
                    a = base + tok * (D // 2) + c // 16 * 8
                    free[page, h, tile, a:a + 8] = True
            t += 1
    assert free.sum() == 16
    d, err = dev(pool), torch.zeros(1, dtype=torch.int32, device=DEV)
    kda().kda_kv4_append(x[:, 0].to(DEV), x[:, 1].to(DEV), cu_of(news).to(DEV), dev(starts, torch.int32), dev(table), d, dev_err=err)
    assert int(err) == 0
    got = d.cpu().numpy()
    assert np.array_equal(got[~free], want[~free])


@pytest.mark.parametrize("dtype,power", [(BF, 118), (BF, 120), (BF, 127), (BF, -120), (FP, 7), (FP, -14)])
def test_gather_at_the_ends_of_the_type(dtype, power):
    """A value in the type's range is read back exactly, also where its block's scale times the tensor's is not in fp32's."""
    H, D, P, n = 2, 64, 16, 20
    rng = np.random.default_rng(82)
    pool, table = make_cache([0], H, D, P, 83, spare=2, max_pages=3)
    table[0, :2] = [1, 0]
    for pos in range(n):
        x = rng.choice([0.0, 0.5, -1, 1.5, -2, 3, 4, -6], (2, H, D)) * 2.0 ** rng.integers(-8, 3)
        x[..., ::16] = np.sign(rng.standard_normal((2, H, D // 16))) * 6 * rng.choice([448.0, 4.0, 2.0 ** -9], (2, H, D // 16))
        ref.store(pool, table[0], pos, x[0], x[1], P)
    k, v = kda().kda_kv4_gather(cu_of([n]).to(DEV), dev([0], torch.int32), n, dev(table), dev(pool), dtype=dtype,
                                k_scale=2.0 ** power, v_scale=2.0 ** power)
    wk, wv = ref.load(pool, table[0], n, P, 2.0 ** power, 2.0 ** power)
    for got, want in ((k, wk), (v, wv)):
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype))


@pytest.mark.parametrize("news,lens", [([1, 1], [9000, 30]), ([3, 5], [9000, 30]), ([90, 40], [5000, 70]), ([600, 550], [3000, 700])])
def test_value_scales_of_every_size(ws, news, lens):
    """Outputs in the type's normal range are as exact with a tiny or a huge tensor scale as with 1."""
    D, P, H, Hq = 64, 64, 8 if news[0] == 600 else 2, 64 if news[0] == 600 else 4
    pool, table = make_cache(lens, H, D, P, 84)
    q = packed_q(news, Hq, D, BF, 85)
    for b, n in enumerate(lens):                              # values around 1000
        for pos in range(0, n, 3):
            ref.store(pool, table[b], pos, np.full((H, D), 0.5), np.full((H, D), 900.0 + pos % 200), P)
    one, want_lse, _ = attend(pool, table, news, lens, q, ws)
    for power in (-127, -118, -105, 100, 114):
        o, lse, err = attend(pool, table, news, lens, q, ws, v_scale=2.0 ** power)
        assert err == 0 and torch.equal(lse, want_lse)
        o, want = o.double() * 2.0 ** -power, one.double()
        # both are one rounding to bf16 of values that differ by fp32 arithmetic; below 2^-126 the type's steps are 2^-133
        step = 2.0 ** -7 * want.abs() + 2.0 ** (-133 - power if power < -100 else -200)
        assert ((o - want).abs() <= step * 1.01).all()
        assert ((o == want) | (want.abs() * 2.0 ** power < 2.0 ** -126)).double().mean() > 0.99

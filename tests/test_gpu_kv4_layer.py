"""The rotated append, the pages' bounds, the picks and the attention over them: bytes and whole numbers bit for bit,
attention within the bounds that kv4_testutil.expected derives."""
import numpy as np
import pytest
import torch

from kv4_testutil import HALF_STEP, check, cu_of, make_cache, packed_q
from oracle import kv4, layer_ops as ref

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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def new_err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# append with rotation
# ---------------------------------------------------------------------------

def turned(x, rope, pos, pairs):
    """The rotation in fp32, each product and sum rounded, in x's type."""
    R = rope.shape[1]
    cos, sin = rope[pos][:, None, :R // 2], rope[pos][:, None, R // 2:]
    f = x.float()
    a, b = (f[..., 0:R:2], f[..., 1:R:2]) if pairs else (f[..., :R // 2], f[..., R // 2:R])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if pairs else torch.cat(y, -1)
    return torch.cat([y.to(x.dtype), x[..., R:]], -1)


def rope_case(news, starts, Hq, H, D, P, dtype, seed):
    lens = [a + n for a, n in zip(starts, news)]
    need = [-(-n // P) for n in lens]
    rng = np.random.default_rng(seed)
    pages = sum(need) + 2
    table = np.full((len(news), max(need) + 1), -1, np.int32)
    order = iter(rng.permutation(pages))
    for b, n in enumerate(need):
        table[b, :n] = [next(order) for _ in range(n)]
    pool = dev(rng.integers(0, 256, (pages, H, P // 16, 18 * D), dtype=np.uint8))
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(sum(news), Hq + 2 * H + 1, D, generator=g) * torch.exp(torch.randn(sum(news), Hq + 2 * H + 1, 1, generator=g))
    qkv = qkv.to(dtype).to(DEV)
    pos = torch.tensor([s + i for s, n in zip(starts, news) for i in range(n)], device=DEV)
    return qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:Hq + 2 * H], dev(table), pool, pos


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("Hq,H,D,P,R", [(3, 3, 64, 16, 32), (8, 1, 64, 32, 64), (10, 2, 128, 16, 128), (16, 8, 128, 64, 64), (5, 1, 128, 256, 96), (32, 2, 128, 16, 32)])
def test_append_rope_is_a_rotation_and_an_append(Hq, H, D, P, R, pairs, dtype):
    news, starts = [1, 0, 37, 16, 5, 1], [0, 3, 30, 16, 15, 4099]
    q, k, v, table, pool, pos = rope_case(news, starts, Hq, H, D, P, dtype, R + Hq)
    rope = kda().make_rope_table(4100, R)
    cu, start = cu_of(news).to(DEV), i32(starts)
    want = pool.clone()
    kda().kda_kv4_append(turned(k, rope, pos, pairs), v, cu, start, table, want, k_scale=2.0, v_scale=0.25)
    err = new_err()
    got = pool.clone()
    out = kda().kda_kv4_append_rope(q, k, v, rope, cu, start, table, got, pairs=pairs, k_scale=2.0, v_scale=0.25, dev_err=err)
    assert int(err) == 0 and torch.equal(got, want)
    assert torch.equal(out, turned(q, rope, pos, pairs))
    # angles in fp64: the table's entries, products and sums are off by 2^-24 each
    exact = ref.rotate(q.double().cpu().numpy(), pos.cpu().numpy(), R, pairs)
    size = np.abs(q.double().cpu().numpy()).max(-1, keepdims=True) * 2
    assert (np.abs(out.double().cpu().numpy() - exact) <= np.abs(exact) * HALF_STEP[dtype] * 1.01 + size * 2.0 ** -22 + 2.0 ** -25).all()
    # in place, in the fused projection's output
    mine = q.clone()
    whole = torch.cat([q, k, v], 1)
    view = whole[:, :Hq]
    assert kda().kda_kv4_append_rope(view, k, v, rope, cu, start, table, got, pairs=pairs, q_out=view) is view
    assert torch.equal(view, out) and torch.equal(whole[:, Hq:], torch.cat([k, v], 1)) and torch.equal(q, mine)


def test_append_rope_of_many_tokens():
    """Several heads a thread: every token of a long piece, ragged requests."""
    news, starts = [900, 1, 700, 63], [100, 5, 0, 64]
    q, k, v, table, pool, pos = rope_case(news, starts, 40, 8, 128, 64, BF, 5)
    rope = kda().make_rope_table(1024, 128)
    cu, start = cu_of(news).to(DEV), i32(starts)
    want, got = pool.clone(), pool.clone()
    kda().kda_kv4_append(turned(k, rope, pos, False), v, cu, start, table, want)
    out = kda().kda_kv4_append_rope(q, k, v, rope, cu, start, table, got)
    assert torch.equal(got, want) and torch.equal(out, turned(q, rope, pos, False))


def test_append_rope_of_nan_and_infinity():
    q, k, v, table, pool, pos = rope_case([4], [3], 2, 1, 64, 16, BF, 6)
    k[0, 0, 3], k[1, 0, 40], v[2, 0, 0], q[3, 0, 1] = float("nan"), float("inf"), float("nan"), float("inf")
    rope = kda().make_rope_table(16, 64)
    cu, start = cu_of([4]).to(DEV), i32([3])
    out = kda().kda_kv4_append_rope(q, k, v, rope, cu, start, table, pool)
    assert torch.equal(out.nan_to_num(7e4), turned(q, rope, pos, False).nan_to_num(7e4))
    gk, gv = kda().kda_kv4_gather(cu, start, 4, table, pool)
    rk = turned(k, rope, pos, False)
    # a NaN takes its block with it; an infinity becomes the largest value, and NaN where it meets a sine of zero
    assert torch.equal(gk.isnan(), rk.isnan().unflatten(-1, (-1, 16)).any(-1, keepdim=True).expand(4, 1, 4, 16).flatten(-2))
    assert gv[2, 0, :16].isnan().all() and gv.isnan().sum() == 16


def test_append_rope_skips_what_it_cannot_place():
    Hq, H, D, P = 4, 2, 64, 16
    q, k, v, table, pool, pos = rope_case([2, 2, 2], [14, 30, 1], Hq, H, D, P, BF, 7)
    rope = kda().make_rope_table(32, 64)
    cu = cu_of([2, 2, 2]).to(DEV)
    sentinel = torch.full_like(q.contiguous(), 5.0)
    # request 0's second page is gone, request 1 passes the table of angles, of the last request only one token is there
    table[0, 0] = 10 ** 6
    cu[3] = 5
    err, got, out = new_err(), pool.clone(), sentinel.clone()
    kda().kda_kv4_append_rope(q, k, v, rope, cu, i32([14, 31, 1]), table, got, q_out=out, dev_err=err)
    assert int(err) == 4 | 32
    at = torch.tensor([14, 15, 31, 31, 1], device=DEV)
    want = turned(q[:5], rope, at, False)
    want[3] = 0
    assert torch.equal(out[:5], want) and torch.equal(out[5], sentinel[5])
    after = pool.clone()
    kda().kda_kv4_append(turned(k, rope, torch.tensor([14, 15, 31, 31, 1, 1], device=DEV), False)[[2, 4]], v[[2, 4]], cu_of([0, 1, 1]).to(DEV),
                         i32([14, 31, 1]), table, after)
    assert torch.equal(got, after)


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------

def records_of(pool, row, length, P):
    """The oracle's records of a row's pages, by head: [(hi, lo, e)] per page."""
    k, _ = kv4.load(pool, row, length, P)
    return [ref.page_bounds(k[a:a + P]) for a in range(0, length, P)]


def packed(record):
    hi, lo, e = record
    out = np.zeros((hi.shape[0], 2 * hi.shape[1] + 16), np.int8)
    out[:, :hi.shape[1]], out[:, hi.shape[1]:2 * hi.shape[1]], out[:, 2 * hi.shape[1]] = hi, lo, e
    return out


@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 16, 1), (128, 64, 2), (64, 256, 1), (128, 32, 9), (64, 128, 2)])
def test_bounds_are_the_oracles(D, P, H):
    lens, news = [1, P, P + 1, 5, 2 * P + 7, 0, 3 * P], [1, P, 2, 5, 2 * P + 7, 0, 1]
    pool, table = make_cache(lens, H, D, P, 11, strength=2.0)
    pool[table[3, 0], 0, 0, :8 * D] = 0x70                     # equal channels
    pool[table[0, 0], 0, 0, :D] = 0                             # all zeros: token 0's codes lie there
    pool[table[0, 0], 0, 0, 0:8 * D] = 0
    pool[table[4, 1], H - 1, 0, 8 * D + 3] = 0x7f              # a NaN among the scales
    bounds = torch.full((len(pool), H, 2 * D + 16), 77, dtype=torch.int8, device=DEV)
    want = bounds.cpu().numpy().copy()
    for b, (n, l) in enumerate(zip(news, lens)):
        rec = records_of(pool, table[b], l, P)
        for j in range((l - n) // P, -(-l // P) if n else 0):
            want[table[b, j]] = packed(rec[j])
    err = new_err()
    start = i32([l - n for l, n in zip(lens, news)])
    kda().kda_kv4_bounds(cu_of(news).to(DEV), start, sum(news), dev(table), dev(pool), bounds, dev_err=err)
    assert int(err) == 0
    got = bounds.cpu().numpy()
    assert (got[table[4, 1], H - 1, 2 * D]) == 127 and np.array_equal(got, want)


def test_bounds_of_long_prompts():
    """Slices of several tokens: each page once, whatever its place in the batch."""
    lens, news = [700, 333, 64], [700, 300, 33]
    pool, table = make_cache(lens, 2, 64, 16, 12)
    bounds = kda().make_kv4_bounds(len(pool), 2, 64)
    want = bounds.cpu().numpy().copy()
    for b, (n, l) in enumerate(zip(news, lens)):
        rec = records_of(pool, table[b], l, 16)
        for j in range((l - n) // 16, -(-l // 16)):
            want[table[b, j]] = packed(rec[j])
    kda().kda_kv4_bounds(cu_of(news).to(DEV), i32([l - n for l, n in zip(lens, news)]), sum(news), dev(table), dev(pool), bounds)
    assert np.array_equal(bounds.cpu().numpy(), want)


def test_bounds_skip_what_they_cannot_place():
    pool, table = make_cache([32, 32], 1, 64, 16, 13)
    bounds = torch.full((len(pool), 1, 144), 9, dtype=torch.int8, device=DEV)
    for starts, tab, bit in (([-3, 200], table, 4), ([0, 0], np.where(table >= 0, len(pool), table), 32), ([0, 0], np.full_like(table, -2), 32)):
        err = new_err()
        kda().kda_kv4_bounds(cu_of([2, 2]).to(DEV), i32(starts), 4, dev(tab), dev(pool), bounds, dev_err=err)
        assert int(err) == bit and (bounds == 9).all()
    err = new_err()                                             # tokens behind the last request
    kda().kda_kv4_bounds(cu_of([0, 0]).to(DEV), i32([0, 0]), 3, dev(table), dev(pool), bounds, dev_err=err)
    assert int(err) == 4 and (bounds == 9).all()


# ---------------------------------------------------------------------------
# picks
# ---------------------------------------------------------------------------

def all_bounds(pool, table, lens, P):
    H, D = pool.shape[1], pool.shape[3] // 18
    out = np.full((len(pool), H, 2 * D + 16), -1, np.int8)
    for b, l in enumerate(lens):
        for j, rec in enumerate(records_of(pool, table[b], l, P)):
            out[table[b, j]] = packed(rec)
    return out


def random_bounds(lens, H, D, P, seed, equal=False):
    """Records and a table without a pool behind them: units differ by page, few values where `equal`."""
    rng = np.random.default_rng(seed)
    need = [-(-n // P) for n in lens]
    pages = sum(need) + 2
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    order = rng.permutation(pages)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    lo = rng.integers(-127, 128, (pages, H, D))
    hi = np.maximum(lo, rng.integers(-127, 128, (pages, H, D)))
    if equal:
        hi, lo = hi * 0 + rng.integers(0, 3, (pages, H, 1)), lo * 0
    rec = np.zeros((pages, H, 2 * D + 16), np.int8)
    rec[..., :D], rec[..., D:2 * D] = hi, lo
    rec[..., 2 * D] = 0 if equal else rng.integers(-3, 2, (pages, H))
    return rec, table


def picks_of(q, news, lens, rec, table, P, count, first, recent):
    H, D = rec.shape[1], q.shape[2]
    G = q.shape[1] // H
    x = q.double().cpu().numpy()
    r64 = rec.astype(int)
    out, t = np.zeros((len(x), H, count), np.int32), 0
    for n, l, row in zip(news, lens, table):
        for i in range(n):
            for h in range(H):
                rows = [None if not 0 <= p < len(rec) else (r64[p, h, :D], r64[p, h, D:2 * D], r64[p, h, 2 * D]) for p in row]
                out[t, h] = ref.pick(x[t, h * G:(h + 1) * G], l - n + i, rows, P, count, first, recent)
            t += 1
    return out


def pick(q, news, lens, rec, table, P, count, first, recent, **kw):
    err = new_err()
    got = kda().kda_kv4_pick(q.to(DEV), cu_of(news).to(DEV), max(news + [1]), i32(lens), dev(table), dev(rec), P, count, first=first,
                             recent=recent, dev_err=err, **kw)
    return got.cpu().numpy(), int(err)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("news,lens,Hq,H,D,P,count,first,recent", [
    ([1], [700], 8, 1, 128, 16, 8, 1, 2),
    ([1, 1, 0, 1, 1], [1, 16, 5, 333, 4000], 12, 4, 128, 16, 5, 0, 1),
    ([1, 1], [900, 2500], 9, 9, 64, 32, 11, 2, 3),
    ([3, 8, 11, 0, 1], [3, 900, 640, 9, 100], 16, 2, 128, 32, 4, 1, 1),
    ([40, 1, 17], [600, 900, 17], 6, 3, 64, 16, 7, 0, 7),
    ([5], [4097], 16, 1, 64, 256, 3, 0, 2),
    ([2, 2], [40000, 9000], 4, 2, 64, 16, 64, 1, 4),            # 2500 pages: a CTA a row
    ([1], [140000], 4, 1, 64, 16, 33, 1, 1),                    # 8750 pages
])
def test_picks_are_the_oracles(news, lens, Hq, H, D, P, count, first, recent, dtype):
    q = packed_q(news, Hq, D, dtype, 3, strength=2.0, extra=1)[:, :Hq]
    for equal in (False, True):
        rec, table = random_bounds(lens, H, D, P, 4, equal)
        rec[0, 0, 2 * D] = 127
        got, err = pick(q, news, lens, rec, table, P, count, first, recent)
        assert err == 0 and np.array_equal(got, picks_of(q, news, lens, rec, table, P, count, first, recent))


def test_picks_in_tables_wider_than_every_kernel():
    """The kernel goes by the table's width: one request of 300 pages in tables of 256 to 40000."""
    lens, count = [300 * 16 - 5], 20
    rec, table = random_bounds(lens, 2, 64, 16, 5)
    q = packed_q([3], 4, 64, BF, 6)
    want = picks_of(q, [3], lens, rec, table, 16, count, 1, 1)
    for width in (301, 1024, 1025, 2048, 2049, 8192, 8193, 32768, 32769, 40000):
        wide = np.full((1, width), -1, np.int32)
        wide[:, :table.shape[1]] = table
        got, err = pick(q, [3], lens, rec, wide, 16, count, 1, 1)
        assert err == 0 and np.array_equal(got, want), width
    rec, table = random_bounds([33000 * 16], 1, 64, 16, 7)      # and one that needs it
    q = packed_q([1], 1, 64, BF, 8)
    got, err = pick(q, [1], [33000 * 16], rec, table, 16, 100, 1, 1)
    r = rec[table[0, :33000], 0].astype(np.int64)
    u, d = ref.asked(q[0].double().numpy())
    s = ((r[:, :64] * u - r[:, 64:128] * d).sum(-1) * 2.0 ** r[:, 128])
    s[0], s[-1] = np.inf, np.inf
    assert np.array_equal(got[0, 0], np.sort(np.lexsort((np.arange(33000), -s))[:100]))


@pytest.mark.parametrize("H,news", [(8, [1] * 80), (2, [2] * 80)])
def test_picks_of_many_requests_in_a_wide_table(H, news):
    """More chunks of pages than CTAs are launched: a CTA takes several runs of a long row."""
    rng = np.random.default_rng(13)
    lens = [int(x) for x in rng.integers(2, 400, 80)]
    lens[3], lens[40], lens[79] = 2099 * 16, 700 * 16 - 3, 1000 * 16 + 1
    rec, table = random_bounds(lens, H, 64, 16, 14)
    q = packed_q(news, 2 * H, 64, BF, 15)
    got, err = pick(q, news, lens, rec, table, 16, 9, 1, 2)
    assert err == 0 and np.array_equal(got, picks_of(q, news, lens, rec, table, 16, 9, 1, 2))


def test_picks_of_queries_that_are_not_numbers():
    lens = [640, 640, 640, 640]
    rec, table = random_bounds(lens, 1, 64, 16, 9)
    q = packed_q([1, 1, 1, 1], 2, 64, BF, 10)
    q[0, 0, 3], q[1, 1, 5], q[2] = float("nan"), float("inf"), 0
    q[3] = q[3] * 2.0 ** -110
    got, err = pick(q, [1] * 4, lens, rec, table, 16, 6, 1, 2)
    assert err == 0 and np.array_equal(got, picks_of(q, [1] * 4, lens, rec, table, 16, 6, 1, 2))
    assert got[:3, 0].tolist() == [[0, 1, 2, 3, 38, 39]] * 3


def test_picks_pass_by_pages_that_are_not_there_and_skip_bad_requests():
    lens = [640, 640, 640]
    rec, table = random_bounds(lens, 2, 64, 16, 11)
    table[0, 3], table[0, 9] = -1, len(rec)
    q = packed_q([1, 1, 1], 4, 64, FP, 12)
    picked = torch.full((3, 2, 8), 55, dtype=torch.int32, device=DEV)
    got, err = pick(q, [1, 1, 1], [640, 10 ** 6, 640], rec, table, 16, 8, 1, 1, picked=picked)
    want = picks_of(q, [1, 1, 1], lens, rec, table, 16, 8, 1, 1)
    assert err == 4 | 32 and np.array_equal(got[[0, 2]], want[[0, 2]]) and (got[1] == 55).all()
    assert not set(got[0].flatten()) & {3, 9}
    # wanted all but one of the candidates: the missing ones come last, the lower first
    got, err = pick(q[:1], [1], [640], rec, table[:1], 16, 39, 1, 1)
    assert err == 32 and got[0, 0].tolist() == [p for p in range(40) if p != 9]
    # rows behind the last request, tokens at negative positions, a request with more tokens than max_q
    picked.fill_(55)
    cu = cu_of([1, 1]).to(DEV)
    kda().kda_kv4_pick(q.to(DEV), cu, 1, i32([640, 0]), dev(table[1:]), dev(rec), 16, 8, picked=picked)
    assert (picked[1] == -1).all() and (picked[2] == 55).all() and (picked[0] != 55).all()
    err = new_err()
    kda().kda_kv4_pick(q.to(DEV), cu_of([2, 1]).to(DEV), 1, i32([640, 640]), dev(table[1:]), dev(rec), 16, 8, picked=picked.fill_(55), dev_err=err)
    assert int(err) == 4 and (picked[:2] == 55).all() and (picked[2] != 55).all()


# ---------------------------------------------------------------------------
# attention over picked pages
# ---------------------------------------------------------------------------

def expected_picked(q, news, lens, pool, table, picked, P, scale, k_scale=1.0, v_scale=1.0):
    """As kv4_testutil.expected, over the picked pages."""
    outs, t = [], 0
    for b, n in enumerate(news):
        k, v = kv4.load(pool, np.maximum(table[b], 0), lens[b], P, k_scale, v_scale)
        top = np.nanmax(np.abs(v)) if v.size and not np.isnan(v).all() else 0.0
        for i in range(n):
            o, lse, a, big = ref.attention_picked(q[t].double().numpy(), k, v, lens[b] - n + i, picked[t], P, scale)
            es = 2 * q.shape[-1] * 2.0 ** -23 * big + 2.0 ** -20
            bo = a * (2.0 ** -11 + 4 * es[..., None]) + 2.0 ** -30 * max(1, lens[b]) * top
            bl = es + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
            outs.append((o, lse, bo, bl))
            t += 1
    return [np.stack(x) for x in zip(*outs)]


def some_picks(news, lens, H, P, count, seed, order=True):
    rng = np.random.default_rng(seed)
    out, t = np.full((sum(news), H, count), -1, np.int32), 0
    for n, l in zip(news, lens):
        for i in range(n):
            pos = l - n + i
            if pos >= 0:
                own = pos // P
                c = min(count, own + 1)
                for h in range(H):
                    r = rng.permutation(own)[:c - 1]
                    out[t, h, :c] = list(np.sort(r) if order else r) + [own]
            t += 1
    return out


def attend(q, news, lens, table, picked, pool, ws, heads, **kw):
    err = new_err()
    o, lse = kda().kda_kv4_attention_picked(q.to(DEV)[:, :heads], cu_of(news).to(DEV), max(news), i32(lens), dev(table), dev(picked), dev(pool),
                                            workspace=ws, dev_err=err, **kw)
    torch.cuda.synchronize()
    return o, lse, int(err)


SHAPES = [
    # news, lens, Hq, Hkv, D, P, count
    ([1], [1], 1, 1, 64, 16, 1),
    ([1], [700], 8, 1, 128, 16, 9),
    ([1, 1, 0, 1], [33, 16, 5, 333], 12, 4, 128, 16, 6),
    ([1] * 5, [900, 17, 64, 65, 400], 10, 2, 64, 32, 7),
    ([1, 1], [2000, 513], 16, 1, 128, 64, 5),
    ([1], [1500], 40, 2, 128, 16, 40),                          # 20 rows a kv head
    ([3, 8, 1], [3, 600, 77], 8, 2, 128, 32, 4),
    ([9], [1100], 3, 3, 64, 256, 3),
    ([20, 2], [300, 40], 16, 2, 64, 16, 11),
    ([1], [4000], 4, 2, 128, 128, 64),                          # more places than pages
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("news,lens,Hq,H,D,P,count", SHAPES)
def test_attention_picked(news, lens, Hq, H, D, P, count, dtype, ws):
    pool, table = make_cache(lens, H, D, P, 21)
    q = packed_q(news, Hq, D, dtype, 22, strength=1.5, extra=2)
    for order in (True, False):
        picked = some_picks(news, lens, H, P, count, 23, order)
        o, lse, err = attend(q, news, lens, table, picked, pool, ws, Hq, k_scale=0.5, v_scale=2.0)
        assert err == 0
        check(o, lse, expected_picked(q[:, :Hq], news, lens, pool, table, picked, P, D ** -0.5, 0.5, 2.0), dtype)


def test_all_pages_are_dense_attention(ws):
    news, lens, H, D, P = [1, 4, 1], [500, 130, 16], 2, 128, 32
    pool, table = make_cache(lens, H, D, P, 24)
    q = packed_q(news, 8, D, BF, 25)
    picked = np.broadcast_to(np.where(np.arange(16) * P < 500, np.arange(16), -1), (6, H, 16)).astype(np.int32).copy()
    o, lse, err = attend(q, news, lens, table, picked, pool, ws, 8)
    dense = kda().kda_kv4_attention(q.to(DEV), cu_of(news).to(DEV), 4, i32(lens), dev(table), dev(pool), workspace=ws)
    assert err == 0 and (o.float() - dense[0].float()).abs().max() <= 2.0 ** -7 and (lse - dense[1]).abs().max() < 1e-5


def test_entries_that_are_missing_or_wrong(ws):
    news, lens, H, D, P = [1, 1, 1], [200, 200, 200], 2, 64, 16
    pool, table = make_cache(lens, H, D, P, 26)
    q = packed_q(news, 4, D, BF, 27)
    picked = some_picks(news, lens, H, P, 5, 28)
    picked[0, 0, 1] = -1                                        # fewer pages
    picked[0, 1] = -1                                           # none: the row sees nothing
    o, lse, err = attend(q, news, lens, table, picked, pool, ws, 4)
    assert err == 0 and not o[0, 2:].any() and (lse[0, 2:] == -np.inf).all()
    check(o, lse, expected_picked(q, news, lens, pool, table, picked, P, D ** -0.5), BF)
    bad = picked.copy()
    bad[1, 0, 0], bad[1, 1, 2], bad[2, 0, 4], bad[2, 1, 3] = 13, -7, 3, 1 << 30
    keep = picked.copy()
    keep[1, 0, 0], keep[1, 1, 2], keep[2, 0, 4], keep[2, 1, 3] = -1, -1, -1, -1
    o, lse, err = attend(q, news, lens, table, bad, pool, ws, 4)
    assert err == 32
    check(o, lse, expected_picked(q, news, lens, pool, table, keep, P, D ** -0.5), BF)
    gone = table.copy()
    gone[0, picked[0, 0, 0]] = len(pool)                        # a page that the table does not have
    keep = picked.copy()
    keep[0, 0, 0] = -1
    o, lse, err = attend(q, news, lens, gone, picked, pool, ws, 4)
    assert err == 32
    check(o, lse, expected_picked(q, news, lens, pool, table, keep, P, D ** -0.5), BF)


def test_rows_that_are_no_ones_and_bad_requests(ws):
    news, lens, H, D, P = [1, 1, 2], [200, 90, 40], 1, 128, 16
    pool, table = make_cache(lens, H, D, P, 29)
    q = packed_q([1] * 6, 8, D, FP, 30)                         # two rows behind the last request
    picked = np.concatenate([some_picks(news, lens, H, P, 4, 31), np.full((2, H, 4), 9, np.int32)])
    o, lse = torch.full((6, 8, D), 3.0, dtype=FP, device=DEV), torch.full((6, 8), 3.0, device=DEV)
    err = new_err()
    kda().kda_kv4_attention_picked(q.to(DEV), cu_of(news).to(DEV), 2, i32([200, -4, 40]), dev(table), dev(picked), dev(pool), o=o, lse=lse,
                                   workspace=ws, dev_err=err)
    assert int(err) == 4 and (o[[1, 4, 5]] == 3).all() and (lse[[1, 4, 5]] == 3).all()
    rows = [0, 2, 3]
    check(o[rows], lse[rows], expected_picked(q[rows], [1, 2], [200, 40], pool, table[[0, 2]], picked[rows], P, D ** -0.5), FP)
    # a token before its cache begins sees nothing
    o, lse, err = attend(q[:2], [2], [1], table[:1], picked[:2] * 0, pool, ws, 8)
    assert err == 0 and not o[0].any() and (lse[0] == -np.inf).all() and torch.isfinite(lse[1]).all()


def test_what_is_not_picked_has_no_influence(ws):
    """NaN scales and codes in other pages, and behind the token in its own, change nothing."""
    news, lens, H, D, P = [1, 3], [300, 150], 2, 128, 32
    pool, table = make_cache(lens, H, D, P, 32)
    q = packed_q(news, 8, D, BF, 33)
    picked = some_picks(news, lens, H, P, 3, 34)
    o, lse, err = attend(q, news, lens, table, picked, pool, ws, 8)
    for h in range(H):
        seen = {int(table[b, p]) for t, b in enumerate([0, 1, 1, 1]) for p in picked[t, h] if p >= 0}
        for page in range(len(pool)):
            if page not in seen:
                pool[page, h] = 255
    o2, lse2, err2 = attend(q, news, lens, table, picked, pool, ws, 8)
    assert err == err2 == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


def test_nan_in_a_picked_page_reaches_who_sees_it(ws):
    news, lens, H, D, P = [2], [66], 1, 64, 32
    pool, table = make_cache(lens, H, D, P, 35)
    D8 = 8 * D
    pool[table[0, 2], 0, 0, D8 + 1 * 4 + 2] = 0x7f             # K of position 65: only the second token sees it
    q = packed_q(news, 4, D, BF, 36)
    picked = some_picks(news, lens, H, P, 3, 37)
    o, lse, err = attend(q, news, lens, table, picked, pool, ws, 4)
    assert err == 0 and torch.isfinite(o[0]).all() and o[1].isnan().all() and lse[1].isnan().all()


# ---------------------------------------------------------------------------
# one layer's step, and streams and graphs
# ---------------------------------------------------------------------------

class Layer:
    """One layer's memory, and its step from the residual to the attention's output."""

    def __init__(self, lens, news, P, count, seed=0):
        self.Hq, self.H, self.D, self.P, self.C, self.count = 8, 2, 128, P, 1024, count
        self.news, self.lens = news, lens
        g = torch.Generator(device=DEV).manual_seed(seed)
        T, M = sum(news), -(-max(lens) // P) + 1
        need = [-(-l // P) for l in lens]
        self.pages = sum(need)
        self.table = torch.full((len(lens), M), -1, dtype=torch.int32, device=DEV)
        order = torch.randperm(self.pages, generator=g, device=DEV).int()
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.pool = kda().make_kv4_pool(self.pages, P, self.H, self.D)
        self.bounds = kda().make_kv4_bounds(self.pages, self.H, self.D)
        self.rope = kda().make_rope_table(max(lens), self.D)
        self.cu, self.start, self.klens = cu_of(news).to(DEV), i32([l - n for l, n in zip(lens, news)]), i32(lens)
        self.x = torch.randn(T, self.C, generator=g, device=DEV).to(BF)
        self.res = torch.randn(T, self.C, generator=g, device=DEV).to(BF)
        self.w = torch.rand(self.C, generator=g, device=DEV).to(BF)
        self.proj = (torch.randn(self.C, (self.Hq + 2 * self.H) * self.D, generator=g, device=DEV) * 0.05).to(BF)
        self.err = new_err()
        old = [l - n for l, n in zip(lens, news)]               # what was there before
        kv = torch.randn(sum(old), 2, self.H, self.D, generator=g, device=DEV).to(BF)
        cu = cu_of(old).to(DEV)
        zero = torch.zeros_like(self.start)
        kda().kda_kv4_append(kv[:, 0], kv[:, 1], cu, zero, self.table, self.pool)
        kda().kda_kv4_bounds(cu, zero, sum(old), self.table, self.pool, self.bounds)
        self.ws = kda().make_kv4_workspace()
        self.pick_ws = torch.empty(kda().kv4_pick_workspace_bytes(T, self.H, M), dtype=torch.uint8, device=DEV)

    def step(self, **kw):
        k = kda()
        y, s, h = k.kda_add_rmsnorm(self.x, self.res, self.w, scales="block", **kw)
        y = (y.float().unflatten(-1, (-1, 128)) * s[..., None]).flatten(-2).to(BF)
        qkv = (y @ self.proj).unflatten(-1, (-1, self.D))
        q, kk, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.H], qkv[:, self.Hq + self.H:]
        q = k.kda_kv4_append_rope(q, kk, v, self.rope, self.cu, self.start, self.table, self.pool, dev_err=self.err, **kw)
        k.kda_kv4_bounds(self.cu, self.start, q.shape[0], self.table, self.pool, self.bounds, dev_err=self.err, **kw)
        picked = k.kda_kv4_pick(q, self.cu, max(self.news), self.klens, self.table, self.bounds, self.P, self.count, workspace=self.pick_ws,
                                dev_err=self.err, **kw)
        o, lse = k.kda_kv4_attention_picked(q, self.cu, max(self.news), self.klens, self.table, picked, self.pool, workspace=self.ws,
                                            dev_err=self.err, **kw)
        return q, picked, o, lse

    def check(self, q, picked, o, lse):
        assert int(self.err) == 0
        pool, table = self.pool.cpu().numpy(), self.table.cpu().numpy()
        rec = all_bounds(pool, table, self.lens, self.P)
        assert np.array_equal(self.bounds.cpu().numpy(), rec)
        want = picks_of(q, self.news, self.lens, rec, table, self.P, self.count, 1, 1)
        assert np.array_equal(picked.cpu().numpy(), want)
        check(o, lse, expected_picked(q.cpu(), self.news, self.lens, pool, table, want, self.P, self.D ** -0.5), BF)


@pytest.mark.parametrize("news,lens,P,count", [([1] * 4, [700, 20, 333, 1], 16, 6), ([3, 1, 5], [260, 90, 5], 32, 3), ([50, 30], [120, 400], 16, 4)])
def test_a_layers_step(news, lens, P, count):
    m = Layer(lens, news, P, count)
    m.check(*m.step())


def test_a_step_in_graphs_that_take_turns():
    """Two layers' captured steps with workspaces of their own run on two streams, and each again with new inputs."""
    a, b = Layer([500, 77], [1, 1], 16, 5, 1), Layer([90, 400, 33], [2, 3, 1], 32, 3, 2)
    graphs = []
    for m in (a, b):
        m.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m.step()
        graphs.append((g, out))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for turn in range(3):
        for m in (a, b):
            m.x.normal_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for m, (_, out) in zip((a, b), graphs):
            m.check(*out)


def test_graphs_that_share_workspaces_run_one_after_the_other():
    a, b = Layer([500, 77], [1, 1], 16, 5, 6), Layer([90, 400, 33], [2, 3, 1], 32, 3, 7)
    b.ws, b.pick_ws = a.ws, torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    a.pick_ws = b.pick_ws
    graphs = []
    for m in (a, b):
        m.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = m.step()
        graphs.append((g, out))
    for turn in range(3):
        for m in (a, b):
            m.x.normal_()
        for g, _ in graphs[::-1] if turn % 2 else graphs:
            g.replay()
        torch.cuda.synchronize()
        for m, (_, out) in zip((a, b), graphs):
            m.check(*out)


def test_pages_past_4_gigabytes(ws):
    """The same step with its pages at the far end of a pool of 6 GB."""
    k, H, D, P, pages = kda(), 8, 128, 256, 20000
    far = torch.zeros(pages, H, P // 16, 18 * D, dtype=torch.uint8, device=DEV)
    near = far[:12].clone()
    g = torch.Generator(device=DEV).manual_seed(8)
    T = 12 * P
    qkv = torch.randn(T, 24, D, generator=g, device=DEV).to(BF)
    rope, cu, start, lens = k.make_rope_table(T, D), i32([0, T]), i32([0]), i32([T])
    outs = []
    for pool, table in ((far, torch.arange(pages - 12, pages, dtype=torch.int32, device=DEV)[None]), (near, torch.arange(12, dtype=torch.int32, device=DEV)[None])):
        err = new_err()
        bounds = k.make_kv4_bounds(len(pool), H, D)
        q = k.kda_kv4_append_rope(qkv[:, :8], qkv[:, 8:16], qkv[:, 16:], rope, cu, start, table, pool, dev_err=err)
        k.kda_kv4_bounds(cu, start, T, table, pool, bounds, dev_err=err)
        picked = k.kda_kv4_pick(q[-3:], i32([0, 3]), 3, lens, table, bounds, P, 5, dev_err=err)
        o, lse = k.kda_kv4_attention_picked(q[-3:], i32([0, 3]), 3, lens, table, picked, pool, workspace=ws, dev_err=err)
        assert int(err) == 0
        outs.append((q, pool[table[0].long()], bounds[table[0].long()], picked, o, lse))
    assert not far[:pages - 12].any()
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_a_step_on_another_stream_is_the_same():
    a, b = Layer([500, 77], [1, 1], 16, 5, 3), Layer([500, 77], [1, 1], 16, 5, 3)
    want = a.step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.step()
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    assert torch.equal(a.pool, b.pool) and torch.equal(a.bounds, b.bounds)


def test_the_same_call_again_is_the_same(ws):
    m = Layer([3000, 2000, 77, 1], [1, 1, 1, 1], 16, 64, 4)
    first = m.step()
    for _ in range(3):
        for x, y in zip(first, m.step()):
            assert torch.equal(x, y)


def test_the_bindings_refuse_what_the_library_would_misread(ws):
    k = kda()
    m = Layer([100, 40], [1, 1], 16, 3, 5)
    q = torch.zeros(2, 8, 128, dtype=BF, device=DEV)
    kv = q[:, :2].contiguous()
    picked = torch.zeros(2, 2, 3, dtype=torch.int32, device=DEV)
    rope = lambda **c: k.kda_kv4_append_rope(*[c.get(n, d) for n, d in dict(q=q, k=kv, v=kv, rope=m.rope, cu=m.cu, start=m.start, table=m.table, pool=m.pool).items()],
                                             **{n: c[n] for n in c if n in ("q_out",)})
    pick_ = lambda **c: k.kda_kv4_pick(*[c.get(n, d) for n, d in dict(q=q, cu=m.cu, max_q=1, lens=m.klens, table=m.table, bounds=m.bounds, page=16, count=3).items()],
                                       **{n: c[n] for n in c if n in ("first", "recent", "picked", "workspace")})
    att = lambda **c: k.kda_kv4_attention_picked(*[c.get(n, d) for n, d in dict(q=q, cu=m.cu, max_q=1, lens=m.klens, table=m.table, picked=picked, pool=m.pool).items()],
                                                 workspace=c.get("workspace", ws))
    bnd = lambda **c: k.kda_kv4_bounds(*[c.get(n, d) for n, d in dict(cu=m.cu, start=m.start, T=2, table=m.table, pool=m.pool, bounds=m.bounds).items()])
    before = m.pool.clone(), m.bounds.clone()
    for bad in (lambda: rope(q=q.float()), lambda: rope(k=kv.half()), lambda: rope(v=kv[:1]), lambda: rope(rope=m.rope.double()), lambda: rope(rope=m.rope[:, :48].contiguous()),
                lambda: rope(rope=m.rope.cpu()), lambda: rope(q_out=q[:1]), lambda: rope(pool=m.pool[:, :1].contiguous()), lambda: rope(cu=m.cu[:2]), lambda: rope(q=q[..., ::2]),
                lambda: rope(q=q.transpose(0, 1)), lambda: pick_(q=q[:, :7]), lambda: pick_(bounds=m.bounds[..., :-16]), lambda: pick_(bounds=m.bounds.view(torch.uint8)),
                lambda: pick_(count=0), lambda: pick_(first=3), lambda: pick_(recent=0), lambda: pick_(page=20), lambda: pick_(picked=picked.long()),
                lambda: pick_(workspace=m.pick_ws[:16]), lambda: pick_(lens=m.klens.long()), lambda: pick_(max_q=0), lambda: att(picked=picked[:1]),
                lambda: att(picked=picked[..., :0]), lambda: att(picked=picked.transpose(0, 1)), lambda: att(q=q[:, :7]), lambda: att(workspace=ws[:64]),
                lambda: att(picked=picked.cpu()), lambda: bnd(bounds=m.bounds[:1]), lambda: bnd(T=-1), lambda: bnd(cu=m.cu.cpu()), lambda: bnd(T=1 << 33)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()
    torch.cuda.synchronize()
    assert torch.equal(m.pool, before[0]) and torch.equal(m.bounds, before[1])
    assert k.kda_kv4_pick(q[:0], i32([0, 0, 0]), 1, m.klens, m.table, m.bounds, 16, 3).shape == (0, 2, 3)
    assert k.kda_kv4_attention_picked(q[:0], i32([0, 0, 0]), 1, m.klens, m.table, picked[:0], m.pool)[0].shape == (0, 8, 128)

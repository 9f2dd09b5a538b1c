"""The paged 4-bit cache on the GPU: append and gather bit for bit, attention within the bounds
that kv4_testutil.expected derives, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from kv4_testutil import check, cu_of, expected, make_cache, packed_q
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


def attend(pool, table, news, lens, q, heads, ws, window=0, scale=None, **kw):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qd = q.to(DEV)[:, :heads]
    o, lse = kda().kda_kv4_attention(qd, cu_of(news).to(DEV), max(news), dev(lens, torch.int32), dev(table), dev(pool),
                                     scale=scale, window=window, workspace=ws, dev_err=err, **kw)
    torch.cuda.synchronize()
    return o, lse, int(err)


# ---------------------------------------------------------------------------
# append and gather
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D,P,H", [(64, 16, 3), (128, 16, 1), (128, 64, 2), (64, 256, 8)])
def test_append_is_the_oracles(dtype, D, P, H):
    news, starts = [1, 0, 37, 16, 5], [0, 3, 30, 16, 15]
    lens = [a + n for a, n in zip(starts, news)]
    pool, table = make_cache([0] * 5, H, D, P, 1, spare=0)
    pages = sum(-(-n // P) for n in lens) + 2
    pool = np.random.default_rng(2).integers(0, 256, (pages, H, P // 16, 18 * D), dtype=np.uint8)
    table = np.full((5, max(-(-n // P) for n in lens) + 1), -1, np.int32)
    order = iter(np.random.default_rng(3).permutation(pages))
    for b, n in enumerate(lens):
        for j in range(-(-n // P)):
            table[b, j] = next(order)
    T = sum(news)
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn(T, 2 * H + 1, D, generator=g) * torch.exp(torch.randn(T, 2 * H + 1, 1, generator=g) * 2)
    qkv = qkv.to(dtype)
    qkv[3, 0, :16] = 0
    qkv[4, 0, 5] = float("nan")
    qkv[5, 1, 7] = float("inf")
    qkv[6, 0, 3] = 60000.0 if dtype == FP else 1e30
    qkv[7, 0, :16] = torch.linspace(-6, 6, 16).to(dtype)
    qkv[8, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -2.5, -5, 0, .125, 3]).to(dtype)
    qkv[9, 0, :16] = 1e-3
    k, v = qkv[:, :H], qkv[:, H:2 * H]
    want = pool.copy()
    t = 0
    for b, n in enumerate(news):
        for i in range(n):
            ref.store(want, table[b], starts[b] + i, k[t].double().numpy(), v[t].double().numpy() / 0.25, P)
            t += 1
    d = dev(pool)
    dq = qkv.to(DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (cu_of(news).to(DEV), dev(starts, torch.int32))
    kda().kda_kv4_append(dq[:, :H], dq[:, H:2 * H], *args, dev(table), d, v_scale=0.25, dev_err=err)
    gk, gv = kda().kda_kv4_gather(*args, T, dev(table), d, dtype=dtype, v_scale=0.25, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    got = d.cpu().numpy()
    # a NaN block's codes say nothing: its scale is NaN
    assert (got != want).sum() <= 16, "%d bytes differ" % (got != want).sum()
    t = 0
    for b, n in enumerate(news):
        wk, wv = ref.load(want, table[b], lens[b], P, 1.0, 0.25)
        for i in range(n):
            for x, w in ((gk, wk), (gv, wv)):
                assert np.array_equal(x[t].double().cpu().numpy(), torch.from_numpy(w[starts[b] + i]).to(dtype).double().numpy(),
                                      equal_nan=True)
            t += 1


def test_append_skips_what_it_cannot_place():
    H, D, P = 2, 64, 16
    pool, table = make_cache([16, 16], H, D, P, 5)
    before = pool.copy()
    x = torch.randn(4, H, D, device=DEV).to(BF)
    cu = cu_of([2, 2]).to(DEV)
    for starts, tab, bit in (([16, 100], table, 32 | 4), ([-5, 0], np.where(table >= 0, len(pool), table), 32 | 4)):
        d = dev(pool)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        kda().kda_kv4_append(x, x, cu, dev(starts, torch.int32), dev(tab), d, dev_err=err)
        gk, gv = kda().kda_kv4_gather(cu, dev(starts, torch.int32), 4, dev(tab), d)
        torch.cuda.synchronize()
        assert int(err) == bit and np.array_equal(d.cpu().numpy(), before) and not gk.any() and not gv.any()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

SHAPES = [
    # news, lens, Hq, Hkv, D, P
    ([1], [1], 1, 1, 128, 16),
    ([1, 1, 1, 1, 1, 1], [1, 15, 16, 17, 0, 300], 8, 1, 128, 16),
    ([1, 0, 1, 1], [64, 64, 65, 127], 6, 2, 64, 32),
    ([1] * 9, [5, 700, 3, 1, 90, 33, 1111, 2, 48], 4, 4, 64, 64),
    ([1, 1, 1], [129, 40, 256], 24, 1, 128, 128),
    ([1, 1], [500, 31], 10, 2, 128, 256),
    ([4, 4, 4], [4, 90, 2], 8, 1, 128, 16),
    ([8, 3, 0, 5], [100, 3, 50, 33], 16, 2, 128, 32),
    ([2, 7], [64, 16], 5, 1, 64, 16),
    ([5, 16], [70, 40], 32, 2, 64, 64),
    ([33, 1, 70], [33, 80, 130], 4, 2, 128, 16),
    ([129], [200], 8, 2, 64, 32),
    ([40, 17], [20, 300], 8, 1, 128, 64),
    ([257, 64], [257, 100], 3, 1, 128, 64),
]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("window", [0, 1, 20])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention(ws, shape, window, dtype):
    news, lens, Hq, Hkv, D, P = SHAPES[shape]
    pool, table = make_cache(lens, Hkv, D, P, 10 + shape)
    q = packed_q(news, Hq, D, dtype, shape, 2.0, extra=2 * Hkv)
    o, lse, err = attend(pool, table, news, lens, q, Hq, ws, window)
    assert err == 0
    check(o, lse, expected(q[:, :Hq], news, lens, pool, table, P, window, D ** -0.5), dtype)


@pytest.mark.parametrize("D,P,window,dtype", [(128, 64, 0, BF), (64, 16, 100, FP)])
def test_large_prompts(ws, D, P, window, dtype):
    """Enough rows that a part of the work holds 256 of them; some of the rows against the oracle."""
    news, lens, Hq, Hkv = [700, 1, 599], [900, 77, 599], 64, 8
    pool, table = make_cache(lens, Hkv, D, P, 17)
    ref.store(pool, table[2], 300, np.full((Hkv, D), np.nan), np.full((Hkv, D), np.nan), P)   # rows 300.. of request 2
    q = packed_q(news, Hq, D, dtype, 18, 2.0)
    o, lse, err = attend(pool, table, news, lens, q, Hq, ws, window)
    assert err == 0
    o2, lse2, _ = attend(pool, table, news, lens, q, Hq, ws, window)
    assert torch.equal(o.view(torch.int16), o2.view(torch.int16))
    at = 0
    for b, n in enumerate(news):
        for i in sorted({0, 1, n // 3, n // 2, 299, 300, 399, 400, n - 2, n - 1} & set(range(n))):
            seen = lens[b] - n + i + 1
            t = at + i
            want = expected(q[t:t + 1], [1], [seen], pool, table[b:b + 1], P, window, D ** -0.5)
            check(o[t:t + 1], lse[t:t + 1], want, dtype)
        at += n


@pytest.mark.parametrize("news", [[1, 1, 1], [6, 6, 2], [90, 20, 64]])
def test_scales_of_every_size(ws, news):
    """Tensor scales, large scores (one token takes all), a negative scale, queries near the type's ends."""
    lens, H, D, P = [300, 40, 77], 2, 128, 16
    for strength, qs, scale, ks, vs, dtype in ((1.0, 1.0, -0.2, 1.0, 1.0, BF), (30.0, 8.0, 0.5, 4.0, 0.125, FP),
                                               (1.0, 1e-30, 0.1, 1.0, 1.0, BF), (1.0, 1e30, 1e-30, 1.0, 2.0, BF),
                                               (1.0, 9000.0, 1e-4, 1.0, 1.0, FP), (1.0, 1.0, 0.0, 0.5, 1.0, BF)):
        pool, table = make_cache(lens, H, D, P, 30, k_scale=ks, v_scale=vs, strength=strength)
        q = packed_q(news, 8, D, dtype, 31, qs)
        o, lse, err = attend(pool, table, news, lens, q, 8, ws, 0, scale, k_scale=ks, v_scale=vs)
        assert err == 0
        check(o, lse, expected(q, news, lens, pool, table, P, 0, scale, ks, vs), dtype)


def test_growing_scores(ws):
    """Keys that match the query better and better: the running maximum moves at every tile."""
    D, P, n = 128, 16, 400
    pool, table = make_cache([n, n], 1, D, P, 40)
    unit = np.ones((1, D))
    for pos in range(n):
        ref.store(pool, table[0], pos, unit * (pos / 40), unit * np.sin(pos), P)
        ref.store(pool, table[1], pos, unit * ((n - pos) / 40), unit * np.cos(pos), P)
    for news in ([1, 1], [3, 5], [100, 80]):
        q = packed_q(news, 8, D, BF, 41, 0.01) + 1
        o, lse, err = attend(pool, table, news, [n, n], q, 8, ws)
        assert err == 0
        check(o, lse, expected(q, news, [n, n], pool, table, P, 0, D ** -0.5), BF)


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [4, 4, 4, 4], [80, 70, 90, 66]])
def test_nan_and_infinity_stay_where_they_are(ws, news):
    """A NaN key or value reaches the rows that see it and no others; a masked one reaches none."""
    lens, D, P, H = [100, 100, 100, 100], 64, 16, 2
    pool, table = make_cache(lens, H, D, P, 50)
    bad = np.ones((H, D)) * 0.5
    nan = bad.copy()
    nan[0, 3] = np.nan
    ref.store(pool, table[0], 20, nan, bad, P)          # head 0 of request 0: a NaN key
    ref.store(pool, table[1], 97, bad, nan, P)          # a NaN value near the end of request 1
    q = packed_q(news, 4, D, BF, 51)
    q[sum(news[:2]), 2, 5] = float("nan")               # one query row of request 2
    q[sum(news[:3]), 0, 5] = float("inf")               # scores of both infinities: NaN
    for window in (0, 30):
        o, lse, err = attend(pool, table, news, lens, q, 4, ws, window)
        assert err == 0
        want = expected(q, news, lens, pool, table, P, window, D ** -0.5)
        got = o.double().cpu().numpy()
        assert np.isnan(want[0]).any() and not np.isnan(want[0]).all()
        # a NaN value is one block of 16 channels; the others of that row stay numbers
        assert np.array_equal(np.isnan(got), np.isnan(want[0]))
        fine = ~np.isnan(want[0])
        assert (np.abs(got - want[0])[fine] <= (want[2] + 2.0 ** -8 * np.abs(want[0]) + 1e-7)[fine]).all()


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [3, 3, 3, 3], [70, 70, 70, 70]])
def test_bad_lengths_and_pages(ws, news):
    lens, D, P, H, Hq = [100, 90, 80, 100], 128, 16, 1, 8
    pool, table = make_cache(lens, H, D, P, 60, max_pages=7)
    q = packed_q(news, Hq, D, BF, 61)
    good = attend(pool, table, news, lens, q, Hq, ws)
    cut = np.cumsum([0] + news)
    # a length past the table, or a negative one: those rows are not written, the others are
    for bad_len in (8 * P + 1, -1, 2 ** 31 - 1):
        o = torch.full((sum(news), Hq, D), 7.0, dtype=BF, device=DEV)
        lse = torch.full((sum(news), Hq), 7.0, device=DEV)
        _, _, err = attend(pool, table, news, [100, bad_len, 80, 100], q, Hq, ws, o=o, lse=lse)
        assert err == 4 and (o[cut[1]:cut[2]] == 7).all() and (lse[cut[1]:cut[2]] == 7).all()
        for b in (0, 2, 3):
            assert torch.equal(o[cut[b]:cut[b + 1]], good[0][cut[b]:cut[b + 1]])
    # a page out of range: its tokens are left out, and the flag says so
    for page in (-1, len(pool), 2 ** 31 - 1):
        t = table.copy()
        t[2, 0] = page
        o, lse, err = attend(pool, t, news, lens, q, Hq, ws)
        assert err == 32
        for b in (0, 1, 3):
            assert torch.equal(o[cut[b]:cut[b + 1]], good[0][cut[b]:cut[b + 1]])
        if news[2] < 60:
            k, v = ref.load(pool, table[2], lens[2], P)
            wo = ref.attention(q[cut[2]:cut[3]].double().numpy(), k[16:], v[16:], 0, D ** -0.5)[0]
            assert np.abs(o[cut[2]:cut[3]].double().cpu().numpy() - wo).max() < 2e-2


def test_no_lse_split_over_many_blocks_and_repeats(ws):
    """A long request among short ones: split over blocks and joined, the same bits on every run."""
    lens, news, D, P, H, Hq = [6001, 3, 200, 0], [1, 1, 1, 1], 128, 64, 2, 16
    pool, table = make_cache(lens, H, D, P, 70)
    q = packed_q(news, Hq, D, BF, 71, 2.0)
    o, lse, err = attend(pool, table, news, lens, q, Hq, ws)
    check(o, lse, expected(q, news, lens, pool, table, P, 0, D ** -0.5), BF)
    for _ in range(5):
        o2, lse2, _ = attend(pool, table, news, lens, q, Hq, ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o3, lse3, _ = attend(pool, table, news, lens, q, Hq, None)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def test_pieces_without_tiles(ws):
    """A narrow window under cut requests: half of the pieces have nothing to read."""
    B, H, G, D, P, window = 30, 2, 4, 64, 16, 16
    lens = [130 + 9 * b for b in range(B)]
    news = [5 + b % 3 for b in range(B)]
    pool, table = make_cache(lens, H, D, P, 60)
    q = packed_q(news, H * G, D, BF, 61)
    want = expected(q, news, lens, pool, table, P, window, D ** -0.5)
    for _ in range(20):
        o, lse, err = attend(pool, table, news, lens, q, H * G, ws, window=window)
        assert err == 0
        check(o, lse, want, BF)


def test_offsets_past_32_bits(ws):
    """Pages that lie more than 2^32 bytes into the pool."""
    H, D, P = 8, 128, 256
    page = H * P // 16 * 18 * D
    pages = (1 << 32) // page + 40
    big = torch.full((pages, H, P // 16, 18 * D), 255, dtype=torch.uint8, device=DEV)
    lens = [700, 300]
    small, table = make_cache(lens, H, D, P, 80, spare=0)
    shift = pages - len(small)
    big[shift:] = dev(small)
    far = np.where(table >= 0, table + shift, -1).astype(np.int32)
    for news in ([1, 1], [80, 70]):
        q = packed_q(news, 16, D, BF, 81)
        a = attend(small, table, news, lens, q, 16, ws)
        o, lse = kda().kda_kv4_attention(q.to(DEV), cu_of(news).to(DEV), max(news), dev(lens, torch.int32), dev(far), big,
                                         workspace=ws)
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)
    x = torch.randn(2, H, D, device=DEV).to(BF)
    cu, start = cu_of([1, 1]).to(DEV), dev([500, 299], torch.int32)
    kda().kda_kv4_append(x, x, cu, start, dev(far), big)
    gk, gv = kda().kda_kv4_gather(cu, start, 2, dev(far), big)
    ns = dev(small)
    kda().kda_kv4_append(x, x, cu, start, dev(table), ns)
    assert torch.equal(big[shift:], ns)
    rk, _ = kda().kda_kv4_gather(cu, start, 2, dev(table), ns)
    assert torch.equal(gk, rk) and torch.equal(gk, gv)


@pytest.mark.parametrize("news", [[1, 1], [70, 90]])
def test_streams_and_graphs(ws, news):
    """Another stream than the tensors' own, and a captured step that is replayed after the cache grew."""
    lens, D, P, H, Hq = [400, 95], 128, 16, 2, 8
    pool, table = make_cache(lens, H, D, P, 90)
    q = packed_q(news, Hq, D, BF, 91)
    want = attend(pool, table, news, lens, q, Hq, ws)
    s = torch.cuda.Stream()
    d = dict(q=q.to(DEV), cu_seqlens=cu_of(news).to(DEV), max_q=max(news), kv_lens=dev(lens, torch.int32),
             page_table=dev(table), pool=dev(pool), workspace=ws)
    s.wait_stream(torch.cuda.current_stream())
    o = torch.empty(sum(news), Hq, D, dtype=BF, device=DEV)
    kda().kda_kv4_attention(**d, o=o, stream=s)
    s.synchronize()
    assert torch.equal(o, want[0])
    graph = torch.cuda.CUDAGraph()
    d["kv_lens"] = dev([90, 95], torch.int32)
    with torch.cuda.stream(s):
        kda().kda_kv4_attention(**d)
    s.synchronize()
    with torch.cuda.graph(graph):
        go, glse = kda().kda_kv4_attention(**d)
    for kv_lens in ([90, 95], lens, [1 + max(news), 20 + max(news)]):
        d["kv_lens"].copy_(dev(kv_lens, torch.int32))
        graph.replay()
        eager = kda().kda_kv4_attention(**d)
        torch.cuda.synchronize()
        # the last lengths run past what was stored: the same NaN in both
        for x, y in zip((go, glse), eager):
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(), y.nan_to_num())


def test_binding_refusals(ws):
    lens, news, D, P, H = [40, 20], [1, 1], 64, 16, 2
    pool, table = make_cache(lens, H, D, P, 95)
    q = packed_q(news, 4, D, BF, 96).to(DEV)
    base = dict(q=q, cu_seqlens=cu_of(news).to(DEV), max_q=1, kv_lens=dev(lens, torch.int32), page_table=dev(table),
                pool=dev(pool), workspace=ws)
    call = lambda **kw: kda().kda_kv4_attention(**{**base, **kw})
    with pytest.raises(TypeError, match="unsupported dtype"):
        call(q=q.float())
    with pytest.raises(ValueError, match="heads and channels must be dense"):
        call(q=q.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="16-byte boundaries"):
        call(q=torch.zeros(2, 4 * D + 4, dtype=BF, device=DEV)[:, :4 * D].view(2, 4, D))
    with pytest.raises(ValueError, match="pool has shape"):
        call(pool=base["pool"][..., :-2].contiguous())
    with pytest.raises(TypeError, match="kv_lens has dtype"):
        call(kv_lens=base["kv_lens"].long())
    with pytest.raises(ValueError, match="cu_seqlens has shape"):
        call(cu_seqlens=base["cu_seqlens"][:2].contiguous())
    with pytest.raises(ValueError, match="page_table must be contiguous"):
        call(page_table=base["page_table"].T.contiguous().T)
    with pytest.raises(kda().KdaError, match="INVALID"):
        call(workspace=ws[:1024])
    with pytest.raises(kda().KdaError, match="INVALID"):
        call(window=-1)
    with pytest.raises(kda().KdaError, match="INVALID"):
        call(k_scale=0.3)
    with pytest.raises(kda().KdaError, match="INVALID"):
        call(q=q[:, :3].contiguous())
    with pytest.raises(ValueError, match="lse has shape"):
        call(lse=torch.zeros(2, 3, device=DEV))
    with pytest.raises(ValueError, match="pool has 2 heads"):
        kda().kda_kv4_append(q, q, base["cu_seqlens"], base["kv_lens"], base["page_table"], base["pool"])
    o, lse = call(q=q[:0], cu_seqlens=torch.zeros(3, dtype=torch.int32, device=DEV))
    assert o.shape == (0, 4, D) and lse.shape == (0, 4)

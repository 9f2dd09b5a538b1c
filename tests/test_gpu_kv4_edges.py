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
    kk, vv = np.repeat(k, G, 1), np.repeat(v, G, 1)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.where(seen[:, None], np.einsum("nhd,thd->nht", q, kk) * scale, -np.inf)
        big = np.where(seen[:, None], np.einsum("nhd,thd->nht", np.abs(q), np.abs(kk)) * abs(scale), 0).max(-1)
        m = np.max(s, -1, keepdims=True)
        p = np.exp(s - np.where(np.isneginf(m), 0, m))
        total = p.sum(-1)
        lse = m[..., 0] + np.log(total)
        # a NaN value reaches the rows that see it, whatever its weight
        bad = np.einsum("nt,thd->nhd", seen.astype(float), np.isnan(vv).astype(float)) > 0
        mean = lambda x: np.einsum("nht,thd->nhd", p, np.nan_to_num(x)) / np.where(total == 0, 1, total)[..., None]
        o, a = np.where(bad, np.nan, mean(vv)), mean(np.abs(vv))
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

"""Builders and error bounds shared by the tests of the paged 4-bit cache."""
import numpy as np
import torch

from oracle import kv4 as ref

# Half a step of each output type, relative to the value.
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def make_cache(lens, H, D, P, seed, spare=3, k_scale=1.0, v_scale=1.0, strength=1.0, max_pages=None):
    """A pool whose rows' pages lie in random order, filled with quantised N(0, 1) rows; all other
    bytes are 0xff (codes -6, scales NaN).  Returns (pool uint8 numpy, table int32 numpy)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // P) for n in lens]
    pages = sum(need) + spare
    M = max_pages or max(need + [1]) + 1
    pool = np.full((pages, H, P // 16, 18 * D), 255, np.uint8)
    order = rng.permutation(pages)
    table = np.full((len(lens), M), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        kv = rng.standard_normal((n, 2, H, D)) * strength
        for pos in range(n):
            ref.store(pool, table[b], pos, kv[pos, 0] / k_scale, kv[pos, 1] / v_scale, P)
    return pool, table


def packed_q(news, Hq, D, dtype, seed, strength=1.0, extra=0):
    """Packed queries [T, Hq, D]: a view of rows of Hq + extra heads."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(sum(news), Hq + extra, D, generator=g) * strength).to(dtype)
    return x


def cu_of(news):
    return torch.tensor([0] + list(np.cumsum(news)), dtype=torch.int32)


def expected(q, news, lens, pool, table, P, window, scale, k_scale=1.0, v_scale=1.0):
    """The oracle's o, lse over the packed rows, with the bound on |error| of each before the
    rounding of o.  The bound's terms:
      - a score is a sum of D products of exact operands in fp32: off by at most
        2 D 2^-23 sum|scale q k| (twice, for truncating accumulators), and 2^-20 relative for the
        exponential and its argument's rounding; a weight's relative error is twice that;
      - a weight is rounded to fp16 once: half a step, 2^-11, and below its smallest normal number
        by 2^-30 of the largest weight;
      - so o is off by that share of the weighted mean of |v|, and lse by the scores' error."""
    outs = []
    at = 0
    for b, n in enumerate(news):
        k, v = ref.load(pool, table[b], lens[b], P, k_scale, v_scale)
        qq = q[at:at + n].double().numpy()
        o, lse, a, big = ref.attention(qq, k, v, window, scale)
        es = 2 * q.shape[-1] * 2.0 ** -23 * big + 2.0 ** -20
        top = np.nanmax(np.abs(v)) if v.size and not np.isnan(v).all() else 0.0
        bo = a * (2.0 ** -11 + 4 * es[..., None]) + 2.0 ** -30 * max(1, lens[b]) * top
        bl = es + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
        outs.append((o, lse, bo, bl))
        at += n
    return [np.concatenate(x) if x else None for x in zip(*outs)]


def check(o, lse, want, dtype):
    wo, wl, bo, bl = want
    go, gl = o.detach().double().cpu().numpy(), lse.detach().double().cpu().numpy()
    assert np.array_equal(np.isnan(go), np.isnan(wo))
    ok = ~np.isnan(wo)
    bad = np.abs(go - wo)[ok] > (bo + HALF_STEP[dtype] * np.abs(wo) * 1.01 + 2.0 ** -24)[ok]
    assert not bad.any(), "o: %d of %d off, worst %.3e" % (bad.sum(), bad.size, np.abs(go - wo)[ok].max())
    empty = wl == -np.inf
    assert np.array_equal(gl == -np.inf, empty)
    ok = ~empty & ~np.isnan(wl)
    assert np.array_equal(np.isnan(gl), np.isnan(wl))
    assert (np.abs(gl - wl)[ok] <= bl[ok]).all(), "lse off by %.3e" % np.abs(gl - wl)[ok].max()

"""Plain fp64 definitions of the operators around the cache's attention (numpy; no code shared with the GPU
path): the residual norm with 8-bit outputs, the position rotation, the bounds of a page's keys, the pages
that a score picks, and attention over them."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from . import kv4

UNBOUNDED = 127


def add_rmsnorm(h, w, eps):
    """y of rows h [T, C] (already added and rounded)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        return h * w / np.sqrt((h * h).mean(-1, keepdims=True) + eps)


def block_scales(y, width):
    """[T, ceil(C / width)] of y [T, C]: max|y| / 448."""
    return np.stack([np.abs(y[:, a:a + width]).max(-1) / 448.0 for a in range(0, y.shape[1], width)], -1)


def rotate(x, pos, R, pairs=False, base=10000.0):
    """x [T, H, D] turned by the angles of pos [T]."""
    x = np.array(x, np.float64)
    angle = np.asarray(pos, np.float64)[:, None] * base ** (-np.arange(0, R, 2) / R)
    z = np.exp(1j * angle)[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    t = (a + 1j * b) * z
    out = x.copy()
    if pairs:
        out[..., 0:R:2], out[..., 1:R:2] = t.real, t.imag
    else:
        out[..., :R // 2], out[..., R // 2:R] = t.real, t.imag
    return out


def unit(top):
    """The least e with top <= 127 x 2^e."""
    e = int(np.floor(np.log2(top / 127))) - 2
    while top > 127 * 2.0 ** e:
        e += 1
    return e


def page_bounds(k):
    """(hi [H, D], lo [H, D], e [H]) of one page's keys k [tokens, H, D]."""
    H, D = k.shape[1:]
    hi, lo, es = np.zeros((H, D), int), np.zeros((H, D), int), np.zeros(H, int)
    for h in range(H):
        if np.isnan(k[:, h]).any():
            es[h] = UNBOUNDED
            continue
        top = np.abs(k[:, h]).max()
        if top > 0:
            es[h] = unit(top)
            hi[h] = np.ceil(k[:, h].max(0) / 2.0 ** es[h])
            lo[h] = np.floor(k[:, h].min(0) / 2.0 ** es[h])
    return hi, lo, es


def _adds_exactly(x):
    """Whether the rows of x >= 0 add up without a rounding in fp64."""
    total, lost = np.zeros(x.shape[1]), np.zeros(x.shape[1])
    for row in x:
        t = total + row
        back = t - total
        lost += np.abs((total - (t - back)) + (row - back))
        total = t
    return not lost.any()


def asked(q):
    """(u, d) whole numbers [D] of one kv head's queries q [G, D]: of the exact sums."""
    q = np.asarray(q, np.float64)
    none = np.zeros(q.shape[1], int), np.zeros(q.shape[1], int)
    if not np.isfinite(q).all():
        return none
    if _adds_exactly(np.abs(q)):
        up, down = np.maximum(q, 0).sum(0), np.maximum(-q, 0).sum(0)
        power = lambda f: 2.0 ** f
    else:
        exact = [[Fraction(float(x)) for x in row] for row in q.T]
        up, down = (np.array([sum((s * x for x in row if s * x > 0), Fraction(0)) for row in exact], object) for s in (1, -1))
        power = lambda f: Fraction(2) ** f
    top = max(up.max(), down.max())
    if (up + down).max() > float(np.finfo(np.float32).max) or top == 0:
        return none
    f = max(unit(float(top)) - 1, -100)
    while top > 127 * power(f):
        f += 1
    return tuple(np.array([round(x / power(f)) for x in side.tolist()], int) for side in (up, down))


def pick(q, pos, records, page_size, count, first, recent):
    """Pages picked for one token at position pos and one kv head: q [G, D]; records a list of (hi [D], lo
    [D], e) of the row's pages, None for one that is out of range.  A list of count, -1 behind."""
    own = pos // page_size if pos >= 0 else -1
    if own + 1 <= count:
        return list(range(own + 1)) + [-1] * (count - own - 1)
    u, d = asked(q)
    scores = []
    for p in range(first, own + 1 - recent):
        if records[p] is None:
            s = -np.inf
        else:
            hi, lo, e = records[p]
            s = np.inf if e == UNBOUNDED else float((u * hi - d * lo).sum()) * 2.0 ** int(e)
        scores.append((-s, p))
    best = sorted(p for _, p in sorted(scores)[:count - first - recent])
    return list(range(first)) + best + list(range(own + 1 - recent, own + 1))


def attention_picked(q, k, v, pos, picked, page_size, scale):
    """One token at position pos: q [Hq, D], k, v [len, H, D], picked [H, count].  Returns o, lse, the
    weighted |v| and the largest sum |scale q k| as kv4.attention does."""
    Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    o, lse, a, big = np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros((Hq, D)), np.zeros(Hq)
    for h in range(H):
        at = [j for p in picked[h] if p >= 0 for j in range(p * page_size, (p + 1) * page_size) if j <= pos]
        if not at:
            continue
        r = kv4.attention(q[None, h * G:(h + 1) * G], k[at, h:h + 1], v[at, h:h + 1], 0, scale)
        for out, x in zip((o, lse, a, big), r):
            out[h * G:(h + 1) * G] = x[0]
    return o, lse, a, big

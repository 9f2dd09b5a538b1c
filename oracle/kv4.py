"""Plain fp64 definitions of the paged 4-bit cache's operators (numpy; no code shared with the
GPU path): the quantisation, the byte layout, attention row by row, and the pages' bookkeeping."""
from __future__ import annotations

import numpy as np

TILE = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)) for e in range(16) for m in range(8)][:127])


def nearest(x, grid):
    """Index of the nearest grid value to x >= 0, ties to the even index, saturating."""
    hi = np.minimum(np.searchsorted(grid, x), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    below, above = x - grid[lo], grid[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def quantise(x):
    """x [..., D] -> (codes 0..15 [..., D], scale bytes [..., D / 16])."""
    blocks = np.asarray(x, np.float64).reshape(x.shape[:-1] + (-1, 16))
    top = np.abs(blocks).max(-1)
    nan = np.isnan(top)
    sb = np.where(nan, 127, nearest(np.minimum(np.where(nan, 0, top) / 6, 448.0), E4M3))
    s = np.where(nan, np.nan, E4M3[np.minimum(sb, 126)])
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s[..., None] > 0, np.abs(blocks) / s[..., None], 0.0)
    code = np.where(np.isnan(y), 7, nearest(np.minimum(np.nan_to_num(y), 6.0), E2M1))
    code = code | ((np.signbit(blocks) & (s[..., None] > 0)).astype(int) << 3)
    return code.reshape(x.shape), sb


def values(code, sb, factor=1.0):
    mag = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(sb == 127, np.nan, E4M3[np.minimum(sb, 126)]) * factor
    return mag * np.repeat(s, 16, axis=-1)


def place(table, pos, page_size):
    """(page, tile, token) of a position of a row."""
    return int(table[pos // page_size]), pos % page_size // TILE, pos % TILE


def store(pool, table, pos, k, v, page_size):
    """Quantise and write one token's k, v [H, D] (already divided by the tensor scales)."""
    D = k.shape[1]
    page, tile, tok = place(table, pos, page_size)
    t = pool[page, :, tile]
    for x, codes_at, scales_at in ((k, 0, 8 * D + tok * (D // 16) + np.arange(D // 16)),
                                   (v, 9 * D, 17 * D + np.arange(D // 16) * TILE + tok)):
        code, sb = quantise(x)
        t[:, codes_at + tok * (D // 2):codes_at + (tok + 1) * (D // 2)] = code[:, 0::2] | (code[:, 1::2] << 4)
        t[:, scales_at] = sb


def load(pool, table, length, page_size, k_scale=1.0, v_scale=1.0):
    """K, V [length, H, D] of a row's first positions."""
    H, D = pool.shape[1], pool.shape[3] // 18
    k, v = np.zeros((length, H, D)), np.zeros((length, H, D))
    if not length:
        return k, v
    pos = np.arange(length)
    t = pool[np.asarray(table)[pos // page_size], :, pos % page_size // TILE]      # [length, H, 18 D]
    tok = pos % TILE
    for out, codes_at, scales_at, factor in (
            (k, 0, 8 * D + tok[:, None] * (D // 16) + np.arange(D // 16), k_scale),
            (v, 9 * D, 17 * D + np.arange(D // 16)[None] * TILE + tok[:, None], v_scale)):
        at = codes_at + tok[:, None] * (D // 2) + np.arange(D // 2)
        byte = np.take_along_axis(t, np.broadcast_to(at[:, None], (length, H, D // 2)), 2).astype(int)
        sb = np.take_along_axis(t, np.broadcast_to(scales_at[:, None], (length, H, D // 16)), 2).astype(int)
        code = np.stack([byte & 15, byte >> 4], -1).reshape(length, H, D)
        out[:] = values(code, sb & 127, factor)
    return k, v


def attention(q, k, v, window=0, scale=1.0):
    """q [n, Hq, D] newest tokens, k, v [len, H, D].  Returns o, lse and, for error bounds, the
    softmax-weighted |v| of each output and the largest sum |scale q k| of each row."""
    n, Hq, D = q.shape
    length, H = k.shape[0], k.shape[1]
    G = Hq // H
    o, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    a, big = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        last = length - n + i
        first = max(0, last + 1 - window) if window else 0
        if last < 0:
            continue
        for h in range(Hq):
            K, V = k[first:last + 1, h // G], v[first:last + 1, h // G]
            with np.errstate(invalid="ignore", over="ignore"):
                s = K @ q[i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                o[i, h] = p @ V / p.sum()
                a[i, h] = p @ np.abs(V) / p.sum()
                lse[i, h] = m + np.log(p.sum())
                big[i, h] = (np.abs(K) @ np.abs(q[i, h])).max() * abs(scale)
    return o, lse, a, big


class Pages:
    """The pages' bookkeeping, one row and one page at a time."""

    def __init__(self, num_pages, rows, max_pages, page_size):
        self.refs = [0] * num_pages
        self.table = [[-1] * max_pages for _ in range(rows)]
        self.lens = [0] * rows
        self.P = page_size

    def held(self, b):
        return -(-self.lens[b] // self.P)

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def alloc(self, grow):
        out = refused = False
        may = [g < 0 and (not (self.lens[b] + g) % self.P or self.refs[self.table[b][(self.lens[b] + g) // self.P]] == 1)
               for b, g in enumerate(grow)]
        for b, g in enumerate(grow):
            if g >= 0:
                continue
            if not may[b]:
                refused = True
                continue
            keep = -(-(self.lens[b] + g) // self.P)
            for j in range(keep, self.held(b)):
                self.refs[self.table[b][j]] -= 1
                self.table[b][j] = -1
            self.lens[b] += g
        for b, g in enumerate(grow):
            if g < 0:
                continue
            have = self.held(b)
            need = -(-(self.lens[b] + g) // self.P) - have
            free = self._free()
            if need and (out or need > len(free)):
                out = True
                continue
            for j in range(need):
                self.table[b][have + j] = free[j]
                self.refs[free[j]] = 1
            self.lens[b] += g
        return out or refused

    def fork(self, src, dst, data):
        """data: list of arrays [num_pages, ...].  Returns True when pages ran out."""
        out = False
        moves = []
        for s, d in zip(src, dst):
            full, part = divmod(self.lens[s], self.P)
            free = self._free()
            if part and (out or not free):
                out = True
                continue
            self.table[d] = self.table[s][:full] + [-1] * (len(self.table[s]) - full)
            for p in self.table[s][:full]:
                self.refs[p] += 1
            if part:
                self.table[d][full] = free[0]
                self.refs[free[0]] = 1
                moves.append((self.table[s][full], free[0]))
            self.lens[d] = self.lens[s]
        for x in data:
            for a, b in moves:
                x[b] = x[a]
        return out

    def free(self, rows):
        for b in rows:
            for p in self.table[b][:self.held(b)]:
                self.refs[p] -= 1
            self.table[b] = [-1] * len(self.table[b])
            self.lens[b] = 0

    def compact(self, data):
        live = sum(r > 0 for r in self.refs)
        to = {}
        holes = [p for p in self._free() if p < live]
        for p in range(live, len(self.refs)):
            if self.refs[p]:
                to[p] = holes[len(to)]
        for x in data:
            for a, b in to.items():
                x[b] = x[a]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return live

"""The paged 4-bit key/value cache: its cases, and the plain form of every operator.

A hybrid model's full-attention layers keep their keys and values in pages of 4-bit codes next to
the recurrent state pools.  A pool is uint8 [pages][Hkv][P / 16][18 D]: for each page and head, tiles
of 16 tokens, each

    K codes [16][D / 2] | K scales [16][D / 16] | V codes [16][D / 2] | V scales [D / 16][16]

Codes are e2m1 (even channel in the low nibble), scales e4m3, one for 16 channels of a token.

``run`` computes with elementary torch operations, or, with ``own`` set, through the library.
"""
import math
import random

import torch

own = False

TILE = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


def _kda():
    import kda_state_gb300
    return kda_state_gb300


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's chat: a single request, one token; what counts is latency
        dict(name="decode_one", kind="attend", B=1, n=1, lo=1037, hi=1037, Hq=64, Hkv=8, D=128, P=16, window=0, dtype="bf16"),
        # a serving batch in mid-flight: every request at another length
        dict(name="decode_batch", kind="attend", B=128, n=1, lo=37, hi=8190, Hq=64, Hkv=8, D=128, P=64, window=0, dtype="bf16"),
        # few requests over very long contexts: the work has to be split over the tokens
        dict(name="decode_long", kind="attend", B=4, n=1, lo=98301, hi=131071, Hq=64, Hkv=8, D=128, P=128, window=0, dtype="bf16"),
        # heads of 64 channels, no sharing of heads, a sliding window inside longer caches
        dict(name="decode_window", kind="attend", B=96, n=1, lo=200, hi=4999, Hq=32, Hkv=32, D=64, P=32, window=1024, dtype="fp16"),
        # verify of 8 draft tokens for 64 requests (the recurrent layers' verify step, same batch)
        dict(name="verify", kind="attend", B=64, n=8, lo=511, hi=6007, Hq=64, Hkv=8, D=128, P=64, window=0, dtype="bf16"),
        # a chunked-prefill piece of 4096 tokens on top of a resumed prefix
        dict(name="prefill_piece", kind="attend", B=2, n=2048, lo=4099, hi=24576, Hq=64, Hkv=8, D=128, P=64, window=0, dtype="bf16"),
        # the new token of each of 384 requests is stored, and read back
        dict(name="append_step", kind="append", B=384, n=1, lo=1, hi=8192, Hkv=8, D=128, P=64, dtype="bf16"),
        # prompts of 64 to 2048 tokens are stored, and read back
        dict(name="append_prompt", kind="append", B=8, n=2048, lo=64, hi=4500, Hkv=8, D=128, P=64, dtype="bf16"),
        # one scheduler step on the pages of 24 layers: growth, forks, a few copies, requests that end
        dict(name="pages_step", kind="pages", B=64, M=96, lo=5, hi=5800, forks=7, copies=5, frees=6, layers=24, Hkv=8, D=128, P=64, pages=3500),
        # a beam step: as many forks as requests
        dict(name="pages_beam", kind="pages", B=256, M=40, lo=3, hi=1200, forks=80, copies=64, frees=120, layers=24, Hkv=8, D=128, P=32, pages=5200),
        # a half-empty pool is compacted, so that its upper part can be given to state slots
        dict(name="compact_half", kind="compact", B=48, M=64, lo=300, hi=4000, layers=24, Hkv=8, D=128, P=64, pages=3001),
        # a pool of a single layer with few requests left in it
        dict(name="compact_few", kind="compact", B=9, M=200, lo=10, hi=3100, layers=1, Hkv=4, D=64, P=16, pages=20011),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "verify", "prefill", "append", "pages", "compact"])
    D = rng.choice([64, 128, 128])
    P = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 5, 8, 8, 16])
    if kind == "decode":
        B, hi = _log(rng, 1, 256), _log(rng, 16, 131072)
        B = max(1, min(B, 400000 // hi))
        return dict(kind="attend", B=B, n=1, lo=rng.randint(1, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, P=P,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), dtype=dtype)
    if kind == "verify":
        n, hi = rng.randint(2, 16), _log(rng, 64, 16384)
        B = max(1, min(_log(rng, 1, 128), 300000 // hi))
        return dict(kind="attend", B=B, n=n, lo=rng.randint(n, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, P=P,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 2048)]), dtype=dtype)
    if kind == "prefill":
        n, B = _log(rng, 17, 2048), rng.randint(1, 4)
        hi = n + rng.choice([0, _log(rng, 1, 8192)])
        return dict(kind="attend", B=B, n=n, lo=rng.randint(n, hi), hi=hi, Hq=Hkv * min(G, 8), Hkv=Hkv, D=D, P=P,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), dtype=dtype)
    if kind == "append":
        n = rng.choice([1, rng.randint(2, 16), _log(rng, 17, 2048)])
        B = max(1, min(_log(rng, 1, 384), 16384 // n))
        hi = n + _log(rng, 1, 4096)
        return dict(kind="append", B=B, n=n, lo=rng.randint(n, hi), hi=hi, Hkv=Hkv, D=D, P=P, dtype=dtype)
    B, M = rng.randint(8, 200), rng.randint(8, 64)
    lo = rng.randint(1, P)
    hi = rng.randint(lo + P, (M - 1) * P)
    c = dict(kind=kind, B=B, M=M, lo=lo, hi=hi, layers=_log(rng, 1, 24), Hkv=Hkv, D=D, P=P)
    if kind == "pages":
        c.update(forks=rng.randint(1, B // 3), copies=rng.randint(1, 40), frees=rng.randint(1, B // 2))
    held = sum(-(-n // P) for n in _page_rows(c)[0])
    c["pages"] = held + 3 * B + 41 + rng.randint(0, held)
    # as many layers as a few GB of pages allow
    c["layers"] = max(1, min(c["layers"], int(4e9 / (c["pages"] * Hkv * P // TILE * 18 * D))))
    return c


def _spread(count, lo, hi):
    """count whole numbers spread over [lo, hi] in no order; the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(count)]


def _requests(c):
    """(new tokens, tokens in the cache with them) of each request."""
    lens = _spread(c["B"], c["lo"], c["hi"])
    if c["n"] <= 16:
        new = [c["n"]] * c["B"]
    else:                                  # prompts: ragged, the longest first in no more than one request
        new = [c["n"]] + _spread(c["B"] - 1, max(1, c["n"] // 32), c["n"])
    if c["kind"] == "append":
        lens = [max(l, n) for l, n in zip(lens, new)]
    return [min(n, l) for n, l in zip(new, lens)], lens


def _seen(n, length, window):
    """(tokens of the cache that some row sees, pairs of a row and a token that it sees)."""
    pairs = 0
    first = length - n                     # row i sees positions up to first + i
    if window:
        full = max(0, n - max(0, window - first - 1))          # rows that see a whole window
        part = n - full
        pairs = full * window + part * (first + 1) + part * (part - 1) // 2
        return length - max(0, first + 1 - window), pairs
    return length, n * (first + 1) + n * (n - 1) // 2


def work(case):
    c = case
    if c["kind"] == "attend":
        new, lens = _requests(c)
        seen = [_seen(n, l, c["window"]) for n, l in zip(new, lens)]
        rows = sum(new) * c["Hq"]
        return {"bytes": sum(s for s, _ in seen) * c["Hkv"] * c["D"] * 9 // 8 + rows * (c["D"] * 4 + 4),
                "flops": 4 * c["D"] * c["Hq"] * sum(p for _, p in seen)}
    if c["kind"] == "append":
        new, _ = _requests(c)
        values = sum(new) * c["Hkv"] * c["D"] * 2              # of k and v: read, stored, fetched, written
        return {"bytes": values * 2 + values * 9 // 16 * 2 + values * 2, "flops": 4 * values}
    page = c["Hkv"] * c["P"] // TILE * 18 * c["D"] * c["layers"]
    if c["kind"] == "pages":
        lens, src, dst, free = _page_rows(c)
        moved = sum(1 for s in src if lens[s] % c["P"]) + c["copies"]
        touched = sum(-(-lens[r] // c["P"]) for r in src + free)
        return {"bytes": 2 * moved * page + 4 * c["pages"] + 16 * touched, "flops": 0}
    refs, table, lens = _scattered(c, 0)
    live = sum(1 for r in refs if r)
    moved = sum(1 for p, r in enumerate(refs) if r and p >= live)
    return {"bytes": 2 * moved * page + 8 * c["pages"] + 8 * c["B"] * c["M"], "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _page_rows(c):
    """Lengths of the rows (a third of them empty), and the rows forked from, forked to, freed."""
    lens = _spread(c["B"], c["lo"], c["hi"])
    empty = c["B"] // 3 + 1
    for i in range(empty):
        lens[i * 3 % c["B"]] = 0
    full = [i for i in range(c["B"]) if lens[i]]
    free_rows = [i for i in range(c["B"]) if not lens[i]]
    dst = free_rows[:c.get("forks", 0)]
    src = [full[(i * 5) % len(full)] for i in range(len(dst))]  # some rows are forked twice
    gone = (dst[::2] + full[::-1])[:c.get("frees", 0)]
    return lens, src, dst, gone


def _scattered(c, seed):
    """refs, page table and lengths of a pool whose rows' pages lie anywhere; neighbours share full pages."""
    rng = random.Random(1000003 * seed + 17)
    lens, _, _, _ = _page_rows(c)
    order = list(range(c["pages"]))
    rng.shuffle(order)
    refs, table, at, last = [0] * c["pages"], [], 0, None
    for b in range(c["B"]):
        need, row = -(-lens[b] // c["P"]), []
        shared = min(2, lens[b] // c["P"], lens[last] // c["P"]) if last is not None and b % 4 == 1 else 0
        for j in range(need):
            if j < shared:
                row.append(table[last][j])
            else:
                row.append(order[at])
                at += 1
            refs[row[-1]] += 1
        table.append(row + [-1] * (c["M"] - need))
        if lens[b]:
            last = b
    return refs, table, lens


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _quantise(x):
    """(codes uint8 [..., D / 2], scales e4m3 [..., D / 16]) of x [..., D]."""
    x = x.float()
    blocks = x.unflatten(-1, (-1, 16))
    scale = (blocks.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = blocks / torch.where(scale.float() == 0, 1.0, scale.float())[..., None]
    y = torch.where(scale.float()[..., None] == 0, 0.0, y)
    a = y.abs()
    # to the nearest of the eight magnitudes, ties to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _rows(g, count, heads, D, dtype, spread=1.0):
    """Keys or values as projections make them: channels of different strength."""
    strength = 0.5 + torch.rand(heads, D, generator=g, device=DEV) * spread
    return (torch.randn(count, heads, D, generator=g, device=DEV) * strength).to(dtype)


def _filled_pool(c, g, pages, table, need):
    """A pool whose held pages carry quantised rows, drawn from a bank of them, and whose others are stale."""
    Hkv, D, P = c["Hkv"], c["D"], c["P"]
    pool = torch.full((pages, Hkv, P // TILE, 18 * D), 255, dtype=torch.uint8, device=DEV)
    held = table[table >= 0].long()
    bank = []
    for strong in (1.0, 0.5):
        codes, scales = _quantise(_rows(g, 8192, 1, D, torch.float32, strong)[:, 0])
        bank.append(torch.cat([codes, scales.view(torch.uint8)], -1))
    for a in range(0, held.numel(), 4096):
        part = held[a:a + 4096]
        shape = (part.numel(), Hkv, P // TILE, TILE)
        k = bank[0][torch.randint(0, 8192, shape, generator=g, device=DEV)]
        v = bank[1][torch.randint(0, 8192, shape, generator=g, device=DEV)]
        pool[part] = torch.cat([k[..., :D // 2].flatten(-2), k[..., D // 2:].flatten(-2),
                                v[..., :D // 2].flatten(-2), v[..., D // 2:].transpose(-1, -2).flatten(-2)], -1)
    return pool


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(7919 * seed + 11)
    s = {"case": c}
    if c["kind"] in ("attend", "append"):
        new, lens = _requests(c)
        M = -(-max(lens) // c["P"]) + 1
        need = [-(-l // c["P"]) for l in lens]
        pages = sum(need) + 5
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((c["B"], M), -1, dtype=torch.int32, device=DEV)
        cells = torch.arange(M, device=DEV)[None] < _i32(need)[:, None]
        table[cells] = perm[:sum(need)]
        s["cu"] = _i32([0] + torch.tensor(new).cumsum(0).tolist())
        s["table"], s["max_new"], T = table, max(new), sum(new)
        s["pool"] = _filled_pool(c, g, pages, table, need)
        s["k_scale"], s["v_scale"] = 1.0, 0.5
        if c["kind"] == "attend":
            s["lens"] = _i32(lens)
            s["scale"] = c["D"] ** -0.5
            # the queries are a view of the fused projection's output, and some look for something
            qkv = torch.randn(T, c["Hq"] + 2 * c["Hkv"], c["D"], generator=g, device=DEV)
            qkv *= 0.5 + 2.0 * torch.rand(T, qkv.shape[1], 1, generator=g, device=DEV)
            s["q"] = qkv.to(DTYPES[c["dtype"]])[:, :c["Hq"]]
            s["workspace"] = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
        else:
            s["start"] = _i32([l - n for l, n in zip(lens, new)])
            s["k"] = _rows(g, T, c["Hkv"], c["D"], DTYPES[c["dtype"]], 4.0)
            s["v"] = _rows(g, T, c["Hkv"], c["D"], DTYPES[c["dtype"]])
        return s
    refs, table, lens = _scattered(c, seed)
    if c["kind"] == "pages":
        _, src, dst, gone = _page_rows(c)
        s["src"], s["dst"], s["gone"] = _i32(src), _i32(dst), _i32(gone)
        # new tokens of this step: one for most rows, a piece for some
        grow = [(1 if b % 5 else c["P"] + 3) if lens[b] and lens[b] + c["P"] + 3 <= c["M"] * c["P"] else 0 for b in range(c["B"])]
        # pages set aside for the prefix cache take copies of pages that rows hold
        free = [p for p, r in enumerate(refs) if not r]
        held = [p for p, r in enumerate(refs) if r]
        to = free[-c["copies"]:]
        s["grow"], s["copy_to"] = _i32(grow), _i32(to)
        s["copy_from"] = _i32([held[(i * 7) % len(held)] for i in range(len(to))])
        for p in to:
            refs[p] = 1
    s["refs"], s["table"], s["lens"] = _i32(refs), _i32(table), _i32(lens)
    shape = (c["pages"], c["Hkv"], c["P"] // TILE, 18 * c["D"])
    s["pools"] = [torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(c["layers"])]
    s["workspace"] = torch.zeros(4 * c["pages"] + 4096, dtype=torch.int32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _values(codes, scales, factor):
    """What codes [..., D / 2] and scales [..., D / 16] stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=codes.device)
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)      # by byte: low, high nibble
    x = pairs[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * (scales.view(torch.float8_e4m3fn).float() * factor)[..., None]).flatten(-2)


def _unpack(tiles, D, k_scale, v_scale):
    """K and V [..., tiles, 16, D] of tiles [..., 18 D]."""
    kc, ks, vc, vs = tiles.split([8 * D, D, 8 * D, D], -1)
    k = _values(kc.unflatten(-1, (TILE, D // 2)), ks.unflatten(-1, (TILE, D // 16)).contiguous(), k_scale)
    v = _values(vc.unflatten(-1, (TILE, D // 2)), vs.unflatten(-1, (D // 16, TILE)).transpose(-1, -2).contiguous(), v_scale)
    return k, v


def _owners(cu, T):
    """(request, index in it) of each of T packed tokens."""
    t = torch.arange(T, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, (t - cu[b]).long()


def _attend(s):
    c, q, table, lens, cu = s["case"], s["q"], s["table"], s["lens"], s["cu"]
    B, Hq, Hkv, D, n = c["B"], c["Hq"], c["Hkv"], c["D"], s["max_new"]
    G, L = Hq // Hkv, table.shape[1] * c["P"]
    tiles = s["pool"][table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3)     # [B, Hkv, L / 16, 18 D]
    k, v = (x.flatten(2, 3) for x in _unpack(tiles, D, s["k_scale"], s["v_scale"]))
    there = (torch.arange(L, device=DEV) < lens[:, None])[:, None, :, None]
    k, v = torch.where(there, k, 0.0), torch.where(there, v, 0.0)
    b, i = _owners(cu, q.shape[0])
    rows = torch.zeros(B, n, Hq, D, device=DEV)
    rows[b, i] = q.float()
    rows = rows.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = (rows @ k.transpose(-1, -2)).view(B, Hkv, G, n, L) * s["scale"]
    new = cu[1:] - cu[:-1]
    last = (lens - new)[:, None] + torch.arange(n, device=DEV)                      # [B, n]
    at = torch.arange(L, device=DEV)
    seen = at <= last[..., None]
    if c["window"]:
        seen &= at > last[..., None] - c["window"]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * n, L) @ v).view(B, Hkv, G, n, D) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[b, i]
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, Hq)[b, i]
    return o.to(q.dtype), lse


def _append(s):
    c, cu, table, pool = s["case"], s["cu"], s["table"], s["pool"]
    D, P = c["D"], c["P"]
    T = s["k"].shape[0]
    b, i = _owners(cu, T)
    pos = s["start"][b].long() + i
    page, tile, tok = table[b, pos // P].long(), pos % P // TILE, pos % TILE
    kc, ks = _quantise(s["k"].float() / s["k_scale"])
    vc, vs = _quantise(s["v"].float() / s["v_scale"])
    shape = pool.shape[:3]
    # the four regions of a tile, as views that index by token
    kcv = pool.as_strided(shape + (TILE, D // 2), pool.stride()[:3] + (D // 2, 1), 0)
    ksv = pool.as_strided(shape + (TILE, D // 16), pool.stride()[:3] + (D // 16, 1), 8 * D)
    vcv = pool.as_strided(shape + (TILE, D // 2), pool.stride()[:3] + (D // 2, 1), 9 * D)
    vsv = pool.as_strided(shape + (TILE, D // 16), pool.stride()[:3] + (1, TILE), 17 * D)
    kcv[page, :, tile, tok] = kc
    ksv[page, :, tile, tok] = ks.view(torch.uint8)
    vcv[page, :, tile, tok] = vc
    vsv[page, :, tile, tok] = vs.view(torch.uint8)
    k = _values(kcv[page, :, tile, tok], ksv[page, :, tile, tok], s["k_scale"])
    v = _values(vcv[page, :, tile, tok], vsv[page, :, tile, tok], s["v_scale"])
    return k.to(s["k"].dtype), v.to(s["v"].dtype)


def _free_order(refs):
    """Free pages first, lowest number first, then the held ones; and how many are free."""
    held = refs > 0
    return torch.argsort(held.to(torch.int8), stable=True), (~held).sum()


def _grow(refs, table, lens, grow, P):
    have, want = (lens + P - 1) // P, (lens + grow + P - 1) // P
    need = want - have
    upto = need.cumsum(0)
    order, free = _free_order(refs)
    served = (upto <= free) | (need == 0)
    col = torch.arange(table.shape[1], device=DEV)
    cell = (col >= have[:, None]) & (col < want[:, None]) & served[:, None]
    pick = order[((upto - need)[:, None] + col - have[:, None]).clamp(0, refs.numel() - 1)]
    table.copy_(torch.where(cell, pick.to(torch.int32), table))
    refs.index_add_(0, pick.flatten(), cell.flatten().to(torch.int32))
    lens += torch.where(served, grow, 0)


def _fork(pools, refs, table, lens, src, dst, P):
    src, dst = src.long(), dst.long()
    full, part = lens[src] // P, lens[src] % P > 0
    order, free = _free_order(refs)
    upto = part.cumsum(0)
    served = (upto <= free) | ~part
    fresh = order[(upto - 1).clamp(0, refs.numel() - 1)]
    col = torch.arange(table.shape[1], device=DEV)
    share = (col < full[:, None]) & served[:, None]
    split = ((col == full[:, None]) & part[:, None]) & served[:, None]
    rows = table[src]
    table[dst] = torch.where(share, rows, torch.where(split, fresh[:, None].to(torch.int32), -1))
    refs.index_add_(0, rows.clamp(min=0).flatten(), share.flatten().to(torch.int32))
    moves = part & served
    old = rows.gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0].long()
    old, new = old[moves], fresh[moves]
    refs[new] = 1
    lens[dst] = torch.where(served, lens[src], 0)
    for pool in pools:
        pool[new] = pool[old]


def _release(refs, table, lens, rows, P):
    rows = rows.long()
    held = torch.arange(table.shape[1], device=DEV) < ((lens[rows] + P - 1) // P)[:, None]
    refs.index_add_(0, table[rows].clamp(min=0).flatten(), -held.flatten().to(torch.int32))
    table[rows] = -1
    lens[rows] = 0


def _compact(pools, refs, table):
    order, free = _free_order(refs)
    live = refs.numel() - free
    page = torch.arange(refs.numel(), device=DEV)
    mover = (refs > 0) & (page >= live)
    to = torch.where(mover, order[(mover.cumsum(0) - 1).clamp(min=0)], page)
    src = mover.nonzero()[:, 0]
    for pool in pools:
        pool[to[src]] = pool[src]
    refs.copy_(torch.zeros_like(refs).index_add_(0, to, refs))
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), -1))
    return live.to(torch.int32).reshape(1)


def run(state):
    s, c = state, state["case"]
    if c["kind"] == "attend":
        if not own:
            return _attend(s)
        return _kda().kda_kv4_attention(s["q"], s["cu"], s["max_new"], s["lens"], s["table"], s["pool"], scale=s["scale"],
                                        window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["workspace"])
    if c["kind"] == "append":
        if not own:
            return _append(s)
        kda = _kda()
        kda.kda_kv4_append(s["k"], s["v"], s["cu"], s["start"], s["table"], s["pool"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return kda.kda_kv4_gather(s["cu"], s["start"], s["k"].shape[0], s["table"], s["pool"], dtype=s["k"].dtype,
                                  k_scale=s["k_scale"], v_scale=s["v_scale"])
    # the bookkeeping changes in place: each pass takes the step from the same beginning
    refs, table, lens = s["refs"].clone(), s["table"].clone(), s["lens"].clone()
    P, pools = c["P"], s["pools"]
    if c["kind"] == "pages":
        if own:
            kda = _kda()
            kda.kda_page_alloc(refs, table, lens, s["grow"], P)
            kda.kda_page_fork(pools, refs, table, lens, s["src"], s["dst"], P, workspace=s["workspace"])
            kda.kda_page_copy(pools, s["copy_from"], s["copy_to"])
            kda.kda_page_free(refs, table, lens, s["gone"], P)
        else:
            _grow(refs, table, lens, s["grow"], P)
            _fork(pools, refs, table, lens, s["src"], s["dst"], P)
            for pool in pools:
                pool[s["copy_to"].long()] = pool[s["copy_from"].long()]
            _release(refs, table, lens, s["gone"], P)
        return [refs, table, lens] + pools
    live = _kda().kda_page_compact(pools, refs, table, workspace=s["workspace"]) if own else _compact(pools, refs, table)
    return [live, refs, table] + pools


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _level(code):
    """e2m1: the value of a 4-bit code, by its fields."""
    sign, exp, man = code // 8, code // 2 % 4, code % 2
    mag = torch.where(exp == 0, 0.5 * man, 2.0 ** (exp - 1.0) * (1 + 0.5 * man))
    return mag * (1.0 - 2.0 * sign)


def _e4m3(byte):
    exp, man = byte // 8, byte % 8
    return torch.where(exp == 0, man * 2.0 ** -9, 2.0 ** (exp - 7.0) * (1 + man / 8.0))


def _cached(pool, row, length, P, D, head, k_side, factor):
    """Keys or values [length, D] of one request and head, token by token from the pool's bytes."""
    t = torch.arange(length, device=pool.device)
    tile = pool[row[t // P].long(), head, t % P // TILE].double()                  # [length, 18 D]
    slot = (t % TILE)[:, None]
    ch = torch.arange(D, device=pool.device)[None]
    base = 0 if k_side else 9 * D
    byte = tile.gather(1, base + slot * (D // 2) + ch // 2)
    code = torch.where(ch % 2 == 0, byte % 16, byte // 16)
    at = 8 * D + slot * (D // 16) + ch // 16 if k_side else 17 * D + ch // 16 * TILE + slot
    return _level(code.floor()) * _e4m3(tile.gather(1, at)) * factor


def exact(case, seed):
    c = case
    if c["kind"] in ("pages", "compact"):
        return None                                  # whole numbers and bytes that are moved
    s = prepare(case, seed)
    if c["kind"] == "append":
        answer = []
        for name in ("k", "v"):
            x = s[name].double() / s[name + "_scale"]
            x = x.view(x.shape[0], x.shape[1], -1, 16)
            want = x.abs().amax(-1, keepdim=True) / 6
            grid = _e4m3(torch.arange(127, device=x.device).double())
            scale = _nearest(want.clamp(max=448.0), grid)
            y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
            mags = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
            answer.append((_nearest(y.abs(), mags) * torch.sign(y) * scale).flatten(-2) * s[name + "_scale"])
        return tuple(answer)
    q, cu, lens = s["q"], s["cu"].tolist(), s["lens"].tolist()
    G = c["Hq"] // c["Hkv"]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(c["B"]):
        n, length = cu[b + 1] - cu[b], lens[b]
        low = max(0, length - n + 1 - c["window"]) if c["window"] else 0
        for h in range(c["Hkv"]):
            k = _cached(s["pool"], s["table"][b], length, c["P"], c["D"], h, True, s["k_scale"])[low:]
            v = _cached(s["pool"], s["table"][b], length, c["P"], c["D"], h, False, s["v_scale"])[low:]
            at = torch.arange(low, length, device=q.device)
            for a in range(0, n, 512):
                z = min(n, a + 512)
                x = torch.einsum("ngd,td->gnt", q[cu[b] + a:cu[b] + z, h * G:(h + 1) * G].double(), k) * s["scale"]
                me = length - n + torch.arange(a, z, device=q.device)[:, None]
                hide = at > me
                if c["window"]:
                    hide |= at <= me - c["window"]
                x = x.masked_fill(hide, -math.inf)
                part = torch.logsumexp(x, -1)
                w = torch.exp(x - torch.where(part == -math.inf, 0.0, part)[..., None])
                o[cu[b] + a:cu[b] + z, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", w, v)
                lse[cu[b] + a:cu[b] + z, h * G:(h + 1) * G] = part.T
    return o, lse


def _nearest(x, grid):
    """The nearest value of an ascending grid, ties to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])

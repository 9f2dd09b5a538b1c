"""An attention layer's serving step around the paged 4-bit cache: its cases, and the plain forms.

The step of one layer: the residual is added and normed, with an output in 8 bits for the projections
(norm); queries and keys are rotated and stored as 4-bit codes (append); the pages that a token attends
to are picked by a score that bounds its products with their keys (pick); attention over them (attend).

A pool is uint8 [pages][Hkv][P / 16][18 D]: for each page and head, tiles of 16 tokens, each

    K codes [16][D / 2] | K scales [16][D / 16] | V codes [16][D / 2] | V scales [D / 16][16]

Codes are e2m1 (even channel in the low nibble), scales e4m3, one for 16 channels of a token.  The bounds
of a page's keys are int8 [pages][Hkv][2 D + 16]: per channel the largest, then the smallest, in units of
2^e, then e.

``run`` computes with elementary torch operations, or, with ``own`` set, through the library.
"""
import math
import random

import torch

own = False

TILE = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"
EPS = 1e-5


def _kda():
    import kda_state_gb300
    return kda_state_gb300


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one user's chat: a single row, 64 heads of 128 channels wide; what counts is latency
        dict(name="norm_one", kind="norm", T=1, C=8192, scales="row", dtype="bf16"),
        # a mixed batch of a smaller model at an odd number of rows, output for 16-bit projections
        dict(name="norm_mixed", kind="norm", T=5003, C=2560, scales="none", dtype="fp16"),
        # the prompts of a full prefill batch, a scale for each 128 channels
        dict(name="norm_prompt", kind="norm", T=16384, C=8192, scales="block", dtype="bf16"),
        # the new token of each of 384 requests is rotated and stored
        dict(name="append_step", kind="append", B=384, n=1, lo=1, hi=8192, Hq=64, Hkv=8, D=128, P=64, R=128, pairs=False, dtype="bf16"),
        # drafts of 64 requests, heads of 64 channels of which half turn, neighbours as pairs
        dict(name="append_drafts", kind="append", B=64, n=8, lo=100, hi=5000, Hq=32, Hkv=32, D=64, P=32, R=32, pairs=True, dtype="fp16"),
        # prompts of 64 to 2048 tokens, far into their contexts
        dict(name="append_prompt", kind="append", B=8, n=2048, lo=64, hi=60000, Hq=64, Hkv=8, D=128, P=64, R=64, pairs=False, dtype="bf16"),
        # one long conversation: the pages of its next token
        dict(name="pick_one", kind="pick", B=1, n=1, lo=131071, hi=131071, Hq=64, Hkv=8, D=128, P=64, count=32, first=1, recent=2, dtype="bf16"),
        # a serving batch, every request at another length, some shorter than what is picked
        dict(name="pick_batch", kind="pick", B=96, n=1, lo=900, hi=16383, Hq=64, Hkv=8, D=128, P=32, count=64, first=1, recent=4, dtype="bf16"),
        # a piece of a prompt on top of its prefix: every token has its own pages
        dict(name="pick_prompt", kind="pick", B=2, n=1024, lo=4099, hi=24576, Hq=32, Hkv=8, D=64, P=64, count=32, first=1, recent=2, dtype="fp16"),
        # the same conversation's attention: 32 of its 2048 pages
        dict(name="attend_one", kind="attend", B=1, n=1, lo=131071, hi=131071, Hq=64, Hkv=8, D=128, P=64, count=32, dtype="bf16"),
        # the batch's attention
        dict(name="attend_batch", kind="attend", B=96, n=1, lo=900, hi=16383, Hq=64, Hkv=8, D=128, P=32, count=64, dtype="bf16"),
        # drafts of 32 requests, each with its own pages of which most are its neighbours' too
        dict(name="attend_drafts", kind="attend", B=32, n=6, lo=3001, hi=20011, Hq=64, Hkv=8, D=128, P=64, count=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "append", "append", "pick", "pick", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "norm":
        C = 8 * _log(rng, 8, 1024)
        T = min(_log(rng, 1, 32768), 16384 * 8192 // C)
        return dict(kind="norm", T=T, C=C, scales=rng.choice(["none", "row", "block"]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    D = rng.choice([64, 128, 128])
    P = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 3, 4, 5, 8, 8, 16])
    if kind == "append":
        n = rng.choice([1, rng.randint(2, 16), _log(rng, 17, 2048)])
        B = max(1, min(_log(rng, 1, 384), 8192 // n))
        hi = n + _log(rng, 1, 32768)
        return dict(kind="append", B=B, n=n, lo=rng.randint(n, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, P=P,
                    R=rng.choice([32, 64] if D == 64 else [32, 64, 96, 128, 128]), pairs=rng.random() < 0.4, dtype=dtype)
    hi = _log(rng, 64, 131072)
    n = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, 512)])
    hi = max(hi, n)
    B = max(1, min(_log(rng, 1, 128), 400000 // hi, 1024 // n))
    c = dict(kind=kind, B=B, n=n, lo=rng.randint(n, hi), hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D, P=P, count=_log(rng, 4, 128), dtype=dtype)
    if kind == "pick":
        c["first"] = rng.randint(0, min(2, c["count"] - 1))
        c["recent"] = rng.randint(1, c["count"] - c["first"])
        return c
    # what the plain form lays out fits the card
    c["B"] = B = max(1, min(B, 300000000 // (n * Hkv * c["count"] * P * D)))
    c["n"] = max(1, min(n, 300000000 // (B * Hkv * c["count"] * P * D)))
    return c


def _spread(count, lo, hi):
    """count whole numbers spread over [lo, hi] in no order; the same for every seed."""
    return [lo + int((hi - lo + 1) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(count)]


def _requests(c):
    """(new tokens, tokens in the cache with them) of each request."""
    lens = _spread(c["B"], c["lo"], c["hi"])
    new = [c["n"]] * c["B"]
    if c["n"] > 16:                        # prompts: ragged
        new = [c["n"]] + _spread(c["B"] - 1, max(1, c["n"] // 32), c["n"])
    return new, [max(l, n) for l, n in zip(lens, new)]


def _shared(c):
    """Of the pages picked, those that all new tokens of a request have in common where they can."""
    return c["count"] * 3 // 4


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["kind"] == "norm":
        cells = c["T"] * c["C"]
        out = {"none": size, "row": 1, "block": 1}[c["scales"]] * cells
        scales = {"none": 0, "row": 4, "block": 4 * -(-c["C"] // 128)}[c["scales"]] * c["T"]
        return {"bytes": 3 * size * cells + out + scales + size * c["C"], "flops": 8 * cells}
    new, lens = _requests(c)
    T, Hkv, D, P = sum(new), c["Hkv"], c["D"], c["P"]
    pages = [[(l - n + i) // P + 1 for i in range(n)] for n, l in zip(new, lens)]      # that each token sees
    if c["kind"] == "append":
        q, kv = T * c["Hq"] * D * 2, 2 * T * Hkv * D * 2
        return {"bytes": 2 * q + kv + 2 * (kv * 9 // 32) + kv + T * c["R"] * 4, "flops": 3 * T * c["R"] * (c["Hq"] + Hkv) + 2 * kv}
    if c["kind"] == "pick":
        touched = sum(p[-1] - (l - n) // P for p, n, l in zip(pages, new, lens))
        seen = sum(map(sum, pages))
        return {"bytes": T * c["Hq"] * D * 2 + sum(p[-1] for p in pages) * Hkv * (2 * D + 16) + touched * Hkv * (P * D * 9 // 16 + 2 * D + 16) +
                T * Hkv * c["count"] * 4, "flops": 4 * D * Hkv * seen}
    read, pairs = 0, 0
    for p, n, l in zip(pages, new, lens):
        each = [min(c["count"], x) for x in p]
        common = min(_shared(c), each[-1])
        read += min(l, (common + sum(x - min(common, x) for x in each)) * P)
        pairs += sum((x - 1) * P + (l - n + i) % P + 1 for i, x in enumerate(each))
    return {"bytes": read * Hkv * D * 9 // 8 + T * c["Hq"] * (D * 4 + 4) + T * Hkv * c["count"] * 4, "flops": 4 * D * c["Hq"] * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

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


def _rows(g, count, heads, D):
    """Keys or values as projections make them: channels of different strength."""
    strength = 0.5 + torch.rand(heads, D, generator=g, device=DEV) * 2.0
    return torch.randn(count, heads, D, generator=g, device=DEV) * strength


def _filled_pool(c, g, pages, table):
    """A pool whose held pages carry quantised rows, drawn from a bank of them with a lean of the page's own, and whose
    others are stale."""
    Hkv, D, P = c["Hkv"], c["D"], c["P"]
    pool = torch.full((pages, Hkv, P // TILE, 18 * D), 255, dtype=torch.uint8, device=DEV)
    held = table[table >= 0].long()
    bank = []
    for side in range(2):
        lean = torch.randn(64, 1, D, generator=g, device=DEV) * 0.8
        codes, scales = _quantise(_rows(g, 8192, 1, D)[:, 0].unflatten(0, (64, 128)) + lean)
        bank.append(torch.cat([codes, scales.view(torch.uint8)], -1).flatten(0, 1))
    for a in range(0, held.numel(), 4096):
        part = held[a:a + 4096]
        shape = (part.numel(), Hkv, P // TILE, TILE)
        lean = 128 * torch.randint(0, 64, shape[:2] + (1, 1), generator=g, device=DEV)
        k = bank[0][lean + torch.randint(0, 128, shape, generator=g, device=DEV)]
        v = bank[1][torch.randint(0, 8192, shape, generator=g, device=DEV)]
        pool[part] = torch.cat([k[..., :D // 2].flatten(-2), k[..., D // 2:].flatten(-2),
                                v[..., :D // 2].flatten(-2), v[..., D // 2:].transpose(-1, -2).flatten(-2)], -1)
    return pool


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(7919 * seed + 23)
    s = {"case": c}
    dt = DTYPES[c["dtype"]]
    if c["kind"] == "norm":
        T, C = c["T"], c["C"]
        # the residual stream is larger than what a layer adds, and some of its channels are much larger
        loud = 1 + 15 * (torch.rand(C, generator=g, device=DEV) < 0.01)
        s["x"] = torch.randn(T, C, generator=g, device=DEV).to(dt)
        s["residual"] = (torch.randn(T, C, generator=g, device=DEV) * 3 * loud).to(dt)
        s["weight"] = (0.5 + torch.rand(C, generator=g, device=DEV)).to(dt)
        return s
    new, lens = _requests(c)
    T, M = sum(new), -(-max(lens) // c["P"]) + 1
    need = [-(-l // c["P"]) for l in lens]
    pages = sum(need) + 5
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["B"], M), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(M, device=DEV)[None] < _i32(need)[:, None]] = perm[:sum(need)]
    s["table"], s["max_new"], s["cu"] = table, max(new), _i32([0] + torch.tensor(new).cumsum(0).tolist())
    s["lens"], s["start"] = _i32(lens), _i32([l - n for l, n in zip(lens, new)])
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    # the queries are a view of the fused projection's output, and some look for something
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV)
    qkv *= 0.5 + 2.0 * torch.rand(T, qkv.shape[1], 1, generator=g, device=DEV)
    qkv = qkv.to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if c["kind"] == "append":
        s["k_scale"], s["v_scale"] = 1.0, 0.5
        s["pool"] = torch.zeros(pages, Hkv, c["P"] // TILE, 18 * D, dtype=torch.uint8, device=DEV)
        angle = torch.arange(max(lens), device=DEV).double()[:, None] * _turns(c["R"])
        s["rope"] = torch.cat([angle.cos(), angle.sin()], -1).float()
        return s
    s["pool"] = _filled_pool(c, g, pages, table)
    if c["kind"] == "pick":
        s["bounds"] = torch.zeros(pages, Hkv, 2 * D + 16, dtype=torch.int8, device=DEV)
        held, P = table.flatten(), c["P"]
        fill = (s["lens"][:, None] - torch.arange(M, device=DEV) * P).clamp(0, P).flatten()
        held, fill = held[held >= 0].long(), fill[held >= 0]
        for a in range(0, held.numel(), 1024):
            s["bounds"][held[a:a + 1024]] = _bounds_of(s["pool"][held[a:a + 1024]], fill[a:a + 1024], D)
        s["workspace"] = torch.zeros(4 * T * Hkv * M + 16 * T + 4096, dtype=torch.uint8, device=DEV)
        return s
    s["k_scale"], s["v_scale"], s["scale"] = 1.0, 0.5, D ** -0.5
    s["workspace"] = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
    # the first page, the own and the one before it, a common part, and the rest each token's own
    b, i = _owners(s["cu"], T)
    mine = (s["start"][b] + i) // c["P"]
    at = torch.arange(M, device=DEV)
    rank = torch.rand(c["B"], Hkv, M, generator=g, device=DEV)
    rank = torch.where(at < ((s["start"] + c["P"] - 1) // c["P"]).clamp(min=1)[:, None, None], rank, -1.0)
    common = torch.zeros(c["B"], Hkv, M, dtype=torch.bool, device=DEV)
    common.scatter_(2, rank.topk(min(M, max(1, _shared(c) - 3)), -1).indices, True)
    score = torch.rand(T, Hkv, M, generator=g, device=DEV) + 2.0 * common[b]
    score += 4.0 * ((at == 0) | (at >= mine[:, None] - 1))[:, None] + 4.0 * (at == mine[:, None])[:, None]
    s["picked"] = _take(torch.where(at <= mine[:, None, None], score, -math.inf), mine, c["count"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _turns(R):
    """Radians a position of each of the R / 2 pairs."""
    return 10000.0 ** (-torch.arange(0, R, 2, device=DEV).double() / R)


def _values(codes, scales, factor):
    """What codes [..., D / 2] and scales [..., D / 16] stand for, in 32 bits."""
    table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device=codes.device)
    pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)      # by byte: low, high nibble
    x = pairs[codes.int()].flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * (scales.view(torch.float8_e4m3fn).float() * factor)[..., None]).flatten(-2)


def _keys(tiles, D, factor):
    """K [..., tiles, 16, D] of tiles [..., 18 D]."""
    return _values(tiles[..., :8 * D].unflatten(-1, (TILE, D // 2)), tiles[..., 8 * D:9 * D].unflatten(-1, (TILE, D // 16)).contiguous(), factor)


def _vals(tiles, D, factor):
    return _values(tiles[..., 9 * D:17 * D].unflatten(-1, (TILE, D // 2)),
                   tiles[..., 17 * D:].unflatten(-1, (D // 16, TILE)).transpose(-1, -2).contiguous(), factor)


def _owners(cu, T):
    """(request, index in it) of each of T packed tokens."""
    t = torch.arange(T, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, (t - cu[b]).long()


def _norm(s):
    c, x, w = s["case"], s["x"], s["weight"].float()
    h = (x.float() + s["residual"].float()).to(x.dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    if c["scales"] == "none":
        return y.to(x.dtype), h
    width = c["C"] if c["scales"] == "row" else 128
    parts = torch.nn.functional.pad(y, (0, -c["C"] % width)).unflatten(-1, (-1, width))
    scale = parts.abs().amax(-1) / 448.0
    code = parts / torch.where(scale == 0, 1.0, scale)[..., None]
    code = code.clamp(-448.0, 448.0).flatten(-2)[:, :c["C"]].to(torch.float8_e4m3fn)
    return code, scale[:, 0] if c["scales"] == "row" else scale, h


def _rotate(x, cos, sin, pairs):
    """x [T, H, D] with its first 2 * cos.shape[-1] channels turned, in x's type."""
    R = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    f = x[..., :R].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if pairs else (f[..., :R // 2], f[..., R // 2:])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if pairs else torch.cat(turned, -1)
    return torch.cat([turned.to(x.dtype), x[..., R:]], -1)


def _append(s):
    c, cu, table, pool = s["case"], s["cu"], s["table"], s["pool"]
    D, P, T = c["D"], c["P"], s["q"].shape[0]
    b, i = _owners(cu, T)
    pos = s["start"][b].long() + i
    cos, sin = s["rope"][pos].chunk(2, -1)
    q, k = _rotate(s["q"], cos, sin, c["pairs"]), _rotate(s["k"], cos, sin, c["pairs"])
    page, tile, tok = table[b, pos // P].long(), pos % P // TILE, pos % TILE
    kc, ks = _quantise(k.float() / s["k_scale"])
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
    return q, k.to(s["k"].dtype), v.to(s["v"].dtype)


def _power(e):
    """2^e, by its bits."""
    return (e.to(torch.int32) + 127 << 23).view(torch.float32)


def _exponent(top):
    """The least e with top <= 127 x 2^e, of finite top > 0."""
    m, e = torch.frexp(top)                               # top = m 2^e, m in [0.5, 1)
    return e.long() - 7 + (m > 127 / 128)


def _bounds_of(tiles, fill, D):
    """Records [pages, Hkv, 2 D + 16] of pages' tiles [pages, Hkv, P / 16, 18 D] with fill [pages] tokens."""
    k = _keys(tiles, D, 1.0).flatten(2, 3)                # [pages, Hkv, P, D]
    there = (torch.arange(k.shape[2], device=k.device) < fill[:, None])[:, None, :, None]
    hi = torch.where(there, k, -math.inf).amax(2)
    lo = torch.where(there, k, math.inf).amin(2)
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1)      # of a NaN: NaN
    nan = top.isnan()
    e = torch.where(top > 0, _exponent(torch.where(top > 0, top, 1.0)), 0)
    unit = _power(e)[..., None]
    hi, lo = (torch.where(nan[..., None], 0.0, x).to(torch.int8) for x in (torch.ceil(hi / unit), torch.floor(lo / unit)))
    end = torch.nn.functional.pad(torch.where(nan, 127, e).to(torch.int8)[..., None], (0, 15))
    return torch.cat([hi, lo, end], -1)


def _take(score, mine, count):
    """The count best of score [T, Hkv, M], ties to the lowest, ascending, -1 behind: int32 [T, Hkv, count]."""
    M = score.shape[-1]
    best = torch.argsort(score, dim=-1, descending=True, stable=True)[..., :count]
    many = (mine + 1).clamp(max=count)
    best = torch.where(torch.arange(best.shape[-1], device=score.device) < many[:, None, None], best, M)
    best = torch.nn.functional.pad(best.sort(-1).values, (0, count - best.shape[-1]), value=M)
    return torch.where(best < M, best, -1).to(torch.int32)


def _wanted(q, Hkv):
    """Whole numbers u, d [T, Hkv, D] that stand for what a kv head's queries ask of channels upwards and downwards."""
    q = q.double().unflatten(1, (Hkv, -1))
    up, down = q.clamp(min=0).sum(2), (-q).clamp(min=0).sum(2)
    top = torch.maximum(up, down).amax(-1)
    good = top.float().isfinite() & (top > 0)
    e = torch.where(good, _exponent(torch.where(good, top, 1.0)), 0).clamp(min=-100)
    unit = _power(e).double()[..., None]
    return (torch.where(good[..., None], torch.round(x / unit), 0.0).float() for x in (up, down))


def _pick(s):
    c, q, table, cu = s["case"], s["q"], s["table"], s["cu"]
    D, P, Hkv, M, T = c["D"], c["P"], c["Hkv"], table.shape[1], q.shape[0]
    b, i = _owners(cu, T)
    mine = s["start"][b] + i.to(torch.int32)
    # the bounds of the pages that the new tokens lie in; where one has several of them, all write the same
    page = table[b, (mine // P).long()].long()
    fill = torch.minimum(s["lens"][b] - mine // P * P, torch.tensor(P, device=DEV))
    s["bounds"][page] = _bounds_of(s["pool"][page], fill, D)
    mine = mine // P
    records = s["bounds"][table.clamp(min=0).long()].transpose(1, 2)               # [B, Hkv, M, 2 D + 16]
    up, down = _wanted(q, Hkv)
    ask = torch.zeros(c["B"], s["max_new"], Hkv, 2 * D, device=DEV)
    ask[b, i] = torch.cat([up, -down], -1)
    # sums of whole numbers below 2^24, times a power of two: exact in 32 bits
    score = ask.transpose(1, 2) @ records[..., :2 * D].float().transpose(-1, -2)   # [B, Hkv, max_new, M]
    e = records[..., None, :, 2 * D]
    score = torch.where(e == 127, math.inf, score * _power(e)).transpose(1, 2)[b, i]
    at = torch.arange(M, device=DEV)
    must = (at < c["first"]) | (at > mine[:, None] - c["recent"])
    rank = torch.argsort(torch.argsort(score, dim=-1, descending=True, stable=True), dim=-1)   # the lowest first among equals
    key = torch.where(must[:, None], 2.0 * M, M - rank.float())
    return [_take(torch.where(at <= mine[:, None, None], key, -1.0).masked_fill((at > mine[:, None])[:, None], -math.inf), mine, c["count"]), s["bounds"]]


def _attend(s):
    c, q, table = s["case"], s["q"], s["table"]
    Hq, Hkv, D, P, T, N = c["Hq"], c["Hkv"], c["D"], c["P"], q.shape[0], c["count"]
    b, i = _owners(s["cu"], T)
    me = s["start"][b].long() + i
    picked = s["picked"].long()
    page = table[b[:, None, None], picked.clamp(min=0)].clamp(min=0).long()
    tiles = s["pool"][page, torch.arange(Hkv, device=DEV)[:, None]].flatten(2, 3)  # [T, Hkv, N P / 16, 18 D]
    at = (picked[..., None] * P + torch.arange(P, device=DEV)).flatten(2)
    seen = ((picked >= 0)[..., None].expand(T, Hkv, N, P).flatten(2) & (at <= me[:, None, None]))[:, :, None]
    rows = q.float().unflatten(1, (Hkv, -1))                                       # [T, Hkv, G, D]
    k = torch.where(seen[:, :, 0, :, None], _keys(tiles, D, s["k_scale"]).flatten(2, 3), 0.0)
    score = ((rows @ k.transpose(-1, -2)) * s["scale"]).masked_fill(~seen, -math.inf)
    del k
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, 0, :, None], _vals(tiles, D, s["v_scale"]).flatten(2, 3), 0.0)
    o = (p @ v) / total
    return o.reshape(T, Hq, D).to(q.dtype), (top + torch.log(total)).reshape(T, Hq)


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _norm, "append": _append, "pick": _pick, "attend": _attend}[c["kind"]](s)
    kda = _kda()
    if c["kind"] == "norm":
        out, scales, h = kda.kda_add_rmsnorm(s["x"], s["residual"], s["weight"], eps=EPS, scales=c["scales"])
        return (out, h) if scales is None else (out, scales, h)
    if c["kind"] == "append":
        q = kda.kda_kv4_append_rope(s["q"], s["k"], s["v"], s["rope"], s["cu"], s["start"], s["table"], s["pool"], pairs=c["pairs"],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"])
        k, v = kda.kda_kv4_gather(s["cu"], s["start"], q.shape[0], s["table"], s["pool"], dtype=q.dtype, k_scale=s["k_scale"],
                                  v_scale=s["v_scale"])
        return q, k, v
    if c["kind"] == "pick":
        kda.kda_kv4_bounds(s["cu"], s["start"], s["q"].shape[0], s["table"], s["pool"], s["bounds"])
        picked = kda.kda_kv4_pick(s["q"], s["cu"], s["max_new"], s["lens"], s["table"], s["bounds"], c["P"], c["count"], first=c["first"],
                                  recent=c["recent"], workspace=s["workspace"])
        return [picked, s["bounds"]]
    return kda.kda_kv4_attention_picked(s["q"], s["cu"], s["max_new"], s["lens"], s["table"], s["picked"], s["pool"], scale=s["scale"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["workspace"])


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


def _nearest(x, grid):
    """The nearest value of an ascending grid, ties to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = x - grid[lo], grid[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])


def _stored(x, factor):
    """What 4-bit codes and their scales keep of x [..., D]."""
    x = (x / factor).unflatten(-1, (-1, 16))
    scale = _nearest((x.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0), _e4m3(torch.arange(127, device=x.device).double()))
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    mags = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (_nearest(y.abs(), mags) * torch.sign(y) * scale).flatten(-2) * factor


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["kind"] == "norm":
        h = s["x"].double() + s["residual"].double()
        f = h.to(s["x"].dtype).double()
        y = f / ((f ** 2).sum(-1, keepdim=True) / c["C"] + EPS).sqrt() * s["weight"].double()
        if c["scales"] == "none":
            return y, h
        width = c["C"] if c["scales"] == "row" else 128
        cut = [y[:, a:a + width] for a in range(0, c["C"], width)]
        scales = [x.abs().max(-1, keepdim=True).values / 448 for x in cut]
        code = torch.cat([x / m for x, m in zip(cut, scales)], -1)
        return code, scales[0][:, 0] if c["scales"] == "row" else torch.cat(scales, -1), h
    cu, start, lens = s["cu"].tolist(), s["start"].tolist(), s["lens"].tolist()
    D, P, B, Hkv = c["D"], c["P"], c["B"], c["Hkv"]
    if c["kind"] == "append":
        pos = torch.cat([start[b] + torch.arange(cu[b + 1] - cu[b], device=DEV) for b in range(B)]).double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos[:, None] * _turns(c["R"]))[:, None]
        half = c["R"] // 2

        def turned(x):
            x = x.double()
            z = torch.complex(x[..., 0:c["R"]:2], x[..., 1:c["R"]:2]) if c["pairs"] else torch.complex(x[..., :half], x[..., half:c["R"]])
            z = z * turn
            z = torch.view_as_real(z).flatten(-2) if c["pairs"] else torch.cat([z.real, z.imag], -1)
            return torch.cat([z, x[..., c["R"]:]], -1)
        k = turned(s["k"]).to(s["k"].dtype).double()           # what a key is stored from has its type
        return turned(s["q"]), _stored(k, s["k_scale"]), _stored(s["v"].double(), s["v_scale"])
    q = s["q"].double()
    G = c["Hq"] // Hkv
    if c["kind"] == "pick":
        return None                                            # whole numbers
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    for b in range(B):
        for h in range(Hkv):
            k = _cached(s["pool"], s["table"][b], lens[b], P, D, h, True, s["k_scale"])
            v = _cached(s["pool"], s["table"][b], lens[b], P, D, h, False, s["v_scale"])
            at = torch.arange(lens[b], device=q.device)
            for t in range(cu[b], cu[b + 1]):
                there = torch.isin(at // P, s["picked"][t, h]) & (at <= start[b] + t - cu[b])
                x = q[t, h * G:(h + 1) * G] @ k[there].T * s["scale"]
                lse[t, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
                o[t, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v[there]
    return o, lse

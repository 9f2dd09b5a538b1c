"""Serving steps of a small hybrid model: a KDA layer's recurrent state beside an attention
layer's paged 4-bit cache, for one batch of requests.

    python examples/hybrid_step.py [--requests 6] [--steps 4] [--seed 0] [--pick COUNT]

Per step every request decodes one token through both layers.  Around the steps: prompts in
pieces, a fork (copy-on-write of pages and of the state slot), a verify of draft tokens of which
a part is accepted, requests that end, and a compaction that hands the pool's upper pages back.
Projections are random numbers: the example shows the calls and their order.

With --pick the attention layer begins with the residual's addition and norm, rotates its queries
and keys on their way into the cache, and reads COUNT pages of each row that a score picks.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_state_gb300 as kda  # noqa: E402

H, HQ, HKV, D, PAGE, MAX_PAGES, PAGES = 4, 16, 2, 128, 64, 40, 200
DEV = "cuda"


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


class Hybrid:
    """The memory of one KDA layer and one attention layer, and a step through both."""

    def __init__(self, rows, seed=0):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        # recurrent layer: a state slot per row
        self.states = torch.zeros(rows, H, D, D, device=DEV)
        # attention layer: pages, who holds them, and each row's list of them
        self.pool = kda.make_kv4_pool(PAGES, PAGE, HKV, D, DEV)
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device=DEV)
        self.table = torch.full((rows, MAX_PAGES), -1, dtype=torch.int32, device=DEV)
        self.lens = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.workspace = kda.make_kv4_workspace(DEV)

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device=DEV).to(torch.bfloat16)

    def attend(self, rows, new):
        """Store `new` tokens of each of `rows` and attend to the cache from them.  Returns (q, k, v, o, lse)."""
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        grow = torch.zeros_like(self.lens)
        grow[rows.long()] = i32(new)
        kda.kda_page_alloc(self.refs, self.table, self.lens, grow, PAGE, dev_err=self.err)
        table, lens = self.table[rows.long()], self.lens[rows.long()]
        qkv = self.rand(sum(new), HQ + 2 * HKV, D)              # the fused projection's output
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        kda.kda_kv4_append(k, v, cu, lens - i32(new), table, self.pool, dev_err=self.err)
        o, lse = kda.kda_kv4_attention(q, cu, max(new), lens, table, self.pool, workspace=self.workspace, dev_err=self.err)
        return q, k, v, o, lse

    def prompt(self, rows, lengths, piece=100):
        """Prompts, `piece` tokens at a time: through the recurrent layer (state to state) and the cache."""
        outs = []
        for at in range(0, max(lengths), piece):
            part = [(int(r), min(piece, n - at)) for r, n in zip(rows.tolist(), lengths) if n > at]
            ids, new = i32([r for r, _ in part]), [n for _, n in part]
            cu = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32)
            T = int(cu[-1])
            kn = torch.nn.functional.normalize(self.rand(T, H, D).float(), dim=-1).to(torch.bfloat16)
            kda.kda_chunk_prefill(self.rand(T, H, D), kn, self.rand(T, H, D), -self.rand(T, H, D).abs(),
                                  torch.rand(T, H, generator=self.g, device=DEV).to(torch.bfloat16), cu.to(DEV), cu,
                                  self.states, ids, ids, dev_err=self.err)
            outs.append(self.attend(ids, new))
        return outs

    def decode(self, rows):
        n = rows.numel()
        kn = torch.nn.functional.normalize(self.rand(n, H, D).float(), dim=-1).to(torch.bfloat16)
        o = kda.kda_decode_step(self.rand(n, H, D), kn, self.rand(n, H, D), -self.rand(n, H, D).abs(),
                                torch.rand(n, H, generator=self.g, device=DEV).to(torch.bfloat16), rows, self.states,
                                dev_err=self.err)
        return o, self.attend(rows, [1] * n)

    def fork(self, src, dst):
        kda.kda_slot_copy([self.states], src, dst, dev_err=self.err)
        kda.kda_page_fork([self.pool], self.refs, self.table, self.lens, src, dst, PAGE, dev_err=self.err)

    def verify(self, rows, drafts, accepted):
        """Attend from the drafts, then take back what was not accepted."""
        out = self.attend(rows, [drafts] * rows.numel())
        back = torch.zeros_like(self.lens)
        back[rows.long()] = i32(accepted) - drafts
        kda.kda_page_alloc(self.refs, self.table, self.lens, back, PAGE, dev_err=self.err)
        return out

    def end(self, rows):
        kda.kda_page_free(self.refs, self.table, self.lens, rows, PAGE, dev_err=self.err)

    def compact(self):
        return kda.kda_page_compact([self.pool], self.refs, self.table, dev_err=self.err)


class SparseHybrid(Hybrid):
    """The same with an attention layer that adds and norms the residual stream, rotates, and reads `count` pages."""

    def __init__(self, rows, count, seed=0):
        super().__init__(rows, seed)
        self.count = count
        self.bounds = kda.make_kv4_bounds(PAGES, HKV, D, DEV)
        self.rope = kda.make_rope_table(MAX_PAGES * PAGE, D, device=DEV)
        self.norm = 1 + 0.1 * self.rand(HQ * D)
        self.proj = self.rand(HQ * D, (HQ + 2 * HKV) * D) / (HQ * D) ** 0.5
        self.residual = None

    def attend(self, rows, new):
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        grow = torch.zeros_like(self.lens)
        grow[rows.long()] = i32(new)
        kda.kda_page_alloc(self.refs, self.table, self.lens, grow, PAGE, dev_err=self.err)
        table, lens, T = self.table[rows.long()], self.lens[rows.long()], sum(new)
        start = lens - i32(new)
        self.residual = self.rand(T, HQ * D)
        y, scales, _ = kda.kda_add_rmsnorm(self.rand(T, HQ * D), self.residual, self.norm, scales="block", residual_out=self.residual)
        y = (y.float().view(T, -1, 128) * scales[..., None]).view(T, -1).to(torch.bfloat16)      # an 8-bit product's operands
        qkv = (y @ self.proj).view(T, HQ + 2 * HKV, D)
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        q = kda.kda_kv4_append_rope(q, k, v, self.rope, cu, start, table, self.pool, q_out=q, dev_err=self.err)
        kda.kda_kv4_bounds(cu, start, T, table, self.pool, self.bounds, dev_err=self.err)
        self.picked = kda.kda_kv4_pick(q, cu, max(new), lens, table, self.bounds, PAGE, self.count, dev_err=self.err)
        o, lse = kda.kda_kv4_attention_picked(q, cu, max(new), lens, table, self.picked, self.pool, workspace=self.workspace,
                                              dev_err=self.err)
        return q, k, v, o, lse

    def rebound(self, rows):
        """The records of all pages that rows hold, anew: a fork's copied page has none, and a compaction moves pages alone."""
        lens = self.lens[rows.long()]
        cu = i32([0] + lens.cumsum(0).tolist())
        kda.kda_kv4_bounds(cu, torch.zeros_like(lens), int(cu[-1]), self.table[rows.long()], self.pool, self.bounds, dev_err=self.err)

    def fork(self, src, dst):
        super().fork(src, dst)
        self.rebound(dst)

    def compact(self):
        live = super().compact()
        self.rebound(torch.arange(self.lens.numel(), dtype=torch.int32, device=DEV))
        return live


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--pick", type=int, default=0, help="pages that a token's attention reads (0: all)")
    a = ap.parse_args(argv)
    n = a.requests
    m = SparseHybrid(n + 2, a.pick, a.seed) if a.pick else Hybrid(n + 2, a.seed)
    rows = i32(list(range(n)))
    m.prompt(rows, [37 + 61 * i for i in range(n)])
    for _ in range(a.steps):
        m.decode(rows)
    m.fork(rows[:2], i32([n, n + 1]))                            # two requests go on in two ways
    rows = i32(list(range(n + 2)))
    m.verify(rows, 8, [1 + i % 8 for i in range(n + 2)])
    for _ in range(a.steps):
        o_state, (_, _, _, o_cache, _) = m.decode(rows)
    m.end(rows[::2].contiguous())
    live = m.compact()
    rows = rows[1::2].contiguous()
    m.decode(rows)
    torch.cuda.synchronize()
    if int(m.err):
        raise SystemExit("device errors: %d" % int(m.err))
    print("rows %d, tokens %s, pages held %d of %d; o(state) rms %.3f, o(cache) rms %.3f" % (
        rows.numel(), m.lens.tolist(), int(live), PAGES, o_state.float().square().mean().sqrt(),
        o_cache.float().square().mean().sqrt()))
    return m


if __name__ == "__main__":
    main()

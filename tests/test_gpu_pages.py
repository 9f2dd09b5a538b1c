"""The pages' bookkeeping on the GPU: equal to the oracle's, number for number and byte for byte."""
import numpy as np
import pytest
import torch

from oracle import kv4 as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()


def kda():
    import kda_state_gb300
    return kda_state_gb300


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """The library's state and the oracle's, side by side."""

    def __init__(self, pages, rows, M, P, layers=2, seed=0, page_shape=(3, 48)):
        rng = np.random.default_rng(seed)
        self.o = ref.Pages(pages, rows, M, P)
        self.data = [rng.integers(0, 256, (pages,) + page_shape, dtype=np.uint8) for _ in range(layers)]
        self.pools = [torch.from_numpy(x.copy()).to(DEV) for x in self.data]
        self.refs, self.table, self.lens = i32(self.o.refs), i32(self.o.table), i32(self.o.lens)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.P = P

    def state(self):
        return self.refs, self.table, self.lens

    def same(self, err=0):
        torch.cuda.synchronize()
        assert int(self.err) == err
        self.err.zero_()
        assert self.refs.tolist() == self.o.refs
        assert self.table.tolist() == self.o.table
        assert self.lens.tolist() == self.o.lens
        for p, x in zip(self.pools, self.data):
            assert np.array_equal(p.cpu().numpy(), x)

    def alloc(self, grow):
        kda().kda_page_alloc(*self.state(), i32(grow), self.P, dev_err=self.err)
        self.same(64 if self.o.alloc(grow) else 0)

    def fork(self, src, dst, **kw):
        kda().kda_page_fork(self.pools, *self.state(), i32(src), i32(dst), self.P, dev_err=self.err, **kw)
        self.same(64 if self.o.fork(src, dst, self.data) else 0)

    def free(self, rows):
        kda().kda_page_free(*self.state(), i32(rows), self.P, dev_err=self.err)
        self.o.free(rows)
        self.same()

    def compact(self, **kw):
        live = kda().kda_page_compact(self.pools, self.refs, self.table, dev_err=self.err, **kw)
        assert int(live) == self.o.compact(self.data)
        self.same()


def test_one_page_at_a_time():
    s = Both(6, 3, 4, 16)
    s.alloc([1, 0, 16])
    s.alloc([15, 17, 1])
    s.free([0])
    s.alloc([0, 0, 31])
    s.fork([1], [0])
    s.compact()


def test_a_pool_that_runs_out():
    s = Both(5, 4, 6, 16)
    s.alloc([33, 17, 20, 0])           # 3 + 2, then none left for the third
    s.alloc([0, 0, 1, 5])
    s.alloc([15, 15, 0, 0])            # fills partial pages: needs nothing
    s.free([1])
    s.alloc([0, 40, 10, 0])            # the second wants 3 of 2: neither it nor the third is served
    s.alloc([0, 0, 10, 0])
    s.fork([0, 2], [1, 3])             # row 0 is full to the page; row 2 takes the last
    s.free([1])
    s.fork([2], [1])                   # nothing left for its partial page
    s.free([0, 1, 2, 3])
    s.compact()


@pytest.mark.parametrize("seed", range(4))
def test_random_steps(seed):
    rng = np.random.default_rng(seed)
    P = [16, 32, 64, 256][seed]
    rows = [5, 40, 130, 9][seed]
    s = Both([60, 300, 1500, 50][seed], rows, 12, P, layers=seed + 1, seed=seed)
    for step in range(40):
        op = rng.integers(5)
        if op <= 1:
            s.alloc([int(rng.integers(0, 2 * P)) if s.o.lens[b] < 10 * P - 1 and rng.random() < .7 else 0 for b in range(rows)])
        elif op == 2:
            full = [b for b in range(rows) if s.o.lens[b]]
            empty = [b for b in range(rows) if not s.o.lens[b]]
            if full and empty:
                n = int(rng.integers(1, len(empty) + 1))
                s.fork([int(x) for x in rng.choice(full, n)], empty[:n])
        elif op == 3:
            s.free([int(x) for x in rng.permutation(rows)[:int(rng.integers(1, rows // 2 + 1))]])
        else:
            s.compact()


def test_rows_shrink():
    s = Both(12, 4, 6, 16)
    s.alloc([40, 33, 16, 0])
    s.alloc([-7, -33, -1, 0])          # a page back, all of them, none
    s.alloc([-1, 0, -15, 96])          # what shrinking frees is there for the growing row
    s.alloc([0, 20, 0, -90])
    s.fork([0], [2])                   # rows 0 and 2 share two full pages
    s.alloc([-3, 0, 5, 0])             # row 0 would write into a shared one: refused
    s.alloc([-16, 0, -21, 0])          # to a border: allowed; row 2 to its own page's start
    s.alloc([-16, 0, 0, 0])
    s.alloc([0, 0, -3, 0])             # now row 2 holds its pages alone


@pytest.mark.parametrize("seed", range(3))
def test_random_steps_with_drafts(seed):
    """Growth by drafts, and back by those not accepted, between forks and ends."""
    rng = np.random.default_rng(50 + seed)
    rows, P = [7, 60, 1100][seed], [16, 32, 16][seed]
    s = Both([40, 200, 4000][seed], rows, 10, P, seed=seed)
    for step in range(25):
        s.alloc([int(rng.integers(1, 9)) if n < 8 * P else 0 for n in s.o.lens])
        s.alloc([-int(rng.integers(0, min(n, 8) + 1)) if rng.random() < .8 else int(n < 8 * P) for n in s.o.lens])
        full = [b for b in range(rows) if s.o.lens[b]]
        s.free([int(x) for x in rng.permutation(full)[:max(1, len(full) // 6)]])
        full = [b for b in range(rows) if s.o.lens[b]]
        empty = [b for b in range(rows) if not s.o.lens[b]]
        if full and empty:
            s.fork([full[0]] * len(empty[:3]), empty[:3])


def test_large_tables_cross_the_scan_steps():
    """More pages than one scan step (16384), more rows than one block (1024)."""
    s = Both(50000, 2500, 20, 16, layers=1, page_shape=(16,))
    rng = np.random.default_rng(7)
    s.alloc([int(x) for x in rng.integers(0, 300, 2500)])
    s.free([int(x) for x in rng.permutation(2500)[:1700]])
    s.alloc([int(x) if n == 0 else 0 for n, x in zip(s.o.lens, rng.integers(0, 250, 2500))])
    s.free([int(x) for x in rng.permutation(2500)[:1800]])
    full = [b for b in range(2500) if s.o.lens[b]]
    empty = [b for b in range(2500) if not s.o.lens[b]]
    n = min(1300, len(empty))
    s.fork([full[i % len(full)] for i in range(n)], empty[:n])
    s.compact()
    s.compact()                         # nothing left to move


@pytest.mark.parametrize("bytes_", [16, 1152, 32768, 100016])
def test_copy(bytes_):
    g = torch.Generator(device=DEV).manual_seed(1)
    pools = [torch.randint(0, 256, (20, bytes_), generator=g, device=DEV, dtype=torch.uint8) for _ in range(3)]
    want = [p.clone() for p in pools]
    src, dst = [3, 3, 19, 0], [4, 18, 1, 2]
    for w in want:
        w[dst] = w[src]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    kda().kda_page_copy(pools, i32(src), i32(dst), dev_err=err)
    assert int(err) == 0 and all(torch.equal(a, b) for a, b in zip(pools, want))
    kda().kda_page_copy(pools, i32([20, -1, 5]), i32([6, 7, 2 ** 31 - 1]), dev_err=err)
    assert int(err) == 32 and all(torch.equal(a, b) for a, b in zip(pools, want))
    halves = [p.view(torch.float16) for p in pools]
    kda().kda_page_copy(halves, i32([5]), i32([6]))
    assert all(torch.equal(p[6], w[5]) for p, w in zip(pools, want))


def test_bad_rows_change_nothing():
    s = Both(40, 6, 5, 16)
    s.alloc([20, 33, 0, 5, 0, 0])
    call = lambda f, *a: (f(*a, dev_err=s.err), torch.cuda.synchronize())
    for src, dst, bit in (([9], [2], 1), ([-1], [2], 1), ([0], [6], 1), ([1], [1], 1), ([0], [3], 4)):
        call(kda().kda_page_fork, s.pools, *s.state(), i32(src), i32(dst), 16)
        s.same(bit)
    for rows, bit in (([6], 1), ([-1], 1)):
        call(kda().kda_page_free, *s.state(), i32(rows), 16)
        s.same(bit)
    for grow in ([0, 0, 81, 0, 0, 0], [0, -34, 0, 0, 0, 0], [0, 0, -1, 0, 0, 0], [0, 0, 0, 2 ** 31 - 1, 0, 0]):
        call(kda().kda_page_alloc, *s.state(), i32(grow), 16)
        s.same(4)
    # an entry that names no page: flagged, the rest of the row goes on
    s.table[1, 1] = 77
    call(kda().kda_page_free, *s.state(), i32([1]), 16)
    assert int(s.err) == 32 and s.lens[1] == 0 and (s.table[1] == -1).all()
    # a page that is free already
    s.err.zero_()
    s.refs[s.table[0, 0]] = 0
    call(kda().kda_page_free, *s.state(), i32([0]), 16)
    assert int(s.err) == 64 and int(s.refs.min()) == 0


def test_refusals():
    s = Both(10, 2, 3, 16)
    with pytest.raises(TypeError, match="refs has dtype"):
        kda().kda_page_alloc(s.refs.long(), s.table, s.lens, s.lens, 16)
    with pytest.raises(ValueError, match="grow has shape"):
        kda().kda_page_alloc(*s.state(), s.lens[:1], 16)
    with pytest.raises(ValueError, match="every pool"):
        kda().kda_page_compact([s.pools[0], s.pools[1][:5]], s.refs, s.table)
    with pytest.raises(kda().KdaError, match="INVALID"):
        kda().kda_page_compact(s.pools, s.refs, s.table, workspace=torch.zeros(8, dtype=torch.int32, device=DEV))
    with pytest.raises(kda().KdaError, match="INVALID"):
        kda().kda_page_free(*s.state(), i32([0]), 24)
    with pytest.raises(ValueError, match="dst has shape"):
        kda().kda_page_copy(s.pools, i32([0]), i32([1, 2]))


def test_captured_step():
    """Growth, fork and free in one graph, replayed from a restored state."""
    s = Both(64, 8, 6, 16)
    s.alloc([20, 33, 0, 5, 64, 0, 0, 1])
    saved = [t.clone() for t in s.state()]
    grow, src, dst, gone = i32([1, 0, 0, 12, 0, 0, 0, 40]), i32([0, 3]), i32([2, 5]), i32([4, 2])
    wsp = torch.zeros(64, dtype=torch.int32, device=DEV)

    def step():
        kda().kda_page_alloc(*s.state(), grow, 16)
        kda().kda_page_fork(s.pools, *s.state(), src, dst, 16, workspace=wsp)
        kda().kda_page_free(*s.state(), gone, 16)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    s.o.alloc([1, 0, 0, 12, 0, 0, 0, 40])
    s.o.fork([0, 3], [2, 5], s.data)
    s.o.free([4, 2])
    for _ in range(3):
        for t, x in zip(s.state(), saved):
            t.copy_(x)
        graph.replay()
        s.same()

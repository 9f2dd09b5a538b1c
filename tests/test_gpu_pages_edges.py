"""The pages' bookkeeping at its edges, equal to the oracle's."""
import numpy as np
import pytest
import torch

from test_gpu_pages import Both, i32, kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()


def consistent(s):
    """Every page is counted once for each entry that names it."""
    held = np.bincount(np.array([p for row in s.o.table for p in row if p >= 0], dtype=int), minlength=len(s.o.refs))
    assert held.tolist() == s.o.refs


def test_rows_forked_to_twice():
    """Of several forks to one row the first is made, wherever the others stand in the list."""
    s = Both(60, 12, 6, 16)
    s.alloc([40, 33, 16, 5, 64, 0, 0, 0, 0, 0, 0, 0])
    fork = lambda src, dst, **kw: (kda().kda_page_fork(s.pools, *s.state(), i32(src), i32(dst), 16, dev_err=s.err), s.same(**kw))
    s.o.fork([0, 3, 4], [5, 6, 7], s.data)
    fork([0, 1, 3, 2, 0, 4, 1], [5, 5, 6, 5, 6, 7, 7], err=4)
    consistent(s)
    # the first has no such source: the second is made
    s.o.fork([2], [8], s.data)
    fork([99, 2, 1], [8, 8, 8], err=1 | 4)
    consistent(s)
    # an empty row is a fork like any other
    fork([9, 0], [10, 10], err=4)
    consistent(s)
    s.free([5, 6, 7, 8])


def test_rows_forked_to_twice_in_a_long_list():
    n = 2600
    s = Both(9000, n + 3, 5, 16, layers=1, page_shape=(16,))
    s.alloc([40, 33, 64] + [0] * n)
    rng = np.random.default_rng(3)
    src, dst = rng.integers(0, 3, n).tolist(), (3 + rng.integers(0, n // 2, n)).tolist()
    first = [i for i in range(n) if dst[i] not in dst[:i]]
    s.o.fork([src[i] for i in first], [dst[i] for i in first], s.data)
    kda().kda_page_fork(s.pools, *s.state(), i32(src), i32(dst), 16, dev_err=s.err)
    s.same(err=4)
    consistent(s)


def test_a_first_fork_without_a_page():
    """The fork that finds no page keeps its row empty, and the later ones to it are still skipped."""
    s = Both(5, 5, 4, 16)
    s.alloc([33, 32, 0, 0, 0])
    kda().kda_page_fork(s.pools, *s.state(), i32([0, 1, 1]), i32([2, 2, 3]), 16, dev_err=s.err)
    s.o.fork([1], [3], s.data)
    s.same(err=64 | 4)
    consistent(s)


@pytest.mark.parametrize("rows", [34, 66])
def test_growth_past_32_bits_of_pages(rows):
    """Rows that together ask for 2^31 (2^32) pages and more: those after the first get none."""
    M, P, N = 1 << 26, 16, 40
    table = torch.full((rows, M), -1, dtype=torch.int32, device=DEV)
    refs, lens, err = i32([0] * N), i32([0] * rows), i32([0])
    kda().kda_page_alloc(refs, table, lens, i32([21] + [1 << 30] * (rows - 2) + [3]), P, dev_err=err)
    assert int(err) == 64
    assert refs.tolist() == [1, 1] + [0] * (N - 2) and lens.tolist() == [21] + [0] * (rows - 1)
    assert table[0, :2].tolist() == [0, 1] and int((table != -1).sum()) == 2

"""The hybrid example with picked pages: records, picks and outputs of every step against the fp64 definitions, through
prompts, decode, a fork, drafts taken back, ends and a compaction."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from kv4_testutil import check
from test_gpu_kv4_layer import all_bounds, expected_picked, picks_of

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from kda_state_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("hybrid_step", os.path.join(ROOT, "examples", "hybrid_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_runs_as_a_program(example, capsys):
    m = example.main(["--requests", "5", "--steps", "2", "--pick", "3"])
    assert "pages held" in capsys.readouterr().out
    held = int((m.refs > 0).sum())
    assert (m.refs[:held] > 0).all() and not m.refs[held:].any()


def test_every_step_picks_by_what_is_stored(example):
    m = example.SparseHybrid(8, 3, 4)

    def follow(rows, new, out):
        q, _, _, o, lse = out
        torch.cuda.synchronize()
        assert int(m.err) == 0
        pool, table, lens = m.pool.cpu().numpy(), m.table.cpu().numpy()[rows], m.lens.cpu().numpy()[rows].tolist()
        rec = all_bounds(pool, table, lens, example.PAGE)
        held = sorted({int(p) for row, n in zip(table, lens) for p in row[:-(-n // example.PAGE)]})
        assert np.array_equal(m.bounds.cpu().numpy()[held], rec[held])
        want = picks_of(q.cpu(), new, lens, rec, table, example.PAGE, 3, 1, 1)
        assert np.array_equal(m.picked.cpu().numpy(), want)
        check(o, lse, expected_picked(q.cpu(), new, lens, pool, table, want, example.PAGE, example.D ** -0.5), torch.bfloat16)

    rows, lengths = [0, 1, 2, 3], [30, 530, 64, 401]
    follow(rows, lengths, m.attend(example.i32(rows), lengths))
    follow(rows, [1] * 4, m.decode(example.i32(rows))[1])
    m.fork(example.i32([1, 3]), example.i32([4, 5]))
    rows = [0, 1, 2, 3, 4, 5]
    follow(rows, [1] * 6, m.decode(example.i32(rows))[1])
    m.verify(example.i32(rows), 8, [1, 8, 3, 5, 2, 7])
    follow(rows, [1] * 6, m.decode(example.i32(rows))[1])
    m.end(example.i32([0, 2, 3]))
    m.compact()
    follow([1, 4, 5], [1] * 3, m.decode(example.i32([1, 4, 5]))[1])

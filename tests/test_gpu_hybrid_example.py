"""The hybrid example end to end: every attention output against fp64 attention over the keys and
values that the cache holds, through prompts, decode, a fork, drafts taken back, ends and a compaction."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from kv4_testutil import check, expected
from oracle import kv4 as ref

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
    m = example.main(["--requests", "5", "--steps", "2"])
    assert "pages held" in capsys.readouterr().out
    held = int((m.refs > 0).sum())
    assert (m.refs[:held] > 0).all() and not m.refs[held:].any()


def test_every_step_attends_to_what_was_stored(example):
    m = example.Hybrid(8, 3)
    history = [np.zeros((0, 2, example.HKV, example.D)) for _ in range(8)]     # k, v of each row as quantised

    def follow(rows, new, out):
        q, k, v, o, lse = out
        at = 0
        for r, n in zip(rows, new):
            kv = np.stack([ref.values(*ref.quantise(x[at:at + n].double().cpu().numpy())) for x in (k, v)], 1)
            history[r] = np.concatenate([history[r], kv])
            at += n
        torch.cuda.synchronize()
        assert int(m.err) == 0
        pool, table, lens = m.pool.cpu().numpy(), m.table.cpu().numpy(), m.lens.tolist()
        for r in range(8):
            assert lens[r] == len(history[r])
            hk, hv = ref.load(pool, table[r], lens[r], example.PAGE)
            assert np.array_equal(hk, history[r][:, 0]) and np.array_equal(hv, history[r][:, 1])
        want = expected(q.cpu(), new, [lens[r] for r in rows], pool, table[rows], example.PAGE, 0, example.D ** -0.5)
        check(o, lse, want, torch.bfloat16)

    rows = [0, 1, 2, 3]
    lengths = [30, 130, 64, 201]
    outs = m.attend(example.i32(rows), lengths)
    follow(rows, lengths, outs)
    _, out = m.decode(example.i32(rows))
    follow(rows, [1] * 4, out)
    m.fork(example.i32([1, 1, 2]), example.i32([4, 5, 6]))
    for a, b in ((1, 4), (1, 5), (2, 6)):
        history[b] = history[a].copy()
        assert torch.equal(m.states[a], m.states[b])
    rows = [0, 1, 2, 3, 4, 5, 6]
    _, out = m.decode(example.i32(rows))
    follow(rows, [1] * 7, out)
    out = m.attend(example.i32(rows), [6] * 7)
    follow(rows, [6] * 7, out)
    kept = [0, 1, 2, 3, 4, 5, 6]
    back = example.i32([k - 6 for k in kept] + [0])
    example.kda.kda_page_alloc(m.refs, m.table, m.lens, back, example.PAGE, dev_err=m.err)
    for r, k in zip(rows, kept):
        history[r] = history[r][:len(history[r]) - 6 + k]
    m.end(example.i32([1, 3]))
    history[1] = history[3] = history[1][:0]
    m.compact()
    rows = [0, 2, 4, 5, 6]
    _, out = m.decode(example.i32(rows))
    follow(rows, [1] * 5, out)

"""Sizes of tensors that the library takes as C ints are not taken modulo 2^32 (CPU: tensors that only claim to be on a
device; nothing is made and nothing called)."""
import pytest
import torch

import kda_state_gb300.binding as binding
from test_stream_buffers import BF, I32, U8, Card, world  # noqa: F401

BIG = 2 ** 32 + 1
POOL, BOUNDS = (8, 2, 1, 1152), (8, 2, 144)


def cards(B=3, M=4):
    return Card(B + 1, dtype=I32), Card(B, dtype=I32), Card(B, M, dtype=I32)


def append_rope(B=3, M=4, rope=(99, 64)):
    cu, start, table = cards(B, M)
    return binding.kda_kv4_append_rope(Card(5, 8, 64, dtype=BF), Card(5, 2, 64, dtype=BF), Card(5, 2, 64, dtype=BF), Card(*rope), cu, start, table,
                                       Card(*POOL, dtype=U8))


def append(B=3, M=4):
    cu, start, table = cards(B, M)
    binding.kda_kv4_append(Card(5, 2, 64, dtype=BF), Card(5, 2, 64, dtype=BF), cu, start, table, Card(*POOL, dtype=U8))


def gather(B=3, M=4):
    cu, start, table = cards(B, M)
    binding.kda_kv4_gather(cu, start, 5, table, Card(*POOL, dtype=U8))


def bounds(B=3, M=4):
    cu, start, table = cards(B, M)
    binding.kda_kv4_bounds(cu, start, 5, table, Card(*POOL, dtype=U8), Card(*BOUNDS, dtype=torch.int8))


def pick(B=3, M=4):
    cu, lens, table = cards(B, M)
    binding.kda_kv4_pick(Card(5, 8, 64, dtype=BF), cu, 1, lens, table, Card(*BOUNDS, dtype=torch.int8), 16, 4, workspace=Card(1 << 12, dtype=U8))


def attention(B=3, M=4):
    cu, lens, table = cards(B, M)
    binding.kda_kv4_attention(Card(5, 8, 64, dtype=BF), cu, 1, lens, table, Card(*POOL, dtype=U8), workspace=Card(1 << 12, dtype=U8))


def attention_picked(B=3, M=4, count=4):
    cu, lens, table = cards(B, M)
    binding.kda_kv4_attention_picked(Card(5, 8, 64, dtype=BF), cu, 1, lens, table, Card(5, 2, count, dtype=I32), Card(*POOL, dtype=U8),
                                     workspace=Card(1 << 12, dtype=U8))


def norm(T=3, C=64):
    binding.kda_add_rmsnorm(Card(T, C, dtype=BF), None, Card(C, dtype=BF))


CASES = [(f, dict(M=BIG)) for f in (append_rope, append, gather, bounds, pick, attention, attention_picked)]
CASES += [(f, dict(B=BIG)) for f in (append_rope, append, gather, bounds, pick, attention, attention_picked)]
CASES += [(append_rope, dict(rope=(BIG, 64))), (append_rope, dict(rope=(4, 2 ** 32 + 64))), (attention_picked, dict(count=BIG)), (norm, dict(T=BIG)),
          (norm, dict(T=2 ** 31)), (norm, dict(C=2 ** 32 + 64))]


@pytest.mark.parametrize("call,sizes", CASES, ids=["%s-%s" % (f.__name__, "-".join(k)) for f, k in CASES])
def test_sizes_past_an_int_are_refused(world, call, sizes):  # noqa: F811
    calls, _ = world
    with pytest.raises(ValueError, match="past 2\\^31 - 1"):
        call(**sizes)
    assert not calls


@pytest.mark.parametrize("call", [append_rope, append, gather, bounds, pick, attention, attention_picked, norm])
def test_usual_sizes_are_taken(world, call):  # noqa: F811
    call()
    assert world[0]

"""Results and buffers of the operators around the cache's attention belong to the stream the call runs on, operands of
another device are refused, and numbers past 32 bits keep their meaning (CPU: tensors that only claim to be on a device)."""
import pytest
import torch

import kda_state_gb300.binding as binding
from test_stream_buffers import BF, CURRENT, I32, SIDE, U8, Card, Stream, world  # noqa: F401

F32 = torch.float32


def norm(stream, **kw):
    return binding.kda_add_rmsnorm(Card(3, 64, dtype=BF), Card(3, 64, dtype=BF), Card(64, dtype=BF), scales="block", stream=stream, **kw)


def append_rope(stream):
    return (binding.kda_kv4_append_rope(Card(5, 8, 64, dtype=BF), Card(5, 2, 64, dtype=BF), Card(5, 2, 64, dtype=BF), Card(99, 64), Card(4, dtype=I32),
                                        Card(3, dtype=I32), Card(3, 4, dtype=I32), Card(8, 2, 1, 1152, dtype=U8), stream=stream),)


def pick(stream, max_q=1, page=16, count=4, **kw):
    return (binding.kda_kv4_pick(Card(5, 8, 64, dtype=BF), Card(4, dtype=I32), max_q, Card(3, dtype=I32), Card(3, 9, dtype=I32),
                                 Card(8, 2, 144, dtype=torch.int8), page, count, workspace=Card(1 << 12, dtype=U8), stream=stream, **kw),)


def attention(stream, max_q=1):
    return binding.kda_kv4_attention_picked(Card(5, 8, 64, dtype=BF), Card(4, dtype=I32), max_q, Card(3, dtype=I32), Card(3, 9, dtype=I32),
                                            Card(5, 2, 4, dtype=I32), Card(8, 2, 1, 1152, dtype=U8), stream=stream)


CALLS = [norm, append_rope, pick, attention]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [SIDE, Stream(SIDE), 0, CURRENT, None])
def test_made_on_the_streams_own(world, call, stream):  # noqa: F811
    calls, made = world
    want = CURRENT if stream is None else getattr(stream, "cuda_stream", stream)
    results = call(stream)
    assert made and all(s == want for s, _, _ in made)
    launched = [args for name, args in calls if not name.endswith("_bytes")]
    assert len(launched) == 1 and launched[0][-1] == want
    for t in results:
        assert getattr(t, "recorded", None) == (CURRENT if want != CURRENT else None)


@pytest.mark.parametrize("call", CALLS)
def test_operands_of_another_device_are_refused(world, monkeypatch, call):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="operands are on cuda:0, the current device is cuda:1"):
        call(None)
    assert not world[0]


@pytest.mark.parametrize("number,passed", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (-2 ** 32, -2 ** 31), (7, 7)])
def test_numbers_past_32_bits_keep_their_meaning(world, number, passed):  # noqa: F811
    calls, _ = world
    pick(None, max_q=number, page=number, first=number, recent=number)
    assert [calls[-1][1][i] for i in (3, 13, 17, 18)] == [passed] * 4
    attention(None, max_q=number)
    assert calls[-1][1][3] == passed
    binding.kda_kv4_bounds(Card(4, dtype=I32), Card(3, dtype=I32), number, Card(3, 9, dtype=I32), Card(8, 2, 1, 1152, dtype=U8),
                           Card(8, 2, 144, dtype=torch.int8))
    assert calls[-1][1][1] == passed


def test_given_results_are_taken(world):  # noqa: F811
    _, made = world
    out, scales, h = Card(3, 64, dtype=torch.float8_e4m3fn), Card(3, 1), Card(3, 64, dtype=BF)
    assert norm(None, out=out, scales_out=scales, residual_out=h) == (out, scales, h) and not made
    for bad in (dict(out=Card(3, 64, dtype=BF)), dict(scales_out=Card(3)), dict(residual_out=Card(3, 64)), dict(out=Card(2, 64, dtype=torch.float8_e4m3fn))):
        with pytest.raises((ValueError, TypeError)):
            norm(None, **bad)

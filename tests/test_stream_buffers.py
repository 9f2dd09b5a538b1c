"""Buffers that a call makes for itself, and results that its caller did not pass, belong to the
stream the call runs on (CPU: tensors that only claim to be on a device, a library that only notes
its calls)."""
import contextlib

import pytest
import torch

import kda_state_gb300.binding as binding

CURRENT, SIDE = 11, 77
BF, I32 = torch.bfloat16, torch.int32


class Card(torch.Tensor):
    """Shape, strides and dtype of a tensor on cuda:0, without memory."""
    addresses = iter(range(1 << 20, 1 << 40, 1 << 12))

    @staticmethod
    def __new__(cls, *shape, dtype=torch.float32, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        t = torch.Tensor._make_wrapper_subclass(cls, tuple(shape), dtype=dtype, device=device or "cuda:0")
        t.address = next(cls.addresses)
        return t

    def record_stream(self, s):
        self.recorded = s.cuda_stream

    def __repr__(self):
        return "Card%s" % (tuple(self.shape),)

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func is torch.Tensor.data_ptr:
            return args[0].address
        return super().__torch_function__(func, types, args, kwargs or {})

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError("no computing here: %s" % func)


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Library:
    """Every entry point succeeds and notes the streams and buffers at that moment."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        def call(*args):
            self.log.append((name, args))
            return 0
        return call if name != "kda_kv4_workspace_bytes" else lambda: 1 << 10


@pytest.fixture
def world(monkeypatch):
    """(calls, made): the library's calls, and of each tensor made its stream, whether it was zeroed, and itself."""
    at, calls, made = [CURRENT], [], []

    @contextlib.contextmanager
    def under(s):
        at.append(s.cuda_stream)
        yield
        at.pop()

    def maker(zeroed):
        def make(*shape, dtype=None, device=None):
            t = Card(*shape, dtype=dtype, device=device)
            made.append((at[-1], zeroed, t))
            return t
        return make

    library = Library(calls)
    monkeypatch.setattr(binding, "lib", lambda: library)
    monkeypatch.setattr(torch, "empty", maker(False))
    monkeypatch.setattr(torch, "zeros", maker(True))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(at[-1]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: at[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return calls, made


def state(N=8, B=3, M=4):
    return dict(refs=Card(N, dtype=I32), page_table=Card(B, M, dtype=I32), lens=Card(B, dtype=I32))


def attention(stream):
    return binding.kda_kv4_attention(Card(3, 8, 64, dtype=BF), Card(4, dtype=I32), 1, Card(3, dtype=I32), Card(3, 4, dtype=I32),
                                     Card(8, 2, 1, 1152, dtype=torch.uint8), stream=stream)


def gather(stream):
    return binding.kda_kv4_gather(Card(4, dtype=I32), Card(3, dtype=I32), 5, Card(3, 4, dtype=I32),
                                  Card(8, 2, 1, 1152, dtype=torch.uint8), stream=stream)


def fork(stream):
    binding.kda_page_fork([Card(8, 64, dtype=torch.uint8)], *state().values(), Card(1, dtype=I32), Card(1, dtype=I32), 16,
                          stream=stream)
    return ()


def compact(stream):
    s = state()
    return (binding.kda_page_compact([Card(8, 64, dtype=torch.uint8)], s["refs"], s["page_table"], stream=stream),)


def heads(*lead):
    return [Card(*lead, 2, 128, dtype=BF) for _ in range(4)] + [Card(*lead, 2, dtype=BF)]


def decode(stream):
    return (binding.kda_decode_step(*heads(3), Card(3, dtype=I32), Card(5, 2, 128, 128), stream=stream),)


def verify_ragged(stream):
    ring = binding.RingBuffers(Card(5, 8, 2, 128, dtype=BF), Card(5, 8, 2, 128, dtype=BF), Card(5, 8, 2, 128), Card(5, 8, 2))
    return (binding.kda_verify_store_inputs_ragged(*heads(7), Card(4, dtype=I32), 4, Card(3, dtype=I32), Card(5, 2, 128, 128),
                                                   ring, stream=stream),)


CALLS = [attention, gather, fork, compact, decode, verify_ragged]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [SIDE, Stream(SIDE), 0, CURRENT, None])
def test_made_on_the_streams_own(world, call, stream):
    calls, made = world
    want = CURRENT if stream is None else getattr(stream, "cuda_stream", stream)
    results = call(stream)
    assert made and all(s == want for s, _, _ in made), "made on %s, launched on %s" % ([s for s, _, _ in made], want)
    (_, args), = calls
    assert getattr(args[-1], "value", args[-1]) in (want, None if want == 0 else want)
    # a result is used on the current stream next: its memory is not given away before that is through
    for t in results:
        assert getattr(t, "recorded", None) == (CURRENT if want != CURRENT else None)


def test_the_workspace_is_zeroed_there(world):
    _, made = world
    attention(SIDE)
    zeroed = [(s, t.numel()) for s, z, t in made if z]
    assert zeroed == [(SIDE, 1 << 10)]


@pytest.mark.parametrize("call", [attention, gather, fork, compact])
@pytest.mark.parametrize("stream", [None, SIDE])
def test_operands_of_another_device_are_refused(world, monkeypatch, call, stream):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="operands are on cuda:0, the current device is cuda:1"):
        call(stream)
    assert not world[0]


U8 = torch.uint8
ALIKE = [Card(8, 64, dtype=U8), Card(8, 8, 8, dtype=U8), Card(8, 64, dtype=torch.int8)]   # pages of 64 bytes


@pytest.mark.parametrize("odd,message", [
    (None, None), (Card(8, 32, dtype=U8), "pools.3.: every pool"), (Card(8, 64, dtype=BF), "pools.3.: every pool"),
    (Card(8, 32, dtype=BF), "pools.3.: every pool"), (Card(8, 64, dtype=U8, device="cuda:1"), "pools.3. is on cuda:1"),
    (torch.ones(8, 64, dtype=U8), "pools.3. must be a CUDA tensor"), (None, "pools.3. is required")])
def test_a_list_of_pools_is_judged_one_way(world, odd, message):
    """Pools are pages of bytes: of one size and element width, whatever their shapes, also where another is at fault."""
    s, one = state(), Card(1, dtype=I32)
    pools = ALIKE + ([odd] if message else [])
    for call in (lambda: binding.kda_page_fork(pools, *s.values(), one, one, 16),
                 lambda: binding.kda_page_compact(pools, s["refs"], s["page_table"]),
                 lambda: binding.kda_page_copy(pools, one, one)):
        world[0].clear()
        if message:
            with pytest.raises(ValueError, match=message):
                call()
            assert not world[0]
        else:
            call()
            assert world[0][0][1][0] == 3 and 64 in world[0][0][1]


@pytest.mark.parametrize("pools", [[Card(9, 64, dtype=U8)], [Card(8, dtype=U8)]])
def test_pools_of_other_pages_are_refused(world, pools):
    s, one = state(), Card(1, dtype=I32)
    for call in (lambda: binding.kda_page_fork(pools, *s.values(), one, one, 16),
                 lambda: binding.kda_page_compact(pools, s["refs"], s["page_table"])):
        with pytest.raises(ValueError, match="every pool"):
            call()
    assert not world[0]


@pytest.mark.parametrize("number,passed", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1),
                                           (2 ** 63 - 1, 2 ** 31 - 1), (-2 ** 32, -2 ** 31), (7, 7)])
def test_numbers_past_32_bits_keep_their_meaning(world, number, passed):
    """A C int would take them modulo 2^32: a window of 2^32 + 5 was one of 5."""
    binding.kda_kv4_attention(Card(3, 8, 64, dtype=BF), Card(4, dtype=I32), number, Card(3, dtype=I32), Card(3, 4, dtype=I32),
                              Card(8, 2, 1, 1152, dtype=U8), window=number, workspace=Card(1 << 10, dtype=U8))
    (_, args), = world[0]
    assert args[3] == passed and args[16] == passed
    s, one = state(), Card(1, dtype=I32)
    world[0].clear()
    binding.kda_page_alloc(*s.values(), s["lens"], number)
    binding.kda_page_free(*s.values(), one, number)
    binding.kda_page_fork(ALIKE, *s.values(), one, one, number)
    assert [args[i] for i, (_, args) in zip((2, 2, 5), world[0])] == [passed] * 3

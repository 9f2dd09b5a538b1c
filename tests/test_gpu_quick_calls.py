"""The plain calls' way to the library gives what the binding's own functions give, and leaves them what it does not take."""
import numpy as np
import pytest
import torch

import kda_state_gb300 as kda
import kda_state_gb300.binding as binding
from kv4_testutil import cu_of, make_cache
from test_quick_calls import CALLS

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()
    kda.lib()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Calls:
    """Calls on one batch, by name, with new buffers each time."""

    def __init__(self):
        self.pool, table = make_cache([100, 37, 5], 2, 64, 16, 1)
        self.table, self.cu, self.start, self.lens = torch.from_numpy(table).to(DEV), cu_of([2, 1, 3]).to(DEV), i32([98, 36, 2]), i32([100, 37, 5])
        g = torch.Generator().manual_seed(2)
        self.qkv = torch.randn(6, 12, 64, generator=g).to(BF).to(DEV)
        self.x, self.r, self.w = (torch.randn(n, 256, generator=g).to(BF).to(DEV) for n in (5, 5, 1))
        self.bounds, self.ws = kda.make_kv4_bounds(len(self.pool), 2, 64), kda.make_kv4_workspace()
        self.rope, self.pick_ws = kda.make_rope_table(120, 64), torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
        kda.kda_kv4_bounds(cu_of([100, 37, 5]).to(DEV), i32([0, 0, 0]), 142, self.table, self.new_pool(), self.bounds)
        self.picked = kda.kda_kv4_pick(self.qkv[:, :8], self.cu, 3, self.lens, self.table, self.bounds, 16, 3)

    def new_pool(self):
        return torch.from_numpy(self.pool).to(DEV)

    def norm(self, **kw):
        return kda.kda_add_rmsnorm(self.x, self.r, self.w[0], **kw)

    def norm_in_place(self):
        r = self.r.clone()
        out = kda.kda_add_rmsnorm(self.x, r, self.w[0], scales="row", residual_out=r)
        assert out[2] is r
        return out

    def norm_alone(self):
        out = kda.kda_add_rmsnorm(self.x, None, self.w[0])
        assert out[2] is self.x and out[1] is None
        return out[:1]

    def rope_append(self, in_place=False):
        pool, qkv = self.new_pool(), self.qkv.clone()
        q = qkv[:, :8]
        out = kda.kda_kv4_append_rope(q, qkv[:, 8:10], qkv[:, 10:], self.rope, self.cu, self.start, self.table, pool, pairs=in_place, k_scale=2,
                                      q_out=q if in_place else None)
        assert (out is q) == in_place
        return out, pool

    def append(self):
        pool = self.new_pool()
        kda.kda_kv4_append(self.qkv[:, 8:10], self.qkv[:, 10:], self.cu, self.start, self.table, pool, v_scale=0.5)
        return pool,

    def gather(self):
        return kda.kda_kv4_gather(self.cu, self.start, 6, self.table, self.new_pool(), dtype=torch.float16, v_scale=0.5)

    def bound(self):
        b = torch.zeros_like(self.bounds)
        kda.kda_kv4_bounds(self.cu, self.start, 6, self.table, self.new_pool(), b)
        return b,

    def pick(self):
        return kda.kda_kv4_pick(self.qkv[:, :8], self.cu, 3, self.lens, self.table, self.bounds, 16, 3, first=0, recent=2, workspace=self.pick_ws),

    def attention(self):
        return kda.kda_kv4_attention(self.qkv[:, :8], self.cu, 3, self.lens, self.table, self.new_pool(), window=40, workspace=self.ws)

    def attention_picked(self):
        return kda.kda_kv4_attention_picked(self.qkv[:, :8], self.cu, 3, self.lens, self.table, self.picked, self.new_pool(), v_scale=2.0,
                                            workspace=self.ws)


ALL = [("norm", {}), ("norm", dict(scales="row")), ("norm", dict(scales="block", eps=1)), ("norm_in_place", {}), ("norm_alone", {}), ("rope_append", {}),
       ("rope_append", dict(in_place=True)), ("append", {}), ("gather", {}), ("bound", {}), ("pick", {}), ("attention", {}), ("attention_picked", {})]


@pytest.mark.parametrize("name,kw", ALL)
def test_both_ways_are_one(monkeypatch, name, kw):
    c = Calls()
    quick, taken = binding._quick, []

    class Spy:
        def __getattr__(self, n):
            def call(*a):
                out = getattr(quick, n)(*a)
                taken.append(out is not None)
                return out
            return call
    monkeypatch.setattr(binding, "_quick", Spy())
    got = getattr(c, name)(**kw)
    assert taken == [True]
    monkeypatch.setattr(binding, "_quick", None)
    want = getattr(c, name)(**kw)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert (x is None and y is None) or (x.dtype == y.dtype and x.shape == y.shape and x.stride() == y.stride() and
                                             torch.equal(x.view(torch.uint8), y.view(torch.uint8)))


def test_the_error_word_is_written_either_way():
    c = Calls()
    for word in (torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)):
        kda.kda_kv4_append(c.qkv[:, 8:10], c.qkv[:, 10:], c.cu, i32([98, 36, 10 ** 6]), c.table, c.new_pool(), dev_err=word)
        assert word.tolist()[0] == 4 and not word[1:].any()
    with pytest.raises((ValueError, TypeError)):
        kda.kda_kv4_append(c.qkv[:, 8:10], c.qkv[:, 10:], c.cu, c.start, c.table, c.new_pool(), dev_err=torch.zeros(1, device=DEV))


def gpu(*spec):
    return torch.zeros(spec[:-1], dtype=spec[-1], device=DEV)


@pytest.mark.parametrize("name,args", CALLS, ids=[n for n, _ in CALLS])
def test_operands_that_do_not_fit_are_left(name, args):
    """Every tensor in turn of another type, shape, layout or place: nothing is launched, None comes back."""
    call = getattr(binding._quick, name)
    for i, arg in enumerate(args(gpu)):
        if not isinstance(arg, torch.Tensor):
            continue
        others = [arg.cpu(), arg.to(torch.float64), arg[:0] if arg.shape[0] else arg, arg.unsqueeze(0),
                  torch.zeros(tuple(arg.shape[:-1]) + (2 * arg.shape[-1],), dtype=arg.dtype, device=DEV)[..., ::2], arg.to(torch.complex64),
                  torch.nn.functional.pad(arg.float(), (0, 8)).to(arg.dtype)]
        for other in others:
            a = list(args(gpu))
            a[i] = other
            if other.shape != arg.shape or other.dtype != arg.dtype or not other.is_contiguous() or not other.is_cuda:
                if name in ("pick", "attention_picked", "attention") and i == len(a) - 2 and other.dim() == 1 and other.dtype == arg.dtype and other.is_contiguous() and other.is_cuda:
                    continue                                     # a workspace may have any size, and is judged by the library
                if other.numel() == 0:
                    continue                                     # nothing to do may be done
                if arg.dtype == torch.int32 and arg.dim() == 2 and other.dim() == 2 and other.dtype == arg.dtype and other.is_cuda and other.is_contiguous():
                    continue                                     # a page table may have any width
                assert call(*a) is None, (i, other.shape, other.dtype)
    torch.cuda.synchronize()


def test_a_subclass_is_left_to_the_binding():
    class Mine(torch.Tensor):
        pass
    c = Calls()
    x = c.x.as_subclass(Mine)
    assert binding._quick.add_rmsnorm(x, c.r, c.w[0], 1e-5, 1, None) is None
    out, s, h = kda.kda_add_rmsnorm(x, c.r, c.w[0], scales="row")
    want = kda.kda_add_rmsnorm(c.x, c.r, c.w[0], scales="row")
    assert torch.equal(out.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])


def test_on_the_current_stream():
    """What a side stream holds back, a plain call made under it waits for."""
    c = Calls()
    want = c.norm(scales="row")
    side = torch.cuda.Stream()
    x = torch.empty_like(c.x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20000000)
        x.copy_(c.x)
        got = kda.kda_add_rmsnorm(x, c.r, c.w[0], scales="row")
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

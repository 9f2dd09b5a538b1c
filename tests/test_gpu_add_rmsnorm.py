"""The residual norm against its fp64 definition, in every type, output and width.

Bounds.  A row's sum of squares is at most 32 additions in a thread, then 10 between threads: off by
(32 + 10 + 1) 2^-24 relative, its root's reciprocal by half of that and 2^-22 of the instruction; the quotient, eps and
the two products add 4 roundings.  Together below 2^-18.  An output is then rounded once: half a step of its type, for
e4m3 2^-4 of a normal value and 2^-10 of a smaller one; its scale is off by the same 2^-18."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()


def kda():
    import kda_state_gb300
    return kda_state_gb300


def inputs(T, C, dtype, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C + extra, generator=g).to(dtype).to(DEV)[:, :C]
    r = (torch.randn(T, C + extra, generator=g) * 3).to(dtype).to(DEV)[:, :C]
    w = (0.5 + torch.rand(C, generator=g)).to(dtype).to(DEV)
    return x, r, w


def check(out, scales, h, x, r, w, mode, eps=1e-5):
    want_h = x if r is None else x + r
    assert torch.equal(h, want_h)
    y = ref.add_rmsnorm(want_h.double().cpu().numpy(), w.double().cpu().numpy(), eps)
    got = out.double().cpu().numpy()
    if mode == "none":
        assert (np.abs(got - y) <= np.abs(y) * (HALF_STEP[x.dtype] * 1.01 + REL) + 2.0 ** -25).all()
        return
    width = y.shape[1] if mode == "row" else 128
    s = ref.block_scales(y, width)
    gs = scales.double().cpu().numpy().reshape(s.shape)
    assert (np.abs(gs - s) <= s * REL).all()
    z = np.where(s == 0, 0.0, 1.0 / np.where(s == 0, 1.0, s)).repeat(width, 1)[:, :y.shape[1]] * y
    assert (np.abs(got - z) <= np.maximum(np.abs(z) * 2.0 ** -4, 2.0 ** -10) + np.abs(z) * 2 * REL).all()


@pytest.mark.parametrize("mode", ["none", "row", "block"])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("T,C", [(1, 8), (3, 64), (5, 264), (6, 512), (7, 1000), (2, 1024), (9, 2168), (4, 4096), (3, 5000), (2, 8192), (1, 16384), (2, 32760)])
def test_norm(T, C, dtype, mode):
    x, r, w = inputs(T, C, dtype, C + T, extra=24)
    out, s, h = kda().kda_add_rmsnorm(x, r, w, scales=mode)
    check(out, s, h, x, r, w, mode)
    out, s, h = kda().kda_add_rmsnorm(x, None, w, eps=1e-3, scales=mode)
    check(out, s, h, x, None, w, mode, 1e-3)


@pytest.mark.parametrize("T", [37, 700, 2500])
@pytest.mark.parametrize("C", [96, 1024, 4096, 7168])
def test_many_rows(T, C):
    x, r, w = inputs(T, C, BF, T)
    for mode in ("none", "block"):
        out, s, h = kda().kda_add_rmsnorm(x, r, w, scales=mode)
        check(out, s, h, x, r, w, mode)


def test_the_residual_in_place():
    for C in (64, 2048, 8192):
        x, r, w = inputs(33, C, BF, 1, extra=8)
        want, s0, h0 = kda().kda_add_rmsnorm(x, r, w, scales="row")
        kept = torch.nn.functional.pad(r, (0, 8)).clone()
        view = kept[:, :C]
        out, s1, h1 = kda().kda_add_rmsnorm(x, view, w, scales="row", residual_out=view)
        assert h1 is view and torch.equal(view, h0) and torch.equal(out.view(torch.uint8), want.view(torch.uint8)) and torch.equal(s0, s1)
        assert not kept[:, C:].any()
        y = x.clone()
        out, _, _ = kda().kda_add_rmsnorm(y, r, w, scales="row", residual_out=y)
        assert torch.equal(y, h0) and torch.equal(out.view(torch.uint8), want.view(torch.uint8))


def test_rows_of_zeros_nan_and_infinity():
    x, r, w = inputs(5, 512, BF, 2)
    x[1], r[1] = 0, 0
    x[2, 5] = float("nan")
    x[3, 300] = float("inf")
    out, s, h = kda().kda_add_rmsnorm(x, r, w, eps=0.0, scales="none")
    o = out.float()
    assert o[1].isnan().all() and o[2].isnan().all() and o[3, 300].isnan() and o[3].nan_to_num(0).abs().max() == 0      # 0 / 0 without eps
    out, s, h = kda().kda_add_rmsnorm(x, r, w, scales="block")
    o = out.float()
    assert not o[1].any() and not s[1].any()
    assert o[2].isnan().all() and s[2].isnan().all()
    assert s[3].isnan().tolist() == [False, False, True, False] and o[3, 256:384].isnan().all()
    assert not o[3, :256].any() and not o[3, 384:].any() and not s[3, :2].any()
    check(out[:1], s[:1], h[:1], x[:1], r[:1], w, "block")
    check(out[4:], s[4:], h[4:], x[4:], r[4:], w, "block")
    out, s, h = kda().kda_add_rmsnorm(x, r, w, scales="row")
    assert out[2:4].float().isnan().all() and s[2:4].isnan().all() and not out[1].float().any() and s[1] == 0


def test_small_rows_keep_their_codes():
    """Values far below the type's usual range: eps rules the root, scales are small numbers."""
    x, r, w = inputs(3, 256, BF, 3)
    for f in (1e-6, 1e-18, 1e-30):
        out, s, h = kda().kda_add_rmsnorm(x * f, r * f, w, scales="row")
        check(out, s, h, x * f, r * f, w, "row")


def test_empty_and_refused():
    x, r, w = inputs(4, 64, BF, 4)
    out, s, h = kda().kda_add_rmsnorm(x[:0], r[:0], w, scales="block")
    assert out.shape == (0, 64) and s.shape == (0, 1) and h.shape == (0, 64)
    k = kda().kda_add_rmsnorm
    for bad in (lambda: k(x.cpu(), r, w), lambda: k(x, r[:3], w), lambda: k(x, r.half(), w), lambda: k(x, r, w[:32]), lambda: k(x.double(), r.double(), w.double()),
                lambda: k(x, r, w, scales="tensor"), lambda: k(x.t(), r.t(), w), lambda: k(x, None, w, residual_out=r), lambda: k(x, r, w.float()),
                lambda: k(x, r, w, out=torch.empty(4, 64, device=DEV)), lambda: k(x, r, w, scales_out=torch.empty(4, device=DEV)),
                lambda: k(x, r, w, scales="row", scales_out=torch.empty(4, 1, device=DEV)), lambda: k(x[:, :60], r[:, :60], w[:60]),
                lambda: k(x[:, 4:], r[:, 4:], w[4:])):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()


def test_on_a_stream_and_in_a_graph():
    x, r, w = inputs(50, 4096, BF, 5)
    want, ws, wh = kda().kda_add_rmsnorm(x, r, w, scales="block")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, s, h = kda().kda_add_rmsnorm(x, r, w, scales="block", stream=side)
    side.synchronize()
    assert torch.equal(out.view(torch.uint8), want.view(torch.uint8)) and torch.equal(h, wh)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, s, h = kda().kda_add_rmsnorm(x, r, w, scales="block")
    x.mul_(2), r.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    check(out, s, h, x, r, w, "block")

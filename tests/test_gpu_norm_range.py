"""The residual norm's 8-bit outputs where products, values or scales leave fp32's normal range.

Bounds: those of test_gpu_add_rmsnorm.py (2^-18 relative for y and the scale, half a step of e4m3).  A y below 2^-126 is
rounded to whole steps of 2^-149, by half of one; so is a scale, whose y is off by 2^-150 / 448 more: together below 2^-149.
Codes are compared with y over the scale that was returned, so that its own rounding does not count twice; y's 2^-150
and the quotient's rounding stay below 2^-149 / scale."""
import numpy as np
import pytest
import torch

from oracle import layer_ops as ref
from test_gpu_add_rmsnorm import BF, DEV, F32, REL, _lib, kda  # noqa: F401

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -149


def check(x, w, mode, eps):
    """Every row is finite and has no residual."""
    out, scales, _ = kda().kda_add_rmsnorm(x, None, w, eps=eps, scales=mode)
    y = ref.add_rmsnorm(x.double().cpu().numpy(), w.double().cpu().numpy(), eps)
    width = y.shape[1] if mode == "row" else 128
    s = ref.block_scales(y, width)
    gs = scales.double().cpu().numpy().reshape(s.shape)
    assert (np.abs(gs - s) <= s * REL + TINY).all()
    wide = gs.repeat(width, 1)[:, :y.shape[1]]
    z = np.where(wide == 0, 0.0, np.clip(y / np.where(wide == 0, 1.0, wide), -448, 448))
    slack = np.abs(z) * 2 * REL + np.where(wide == 0, 0.0, TINY / np.where(wide == 0, 1.0, wide))
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - z) <= np.maximum(np.abs(z) * 2.0 ** -4, 2.0 ** -10) + slack).all()
    return got, gs


def faint(T, C, dtype, seed, size):
    """Rows of `size`, with zeros among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g) * size
    x[:, 5::7] = 0
    return x.to(dtype).to(DEV)


def weights(C, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return ((0.5 + torch.rand(C, generator=g)) * size).to(dtype).to(DEV)


@pytest.mark.parametrize("mode", ["row", "block"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [8, 200, 1024, 4096, 8192, 20000])
def test_faint_rows(C, dtype, mode):
    for size in (1e-33, 1.3e-36, 1e-36, 1e-37, 3e-38, 1e-39):
        got, s = check(faint(3, C, dtype, C, size), weights(C, dtype, 1), mode, 1e-5)
        assert (np.abs(got) == 448).any(-1).all() and (s > 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [512, 3000, 16384])
def test_a_faint_block_in_a_usual_row(C, dtype):
    x = torch.randn(2, C, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    w = weights(C, dtype, 2)
    x[:, 128:256] = faint(2, 128, dtype, 4, 1e-37)
    x[1, 256:384] = 0
    x[0, 256:384] *= 1e-30
    got, s = check(x, w, "block", 1e-5)
    assert not s[1, 2] and not got[1, 256:384].any() and (s[:, 1] > 0).all()


def test_the_definitions_own_numbers():
    x = torch.ones(1, 256, dtype=BF, device=DEV)
    x[0, :128] = 0
    x[0, 3], x[0, 9] = 1e-37, -3e-38
    out, s, _ = kda().kda_add_rmsnorm(x, None, torch.ones(256, dtype=BF, device=DEV), scales="block")
    o = out.float()[0]
    assert o[3] == 448 and o[9] == -128 and o[:128].count_nonzero() == 2 and (o[128:] == 448).all() and s[0, 0] > 0


@pytest.mark.parametrize("mode", ["row", "block"])
@pytest.mark.parametrize("C", [256, 2048, 9000])
def test_products_past_fp32(C, mode):
    """h w overflows or vanishes, h w / rms does not."""
    for h, w, eps in ((1e10, 1e32, 1e-5), (1e16, 1e27, 1e-5), (1e-18, 1e-25, 0.0), (1e-17, 1e-24, 0.0)):
        x = faint(3, C, F32, 7, h)
        got, s = check(x, weights(C, F32, 8, w), mode, eps)
        assert (s > 0).all() and (np.abs(got) == 448).any(-1).all()


@pytest.mark.parametrize("mode", ["row", "block"])
def test_scales_of_few_bits(mode):
    for w in (1e-36, 1e-38, 2e-40, 1e-43):
        check(faint(3, 640, F32, 9, 1.0), weights(640, F32, 10, w), mode, 1e-5)


def test_an_infinite_weight_is_its_blocks_alone():
    x = faint(2, 512, F32, 11, 1.0)
    w = weights(512, F32, 12)
    w[130] = float("inf")
    out, s, _ = kda().kda_add_rmsnorm(x, None, w, scales="block")
    assert s.isnan().tolist() == [[False, True, False, False]] * 2 and out.float().isnan().sum(-1).tolist() == [128, 128]
    out, s, _ = kda().kda_add_rmsnorm(x, None, w, scales="row")
    assert s.isnan().all() and out.float().isnan().all()


@pytest.mark.parametrize("mode", ["row", "block"])
@pytest.mark.parametrize("C", [96, 1000, 4096, 9000])
def test_the_residuals_forms_are_one(C, mode):
    """With the sum kept, kept in place (of either operand) or not at all, in faint rows and blocks and in usual ones."""
    x, r, w = faint(4, C, BF, 13, 1.0), faint(4, C, BF, 14, 1.0), weights(C, BF, 15)
    for t in (x, r):
        t[0] *= 1e-37
        t[1, 128:256] *= 1e-37
        t[2] = 0
    h = x + r
    want = kda().kda_add_rmsnorm(h, None, w, scales=mode)
    same = lambda out, s: torch.equal(out.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1])
    out, s, kept = kda().kda_add_rmsnorm(x, r, w, scales=mode)
    assert same(out, s) and torch.equal(kept, h)
    for into in (0, 1):
        pair = [x.clone(), r.clone()]
        out, s, kept = kda().kda_add_rmsnorm(*pair, w, scales=mode, residual_out=pair[into])
        assert same(out, s) and kept is pair[into] and torch.equal(kept, h)
    out, s = torch.empty_like(want[0]), torch.empty_like(want[1])
    status = kda().lib().kda_add_rmsnorm(0, 4, C, x.data_ptr(), C, r.data_ptr(), C, w.data_ptr(), 1e-5, 1 if mode == "row" else 2, None, 0,
                                         out.data_ptr(), s.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0 and same(out, s)

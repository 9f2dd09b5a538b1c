"""The residual norm at the largest number of rows that a call takes."""
import pytest
import torch

from test_gpu_add_rmsnorm import BF, DEV, _lib, kda  # noqa: F401

pytestmark = pytest.mark.gpu


def test_as_many_rows_as_an_int_counts():
    """2^31 - 1 rows of 8 channels (63 GB)."""
    T = 2 ** 31 - 1
    x = torch.zeros(T, 8, dtype=BF, device=DEV)
    x[0], x[T // 2], x[-1] = 1, 2, torch.arange(8, device=DEV)
    w = torch.ones(8, dtype=BF, device=DEV)
    out, s, h = kda().kda_add_rmsnorm(x, None, w, scales="row")
    want, ws, _ = kda().kda_add_rmsnorm(x[[0, T // 2, T - 1]], None, w, scales="row")
    at = torch.tensor([0, T // 2, T - 1], device=DEV)
    assert torch.equal(out[at].view(torch.uint8), want.view(torch.uint8)) and torch.equal(s[at], ws)
    assert int((s != 0).sum()) == 3
    del x, out, s, h
    torch.cuda.empty_cache()

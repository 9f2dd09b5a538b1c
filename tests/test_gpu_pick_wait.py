"""The picks' bounded wait on the GPU: where the first records never all arrive the scores report KDA_DEVERR_TIMEOUT and
return, and the next call gives what it gave before."""
import numpy as np
import pytest
import torch

from test_gpu_kv4_layer import BF, DEV, _lib, cu_of, dev, i32, kda, new_err, packed_q, random_bounds  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,D,longest", [(1, 8, 128, 700), (5, 3, 64, 3000), (80, 8, 64, 33600), (3, 1, 128, 20000)])
def test_waits_run_out_and_the_next_call_is_as_before(B, H, D, longest):
    rng = np.random.default_rng(41)
    lens = [longest] + [int(x) for x in rng.integers(1, longest, B - 1)]
    rec, table = random_bounds(lens, H, D, 16, 42)
    q = packed_q([1] * B, 2 * H, D, BF, 43).to(DEV)
    err, ws = new_err(), torch.empty(kda().kv4_pick_workspace_bytes(B, H, table.shape[1]), dtype=torch.uint8, device=DEV)
    cu, kl, tab, bounds = cu_of([1] * B).to(DEV), i32(lens), dev(table), dev(rec)
    want = kda().kda_kv4_pick(q, cu, 1, kl, tab, bounds, 16, 9, workspace=ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kda().kda_selftest_kv4_pick_wait(q, cu, kl, tab, bounds, 16, 9, ws, err, wait_us=2000)
    torch.cuda.synchronize()
    assert int(err) == kda().KDA_DEVERR_TIMEOUT
    err.zero_()
    for _ in range(3):
        got = kda().kda_kv4_pick(q, cu, 1, kl, tab, bounds, 16, 9, workspace=ws, dev_err=err)
        torch.cuda.synchronize()
        assert int(err) == 0 and torch.equal(got, want)

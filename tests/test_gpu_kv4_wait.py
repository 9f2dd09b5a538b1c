"""The cache attention's bounded waits on the GPU: where the first codes never arrive every kernel reports
KDA_DEVERR_TIMEOUT and returns, and the next launch gives what it gave before."""
import pytest
import torch

from kv4_testutil import cu_of, make_cache, packed_q

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from kda_state_gb300 import _build
    _build.build()


@pytest.mark.parametrize("news,lens,Hq,Hkv,D", [
    ([1, 1, 0, 1], [300, 40, 3, 6000], 8, 2, 128),            # few rows: 8
    ([4, 1, 3], [300, 40, 2000], 8, 2, 64),                   # few rows: 16
    ([90, 20, 64], [500, 20, 2600], 4, 2, 128),               # tiles of 128 rows, requests cut along the tokens
    ([90] * 40, [300] * 40, 32, 4, 64),                       # tiles of 128 rows, several parts a CTA
    ([700, 599], [900, 599], 64, 8, 128),                     # tiles of 256 rows
    ([700, 599], [900, 599], 64, 8, 64),
])
def test_waits_run_out_and_the_next_launch_is_as_before(news, lens, Hq, Hkv, D):
    import kda_state_gb300 as kda
    pool, table = make_cache(lens, Hkv, D, 64, 1)
    q = packed_q(news, Hq, D, torch.bfloat16, 2).to(DEV)
    ws, err = kda.make_kv4_workspace(), torch.zeros(1, dtype=torch.int32, device=DEV)
    args = (q, cu_of(news).to(DEV), max(news), torch.tensor(lens, dtype=torch.int32, device=DEV),
            torch.from_numpy(table).to(DEV), torch.from_numpy(pool).to(DEV))
    want = kda.kda_kv4_attention(*args, workspace=ws, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    kda.kda_selftest_kv4_wait(*args, ws, err, wait_us=2000)
    torch.cuda.synchronize()
    assert int(err) == kda.KDA_DEVERR_TIMEOUT
    ws.zero_()
    err.zero_()
    for _ in range(3):
        o, lse = kda.kda_kv4_attention(*args, workspace=ws, dev_err=err)
        torch.cuda.synchronize()
        assert int(err) == 0 and torch.equal(o, want[0]) and torch.equal(lse, want[1])

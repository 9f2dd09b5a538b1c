"""Refusals of the picks' wait self-test that need no GPU."""
import pytest

from test_layer_host import FAKE, INVALID, L, PICK, UNSUPPORTED, call  # noqa: F401

GOOD = {k: v for k, v in PICK.items() if k not in ("err", "stream")}
GOOD.update(max_q=1, err=FAKE, wait_us=1000, stream=None)


@pytest.mark.parametrize("status,change", [
    (INVALID, dict(err=None)), (INVALID, dict(wait_us=0)), (INVALID, dict(wait_us=2000001)), (INVALID, dict(T=0)), (INVALID, dict(max_q=2)),
    (INVALID, dict(count=5)), (INVALID, dict(ws_bytes=16)), (INVALID, dict(q=None)), (INVALID, dict(bounds=None)), (UNSUPPORTED, dict(D=96)),
])
def test_pick_wait(L, status, change):  # noqa: F811
    assert call(L.kda_selftest_kv4_pick_wait, GOOD, **change) == status

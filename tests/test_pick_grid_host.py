"""Batches that are past a launch's grid are refused as arguments, before anything is launched (no GPU)."""
import pytest

from test_layer_host import INVALID, L, PICK, call  # noqa: F401

BIG = dict(ws_bytes=1 << 50, D=64, count=4, max_pages=5)


@pytest.mark.parametrize("change", [
    dict(B=1 << 20, T=1 << 20, max_q=1 << 20, Hq=1, Hkv=1, qs=64),
    dict(B=131072, T=262144, max_q=131072, Hq=2, Hkv=1, qs=128),
    dict(B=2, T=2, max_q=2, Hq=131071, Hkv=131071, qs=131071 * 64),
    dict(B=1, T=1, max_q=1, Hq=524281, Hkv=524281, qs=524281 * 64),
])
def test_refused(L, change):  # noqa: F811
    assert call(L.kda_kv4_pick, PICK, **{**BIG, **change}) == INVALID

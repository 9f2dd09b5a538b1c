"""Refusals of the paged 4-bit cache's entry points at the ends of their ranges (CPU; no call here gets past the checks,
or has any work)."""
import pytest

from test_kv4_host import APP, ATT, GAT, L  # noqa: F401  (L: the fixture)


@pytest.mark.parametrize("scale", [2.0 ** -149, 2.0 ** -128])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_scales_without_a_reciprocal_are_refused(L, which, scale):  # noqa: F811
    for call, args in ((L.kda_kv4_append, APP), (L.kda_kv4_gather, GAT), (L.kda_kv4_attention, ATT)):
        assert call(*{**args, which: scale}.values()) == -1
        for fine in (2.0 ** -127, 2.0 ** -126, 2.0 ** 127):
            assert call(*{**args, which: fine, "T": 0}.values()) == 0


@pytest.mark.parametrize("change", [dict(H=1 << 25, T=1), dict(H=(1 << 31) - 1, T=1)])
def test_rows_past_32_bits_are_refused(L, change):  # noqa: F811
    """Heads times channels of a token index in 32 bits."""
    wide = 1 << 40
    h = change["H"]
    assert L.kda_kv4_append(*{**APP, **change, "kst": wide, "vst": wide}.values()) == -1
    assert L.kda_kv4_gather(*{**GAT, **change}.values()) == -1
    assert L.kda_kv4_attention(*{**ATT, "T": 1, "Hq": h, "Hkv": h, "qs": wide}.values()) == -1
    assert L.kda_kv4_attention(*{**ATT, "T": 1, "Hq": h, "Hkv": 1, "qs": wide}.values()) == -1


def test_selftest_kv4_wait_refuses(L):  # noqa: F811
    from test_kv4_host import FAKE
    names = ("dt", "B", "T", "max_q", "Hq", "Hkv", "D", "q", "qs", "cu", "lens", "table", "M", "P", "pool", "pages", "o", "ws", "wsb")
    call = lambda err=FAKE, us=1000, **kw: L.kda_selftest_kv4_wait(*({**ATT, **kw}[n] for n in names), err, us, None)
    for kw in (dict(err=None), dict(us=0), dict(us=2000001), dict(T=0), dict(ws=None), dict(q=None), dict(wsb=1)):
        assert call(**kw) == -1
    assert call(D=96) == -2

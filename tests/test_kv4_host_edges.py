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

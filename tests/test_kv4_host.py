"""The paged 4-bit cache's entry points refuse bad arguments before anything is launched (CPU)."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(4096)          # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(4100)
WS = 16 << 20


@pytest.fixture(scope="module")
def L():
    from kda_state_gb300 import _build
    _build.build()
    import kda_state_gb300 as kda
    return kda.lib()


ATT = dict(dt=0, B=2, T=2, max_q=1, Hq=8, Hkv=2, D=128, q=FAKE, qs=1024, cu=FAKE, lens=FAKE, table=FAKE, M=4, P=16,
           pool=FAKE, pages=8, window=0, scale=0.1, ks=1.0, vs=1.0, o=FAKE, lse=None, ws=FAKE, wsb=WS, err=None, st=None)
APP = dict(dt=2, B=2, T=2, H=2, D=64, k=FAKE, kst=128, v=FAKE, vst=128, cu=FAKE, start=FAKE, table=FAKE, M=4, P=32,
           pool=FAKE, pages=8, ks=1.0, vs=1.0, err=None, st=None)
GAT = dict(dt=0, B=2, T=2, H=2, D=64, k=FAKE, v=FAKE, cu=FAKE, start=FAKE, table=FAKE, M=4, P=32, pool=FAKE, pages=8,
           ks=1.0, vs=1.0, err=None, st=None)


@pytest.mark.parametrize("change, status", [
    (dict(dt=1), -2), (dict(dt=7), -2), (dict(D=96), -2), (dict(D=0), -2), (dict(B=-1), -1), (dict(T=-1), -1),
    (dict(max_q=-1), -1), (dict(max_q=0), -1), (dict(Hq=7), -1), (dict(Hq=1), -1), (dict(Hkv=0), -1), (dict(M=0), -1),
    (dict(P=24), -1), (dict(P=8), -1), (dict(P=512), -1), (dict(pages=0), -1), (dict(window=-1), -1),
    (dict(scale=float("nan")), -1), (dict(ks=3.0), -1), (dict(vs=0.0), -1), (dict(vs=-1.0), -1),
    (dict(ks=float("inf")), -1), (dict(q=None), -1), (dict(cu=None), -1), (dict(lens=None), -1), (dict(table=None), -1),
    (dict(pool=None), -1), (dict(o=None), -1), (dict(ws=None), -1), (dict(wsb=WS - 1), -1), (dict(q=ODD), -1),
    (dict(pool=ODD), -1), (dict(o=ODD), -1), (dict(ws=ODD), -1), (dict(qs=1023), -1), (dict(qs=1028), -1),
    (dict(B=0), -1), (dict(M=1 << 30, P=256), -1), (dict(T=1 << 30), -1)])
def test_attention_refuses(L, change, status):
    assert L.kda_kv4_attention(*{**ATT, **change}.values()) == status


def test_nothing_to_do_is_not_an_error(L):
    assert L.kda_kv4_attention(*{**ATT, "T": 0}.values()) == 0
    assert L.kda_kv4_attention(*{**ATT, "T": 0, "B": 0, "max_q": 0}.values()) == 0
    assert L.kda_kv4_append(*{**APP, "T": 0}.values()) == 0
    assert L.kda_kv4_gather(*{**GAT, "T": 0}.values()) == 0
    assert L.kda_page_alloc(0, 4, 16, 8, FAKE, None, None, None, None, None) == 0


@pytest.mark.parametrize("change, status", [
    (dict(dt=1), -2), (dict(D=32), -2), (dict(B=-1), -1), (dict(H=0), -1), (dict(P=48), -1), (dict(M=0), -1),
    (dict(pages=0), -1), (dict(ks=1.5), -1), (dict(vs=float("nan")), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(cu=None), -1), (dict(start=None), -1), (dict(table=None), -1), (dict(pool=None), -1), (dict(pool=ODD), -1),
    (dict(k=ODD), -1), (dict(v=ODD), -1), (dict(B=0), -1), (dict(T=1 << 30, H=4, kst=256, vst=256), -1)])
def test_append_and_gather_refuse(L, change, status):
    assert L.kda_kv4_append(*{**APP, **change}.values()) == status
    assert L.kda_kv4_gather(*{**GAT, **{n: x for n, x in change.items() if n in GAT}}.values()) == status


def test_append_refuses_strides(L):
    for change in (dict(kst=127), dict(kst=64), dict(vst=132), dict(vst=-128)):
        assert L.kda_kv4_append(*{**APP, **change}.values()) == -1


def test_pages_refuse(L):
    pools = (ctypes.c_void_p * 2)(4096, 8192)
    bad_pools = (ctypes.c_void_p * 2)(4096, 8200)
    alloc = dict(B=2, M=4, P=16, N=8, refs=FAKE, table=FAKE, lens=FAKE, grow=FAKE, err=None, st=None)
    for c in (dict(B=-1), dict(M=0), dict(P=17), dict(N=0), dict(refs=None), dict(table=None), dict(lens=None),
              dict(grow=None), dict(M=1 << 28)):
        assert L.kda_page_alloc(*{**alloc, **c}.values()) == -1
    free = dict(B=2, M=4, P=16, N=8, refs=FAKE, table=FAKE, lens=FAKE, rows=FAKE, n=1, err=None, st=None)
    for c in (dict(n=-1), dict(rows=None), dict(refs=None), dict(P=0)):
        assert L.kda_page_free(*{**free, **c}.values()) == -1
    assert L.kda_page_free(*{**free, "n": 0}.values()) == 0
    fork = dict(L=2, pools=pools, bytes=1152, B=2, M=4, P=16, N=8, refs=FAKE, table=FAKE, lens=FAKE, src=FAKE, dst=FAKE,
                n=1, ws=FAKE, wsn=2, err=None, st=None)
    for c in (dict(L=0), dict(L=257), dict(pools=None), dict(pools=bad_pools), dict(bytes=0), dict(bytes=1160), dict(n=-1),
              dict(src=None), dict(dst=None), dict(ws=None), dict(wsn=1), dict(lens=None)):
        assert L.kda_page_fork(*{**fork, **c}.values()) == -1
    assert L.kda_page_fork(*{**fork, "n": 0}.values()) == 0
    comp = dict(L=2, pools=pools, bytes=1152, B=2, M=4, N=8, refs=FAKE, table=FAKE, live=FAKE, ws=FAKE, wsn=40, err=None,
                st=None)
    for c in (dict(L=0), dict(bytes=8), dict(B=-1), dict(M=0), dict(N=0), dict(refs=None), dict(table=None), dict(live=None),
              dict(ws=None), dict(wsn=39)):
        assert L.kda_page_compact(*{**comp, **c}.values()) == -1
    copy = dict(L=2, pools=pools, bytes=1152, N=8, src=FAKE, dst=FAKE, n=1, err=None, st=None)
    for c in (dict(L=0), dict(pools=bad_pools), dict(bytes=4), dict(N=0), dict(n=-1), dict(src=None), dict(dst=None)):
        assert L.kda_page_copy(*{**copy, **c}.values()) == -1
    assert L.kda_page_copy(*{**copy, "n": 0}.values()) == 0


def test_binding_refuses_host_tensors_and_sizes(L):
    import kda_state_gb300 as kda
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        kda.kda_page_alloc(i, i[:, None], i, i, 16)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        kda.kda_kv4_attention(torch.zeros(2, 4, 64, dtype=torch.bfloat16), i, 1, i, i[:, None], i)
    with pytest.raises(ValueError, match="non-empty list"):
        kda.kda_page_copy([], i, i)
    with pytest.raises(ValueError, match="page_size"):
        kda.make_kv4_pool(4, 20, 2, 64, device="cpu")
    assert kda.make_kv4_pool(4, 32, 2, 64, device="cpu").shape == (4, 2, 2, 1152)
    assert kda.kv4_tile_bytes(128) == 2304 and kda.kv4_workspace_bytes() == WS

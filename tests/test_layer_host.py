"""Refusals of the residual norm, the rotated append, page bounds, picks and the attention over them that need no GPU:
bad arguments return an error before anything is launched."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(4096)   # never dereferenced
ODD = ctypes.c_void_p(4104)    # 8 bytes past a 16-byte boundary
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def L():
    from kda_state_gb300 import _build
    _build.build()
    import kda_state_gb300 as kda
    return kda.lib()


def call(fn, good, **changes):
    args = dict(good)
    for name, value in changes.items():
        assert name in args, name
        args[name] = value
    return fn(*args.values())


NORM = dict(dt=0, tokens=3, C=64, x=FAKE, xs=64, residual=FAKE, rs=64, w=FAKE, eps=1e-5, mode=1, sum=FAKE, hs=64, out=FAKE,
            scales=FAKE, stream=None)


@pytest.mark.parametrize("status,change", [
    (UNSUPPORTED, dict(dt=7)), (UNSUPPORTED, dict(mode=3)), (INVALID, dict(tokens=-1)), (INVALID, dict(C=0)), (INVALID, dict(C=60)),
    (INVALID, dict(C=32776, xs=32776, rs=32776, hs=32776)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))),
    (INVALID, dict(x=None)), (INVALID, dict(w=None)), (INVALID, dict(out=None)), (INVALID, dict(scales=None)),
    (INVALID, dict(residual=None)), (INVALID, dict(x=ODD)), (INVALID, dict(sum=ODD)), (INVALID, dict(w=ODD)), (INVALID, dict(out=ODD)),
    (INVALID, dict(xs=63)), (INVALID, dict(xs=68)), (INVALID, dict(rs=32)), (INVALID, dict(hs=66)),
    (0, dict(tokens=0, x=None, w=None, out=None)),
])
def test_norm(L, status, change):
    assert call(L.kda_add_rmsnorm, NORM, **change) == status


ROPE = dict(dt=0, B=2, T=3, Hq=4, Hkv=2, D=64, R=64, pairs=0, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, rope=FAKE, positions=50,
            cu=FAKE, start=FAKE, table=FAKE, max_pages=5, page_size=16, pool=FAKE, num_pages=9, k_scale=1.0, v_scale=0.5, out=FAKE,
            os=256, err=None, stream=None)


@pytest.mark.parametrize("status,change", [
    (UNSUPPORTED, dict(dt=1)), (UNSUPPORTED, dict(D=96)), (INVALID, dict(R=0)), (INVALID, dict(R=48)), (INVALID, dict(R=96)),
    (INVALID, dict(positions=0)), (INVALID, dict(Hq=0)), (INVALID, dict(Hkv=0)), (INVALID, dict(page_size=24)), (INVALID, dict(k_scale=3.0)),
    (INVALID, dict(v_scale=0.0)), (INVALID, dict(B=0)), (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)),
    (INVALID, dict(rope=None)), (INVALID, dict(out=None)), (INVALID, dict(cu=None)), (INVALID, dict(pool=None)), (INVALID, dict(rope=ODD)),
    (INVALID, dict(q=ODD)), (INVALID, dict(qs=255)), (INVALID, dict(ks=64)), (INVALID, dict(os=128)), (INVALID, dict(os=264)),
    (INVALID, dict(T=1 << 28)), (0, dict(T=0)),
])
def test_append_rope(L, status, change):
    assert call(L.kda_kv4_append_rope, ROPE, **change) == status


BOUNDS = dict(B=2, T=3, H=2, D=64, cu=FAKE, start=FAKE, table=FAKE, max_pages=5, page_size=16, pool=FAKE, num_pages=9, bounds=FAKE,
              err=None, stream=None)


@pytest.mark.parametrize("status,change", [
    (UNSUPPORTED, dict(D=32)), (INVALID, dict(B=-1)), (INVALID, dict(T=-1)), (INVALID, dict(H=0)), (INVALID, dict(page_size=512)),
    (INVALID, dict(cu=None)), (INVALID, dict(start=None)), (INVALID, dict(table=None)), (INVALID, dict(pool=ODD)),
    (INVALID, dict(bounds=None)), (INVALID, dict(bounds=ODD)), (0, dict(T=0, bounds=None)),
])
def test_bounds(L, status, change):
    assert call(L.kda_kv4_bounds, BOUNDS, **change) == status


PICK = dict(dt=2, B=2, T=3, max_q=2, Hq=4, Hkv=2, D=64, q=FAKE, qs=256, cu=FAKE, lens=FAKE, table=FAKE, max_pages=5, page_size=16,
            bounds=FAKE, num_pages=9, count=4, first=1, recent=1, picked=FAKE, ws=FAKE, ws_bytes=1 << 20, err=None, stream=None)


@pytest.mark.parametrize("status,change", [
    (UNSUPPORTED, dict(dt=1)), (UNSUPPORTED, dict(D=256)), (INVALID, dict(Hq=5)), (INVALID, dict(Hq=1)), (INVALID, dict(max_q=0)),
    (INVALID, dict(count=0)), (INVALID, dict(first=-1)), (INVALID, dict(recent=0)), (INVALID, dict(first=4)),
    (INVALID, dict(first=2, recent=3)), (INVALID, dict(first=0x7fffffff, recent=0x7fffffff)), (INVALID, dict(page_size=8)),
    (INVALID, dict(max_pages=1 << 27)), (INVALID, dict(q=ODD)), (INVALID, dict(qs=128)), (INVALID, dict(lens=None)),
    (INVALID, dict(bounds=ODD)), (INVALID, dict(picked=None)), (INVALID, dict(ws=None)), (INVALID, dict(ws=ODD)),
    (INVALID, dict(ws_bytes=100)), (0, dict(T=0, q=None, ws=None)),
])
def test_pick(L, status, change):
    assert call(L.kda_kv4_pick, PICK, **change) == status


def test_pick_workspace_covers_every_score(L):
    assert L.kda_kv4_pick_workspace_bytes(3, 2, 5) >= 3 * 2 * 5 * 4
    assert L.kda_kv4_pick_workspace_bytes(4096, 8, 8192) >= 4096 * 8 * 8192 * 4
    assert L.kda_kv4_pick_workspace_bytes(-1, 2, 5) == 0 and L.kda_kv4_pick_workspace_bytes(1 << 30, 4, 5) == 0


ATTEND = dict(dt=0, B=2, T=3, max_q=2, Hq=4, Hkv=2, D=64, q=FAKE, qs=256, cu=FAKE, lens=FAKE, table=FAKE, max_pages=5, page_size=16,
              picked=FAKE, count=4, pool=FAKE, num_pages=9, scale=0.125, k_scale=1.0, v_scale=1.0, o=FAKE, lse=None, ws=FAKE,
              ws_bytes=16 << 20, err=None, stream=None)


@pytest.mark.parametrize("status,change", [
    (UNSUPPORTED, dict(dt=1)), (INVALID, dict(count=0)), (INVALID, dict(picked=None)), (INVALID, dict(Hq=3)), (INVALID, dict(o=ODD)),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(k_scale=0.3)), (INVALID, dict(ws_bytes=16)), (INVALID, dict(pool=None)),
    (0, dict(T=0, picked=None, q=None)),
])
def test_attention_picked(L, status, change):
    assert call(L.kda_kv4_attention_picked, ATTEND, **change) == status

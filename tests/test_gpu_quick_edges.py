"""The plain calls' way to the library: what other threads may do meanwhile, and sizes past 32 bits."""
import ctypes
import threading
import time

import pytest
import torch

import kda_state_gb300 as kda
import kda_state_gb300.binding as binding
from test_gpu_quick_calls import Calls, _lib  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


def addresses():
    L = kda.lib()
    return [ctypes.cast(fn, ctypes.c_void_p).value for fn in (
        L.kda_add_rmsnorm, L.kda_kv4_append_rope, L.kda_kv4_bounds, L.kda_kv4_pick, L.kda_kv4_attention_picked, L.kda_kv4_append,
        L.kda_kv4_gather, L.kda_kv4_attention)]


def test_other_threads_run_while_a_call_is_in_the_library():
    """In place of the append stands the C library's sleep (its first argument, the type's number, is 2 for fp16)."""
    c = Calls()
    k, v = c.qkv[:, 8:10].half(), c.qkv[:, 10:].half()
    where = addresses()
    sleeping = list(where)
    sleeping[5] = ctypes.cast(ctypes.CDLL(None).sleep, ctypes.c_void_p).value
    seen, stop = [], threading.Event()

    def other():
        while not stop.is_set():
            seen.append(time.monotonic())
            time.sleep(0.01)
    worker = threading.Thread(target=other)
    binding._quick.bind(*sleeping)
    try:
        worker.start()
        t0 = time.monotonic()
        assert binding._quick.append(k, v, c.cu, c.start, c.table, c.new_pool(), 1.0, 1.0, None) is True
        t1 = time.monotonic()
    finally:
        binding._quick.bind(*where)
        stop.set()
        worker.join()
    assert t1 - t0 > 1.5 and sum(t0 + 0.2 < t < t1 - 0.2 for t in seen) > 10


def test_a_table_wider_than_32_bits_count_is_refused():
    """[1, 2^32 + 1] (17 GB): not taken for a table of one page."""
    c = Calls()
    k, v, pool = c.qkv[:1, 8:10], c.qkv[:1, 10:], c.new_pool()
    table = torch.zeros(1, 2 ** 32 + 1, dtype=torch.int32, device=DEV)
    cu, zero = torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    before = pool.clone()
    assert binding._quick.append(k, v, cu, zero, table, pool, 1.0, 1.0, None) is None
    for call in (lambda: kda.kda_kv4_attention(c.qkv[:1, :8], cu, 1, zero + 1, table, pool, workspace=c.ws),
                 lambda: kda.kda_kv4_pick(c.qkv[:1, :8], cu, 1, zero + 1, table, c.bounds, 16, 3, workspace=c.pick_ws)):
        with pytest.raises((ValueError, RuntimeError, ctypes.ArgumentError)):
            call()
    torch.cuda.synchronize()
    assert torch.equal(pool, before)
    del table
    torch.cuda.empty_cache()


def test_calls_of_several_threads():
    """Each thread on a stream of its own, with operands and workspaces of its own."""
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                c = Calls()
                want = c.norm(scales="block"), c.rope_append(), c.pick(), c.attention(), c.attention_picked()
                for _ in range(100):
                    got = c.norm(scales="block"), c.rope_append(), c.pick(), c.attention(), c.attention_picked()
                    for x, y in zip(sum(map(tuple, got), ()), sum(map(tuple, want), ())):
                        if not torch.equal(x.view(torch.uint8), y.view(torch.uint8)):
                            wrong.append(i)
        except Exception as e:             # noqa: BLE001
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong

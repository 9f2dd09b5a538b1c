"""The plain calls' way to the library: what other threads may do meanwhile, and sizes past 32 bits."""
import ctypes
import threading
import time

import pytest

import kda_state_gb300 as kda
import kda_state_gb300.binding as binding
from test_gpu_quick_calls import Calls, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


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

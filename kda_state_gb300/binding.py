"""ctypes binding of libkda.so: the C entry points under the same names.

Argument marshalling only -- every step of the KDA path runs in the library's
CUDA kernels.  Tensors are torch tensors on the current CUDA device (PyTorch
supplies device memory and streams); shapes follow include/kda.h.  If the
library is missing the calls raise: there is no other implementation.

Errors that depend on device data (a slot id out of range, inconsistent
cu_seqlens, an accept length above the window, a wait that gave up) are found
by the kernels, which skip the affected unit and set KDA_DEVERR_* bits in
``dev_err``.  The calls never synchronise, so those bits cannot be raised here:
pass a zeroed int32 device tensor as ``dev_err`` and read it after the stream
has synchronised.  With ``dev_err=None`` (the default) such units are skipped
without a report.
"""
from __future__ import annotations

import array
import ctypes
import importlib.machinery
import importlib.util
import os
import warnings
from dataclasses import dataclass

import torch

from . import _build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
QUICK_PATH = os.path.join(_HERE, "_quick.so")

KDA_OK = 0
KDA_ERR_INVALID_ARG = -1
KDA_ERR_UNSUPPORTED = -2
KDA_ERR_CUDA = -3
KDA_DTYPE_BF16 = 0
KDA_DTYPE_FP32 = 1
KDA_DTYPE_FP16 = 2
KDA_DEVERR_SLOT_RANGE = 1
KDA_DEVERR_ACCEPT_RANGE = 2
KDA_DEVERR_SEQLENS = 4
KDA_DEVERR_RANGE = 8
KDA_DEVERR_TIMEOUT = 16
KDA_DEVERR_PAGE_RANGE = 32
KDA_DEVERR_PAGES = 64
KDA_NORM_TYPE = 0
KDA_NORM_E4M3_ROW = 1
KDA_NORM_E4M3_BLOCK = 2
KDA_MAX_LAYERS = 256
K_DIM = 128
V_DIM = 128

_DT = {torch.bfloat16: KDA_DTYPE_BF16, torch.float32: KDA_DTYPE_FP32}

_lib = None
# The plain calls' way to the library (csrc/kda_quick.cpp), once that is loaded: it does what the functions here do for
# exact torch tensors on the current device and stream, and returns None for whatever it does not take.
_quick = None


def _load_quick(L):
    """The module, or None with a warning: it is a faster way, and only into the interpreter and torch it was built for."""
    try:
        had, key = _build.quick_built_for(), _build.quick_key()
        if had != key or not os.path.exists(QUICK_PATH):
            raise ImportError("it is built for %s, this is %s" % (had or "nothing", key) if had != key else "it is not there")
        loader = importlib.machinery.ExtensionFileLoader("_quick", QUICK_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_quick", QUICK_PATH, loader=loader))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn("calls take longer without %s (%s); run __graft_entry__.build()" % (QUICK_PATH, e), RuntimeWarning)
        return None
    module.bind(*[ctypes.cast(fn, ctypes.c_void_p).value for fn in (
        L.kda_add_rmsnorm, L.kda_kv4_append_rope, L.kda_kv4_bounds, L.kda_kv4_pick, L.kda_kv4_attention_picked,
        L.kda_kv4_append, L.kda_kv4_gather, L.kda_kv4_attention)])
    return module


class KdaError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__("%s failed: %s (%d)" % (fn, kda_status_string(status), status))
        self.status = status


class kda_ring(ctypes.Structure):
    """Mirror of the C struct ``kda_ring`` (one layer's ReplaySSM input ring)."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("decay", ctypes.c_void_p),
                ("beta", ctypes.c_void_p), ("ring_len", ctypes.c_int), ("reserved", ctypes.c_int)]


def lib() -> ctypes.CDLL:
    """Load libkda.so (built by ``kda_state_gb300._build.build()``)."""
    global _lib, _quick
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkda.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, ip = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
        L.kda_chunk_prefill.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, ip, ip, vp, i, ip, ip,
                                        ip, vp, f, ip, vp]
        L.kda_chunk_prefill_checkpoints.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, ip, ip,
                                                    vp, i, ip, ip, ip, i, ip, i, vp, f, ip, vp]
        L.kda_decode_step.argtypes = [i, i, i, i, i, vp, vp, vp, vp, vp, ip, vp, i, vp, f, ip, vp]
        L.kda_verify_store_inputs.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, ip, vp, i,
                                              ctypes.POINTER(kda_ring), ip, vp, f, ip, vp]
        L.kda_verify_store_inputs_ragged.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, ip, i,
                                                     ip, vp, i, ctypes.POINTER(kda_ring), ip, vp,
                                                     f, ip, vp]
        L.kda_replay_fold.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_void_p),
                                      ctypes.POINTER(kda_ring), i, i, ip, ip, ip, ip, vp]
        L.kda_verify_snapshot.argtypes = [i, i, i, i, i, i, vp, vp, vp, vp, vp, ip, vp, i, vp, ip,
                                          i, vp, f, ip, vp]
        L.kda_snapshot_commit.argtypes = [i, i, i, i, i, i, ctypes.POINTER(ctypes.c_void_p),
                                          ctypes.POINTER(ctypes.c_void_p), i, i, ip, ip, ip, ip,
                                          vp]
        ll = ctypes.c_longlong
        L.kda_conv_prologue.argtypes = [i, i, i, i, i, vp, vp, vp, ll, vp, vp, vp, i, ip, ip, ip, ip,
                                        vp, vp, vp, vp, f, ip, vp]
        L.kda_gated_rmsnorm.argtypes = [i, i, i, i, vp, ll, ll, vp, vp, f, vp, vp]
        L.kda_decode_fused.argtypes = [i, i, i, i, i, vp, vp, vp, ll, vp, vp, vp, vp, vp, vp, ip, vp,
                                       i, vp, f, f, f, ip, vp]
        L.kda_slot_copy.argtypes = [i, ctypes.POINTER(ctypes.c_void_p), ctypes.c_size_t, i, ip, ip,
                                    i, ip, vp]
        sz = ctypes.c_size_t
        L.kda_kv4_append.argtypes = [i, i, i, i, i, vp, ll, vp, ll, ip, ip, ip, i, i, vp, i, f, f, ip,
                                     vp]
        L.kda_kv4_gather.argtypes = [i, i, i, i, i, vp, vp, ip, ip, ip, i, i, vp, i, f, f, ip, vp]
        L.kda_kv4_workspace_bytes.argtypes = []
        L.kda_kv4_workspace_bytes.restype = sz
        L.kda_kv4_attention.argtypes = [i, i, i, i, i, i, i, vp, ll, ip, ip, ip, i, i, vp, i, i, f, f,
                                        f, vp, vp, vp, sz, ip, vp]
        L.kda_selftest_kv4_wait.argtypes = [i, i, i, i, i, i, i, vp, ll, ip, ip, ip, i, i, vp, i, vp, vp,
                                            sz, ip, i, vp]
        L.kda_kv4_append_rope.argtypes = [i, i, i, i, i, i, i, i, vp, ll, vp, ll, vp, ll, vp, i, ip, ip, ip,
                                          i, i, vp, i, f, f, vp, ll, ip, vp]
        L.kda_kv4_bounds.argtypes = [i, i, i, i, ip, ip, ip, i, i, vp, i, vp, ip, vp]
        L.kda_kv4_pick_workspace_bytes.argtypes = [i, i, i]
        L.kda_kv4_pick_workspace_bytes.restype = sz
        L.kda_kv4_pick.argtypes = [i, i, i, i, i, i, i, vp, ll, ip, ip, ip, i, i, vp, i, i, i, i, ip, vp, sz,
                                   ip, vp]
        L.kda_selftest_kv4_pick_wait.argtypes = [i, i, i, i, i, i, i, vp, ll, ip, ip, ip, i, i, vp, i, i, i, i, ip, vp, sz,
                                                 ip, i, vp]
        L.kda_kv4_attention_picked.argtypes = [i, i, i, i, i, i, i, vp, ll, ip, ip, ip, i, i, ip, i, vp, i, f,
                                               f, f, vp, vp, vp, sz, ip, vp]
        L.kda_add_rmsnorm.argtypes = [i, i, i, vp, ll, vp, ll, vp, f, i, vp, ll, vp, vp, vp]
        L.kda_page_alloc.argtypes = [i, i, i, i, ip, ip, ip, ip, ip, vp]
        L.kda_page_fork.argtypes = [i, vp, sz, i, i, i, i, ip, ip, ip, ip, ip, i, vp, sz, ip, vp]
        L.kda_page_free.argtypes = [i, i, i, i, ip, ip, ip, ip, i, ip, vp]
        L.kda_page_compact.argtypes = [i, vp, sz, i, i, i, ip, ip, ip, vp, sz, ip, vp]
        L.kda_page_copy.argtypes = [i, vp, sz, i, ip, ip, i, ip, vp]
        L.kda_selftest_bounded_wait.argtypes = [ip, i, vp]
        L.kda_selftest_prefill_wait.argtypes = [i, i, i, vp, vp, vp, vp, vp, ip, ip, vp, i, ip, ip,
                                                vp, ip, i, vp]
        for fn in ("kda_chunk_prefill", "kda_chunk_prefill_checkpoints", "kda_decode_step", "kda_verify_store_inputs",
                   "kda_verify_store_inputs_ragged", "kda_verify_snapshot",
                   "kda_snapshot_commit", "kda_conv_prologue", "kda_gated_rmsnorm",
                   "kda_decode_fused",
                   "kda_add_rmsnorm", "kda_kv4_append_rope", "kda_kv4_bounds", "kda_kv4_pick",
                   "kda_kv4_attention_picked", "kda_kv4_append", "kda_kv4_gather", "kda_kv4_attention", "kda_page_alloc",
                   "kda_page_fork", "kda_page_free", "kda_page_compact", "kda_page_copy",
                   "kda_replay_fold", "kda_slot_copy", "kda_selftest_bounded_wait",
                   "kda_selftest_prefill_wait", "kda_selftest_kv4_wait", "kda_selftest_kv4_pick_wait"):
            getattr(L, fn).restype = ctypes.c_int
        L.kda_status_string.argtypes = [ctypes.c_int]
        L.kda_status_string.restype = ctypes.c_char_p
        _quick = _load_quick(L)
        _lib = L
    return _lib


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _make(stream, shape, dtype, device, zero=False, result=True):
    """A result that the caller did not pass, or (``result`` false) a buffer for the call alone.

    Made, zeroed and given back on the stream that the call runs on: on the current one nothing
    would order the zeroing before the kernels, or a later owner of the memory after them.  A
    result is used on the current stream next, so that one holds its memory too."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else
                  torch.cuda.default_stream(device))
    current = torch.cuda.current_stream(device)
    if current.cuda_stream == stream.cuda_stream:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = make(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(current)
    return t


def _check(fn, status):
    if status != KDA_OK:
        raise KdaError(fn, status)


def _dt(t):
    if t.dtype not in _DT:
        raise TypeError("unsupported dtype %s (bf16 or fp32)" % t.dtype)
    return _DT[t.dtype]


I32 = torch.int32
F32 = torch.float32


def _need(t, name, shape=None, dtype=None, device=None, dense=True, optional=False):
    """Check one tensor argument against the layout include/kda.h states (the C
    side receives a bare pointer and cannot): a CUDA tensor, on ``device`` when
    given, of ``dtype``, of ``shape`` (None matches any size) and, when
    ``dense``, contiguous.  Raises ValueError / TypeError before anything is
    launched."""
    if t is None:
        if optional:
            return
        raise ValueError("%s is required" % name)
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the other operands on %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if shape is not None and (t.dim() != len(shape) or
                              any(e is not None and e != n for e, n in zip(shape, t.shape))):
        raise ValueError("%s has shape %s, expected [%s]" % (
            name, list(t.shape), ", ".join("*" if e is None else str(e) for e in shape)))
    if dense and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _need_err(dev_err, device):
    """dev_err: None or a device int32 tensor of at least one element."""
    _need(dev_err, "dev_err", dtype=I32, device=device, optional=True)
    if dev_err is not None and dev_err.numel() < 1:
        raise ValueError("dev_err needs at least one element")


def _need_ring(ring, H, K, V, dtype, device, name="ring"):
    """A ring's four buffers: k, v [S, R, H, K|V] in the input dtype, decay
    [S, R, H, K] and beta [S, R, H] in fp32, one slot count and ring length."""
    _need(ring.k, name + ".k", (None, None, H, K), dtype, device)
    S, R = ring.k.shape[0], ring.k.shape[1]
    _need(ring.v, name + ".v", (S, R, H, V), dtype, device)
    _need(ring.decay, name + ".decay", (S, R, H, K), F32, device)
    _need(ring.beta, name + ".beta", (S, R, H), F32, device)


def _need_inputs(q, k, v, gk, beta, lead):
    """q, k, gk [*lead, H, K] and v [*lead, H, V], beta [*lead, H], one dtype
    (bf16 or fp32), dense, on q's device.  Returns (dtype, device, H, K, V)."""
    _need(q, "q", tuple(lead) + (None, None))
    dt, dev = q.dtype, q.device
    _dt(q)
    H, K = q.shape[-2], q.shape[-1]
    _need(k, "k", tuple(lead) + (H, K), dt, dev)
    _need(gk, "gk", tuple(lead) + (H, K), dt, dev)
    _need(v, "v", tuple(lead) + (H, None), dt, dev)
    _need(beta, "beta", tuple(lead) + (H,), dt, dev)
    return dt, dev, H, K, v.shape[-1]


# ---------------------------------------------------------------------------
# ReplaySSM ring helpers
# ---------------------------------------------------------------------------

def ring_len_for(gamma: int) -> int:
    """Ring length for gamma draft tokens: the smallest power of two that is at
    least 2 (gamma + 1) (gamma = 5 -> 12 -> 16)."""
    need = 2 * (int(gamma) + 1)
    r = 1
    while r < need:
        r <<= 1
    return r


def state_bytes(K: int = K_DIM, V: int = V_DIM) -> int:
    """Bytes of one (request, layer, head) fp32 state: 64 KB at K = V = 128."""
    return K * V * 4


def record_bytes(dtype=torch.bfloat16, K: int = K_DIM, V: int = V_DIM) -> int:
    """Bytes of one stored ring record: k and v in the input dtype, exp(gk) and
    beta in fp32 (1028 B for bf16 at K = V = 128)."""
    es = torch.tensor([], dtype=dtype).element_size()
    return K * es + V * es + K * 4 + 4


@dataclass
class RingBuffers:
    """One layer's ring: k, v [num_slots, R, H, K|V] (input dtype), decay
    [num_slots, R, H, K] and beta [num_slots, R, H] (fp32)."""
    k: torch.Tensor
    v: torch.Tensor
    decay: torch.Tensor
    beta: torch.Tensor

    @property
    def ring_len(self) -> int:
        return self.k.shape[1]

    def descriptor(self) -> kda_ring:
        return kda_ring(self.k.data_ptr(), self.v.data_ptr(), self.decay.data_ptr(),
                        self.beta.data_ptr(), self.ring_len, 0)


def make_ring(num_slots: int, ring_len: int, H: int, dtype=torch.bfloat16, device="cuda",
              K: int = K_DIM, V: int = V_DIM) -> RingBuffers:
    return RingBuffers(torch.zeros(num_slots, ring_len, H, K, dtype=dtype, device=device),
                       torch.zeros(num_slots, ring_len, H, V, dtype=dtype, device=device),
                       torch.zeros(num_slots, ring_len, H, K, dtype=torch.float32, device=device),
                       torch.zeros(num_slots, ring_len, H, dtype=torch.float32, device=device))


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def _need_prefill_common(cu_seqlens, N, state_pool, H, K, V, init_slot, out_slot, snap_slot,
                         dev_err, dev):
    if N < 0:
        raise ValueError("cu_seqlens_host needs N + 1 >= 1 entries")
    _need(cu_seqlens, "cu_seqlens", (N + 1,), I32, dev)
    _need(state_pool, "state_pool", (None, H, K, V), F32, dev)
    _need(init_slot, "init_slot", (N,), I32, dev)
    _need(out_slot, "out_slot", (N,), I32, dev)
    _need(snap_slot, "snap_slot", (N,), I32, dev, optional=True)
    _need_err(dev_err, dev)


def kda_chunk_prefill(q, k, v, gk, beta, cu_seqlens, cu_seqlens_host, state_pool, init_slot,
                      out_slot, snap_slot=None, o=None, scale: float = 1.0, dev_err=None,
                      stream=None):
    """q/k/gk [T, H, K], v [T, H, V], beta [T, H] on the device; cu_seqlens int32
    [N+1] on the device and its host copy; state_pool fp32 [slots, H, K, V];
    init_slot / out_slot / snap_slot int32 [N] on the device.  Returns o."""
    _need(q, "q", (None, None, None))
    T = q.shape[0]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (T,))
    host = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    N = host.numel() - 1
    _need_prefill_common(cu_seqlens, N, state_pool, H, K, V, init_slot, out_slot, snap_slot,
                         dev_err, dev)
    if o is None:
        o = _make(stream, (T, H, V), q.dtype, q.device)
    _need(o, "o", (T, H, V), dt, dev)
    hp = host.numpy().ctypes.data_as(ctypes.c_void_p)
    _check("kda_chunk_prefill", lib().kda_chunk_prefill(
        _dt(q), N, T, H, K, V, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(cu_seqlens), hp,
        _p(state_pool), state_pool.shape[0], _p(init_slot), _p(out_slot), _p(snap_slot), _p(o),
        float(scale), _p(dev_err), _stream(stream)))
    return o


def kda_chunk_prefill_checkpoints(q, k, v, gk, beta, cu_seqlens, cu_seqlens_host, state_pool,
                                  init_slot, out_slot, ckpt_interval: int, ckpt_slots,
                                  snap_slot=None, o=None, scale: float = 1.0, dev_err=None,
                                  stream=None):
    """``kda_chunk_prefill`` that also writes the state after every
    ``ckpt_interval`` tokens of sequence n into slot ``ckpt_slots[n, m]``
    (int32 [N, max_ckpts] on the device, -1 skips).  Returns o."""
    _need(q, "q", (None, None, None))
    T = q.shape[0]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (T,))
    host = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    N = host.numel() - 1
    _need_prefill_common(cu_seqlens, N, state_pool, H, K, V, init_slot, out_slot, snap_slot,
                         dev_err, dev)
    _need(ckpt_slots, "ckpt_slots", (N, None), I32, dev)
    if o is None:
        o = _make(stream, (T, H, V), q.dtype, q.device)
    _need(o, "o", (T, H, V), dt, dev)
    hp = host.numpy().ctypes.data_as(ctypes.c_void_p)
    _check("kda_chunk_prefill_checkpoints", lib().kda_chunk_prefill_checkpoints(
        _dt(q), N, T, H, K, V, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(cu_seqlens), hp,
        _p(state_pool), state_pool.shape[0], _p(init_slot), _p(out_slot), _p(snap_slot),
        int(ckpt_interval), _p(ckpt_slots), ckpt_slots.shape[1], _p(o), float(scale),
        _p(dev_err), _stream(stream)))
    return o


def kda_decode_step(q, k, v, gk, beta, slot_ids, state_pool, o=None, scale: float = 1.0,
                    dev_err=None, stream=None):
    """q/k/gk [B, H, K], v [B, H, V], beta [B, H]; slot_ids int32 [B].  Updates the
    pool in place and returns o [B, H, V]."""
    _need(q, "q", (None, None, None))
    B = q.shape[0]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (B,))
    _need(slot_ids, "slot_ids", (B,), I32, dev)
    _need(state_pool, "state_pool", (None, H, K, V), F32, dev)
    _need_err(dev_err, dev)
    if o is None:
        o = _make(stream, (B, H, V), q.dtype, q.device)
    _need(o, "o", (B, H, V), dt, dev)
    _check("kda_decode_step", lib().kda_decode_step(
        _dt(q), B, H, K, V, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(slot_ids), _p(state_pool),
        state_pool.shape[0], _p(o), float(scale), _p(dev_err), _stream(stream)))
    return o


def kda_verify_store_inputs(q, k, v, gk, beta, slot_ids, state_pool, ring: RingBuffers,
                            ring_base=None, o=None, scale: float = 1.0, dev_err=None, stream=None):
    """q/k/gk [B, G, H, K], v [B, G, H, V], beta [B, G, H]; reads the pool, never
    writes it; stores the G records into ``ring``.  Returns o [B, G, H, V]."""
    _need(q, "q", (None, None, None, None))
    B, G = q.shape[0], q.shape[1]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (B, G))
    _need(slot_ids, "slot_ids", (B,), I32, dev)
    _need(state_pool, "state_pool", (None, H, K, V), F32, dev)
    _need_ring(ring, H, K, V, dt, dev)
    _need(ring_base, "ring_base", (B,), I32, dev, optional=True)
    _need_err(dev_err, dev)
    if o is None:
        o = _make(stream, (B, G, H, V), q.dtype, q.device)
    _need(o, "o", (B, G, H, V), dt, dev)
    desc = ring.descriptor()
    _check("kda_verify_store_inputs", lib().kda_verify_store_inputs(
        _dt(q), B, G, H, K, V, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(slot_ids),
        _p(state_pool), state_pool.shape[0], ctypes.byref(desc), _p(ring_base), _p(o),
        float(scale), _p(dev_err), _stream(stream)))
    return o


def kda_verify_store_inputs_ragged(q, k, v, gk, beta, cu_drafts, G_max: int, slot_ids,
                                   state_pool, ring: RingBuffers, ring_base=None, o=None,
                                   scale: float = 1.0, dev_err=None, stream=None):
    """Verify with G_b <= G_max drafts per request: q/k/gk [T, H, K], v [T, H, V],
    beta [T, H] packed by cu_drafts (device int32 [B+1]).  Reads the pool, never
    writes it; stores request b's G_b records into ``ring``.  Returns o [T, H, V]
    (rows of no request are left as they were)."""
    _need(q, "q", (None, None, None))
    T = q.shape[0]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (T,))
    _need(cu_drafts, "cu_drafts", (None,), I32, dev)
    B = cu_drafts.numel() - 1
    if B < 0:
        raise ValueError("cu_drafts needs B + 1 >= 1 entries")
    _need(slot_ids, "slot_ids", (B,), I32, dev)
    _need(state_pool, "state_pool", (None, H, K, V), F32, dev)
    _need_ring(ring, H, K, V, dt, dev)
    _need(ring_base, "ring_base", (B,), I32, dev, optional=True)
    _need_err(dev_err, dev)
    if o is None:
        o = _make(stream, (T, H, V), q.dtype, q.device, zero=True)
    _need(o, "o", (T, H, V), dt, dev)
    desc = ring.descriptor()
    _check("kda_verify_store_inputs_ragged", lib().kda_verify_store_inputs_ragged(
        _dt(q), B, int(G_max), H, K, V, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(cu_drafts), T,
        _p(slot_ids), _p(state_pool), state_pool.shape[0], ctypes.byref(desc), _p(ring_base),
        _p(o), float(scale), _p(dev_err), _stream(stream)))
    return o


def kda_replay_fold(state_pools, rings, slot_ids, accept_len, max_accept: int, ring_base=None,
                    dev_err=None, stream=None):
    """Fold the accepted prefixes of every layer in one launch.  state_pools: list
    of L fp32 pools [slots, H, K, V]; rings: list of L RingBuffers."""
    L = len(state_pools)
    if L != len(rings) or L == 0:
        raise ValueError("state_pools and rings must be non-empty lists of equal length")
    _need(state_pools[0], "state_pools[0]", (None, None, None, None), F32)
    S, H, K, V = state_pools[0].shape
    dev = state_pools[0].device
    for i, p in enumerate(state_pools):
        _need(p, "state_pools[%d]" % i, (S, H, K, V), F32, dev)
    dt = rings[0].k.dtype
    if dt not in _DT:
        raise TypeError("unsupported ring dtype %s (bf16 or fp32)" % dt)
    for i, r in enumerate(rings):
        _need_ring(r, H, K, V, dt, dev, "rings[%d]" % i)
    _need(slot_ids, "slot_ids", (None,), I32, dev)
    B = slot_ids.numel()
    _need(accept_len, "accept_len", (B,), I32, dev)
    _need(ring_base, "ring_base", (B,), I32, dev, optional=True)
    _need_err(dev_err, dev)
    ptrs = (ctypes.c_void_p * L)(*[p.data_ptr() for p in state_pools])
    descs = (kda_ring * L)(*[r.descriptor() for r in rings])
    _check("kda_replay_fold", lib().kda_replay_fold(
        _DT[rings[0].k.dtype], L, B, H, K, V, ptrs, descs, S, int(max_accept), _p(slot_ids),
        _p(accept_len), _p(ring_base), _p(dev_err), _stream(stream)))


def kda_verify_snapshot(q, k, v, gk, beta, slot_ids, state_pool, snaps, snap_ids, o=None,
                        scale: float = 1.0, dev_err=None, stream=None):
    """Snapshot-per-step verify: q/k/gk [B, G, H, K], v [B, G, H, V], beta
    [B, G, H]; writes the state after draft step i of request b to
    snaps[snap_ids[b], i] (snaps fp32 [num_snap_slots, G, H, K, V]); never writes
    the pool.  Returns o [B, G, H, V]."""
    _need(q, "q", (None, None, None, None))
    B, G = q.shape[0], q.shape[1]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (B, G))
    _need(slot_ids, "slot_ids", (B,), I32, dev)
    _need(state_pool, "state_pool", (None, H, K, V), F32, dev)
    _need(snaps, "snaps", (None, G, H, K, V), F32, dev)
    _need(snap_ids, "snap_ids", (B,), I32, dev)
    _need_err(dev_err, dev)
    if o is None:
        o = _make(stream, (B, G, H, V), q.dtype, q.device)
    _need(o, "o", (B, G, H, V), dt, dev)
    _check("kda_verify_snapshot", lib().kda_verify_snapshot(
        _dt(q), B, G, H, K, V, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(slot_ids),
        _p(state_pool), state_pool.shape[0], _p(snaps), _p(snap_ids), snaps.shape[0], _p(o),
        float(scale), _p(dev_err), _stream(stream)))
    return o


def kda_snapshot_commit(state_pools, snaps, slot_ids, snap_ids, accept_len, dev_err=None,
                        stream=None):
    """Copy snapshot accept_len[b]-1 over slot slot_ids[b] in every layer, one
    launch.  state_pools / snaps: lists of L pools [slots, H, K, V] and snapshot
    buffers [num_snap_slots, G, H, K, V]."""
    L = len(state_pools)
    if L != len(snaps) or L == 0:
        raise ValueError("state_pools and snaps must be non-empty lists of equal length")
    _need(state_pools[0], "state_pools[0]", (None, None, None, None), F32)
    S, H, K, V = state_pools[0].shape
    dev = state_pools[0].device
    _need(snaps[0], "snaps[0]", (None, None, H, K, V), F32, dev)
    NS, G = snaps[0].shape[0], snaps[0].shape[1]
    for i in range(L):
        _need(state_pools[i], "state_pools[%d]" % i, (S, H, K, V), F32, dev)
        _need(snaps[i], "snaps[%d]" % i, (NS, G, H, K, V), F32, dev)
    _need(slot_ids, "slot_ids", (None,), I32, dev)
    B = slot_ids.numel()
    _need(snap_ids, "snap_ids", (B,), I32, dev)
    _need(accept_len, "accept_len", (B,), I32, dev)
    _need_err(dev_err, dev)
    pp = (ctypes.c_void_p * L)(*[p.data_ptr() for p in state_pools])
    sp = (ctypes.c_void_p * L)(*[p.data_ptr() for p in snaps])
    _check("kda_snapshot_commit", lib().kda_snapshot_commit(
        L, B, H, K, V, G, pp, sp, S, NS, _p(slot_ids), _p(snap_ids),
        _p(accept_len), _p(dev_err), _stream(stream)))


# ---------------------------------------------------------------------------
# fused prologue / epilogue around the recurrence
# ---------------------------------------------------------------------------

CONV_WIDTH = 4          # KDA_CONV_WIDTH
EPS_L2 = 1e-6           # q, k L2 norm
EPS_NORM = 1e-5         # gated RMSNorm of o


def _raw_stride(q_raw, k_raw, v_raw, K):
    """Token stride (elements) shared by three [T, H, K] raw views whose head
    and channel axes are dense (e.g. slices of one fused projection output)."""
    st = q_raw.stride(0)
    for x in (q_raw, k_raw, v_raw):
        if x.stride(-1) != 1 or x.stride(-2) != K or x.stride(0) != st:
            raise ValueError("q_raw, k_raw, v_raw need dense [H, K] rows and one token stride")
    return st


def make_conv_state(num_slots: int, H: int, dtype=torch.bfloat16, device="cuda", K: int = K_DIM):
    """Conv state pool [num_slots, W-1, 3, H, K] (zeros)."""
    return torch.zeros(num_slots, CONV_WIDTH - 1, 3, H, K, dtype=dtype, device=device)


def kda_conv_prologue(q_raw, k_raw, v_raw, b_raw, conv_w, conv_state, init_slot, out_slot,
                      cu_seqlens, cu_seqlens_host, eps_l2: float = EPS_L2, out=None, dev_err=None,
                      stream=None):
    """Short conv + SiLU of q, k, v ([T, H, K] views sharing a token stride), L2
    norm of q and k, beta = sigmoid(b_raw [T, H]); conv_w [3, H, K, W];
    conv_state [slots, W-1, 3, H, K] read at init_slot and written at out_slot
    (int32 [N] on the device, -1: zeros / none).  Returns (q, k, v, beta)."""
    _need(q_raw, "q_raw", (None, None, None), dense=False)
    T, H, K = q_raw.shape
    dt, dev = q_raw.dtype, q_raw.device
    _dt(q_raw)
    _need(k_raw, "k_raw", (T, H, K), dt, dev, dense=False)
    _need(v_raw, "v_raw", (T, H, K), dt, dev, dense=False)
    st = _raw_stride(q_raw, k_raw, v_raw, K)
    host = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    N = host.numel() - 1
    if N < 0:
        raise ValueError("cu_seqlens_host needs N + 1 >= 1 entries")
    _need(b_raw, "b_raw", (T, H), dt, dev)
    _need(conv_w, "conv_w", (3, H, K, CONV_WIDTH), dt, dev)
    _need(conv_state, "conv_state", (None, CONV_WIDTH - 1, 3, H, K), dt, dev)
    _need(init_slot, "init_slot", (N,), I32, dev)
    _need(out_slot, "out_slot", (N,), I32, dev)
    _need(cu_seqlens, "cu_seqlens", (N + 1,), I32, dev)
    _need_err(dev_err, dev)
    if out is None:
        out = tuple(_make(stream, shape, q_raw.dtype, q_raw.device)
                    for shape in ((T, H, K), (T, H, K), (T, H, K), (T, H)))
    q, k, v, beta = out
    for name, t in (("out[0]", q), ("out[1]", k), ("out[2]", v)):
        _need(t, name, (T, H, K), dt, dev)
    _need(beta, "out[3]", (T, H), dt, dev)
    hp = host.numpy().ctypes.data_as(ctypes.c_void_p)
    _check("kda_conv_prologue", lib().kda_conv_prologue(
        _dt(q_raw), N, T, H, K, _p(q_raw), _p(k_raw), _p(v_raw), st, _p(b_raw), _p(conv_w),
        _p(conv_state), conv_state.shape[0], _p(init_slot), _p(out_slot), _p(cu_seqlens), hp,
        _p(q), _p(k), _p(v), _p(beta), float(eps_l2), _p(dev_err), _stream(stream)))
    return q, k, v, beta


def kda_gated_rmsnorm(o, gate, w_norm, eps: float = EPS_NORM, out=None, stream=None):
    """out = w_norm * o / sqrt(mean o^2 + eps) * sigmoid(gate) per [token, head]
    row; o [T, H, V] may be strided (channel axis dense)."""
    _need(o, "o", (None, None, None), dense=False)
    T, H, V = o.shape
    dt, dev = o.dtype, o.device
    _dt(o)
    if o.stride(-1) != 1:
        raise ValueError("o needs a dense channel axis")
    _need(gate, "gate", (T, H, V), dt, dev)
    _need(w_norm, "w_norm", (V,), dt, dev)
    if out is None:
        out = _make(stream, (T, H, V), o.dtype, o.device)
    _need(out, "out", (T, H, V), dt, dev)
    _check("kda_gated_rmsnorm", lib().kda_gated_rmsnorm(
        _dt(o), T, H, V, _p(o), o.stride(0), o.stride(1), _p(gate), _p(w_norm), float(eps),
        _p(out), _stream(stream)))
    return out


_NORM_DT = {torch.bfloat16: KDA_DTYPE_BF16, torch.float16: KDA_DTYPE_FP16, torch.float32: KDA_DTYPE_FP32}
_NORM_BYTES = {torch.bfloat16: 2, torch.float16: 2, torch.float32: 4}
_NORM_OUT = {"none": KDA_NORM_TYPE, "row": KDA_NORM_E4M3_ROW, "block": KDA_NORM_E4M3_BLOCK}
NORM_BLOCK = 128      # channels of a scale


def _norm_rows(t, name, dtype, shape, dev):
    """[tokens, C] whose channels are dense and whose rows may be strided.  Returns the address and the
    stride between rows, in elements."""
    try:
        same = t.dtype is dtype and t.shape == shape and t.get_device() == dev
    except AttributeError:
        same = False
    if not same:
        _need(t, name, shape, dtype, torch.device("cuda", dev), dense=False)
    stride, one = t.stride()
    if shape[0] <= 1:
        stride = shape[1]
    at = t.data_ptr()
    if one != 1 or stride < shape[1] or stride * _NORM_BYTES[dtype] % 16 != 0 or at % 16 != 0:
        raise ValueError("%s: channels must be dense, rows start on 16-byte boundaries and not overlap" % name)
    return at, stride


def kda_add_rmsnorm(x, residual, weight, eps: float = EPS_NORM, scales: str = "none", residual_out=None,
                    out=None, scales_out=None, stream=None):
    """The norm that a layer begins with: h = x + residual (x [T, C] and residual bf16, fp16 or fp32,
    rows may be strided; h is rounded to their dtype; residual None: h = x) and
    y = weight * h / sqrt(mean h^2 + eps).  ``scales``: "none" for y in the dtype, "row" or "block" for
    e4m3 codes with fp32 scales of a row [T] or of 128 channels [T, ceil(C / 128)].  Returns (out,
    scales or None, h); ``residual_out`` takes h and may be ``residual`` itself."""
    if _quick is not None and stream is None and out is None and scales_out is None and scales in _NORM_OUT:
        done = _quick.add_rmsnorm(x, residual, weight, eps, _NORM_OUT[scales], residual_out)
        if done is not None:
            return done
    shape, dev = _first(x, "x", 2)
    dtype = x.dtype
    if dtype not in _NORM_DT:
        raise TypeError("unsupported dtype %s (bf16, fp16 or fp32)" % dtype)
    if scales not in _NORM_OUT:
        raise ValueError('scales is "none", "row" or "block", not %r' % (scales,))
    T, C = shape
    _sizes("x", T, C)
    xa, xs = _norm_rows(x, "x", dtype, shape, dev)
    wa = _ptr(weight, "weight", (C,), dtype, dev)
    at, kind = x.device, dtype if scales == "none" else torch.float8_e4m3fn
    ra = ha = sa = None
    rs = hs = 0
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
        residual_out = x
    else:
        ra, rs = _norm_rows(residual, "residual", dtype, shape, dev)
        if residual_out is None:
            residual_out = torch.empty(shape, dtype=dtype, device=at) if stream is None else _make(stream, shape, dtype, at)
            ha, hs = residual_out.data_ptr(), C
        else:
            ha, hs = _norm_rows(residual_out, "residual_out", dtype, shape, dev)
    if out is None:
        out = torch.empty(shape, dtype=kind, device=at) if stream is None else _make(stream, shape, kind, at)
        oa = out.data_ptr()
    else:
        oa = _ptr(out, "out", shape, kind, dev)
    if scales == "none":
        if scales_out is not None:
            raise ValueError('scales_out needs scales "row" or "block"')
    else:
        sshape = (T,) if scales == "row" else (T, (C + NORM_BLOCK - 1) // NORM_BLOCK)
        if scales_out is None:
            scales_out = torch.empty(sshape, dtype=F32, device=at) if stream is None else _make(stream, sshape, F32, at)
            sa = scales_out.data_ptr()
        else:
            sa = _ptr(scales_out, "scales_out", sshape, F32, dev)
    status = lib().kda_add_rmsnorm(_NORM_DT[dtype], T, C, xa, xs, ra, rs, wa, eps, _NORM_OUT[scales],
                                   ha, hs, oa, sa, _stream_of(stream, dev))
    if status:
        _check("kda_add_rmsnorm", status)
    return out, scales_out, residual_out


def kda_decode_fused(q_raw, k_raw, v_raw, gk, b_raw, conv_w, conv_state, gate, w_norm, slot_ids,
                     state_pool, out=None, scale: float = 1.0, eps_l2: float = EPS_L2,
                     eps_norm: float = EPS_NORM, dev_err=None, stream=None):
    """Conv + KDA + onorm for one token per request: raw q, k, v [B, H, K]
    (views sharing a token stride), gk, gate [B, H, K], b_raw [B, H]; the
    slot's conv state and KDA state are updated in place.  Returns out [B, H, V]."""
    _need(q_raw, "q_raw", (None, None, None), dense=False)
    B, H, K = q_raw.shape
    dt, dev = q_raw.dtype, q_raw.device
    _dt(q_raw)
    _need(k_raw, "k_raw", (B, H, K), dt, dev, dense=False)
    _need(v_raw, "v_raw", (B, H, K), dt, dev, dense=False)
    _need(state_pool, "state_pool", (None, H, K, None), F32, dev)
    V = state_pool.shape[-1]
    st = _raw_stride(q_raw, k_raw, v_raw, K)
    _need(gk, "gk", (B, H, K), dt, dev)
    _need(b_raw, "b_raw", (B, H), dt, dev)
    _need(conv_w, "conv_w", (3, H, K, CONV_WIDTH), dt, dev)
    _need(conv_state, "conv_state", (None, CONV_WIDTH - 1, 3, H, K), dt, dev)
    _need(gate, "gate", (B, H, V), dt, dev)
    _need(w_norm, "w_norm", (V,), dt, dev)
    _need(slot_ids, "slot_ids", (B,), I32, dev)
    _need_err(dev_err, dev)
    if out is None:
        out = _make(stream, (B, H, V), q_raw.dtype, q_raw.device)
    _need(out, "out", (B, H, V), dt, dev)
    _check("kda_decode_fused", lib().kda_decode_fused(
        _dt(q_raw), B, H, K, V, _p(q_raw), _p(k_raw), _p(v_raw), st, _p(gk), _p(b_raw),
        _p(conv_w), _p(conv_state), _p(gate), _p(w_norm), _p(slot_ids), _p(state_pool),
        state_pool.shape[0], _p(out), float(scale), float(eps_l2), float(eps_norm), _p(dev_err),
        _stream(stream)))
    return out


def kda_slot_copy(pools, src, dst, dev_err=None, stream=None):
    """dst[i] <- src[i] in every pool of the list (int32 device index tensors)."""
    P = len(pools)
    if P == 0:
        raise ValueError("pools must be a non-empty list")
    _need(pools[0], "pools[0]", None, F32)
    dev = pools[0].device
    if pools[0].dim() < 1:
        raise ValueError("pools[0] needs a slot axis")
    for i, p in enumerate(pools):
        _need(p, "pools[%d]" % i, tuple(pools[0].shape), F32, dev)
    _need(src, "src", (None,), I32, dev)
    _need(dst, "dst", (src.numel(),), I32, dev)
    _need_err(dev_err, dev)
    ptrs = (ctypes.c_void_p * P)(*[p.data_ptr() for p in pools])
    slot_elems = pools[0][0].numel()
    _check("kda_slot_copy", lib().kda_slot_copy(
        P, ptrs, slot_elems, pools[0].shape[0], _p(src), _p(dst), src.numel(), _p(dev_err),
        _stream(stream)))


# ---------------------------------------------------------------------------
# the paged 4-bit key/value cache
# ---------------------------------------------------------------------------

# These calls are short next to the host's share of them: each argument is checked with a few
# attribute reads, and only one that fails goes through _need for its message.

KV_TILE = 16          # tokens of a tile
_KV_DT = {torch.bfloat16: KDA_DTYPE_BF16, torch.float16: KDA_DTYPE_FP16}
_U8 = torch.uint8
_numel, _width, _device_of = torch.Tensor.numel, torch.Tensor.element_size, torch.Tensor.get_device
_dense, _address = torch.Tensor.is_contiguous, torch.Tensor.data_ptr


def kv4_tile_bytes(D: int = K_DIM) -> int:
    """Bytes of 16 tokens of one head: codes and scales of K and V (4.5 bits a value)."""
    return 18 * int(D)


def make_kv4_pool(num_pages: int, page_size: int, H_kv: int, D: int = K_DIM, device="cuda"):
    """One layer's pool, uint8 [num_pages, H_kv, page_size / 16, 18 D]."""
    if page_size not in (16, 32, 64, 128, 256):
        raise ValueError("page_size is 16, 32, 64, 128 or 256, not %r" % (page_size,))
    return torch.zeros(num_pages, H_kv, page_size // KV_TILE, kv4_tile_bytes(D), dtype=torch.uint8,
                       device=device)


def kv4_workspace_bytes() -> int:
    return int(lib().kda_kv4_workspace_bytes())


def make_kv4_workspace(device="cuda"):
    """The attention's workspace, for one call at a time (zeroed, as its first call needs it)."""
    return torch.zeros(kv4_workspace_bytes(), dtype=torch.uint8, device=device)


def _kv_dt(dtype):
    if dtype not in _KV_DT:
        raise TypeError("unsupported dtype %s (bf16 or fp16)" % dtype)
    return _KV_DT[dtype]


def _ptr(t, name, shape, dtype, dev):
    """The address of a dense tensor of this shape and dtype on CUDA device number dev."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, shape, dtype, torch.device("cuda", dev))
    return t.data_ptr()


def _int(x):
    """A number as a C int, at its ends where it is past them (ctypes would take it modulo 2^32)."""
    return x if -0x80000000 <= x <= 0x7fffffff else 0x7fffffff if x > 0 else -0x80000000


def _sizes(name, *sizes):
    """A tensor's sizes that the library takes as C ints."""
    if any(n >> 31 for n in sizes):
        raise ValueError("%s: a size is past 2^31 - 1 (%s)" % (name, ", ".join(map(str, sizes))))


def _err_ptr(dev_err, dev):
    if dev_err is None:
        return None
    _need_err(dev_err, torch.device("cuda", dev))
    return dev_err.data_ptr()


def _stream_of(stream, dev):
    """The stream argument as a handle, by default the current one.  The library launches on the current
    device, which has to be the operands'."""
    if torch._C._cuda_getDevice() != dev:
        raise ValueError("the operands are on cuda:%d, the current device is cuda:%d" % (dev, torch._C._cuda_getDevice()))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _first(t, name, dims):
    """The operand that sets the device, a CUDA tensor of ``dims`` dimensions.  Returns its shape and
    the device's number."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != dims:
        _need(t, name, (None,) * dims, dense=False)
    return t.shape, t.get_device()


def _rows(t, name, dtype, shape, dev):
    """[tokens, heads, D] whose heads are dense and whose tokens may be strided.  Returns the
    address and the stride between tokens, in elements."""
    try:
        same = t.dtype is dtype and t.shape == shape and t.get_device() == dev
    except AttributeError:
        same = False
    if not same:
        _need(t, name, shape, dtype, torch.device("cuda", dev), dense=False)
    T, H, D = shape
    stride, head, one = t.stride()
    if T <= 1:
        stride = H * D
    at = t.data_ptr()
    if one != 1 or (H > 1 and head != D):
        raise ValueError("%s: heads and channels must be dense (only tokens may be strided)" % name)
    if stride < H * D or stride % 8 != 0 or at % 16 != 0:
        raise ValueError("%s: tokens must start on 16-byte boundaries and not overlap" % name)
    return at, stride


def _pool(pool, D, dev):
    """uint8 [num_pages, H_kv, page_size / 16, 18 D].  Returns (address, num_pages, H_kv, page_size)."""
    shape = pool.shape if isinstance(pool, torch.Tensor) else ()
    if len(shape) != 4 or shape[3] != 18 * D:
        _need(pool, "pool", (None, None, None, 18 * D), _U8, torch.device("cuda", dev))
    return _ptr(pool, "pool", shape, _U8, dev), shape[0], shape[1], shape[2] * KV_TILE


def _table(page_table, dev):
    """int32 [B, max_pages].  Returns (address, B, max_pages)."""
    shape = page_table.shape if isinstance(page_table, torch.Tensor) else ()
    if len(shape) != 2:
        shape = (None, None)
    at = _ptr(page_table, "page_table", shape, I32, dev)
    _sizes("page_table", *shape)
    return (at,) + tuple(shape)


def kda_kv4_append(k, v, cu_seqlens, start, page_table, pool, k_scale: float = 1.0,
                   v_scale: float = 1.0, dev_err=None, stream=None):
    """Store the packed new tokens' k, v [T, H_kv, D] (bf16 or fp16; tokens may be
    strided) as 4-bit codes: token i of request b at position start[b] + i of the
    pages that row b of page_table (int32 [B, max_pages]) names.  cu_seqlens int32
    [B + 1], start int32 [B]; the scales are powers of two.  Writes the pool in place."""
    if _quick is not None and stream is None and _quick.append(k, v, cu_seqlens, start, page_table, pool, k_scale, v_scale, dev_err):
        return
    shape, dev = _first(k, "k", 3)
    dtype = k.dtype
    dt = _kv_dt(dtype)
    T, H, D = shape
    ka, ks = _rows(k, "k", dtype, shape, dev)
    va, vs = _rows(v, "v", dtype, shape, dev)
    pa, pages, Hp, page_size = _pool(pool, D, dev)
    if Hp != H:
        raise ValueError("pool has %d heads, k has %d" % (Hp, H))
    ta, B, M = _table(page_table, dev)
    status = lib().kda_kv4_append(
        dt, B, T, H, D, ka, ks, va, vs, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(start, "start", (B,), I32, dev), ta, M, page_size, pa, pages, k_scale, v_scale,
        _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_kv4_append", status)


def kda_kv4_gather(cu_seqlens, start, total_tokens: int, page_table, pool, dtype=torch.bfloat16,
                   k=None, v=None, k_scale: float = 1.0, v_scale: float = 1.0, dev_err=None,
                   stream=None):
    """Read tokens back as the values they stand for: positions start[b] + i of request b
    into packed k, v [total_tokens, H_kv, D].  Returns (k, v)."""
    if _quick is not None and stream is None and k is None and v is None:
        done = _quick.gather(cu_seqlens, start, total_tokens, page_table, pool, dtype, k_scale, v_scale, dev_err)
        if done is not None:
            return done
    dt = _kv_dt(dtype)
    shape, dev = _first(pool, "pool", 4)
    D, T = shape[3] // 18, int(total_tokens)
    pa, pages, H, page_size = _pool(pool, D, dev)
    ta, B, M = _table(page_table, dev)
    if k is None:
        k = _make(stream, (T, H, D), dtype, pool.device) if stream is not None else torch.empty(
            T, H, D, dtype=dtype, device=pool.device)
        ka = k.data_ptr()
    else:
        ka = _ptr(k, "k", (T, H, D), dtype, dev)
    if v is None:
        v = _make(stream, (T, H, D), dtype, pool.device) if stream is not None else torch.empty(
            T, H, D, dtype=dtype, device=pool.device)
        va = v.data_ptr()
    else:
        va = _ptr(v, "v", (T, H, D), dtype, dev)
    status = lib().kda_kv4_gather(
        dt, B, T, H, D, ka, va,
        _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev), _ptr(start, "start", (B,), I32, dev),
        ta, M, page_size, pa, pages, k_scale, v_scale, _err_ptr(dev_err, dev),
        _stream_of(stream, dev))
    _check("kda_kv4_gather", status)
    return k, v


def kda_kv4_attention(q, cu_seqlens, max_q: int, kv_lens, page_table, pool, scale=None,
                      window: int = 0, k_scale: float = 1.0, v_scale: float = 1.0, o=None, lse=None,
                      workspace=None, dev_err=None, stream=None):
    """Causal attention of the packed newest tokens' q [T, H_q, D] (bf16 or fp16; tokens
    may be strided) over the cache; kv_lens int32 [B] counts each request's cached
    tokens, the new ones included, and no request has more than max_q new ones.
    ``window`` > 0 lets a token see that many positions, its own among them; ``scale``
    defaults to D ** -0.5.  ``workspace``: ``make_kv4_workspace()``, kept by the caller
    (one for each stream); a call without one makes its own.  Returns (o, lse), o in
    q's dtype and lse fp32 [T, H_q]; a row that sees nothing has o = 0, lse = -inf."""
    if _quick is not None and stream is None and o is None and lse is None and workspace is not None:
        done = _quick.attention(q, cu_seqlens, max_q, kv_lens, page_table, pool, scale, window, k_scale, v_scale, workspace, dev_err)
        if done is not None:
            return done
    shape, dev = _first(q, "q", 3)
    dtype = q.dtype
    dt = _kv_dt(dtype)
    T, H, D = shape
    qa, qs = _rows(q, "q", dtype, shape, dev)
    pa, pages, H_kv, page_size = _pool(pool, D, dev)
    ta, B, M = _table(page_table, dev)
    if o is None:
        o = _make(stream, shape, dtype, q.device) if stream is not None else torch.empty(
            shape, dtype=dtype, device=q.device)
        oa = o.data_ptr()
    else:
        oa = _ptr(o, "o", shape, dtype, dev)
    if lse is None:
        lse = _make(stream, (T, H), F32, q.device) if stream is not None else torch.empty(
            T, H, dtype=F32, device=q.device)
        la = lse.data_ptr()
    else:
        la = _ptr(lse, "lse", (T, H), F32, dev)
    if workspace is None:
        workspace = _make(stream, (kv4_workspace_bytes(),), _U8, q.device, zero=True, result=False)
    (wb,), _ = _first(workspace, "workspace", 1)
    if (max_q | window) >> 31:
        max_q, window = _int(max_q), _int(window)
    status = lib().kda_kv4_attention(
        dt, B, T, max_q, H, H_kv, D, qa, qs, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(kv_lens, "kv_lens", (B,), I32, dev), ta, M, page_size, pa, pages, window,
        D ** -0.5 if scale is None else scale, k_scale, v_scale, oa, la,
        _ptr(workspace, "workspace", (wb,), _U8, dev), wb,
        _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_kv4_attention", status)
    return o, lse


def make_rope_table(positions: int, R: int, base: float = 10000.0, device="cuda"):
    """The angles that ``kda_kv4_append_rope`` turns by: fp32 [positions, R], R / 2 cosines and R / 2 sines of
    p base^(-2 i / R) each, computed in 64 bits."""
    turns = float(base) ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * turns
    return torch.cat([angle.cos(), angle.sin()], -1).float()


def kda_kv4_append_rope(q, k, v, rope, cu_seqlens, start, page_table, pool, pairs: bool = False,
                        k_scale: float = 1.0, v_scale: float = 1.0, q_out=None, dev_err=None, stream=None):
    """``kda_kv4_append`` of k, v [T, H_kv, D] with the position rotation on the way: the first R channels of
    each head of q [T, H_q, D] and k turn by their token's row of ``rope`` (fp32 [positions, R]:
    ``make_rope_table``), as pairs (c, c + R / 2) or, with ``pairs``, (2 c, 2 c + 1).  q, k and v may be views
    of a fused projection's output.  Returns the rotated q; ``q_out`` takes it and may be q itself."""
    if _quick is not None and stream is None:
        done = _quick.append_rope(q, k, v, rope, cu_seqlens, start, page_table, pool, pairs, k_scale, v_scale, q_out, dev_err)
        if done is not None:
            return done
    shape, dev = _first(q, "q", 3)
    dtype = q.dtype
    dt = _kv_dt(dtype)
    T, Hq, D = shape
    pa, pages, H, page_size = _pool(pool, D, dev)
    kshape = (T, H, D)
    qa, qs = _rows(q, "q", dtype, shape, dev)
    ka, ks = _rows(k, "k", dtype, kshape, dev)
    va, vs = _rows(v, "v", dtype, kshape, dev)
    rshape, _ = _first(rope, "rope", 2)
    _sizes("rope", *rshape)
    ta, B, M = _table(page_table, dev)
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=q.device) if stream is None else _make(
            stream, shape, dtype, q.device)
        oa, os_ = q_out.data_ptr(), Hq * D
    else:
        oa, os_ = _rows(q_out, "q_out", dtype, shape, dev)
    status = lib().kda_kv4_append_rope(
        dt, B, T, Hq, H, D, rshape[1], 1 if pairs else 0, qa, qs, ka, ks, va, vs,
        _ptr(rope, "rope", rshape, F32, dev), rshape[0],
        _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev), _ptr(start, "start", (B,), I32, dev), ta, M,
        page_size, pa, pages, k_scale, v_scale, oa, os_, _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_kv4_append_rope", status)
    return q_out


def kv4_bounds_bytes(D: int = K_DIM) -> int:
    """Bytes of one page and head's record of bounds."""
    return 2 * int(D) + 16


def make_kv4_bounds(num_pages: int, H_kv: int, D: int = K_DIM, device="cuda"):
    """One layer's records of its pages' keys, int8 [num_pages, H_kv, 2 D + 16]."""
    return torch.zeros(num_pages, H_kv, kv4_bounds_bytes(D), dtype=torch.int8, device=device)


def kda_kv4_bounds(cu_seqlens, start, total_tokens: int, page_table, pool, bounds, dev_err=None, stream=None):
    """Bring the records of the pages up to date that hold positions start[b] .. of each request's new tokens
    (cu_seqlens int32 [B + 1]), after those were appended.  ``bounds``: ``make_kv4_bounds()``, in place."""
    if _quick is not None and stream is None and _quick.bounds(cu_seqlens, start, total_tokens, page_table, pool, bounds, dev_err):
        return
    shape, dev = _first(pool, "pool", 4)
    D = shape[3] // 18
    pa, pages, H, page_size = _pool(pool, D, dev)
    ta, B, M = _table(page_table, dev)
    status = lib().kda_kv4_bounds(
        B, _int(int(total_tokens)), H, D, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(start, "start", (B,), I32, dev), ta, M, page_size, pa, pages,
        _ptr(bounds, "bounds", (pages, H, 2 * D + 16), torch.int8, dev), _err_ptr(dev_err, dev),
        _stream_of(stream, dev))
    _check("kda_kv4_bounds", status)


def kv4_pick_workspace_bytes(total_tokens: int, H_kv: int, max_pages: int) -> int:
    return int(lib().kda_kv4_pick_workspace_bytes(_int(total_tokens), _int(H_kv), _int(max_pages)))


def kda_kv4_pick(q, cu_seqlens, max_q: int, kv_lens, page_table, bounds, page_size: int, count: int,
                 first: int = 1, recent: int = 1, picked=None, workspace=None, dev_err=None, stream=None):
    """The pages that each new token attends to, by kv head: ``count`` of those up to its own, the ``first`` and
    the ``recent`` ones (its own among them) and of the others those whose score is highest, or all of them where
    they are no more.  q [T, H_q, D], as it is attended with; cu_seqlens, max_q and kv_lens as in
    ``kda_kv4_attention``; ``bounds`` from ``kda_kv4_bounds``.  Returns int32 [T, H_kv, count]: numbers of pages in
    the request's row, ascending, then -1.  ``workspace``: uint8, ``kv4_pick_workspace_bytes(T, H_kv, max_pages)`` at
    least, kept by the caller (one for each stream); a call without one makes its own."""
    if _quick is not None and stream is None and picked is None and workspace is not None:
        done = _quick.pick(q, cu_seqlens, max_q, kv_lens, page_table, bounds, page_size, count, first, recent, workspace, dev_err)
        if done is not None:
            return done
    shape, dev = _first(q, "q", 3)
    dtype = q.dtype
    dt = _kv_dt(dtype)
    T, Hq, D = shape
    qa, qs = _rows(q, "q", dtype, shape, dev)
    (pages, H, _), _ = _first(bounds, "bounds", 3)
    ba = _ptr(bounds, "bounds", (pages, H, 2 * D + 16), torch.int8, dev)
    ta, B, M = _table(page_table, dev)
    if (max_q | page_size | count | first | recent) >> 31:
        max_q, page_size, count, first, recent = map(_int, (max_q, page_size, count, first, recent))
    if picked is None:
        picked = torch.empty((T, H, count), dtype=I32, device=q.device) if stream is None else _make(
            stream, (T, H, count), I32, q.device)
        oa = picked.data_ptr()
    else:
        oa = _ptr(picked, "picked", (T, H, count), I32, dev)
    if workspace is None:
        workspace = _make(stream, (kv4_pick_workspace_bytes(T, H, M),), _U8, q.device, result=False)
    (wb,), _ = _first(workspace, "workspace", 1)
    status = lib().kda_kv4_pick(
        dt, B, T, max_q, Hq, H, D, qa, qs, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(kv_lens, "kv_lens", (B,), I32, dev), ta, M, page_size, ba, pages, count, first, recent, oa,
        _ptr(workspace, "workspace", (wb,), _U8, dev), wb, _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_kv4_pick", status)
    return picked


def kda_kv4_attention_picked(q, cu_seqlens, max_q: int, kv_lens, page_table, picked, pool, scale=None,
                             k_scale: float = 1.0, v_scale: float = 1.0, o=None, lse=None, workspace=None,
                             dev_err=None, stream=None):
    """``kda_kv4_attention`` over the pages that ``picked`` (int32 [T, H_kv, count], of ``kda_kv4_pick``) names for
    each token and kv head.  Returns (o, lse)."""
    if _quick is not None and stream is None and o is None and lse is None and workspace is not None:
        done = _quick.attention_picked(q, cu_seqlens, max_q, kv_lens, page_table, picked, pool, scale, k_scale, v_scale, workspace,
                                       dev_err)
        if done is not None:
            return done
    shape, dev = _first(q, "q", 3)
    dtype = q.dtype
    dt = _kv_dt(dtype)
    T, H, D = shape
    qa, qs = _rows(q, "q", dtype, shape, dev)
    pa, pages, H_kv, page_size = _pool(pool, D, dev)
    ta, B, M = _table(page_table, dev)
    pshape, _ = _first(picked, "picked", 3)
    count = pshape[2]
    _sizes("picked", count)
    if o is None:
        o = torch.empty(shape, dtype=dtype, device=q.device) if stream is None else _make(stream, shape, dtype, q.device)
        oa = o.data_ptr()
    else:
        oa = _ptr(o, "o", shape, dtype, dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=F32, device=q.device) if stream is None else _make(stream, (T, H), F32, q.device)
        la = lse.data_ptr()
    else:
        la = _ptr(lse, "lse", (T, H), F32, dev)
    if workspace is None:
        workspace = _make(stream, (kv4_workspace_bytes(),), _U8, q.device, zero=True, result=False)
    (wb,), _ = _first(workspace, "workspace", 1)
    status = lib().kda_kv4_attention_picked(
        dt, B, T, _int(max_q), H, H_kv, D, qa, qs, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(kv_lens, "kv_lens", (B,), I32, dev), ta, M, page_size,
        _ptr(picked, "picked", (T, H_kv, count), I32, dev), count, pa, pages,
        D ** -0.5 if scale is None else scale, k_scale, v_scale, oa, la,
        _ptr(workspace, "workspace", (wb,), _U8, dev), wb, _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_kv4_attention_picked", status)
    return o, lse


def _page_state(refs, page_table, lens):
    """refs int32 [num_pages], page_table int32 [B, max_pages], lens int32 [B].  Returns their
    addresses, (B, max_pages, num_pages) and the device's number."""
    (N,), dev = _first(refs, "refs", 1)
    ta, B, M = _table(page_table, dev)
    return (_ptr(refs, "refs", (N,), I32, dev), ta,
            None if lens is None else _ptr(lens, "lens", (B,), I32, dev), B, M, N, dev)


def _page_pools(pools, num_pages, dev):
    """Layers' pools [num_pages, ...], dense, of one size and element width (their shapes do not matter).  Returns (the array of their addresses, its
    address, bytes of a page); the array has to outlive the call."""
    if len(pools) == 0:
        raise ValueError("pools must be a non-empty list")
    try:
        shape, sizes, widths = pools[0].shape, list(map(_numel, pools)), list(map(_width, pools))
        one = (sizes.count(sizes[0]) == widths.count(widths[0]) == len(pools) and
               len(shape) >= 2 and shape[0] == num_pages and
               set(map(_device_of, pools)) == {dev} and all(map(_dense, pools)))
    except (AttributeError, TypeError):
        one = False
    if not one:
        for n, q in enumerate(pools):
            _need(q, "pools[%d]" % n, device=torch.device("cuda", dev))
            p = pools[0]
            if p.dim() < 2 or p.shape[0] != num_pages or q.numel() != p.numel() or q.element_size() != p.element_size():
                raise ValueError("pools[%d]: every pool is [%d, ...] of one size and element width" % (
                    n, num_pages))
    ptrs = array.array("Q", map(_address, pools))
    p = pools[0]
    return ptrs, ptrs.buffer_info()[0], p.numel() // num_pages * p.element_size()


def kda_page_alloc(refs, page_table, lens, grow, page_size: int, dev_err=None, stream=None):
    """Row b grows by grow[b] tokens (int32 [B]): the pages that takes are the lowest free
    ones, rows in order; a negative grow takes tokens back and lets go of their pages.  refs int32 [num_pages] (holders of each page, 0: free),
    page_table int32 [B, max_pages], lens int32 [B]; all three change in place."""
    ra, ta, la, B, M, N, dev = _page_state(refs, page_table, lens)
    status = lib().kda_page_alloc(B, M, _int(page_size), N, ra, ta, la, _ptr(grow, "grow", (B,), I32, dev),
                                  _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_page_alloc", status)


def kda_page_fork(pools, refs, page_table, lens, src, dst, page_size: int, workspace=None,
                  dev_err=None, stream=None):
    """Copy-on-write: row dst[i] (empty, named once) also holds row src[i]'s full pages, and gets a
    copy of its partial last page in every pool of the list.  ``workspace``: int32, at
    least 2 n; a call without one makes its own."""
    ra, ta, la, B, M, N, dev = _page_state(refs, page_table, lens)
    keep, ptrs, page_bytes = _page_pools(pools, N, dev)
    (n,), _ = _first(src, "src", 1)
    if workspace is None:
        workspace = _make(stream, (2 * n,), I32, refs.device, result=False)
    (wn,), _ = _first(workspace, "workspace", 1)
    status = lib().kda_page_fork(
        len(pools), ptrs, page_bytes, B, M, _int(page_size), N, ra, ta, la, _ptr(src, "src", (n,), I32, dev),
        _ptr(dst, "dst", (n,), I32, dev), n, _ptr(workspace, "workspace", (wn,), I32, dev), wn,
        _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_page_fork", status)


def kda_page_free(refs, page_table, lens, rows, page_size: int, dev_err=None, stream=None):
    """Rows (int32 [n], distinct) let go of their pages; those nobody holds are free."""
    ra, ta, la, B, M, N, dev = _page_state(refs, page_table, lens)
    (n,), _ = _first(rows, "rows", 1)
    status = lib().kda_page_free(B, M, _int(page_size), N, ra, ta, la, _ptr(rows, "rows", (n,), I32, dev), n,
                                 _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_page_free", status)


def kda_page_compact(pools, refs, page_table, live=None, workspace=None, dev_err=None, stream=None):
    """Move the held pages above the number of held pages into the free ones below, in
    every pool; refs and page_table follow.  Returns live, int32 [1] on the device: the
    pages from there on are free.  ``workspace``: int32, at least 3 num_pages + 16."""
    ra, ta, _, B, M, N, dev = _page_state(refs, page_table, None)
    keep, ptrs, page_bytes = _page_pools(pools, N, dev)
    if live is None:
        live = _make(stream, (1,), I32, refs.device)
    if workspace is None:
        workspace = _make(stream, (3 * N + 16,), I32, refs.device, result=False)
    (wn,), _ = _first(workspace, "workspace", 1)
    status = lib().kda_page_compact(
        len(pools), ptrs, page_bytes, B, M, N, ra, ta, _ptr(live, "live", (1,), I32, dev),
        _ptr(workspace, "workspace", (wn,), I32, dev), wn, _err_ptr(dev_err, dev),
        _stream_of(stream, dev))
    _check("kda_page_compact", status)
    return live


def kda_page_copy(pools, src, dst, dev_err=None, stream=None):
    """Page dst[i] <- page src[i] in every pool of the list (int32 device index tensors)."""
    if len(pools) == 0:
        raise ValueError("pools must be a non-empty list")
    (n,), dev = _first(src, "src", 1)
    if not isinstance(pools[0], torch.Tensor) or pools[0].dim() < 1:
        raise ValueError("pools[0] needs a page axis")
    N = pools[0].shape[0]
    keep, ptrs, page_bytes = _page_pools(pools, N, dev)
    status = lib().kda_page_copy(
        len(pools), ptrs, page_bytes, N, _ptr(src, "src", (n,), I32, dev),
        _ptr(dst, "dst", (n,), I32, dev), n, _err_ptr(dev_err, dev), _stream_of(stream, dev))
    _check("kda_page_copy", status)


def kda_selftest_bounded_wait(dev_err, wait_us: int = 2000, stream=None):
    """One CTA waits, with the kernels' bounded-wait loop, on a barrier nothing
    arrives at; after wait_us it sets KDA_DEVERR_TIMEOUT in dev_err (a device
    int32 tensor) and returns."""
    _need(dev_err, "dev_err", dtype=I32)
    if dev_err.numel() < 1:
        raise ValueError("dev_err needs at least one element")
    _check("kda_selftest_bounded_wait", lib().kda_selftest_bounded_wait(_p(dev_err), int(wait_us),
                                                                       _stream(stream)))


def kda_selftest_prefill_wait(q, k, v, gk, beta, cu_seqlens, cu_seqlens_host, state_pool,
                              init_slot, out_slot, dev_err, o=None, wait_us: int = 1000,
                              stream=None):
    """The bf16 chunked prefill with the first chunk's q, k, gk never requested:
    every unit's first wait gives up after wait_us, sets KDA_DEVERR_TIMEOUT in
    dev_err and the unit writes no slot.  Arguments as ``kda_chunk_prefill``
    (bf16 only).  Returns o (not written by the abandoned units)."""
    _need(q, "q", (None, None, None), dtype=torch.bfloat16)
    T = q.shape[0]
    dt, dev, H, K, V = _need_inputs(q, k, v, gk, beta, (T,))
    host = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    N = host.numel() - 1
    _need_prefill_common(cu_seqlens, N, state_pool, H, K, V, init_slot, out_slot, None, dev_err,
                         dev)
    if dev_err is None:
        raise ValueError("dev_err is required")
    if o is None:
        o = _make(stream, (T, H, V), q.dtype, q.device)
    _need(o, "o", (T, H, V), dt, dev)
    hp = host.numpy().ctypes.data_as(ctypes.c_void_p)
    _check("kda_selftest_prefill_wait", lib().kda_selftest_prefill_wait(
        N, T, H, _p(q), _p(k), _p(v), _p(gk), _p(beta), _p(cu_seqlens), hp, _p(state_pool),
        state_pool.shape[0], _p(init_slot), _p(out_slot), _p(o), _p(dev_err), int(wait_us),
        _stream(stream)))
    return o


def kda_selftest_kv4_wait(q, cu_seqlens, max_q: int, kv_lens, page_table, pool, workspace, dev_err, o=None,
                          wait_us: int = 1000, stream=None):
    """The cache attention with first codes that never arrive: its waits give up after wait_us and set
    KDA_DEVERR_TIMEOUT in dev_err.  Arguments as ``kda_kv4_attention``; zero the workspace
    afterwards.  Returns o (not valid)."""
    shape, dev = _first(q, "q", 3)
    dt = _kv_dt(q.dtype)
    T, H, D = shape
    qa, qs = _rows(q, "q", q.dtype, shape, dev)
    pa, pages, H_kv, page_size = _pool(pool, D, dev)
    ta, B, M = _table(page_table, dev)
    if dev_err is None:
        raise ValueError("dev_err is required")
    if o is None:
        o = _make(stream, shape, q.dtype, q.device)
    (wb,), _ = _first(workspace, "workspace", 1)
    _check("kda_selftest_kv4_wait", lib().kda_selftest_kv4_wait(
        dt, B, T, _int(max_q), H, H_kv, D, qa, qs, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(kv_lens, "kv_lens", (B,), I32, dev), ta, M, page_size, pa, pages, _ptr(o, "o", shape, q.dtype, dev),
        _ptr(workspace, "workspace", (wb,), _U8, dev), wb, _err_ptr(dev_err, dev), int(wait_us),
        _stream_of(stream, dev)))
    return o


def kda_selftest_kv4_pick_wait(q, cu_seqlens, kv_lens, page_table, bounds, page_size: int, count: int, workspace, dev_err,
                               wait_us: int = 1000, stream=None):
    """The picks of single tokens with first records that never all arrive: the scores' waits give up after wait_us
    and set KDA_DEVERR_TIMEOUT in dev_err.  Arguments as ``kda_kv4_pick``.  Returns the picks (not valid)."""
    shape, dev = _first(q, "q", 3)
    dt = _kv_dt(q.dtype)
    T, Hq, D = shape
    qa, qs = _rows(q, "q", q.dtype, shape, dev)
    (pages, H, _), _ = _first(bounds, "bounds", 3)
    ta, B, M = _table(page_table, dev)
    if dev_err is None:
        raise ValueError("dev_err is required")
    picked = _make(stream, (T, H, count), I32, q.device)
    (wb,), _ = _first(workspace, "workspace", 1)
    _check("kda_selftest_kv4_pick_wait", lib().kda_selftest_kv4_pick_wait(
        dt, B, T, 1, Hq, H, D, qa, qs, _ptr(cu_seqlens, "cu_seqlens", (B + 1,), I32, dev),
        _ptr(kv_lens, "kv_lens", (B,), I32, dev), ta, M, _int(page_size),
        _ptr(bounds, "bounds", (pages, H, 2 * D + 16), torch.int8, dev), pages, _int(count), 1, 1, picked.data_ptr(),
        _ptr(workspace, "workspace", (wb,), _U8, dev), wb, _err_ptr(dev_err, dev), int(wait_us), _stream_of(stream, dev)))
    return picked

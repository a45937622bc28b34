"""Packed LoRA fine-tuning for NVIDIA B200 (sm_100a): Python binding of the C ABI.

This module only marshals arguments into ``libplora.so`` (built from
``csrc/`` by ``packed_lora_fine_b200.build``); every step of the computation
runs in the library's CUDA kernels.  The functions keep the C names of
``include/plora.h``: ``plora_create``, ``plora_forward``, ``plora_backward``,
``plora_check``, ``plora_saved_bytes``, ``plora_debug_unpack_saved``,
``plora_destroy``.  Tensors are passed as device pointers (ints); PyTorch is
only a convenient owner of device memory and streams.

There is no fallback: if the library is missing, importing the binding
raises ``ImportError``.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import itertools
import os
from typing import Iterable, List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# PLORA_LIBRARY may name another build of the library (the PLORA_DEBUG build with device-side bounds
# checks, libplora_debug.so); a missing file still raises ImportError.
LIB_PATH = os.environ.get("PLORA_LIBRARY") or os.path.join(_HERE, "libplora.so")

PLORA_OK = 0
PLORA_ERR_INVALID_ARG = 1
PLORA_ERR_UNSUPPORTED = 2
PLORA_ERR_OOM = 3
PLORA_ERR_CUDA = 4
PLORA_ERR_TIMEOUT = 5
PLORA_ERR_BOUNDS = 6
PLORA_BF16 = 0
PLORA_FP32 = 1
PLORA_FLAG_SIMT = 1
PLORA_FLAG_UNFUSED = 2
PLORA_FLAG_BASE_PAIR = 4
PLORA_MAX_RANK = 256
PLORA_MAX_ADAPTERS = 4096
PLORA_MAX_OUT_BLOCKS = 8
PLORA_STATIC_SCRATCH_BYTES = 16 << 20
PLORA_ACT_NONE, PLORA_ACT_RELU, PLORA_ACT_GELU, PLORA_ACT_GELU_TANH, PLORA_ACT_SILU = range(5)
PLORA_MUON_SCALE_NONE, PLORA_MUON_SCALE_ROWS, PLORA_MUON_SCALE_RMS = range(3)
PLORA_MUON_MAX_STEPS = 16
ACTIVATIONS = {"none": PLORA_ACT_NONE, "relu": PLORA_ACT_RELU, "gelu": PLORA_ACT_GELU,
               "gelu_tanh": PLORA_ACT_GELU_TANH, "silu": PLORA_ACT_SILU}
MUON_SCALES = {"none": PLORA_MUON_SCALE_NONE, "rows": PLORA_MUON_SCALE_ROWS, "rms": PLORA_MUON_SCALE_RMS}
MUON_COEFFS = (3.4445, -4.7750, 2.0315)

EXPORTED = ("plora_create", "plora_destroy", "plora_saved_bytes", "plora_forward", "plora_backward",
            "plora_check", "plora_status_string", "plora_last_error", "plora_debug_unpack_saved",
            "plora_version", "plora_debug_schedule", "plora_profile_enable", "plora_profile_read",
            "plora_grad_B_static", "plora_adamw_step", "plora_debug_timeout_probe", "plora_device_info",
            "plora_capture_reserve", "plora_capture_release", "plora_partition", "plora_debug_build",
            "plora_layer_create", "plora_layer_destroy", "plora_layer_handle", "plora_layer_saved_bytes",
            "plora_layer_forward", "plora_layer_backward", "plora_layer_check", "plora_layer_last_error",
            "plora_epilogue_saved_bytes", "plora_epilogue_work_bytes", "plora_forward_epilogue", "plora_backward_epilogue",
            "plora_muon_work_bytes", "plora_muon_step")


class plora_config(ctypes.Structure):
    _fields_ = [("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("max_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("max_tokens", ctypes.c_int64), ("n_out_blocks", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("out_block_end", ctypes.c_int64 * PLORA_MAX_OUT_BLOCKS)]


def make_config(d_in, d_out, dtype, max_adapters, max_rank, max_tokens, flags=0, out_blocks=None):
    """plora_config; out_blocks: the output widths of P >= 2 shared-input projections stacked in W
    (their sum is d_out), or None for one projection."""
    cfg = plora_config(d_in, d_out, dtype, max_adapters, max_rank, flags, max_tokens)
    if out_blocks is not None and len(out_blocks) > 1:
        cfg.n_out_blocks = len(out_blocks)
        end = 0
        for b, w in enumerate(out_blocks):
            end += int(w)
            cfg.out_block_end[b] = end
    return cfg


class plora_adapter(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("scale", ctypes.c_float), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("dA", ctypes.c_void_p), ("dB", ctypes.c_void_p)]


class plora_adamw_state(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int32),
                ("A_master", ctypes.c_void_p), ("B_master", ctypes.c_void_p), ("mA", ctypes.c_void_p),
                ("vA", ctypes.c_void_p), ("mB", ctypes.c_void_p), ("vB", ctypes.c_void_p)]


class plora_epilogue(ctypes.Structure):
    _fields_ = [("activation", ctypes.c_int32), ("inference", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("dbias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("Z", ctypes.c_void_p),
                ("work", ctypes.c_void_p)]


class plora_muon_state(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("eps", ctypes.c_float), ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("ns_steps", ctypes.c_int32), ("nesterov", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("A_master", ctypes.c_void_p), ("B_master", ctypes.c_void_p),
                ("mA", ctypes.c_void_p), ("mB", ctypes.c_void_p)]


class PloraError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{status_string(status)}: {message}")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libplora.so (raises ImportError if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libplora.so not built at {path}; run packed_lora_fine_b200.build.build()")
    lib = ctypes.CDLL(path)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    H = ctypes.c_void_p
    lib.plora_create.argtypes = [ctypes.POINTER(H), ctypes.POINTER(plora_config)]
    lib.plora_destroy.argtypes = [H]
    lib.plora_saved_bytes.argtypes = [H, I32, P, P, ctypes.POINTER(ctypes.c_size_t)]
    lib.plora_forward.argtypes = [H, P, P, P, I32, P, P, P, P]
    lib.plora_backward.argtypes = [H, P, P, P, P, I32, P, P, P, P]
    lib.plora_check.argtypes = [H, P]
    lib.plora_status_string.argtypes = [ctypes.c_int]
    lib.plora_status_string.restype = ctypes.c_char_p
    lib.plora_last_error.argtypes = [H]
    lib.plora_last_error.restype = ctypes.c_char_p
    lib.plora_debug_unpack_saved.argtypes = [H, I32, P, P, P, I32, P, P]
    lib.plora_debug_schedule.argtypes = [ctypes.POINTER(plora_config), I32, P, P, I32, I32, P, I64,
                                         ctypes.POINTER(ctypes.c_int64)]
    lib.plora_debug_schedule.restype = ctypes.c_int
    lib.plora_profile_enable.argtypes = [H, I32]
    lib.plora_profile_enable.restype = ctypes.c_int
    lib.plora_profile_read.argtypes = [H, I32, ctypes.POINTER(I32), P, P, P]
    lib.plora_profile_read.restype = ctypes.c_int
    lib.plora_capture_reserve.argtypes = [H, I32]
    lib.plora_capture_reserve.restype = ctypes.c_int
    lib.plora_capture_release.argtypes = [H]
    lib.plora_capture_release.restype = ctypes.c_int
    lib.plora_device_info.argtypes = [H, P, I32, ctypes.POINTER(I32)]
    lib.plora_device_info.restype = ctypes.c_int
    lib.plora_debug_timeout_probe.argtypes = [H, I64, P]
    lib.plora_debug_timeout_probe.restype = ctypes.c_int
    lib.plora_adamw_step.argtypes = [H, I32, P, P, P]
    lib.plora_adamw_step.restype = ctypes.c_int
    lib.plora_epilogue_work_bytes.argtypes = [H, I32, P, P, ctypes.POINTER(ctypes.c_size_t)]
    lib.plora_epilogue_saved_bytes.argtypes = [H, I32, P, P, P, ctypes.POINTER(ctypes.c_size_t)]
    lib.plora_forward_epilogue.argtypes = [H, P, P, P, I32, P, P, P, P, P]
    lib.plora_backward_epilogue.argtypes = [H, P, P, P, P, I32, P, P, P, P, P]
    lib.plora_muon_work_bytes.argtypes = [H, I32, P, ctypes.POINTER(ctypes.c_size_t)]
    lib.plora_muon_step.argtypes = [H, I32, P, P, P, P]
    for fn in ("plora_epilogue_work_bytes", "plora_epilogue_saved_bytes", "plora_forward_epilogue", "plora_backward_epilogue",
               "plora_muon_work_bytes", "plora_muon_step"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.plora_grad_B_static.argtypes = [ctypes.POINTER(plora_config), P, I32, P, P, P, P]
    lib.plora_grad_B_static.restype = ctypes.c_int
    lib.plora_version.argtypes = []
    lib.plora_version.restype = ctypes.c_int32
    lib.plora_debug_build.argtypes = []
    lib.plora_debug_build.restype = ctypes.c_int32
    lib.plora_layer_create.argtypes = [ctypes.POINTER(H), I32, P]
    lib.plora_layer_destroy.argtypes = [H]
    lib.plora_layer_handle.argtypes = [H, I32, ctypes.POINTER(H)]
    lib.plora_layer_saved_bytes.argtypes = [H, I32, P, P, P]
    lib.plora_layer_forward.argtypes = [H, I32, P, P, P]
    lib.plora_layer_backward.argtypes = [H, I32, P, P, P]
    lib.plora_layer_check.argtypes = [H, P]
    lib.plora_layer_last_error.argtypes = [H]
    lib.plora_layer_last_error.restype = ctypes.c_char_p
    for fn in ("plora_layer_create", "plora_layer_destroy", "plora_layer_handle", "plora_layer_saved_bytes",
               "plora_layer_forward", "plora_layer_backward", "plora_layer_check"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.plora_partition.argtypes = [I32, P, P, I64, I64, ctypes.c_double, ctypes.c_double, I32, P, P]
    lib.plora_partition.restype = ctypes.c_int
    for fn in ("plora_create", "plora_destroy", "plora_saved_bytes", "plora_forward", "plora_backward",
               "plora_check", "plora_debug_unpack_saved"):
        getattr(lib, fn).restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(s: int) -> str:
    return load().plora_status_string(int(s)).decode()


def _raise(h, s: int):
    if s != PLORA_OK:
        msg = load().plora_last_error(h).decode() if h else ""
        raise PloraError(s, msg)


def _offsets(off) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(off, dtype=np.int64))


def make_table(ranks: Sequence[int], scales: Sequence[float], A: Sequence[int], B: Sequence[int],
               dA: Optional[Sequence[int]] = None, dB: Optional[Sequence[int]] = None):
    """Build a host plora_adapter[] from ranks, scales and device pointers (ints)."""
    n = len(ranks)
    return (plora_adapter * max(1, n))(*[
        (int(ranks[i]), float(scales[i]), int(A[i]), int(B[i]), None if dA is None else int(dA[i]),
         None if dB is None else int(dB[i])) for i in range(n)])


# ---------------------------------------------------------------- C names
def plora_create(d_in: int, d_out: int, dtype: int, max_adapters: int, max_rank: int, max_tokens: int,
                 flags: int = 0, out_blocks=None) -> int:
    lib = load()
    cfg = make_config(d_in, d_out, dtype, max_adapters, max_rank, max_tokens, flags, out_blocks)
    h = ctypes.c_void_p()
    s = lib.plora_create(ctypes.byref(h), ctypes.byref(cfg))
    if s != PLORA_OK:
        raise PloraError(s, "plora_create")
    return h.value


def plora_create_status(cfg: plora_config):
    """Raw form: returns (status, handle-or-None)."""
    h = ctypes.c_void_p()
    s = load().plora_create(ctypes.byref(h), ctypes.byref(cfg))
    return s, h.value


def plora_destroy(h: int) -> None:
    _raise(None, load().plora_destroy(h))


def plora_saved_bytes(h: int, n: int, off, tab) -> int:
    off = _offsets(off)
    out = ctypes.c_size_t(0)
    _raise(h, load().plora_saved_bytes(h, n, off.ctypes.data, ctypes.addressof(tab), ctypes.byref(out)))
    return int(out.value)


def plora_forward(h: int, X: int, W: int, Y: int, n: int, off, tab, saved: int, stream: int = 0,
                  check: bool = True) -> int:
    off = _offsets(off)
    s = load().plora_forward(h, X, W, Y, n, off.ctypes.data, ctypes.addressof(tab), saved, stream)
    if check:
        _raise(h, s)
    return s


def plora_backward(h: int, X: int, W: int, dY: int, dX: Optional[int], n: int, off, tab, saved: int,
                   stream: int = 0, check: bool = True) -> int:
    off = _offsets(off)
    s = load().plora_backward(h, X, W, dY, dX or None, n, off.ctypes.data, ctypes.addressof(tab), saved, stream)
    if check:
        _raise(h, s)
    return s


def plora_check(h: int, stream: int = 0) -> int:
    return load().plora_check(h, stream)


def plora_last_error(h: int) -> str:
    return load().plora_last_error(h).decode()


def plora_debug_unpack_saved(h: int, n: int, off, tab, saved: int, i: int, H_out: int, stream: int = 0) -> None:
    off = _offsets(off)
    _raise(h, load().plora_debug_unpack_saved(h, n, off.ctypes.data, ctypes.addressof(tab), saved, i, H_out,
                                              stream))


def plora_debug_schedule(cfg: plora_config, n: int, off, tab, grads: bool, which: int):
    """Returns (status, int32 numpy array) of the host schedule; see include/plora.h."""
    lib = load()
    off = _offsets(off)
    cnt = ctypes.c_int64(0)
    tptr = ctypes.addressof(tab) if tab is not None else None
    s = lib.plora_debug_schedule(ctypes.byref(cfg), n, off.ctypes.data, tptr, int(grads), which, None, 0,
                                 ctypes.byref(cnt))
    if s != PLORA_OK:
        return s, None
    buf = np.zeros(max(1, cnt.value), dtype=np.int32)
    s = lib.plora_debug_schedule(ctypes.byref(cfg), n, off.ctypes.data, tptr, int(grads), which,
                                 buf.ctypes.data, cnt.value, ctypes.byref(cnt))
    return s, buf[:cnt.value]


def plora_profile_enable(h: int, enable: bool) -> None:
    _raise(h, load().plora_profile_enable(h, int(bool(enable))))


def plora_profile_read(h: int) -> dict:
    """{kernel kind: (launches, total device ms)} since the last read."""
    lib = load()
    cap = 32
    n = ctypes.c_int32(0)
    names = (ctypes.c_char_p * cap)()
    launches = (ctypes.c_int64 * cap)()
    ms = (ctypes.c_double * cap)()
    _raise(h, lib.plora_profile_read(h, cap, ctypes.byref(n), names, launches, ms))
    return {names[k].decode(): (int(launches[k]), float(ms[k])) for k in range(min(n.value, cap))}


def plora_capture_reserve(h: int, n: int) -> None:
    """Reserve n schedule slots for calls captured into CUDA graphs (one per captured call)."""
    _raise(h, load().plora_capture_reserve(h, int(n)))


def plora_capture_release(h: int) -> None:
    """Free the capture slots (only once no graph holding this handle's captured calls replays)."""
    _raise(h, load().plora_capture_release(h))


def plora_device_info(h: int) -> dict:
    """SMs of the handle's device, the co-resident 2-SM clusters of the pair base GEMMs, and this
    build's single-SM base-GEMM tile rows and rasterisation windows."""
    out = (ctypes.c_int32 * 6)()
    cnt = ctypes.c_int32(0)
    _raise(h, load().plora_device_info(h, ctypes.cast(out, ctypes.c_void_p), 6, ctypes.byref(cnt)))
    return {"sms": int(out[0]), "pairs_fwd": int(out[1]), "pairs_dx": int(out[2]), "base_rows": int(out[3]),
            "window_rows": int(out[4]), "dx_window_rows": int(out[5])}


# Nominal B200 peaks for the partition cost model (dense bf16 tensor FLOP/s, HBM bytes/s); only their
# ratio matters for the balance.
PARTITION_FLOPS = 2.25e15
PARTITION_BYTES = 8.0e12


def plora_partition(counts, ranks, d_in: int, d_out: int, n_parts: int, flops_per_s: float = PARTITION_FLOPS,
                    bytes_per_s: float = PARTITION_BYTES):
    """Assign each adapter to one of n_parts GPUs (longest processing time first over the per-adapter
    cost of include/plora.h).  Returns (owner int32[n], part_cost float64[n_parts]); raises PloraError."""
    counts = np.ascontiguousarray(counts, dtype=np.int64)
    ranks = np.ascontiguousarray(ranks, dtype=np.int32)
    n = len(counts)
    owner = np.full(n, -1, np.int32)
    cost = np.zeros(max(1, int(n_parts)), np.float64)
    st = load().plora_partition(n, counts.ctypes.data, ranks.ctypes.data, int(d_in), int(d_out), float(flops_per_s),
                                float(bytes_per_s), int(n_parts), owner.ctypes.data, cost.ctypes.data)
    if st != PLORA_OK:
        raise PloraError(st, "plora_partition")
    return owner, cost[:n_parts]


def shard(owner, off, part: int):
    """Part `part`'s share of a packed adapter set: (adapter ids in increasing order, their local
    offsets int64[k+1] into the part's own packed token buffer, and the global row ranges
    [(off[i], off[i+1])] to gather that buffer from).  Index bookkeeping only."""
    owner = np.asarray(owner)
    off = np.asarray(off, dtype=np.int64)
    ids = np.nonzero(owner == part)[0].astype(np.int64)
    counts = off[ids + 1] - off[ids]
    local = np.zeros(len(ids) + 1, np.int64)
    local[1:] = np.cumsum(counts)
    return ids, local, [(int(off[i]), int(off[i + 1])) for i in ids]


def plora_grad_B_static(cfg: plora_config, dY: int, n: int, off, tab, saved: int, stream: int = 0) -> int:
    """dB of every adapter without allocating (scratch in a static device array). Returns the status."""
    off = _offsets(off)
    return int(load().plora_grad_B_static(ctypes.byref(cfg), dY, n, off.ctypes.data, ctypes.addressof(tab),
                                          saved, stream))


def make_adamw_states(hparams, A_master, B_master, mA, vA, mB, vB):
    """Host plora_adamw_state[] from per-adapter dicts (lr, beta1, beta2, eps, weight_decay, step) and device
    pointers (ints; A_master / B_master may be None for an fp32 handle)."""
    n = len(hparams)
    st = (plora_adamw_state * max(1, n))()
    for i, hp in enumerate(hparams):
        st[i].lr = float(hp["lr"])
        st[i].beta1 = float(hp.get("beta1", 0.9))
        st[i].beta2 = float(hp.get("beta2", 0.999))
        st[i].eps = float(hp.get("eps", 1e-8))
        st[i].weight_decay = float(hp.get("weight_decay", 0.01))
        st[i].step = int(hp["step"])
        st[i].A_master = A_master[i] if A_master is not None else None
        st[i].B_master = B_master[i] if B_master is not None else None
        st[i].mA, st[i].vA, st[i].mB, st[i].vB = mA[i], vA[i], mB[i], vB[i]
    return st


def plora_adamw_step(h: int, n: int, tab, states, stream: int = 0, check: bool = True) -> int:
    s = load().plora_adamw_step(h, n, ctypes.addressof(tab), ctypes.addressof(states), stream)
    if check:
        _raise(h, s)
    return s


def make_muon_states(hparams, A_master, B_master, mA, mB):
    """Host plora_muon_state[] from per-adapter dicts (lr; momentum 0.95, nesterov True, weight_decay 0,
    eps 1e-7, ns_steps 5, coeffs MUON_COEFFS, scale "rows": "none", "rows" or "rms") and device pointers
    (ints; A_master / B_master None for an fp32 handle)."""
    st = (plora_muon_state * max(1, len(hparams)))()
    for i, hp in enumerate(hparams):
        st[i].lr = float(hp["lr"])
        st[i].momentum = float(hp.get("momentum", 0.95))
        st[i].weight_decay = float(hp.get("weight_decay", 0.0))
        st[i].eps = float(hp.get("eps", 1e-7))
        st[i].a, st[i].b, st[i].c = (float(x) for x in hp.get("coeffs", MUON_COEFFS))
        st[i].ns_steps = int(hp.get("ns_steps", 5))
        st[i].nesterov = int(bool(hp.get("nesterov", True)))
        st[i].scale = MUON_SCALES[hp.get("scale", "rows")]
        st[i].A_master = A_master[i] if A_master is not None else None
        st[i].B_master = B_master[i] if B_master is not None else None
        st[i].mA, st[i].mB = mA[i], mB[i]
    return st


def plora_muon_work_bytes(h: int, n: int, tab) -> int:
    out = ctypes.c_size_t(0)
    _raise(h, load().plora_muon_work_bytes(h, n, ctypes.addressof(tab), ctypes.byref(out)))
    return int(out.value)


def plora_muon_step(h: int, n: int, tab, states, work: int, stream: int = 0, check: bool = True) -> int:
    s = load().plora_muon_step(h, n, ctypes.addressof(tab), ctypes.addressof(states), work or None, stream)
    if check:
        _raise(h, s)
    return s


def make_epilogue(activation="none", bias=None, dbias=None, residual=None, Z=None, work=None,
                  inference=False) -> plora_epilogue:
    """plora_epilogue from an activation's name (or number) and device pointers (ints); bias and dbias are
    lists with one pointer (or None) per adapter, or None."""
    ep = plora_epilogue()
    if isinstance(activation, str) and activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    ep.activation = ACTIVATIONS[activation] if isinstance(activation, str) else int(activation)
    keep = []
    for name, ptrs in (("bias", bias), ("dbias", dbias)):
        if ptrs is not None:
            arr = (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)
            keep.append(arr)
            setattr(ep, name, ctypes.addressof(arr))
    ep.residual, ep.Z, ep.work = residual or None, Z or None, work or None
    ep.inference = int(inference)
    ep._keep = keep
    return ep


def plora_epilogue_work_bytes(h: int, n: int, off, ep: plora_epilogue) -> int:
    off = _offsets(off)
    out = ctypes.c_size_t(0)
    _raise(h, load().plora_epilogue_work_bytes(h, n, off.ctypes.data, ctypes.addressof(ep), ctypes.byref(out)))
    return int(out.value)


def plora_epilogue_saved_bytes(h: int, n: int, off, tab, ep: plora_epilogue) -> int:
    off = _offsets(off)
    out = ctypes.c_size_t(0)
    _raise(h, load().plora_epilogue_saved_bytes(h, n, off.ctypes.data, ctypes.addressof(tab), ctypes.addressof(ep),
                                                ctypes.byref(out)))
    return int(out.value)


def plora_forward_epilogue(h: int, X: int, W: int, Y: int, n: int, off, tab, saved: int, ep: plora_epilogue,
                           stream: int = 0, check: bool = True) -> int:
    off = _offsets(off)
    s = load().plora_forward_epilogue(h, X, W, Y, n, off.ctypes.data, ctypes.addressof(tab), saved,
                                      ctypes.addressof(ep), stream)
    if check:
        _raise(h, s)
    return s


def plora_backward_epilogue(h: int, X: int, W: int, dY: int, dX: Optional[int], n: int, off, tab, saved: int,
                            ep: plora_epilogue, stream: int = 0, check: bool = True) -> int:
    off = _offsets(off)
    s = load().plora_backward_epilogue(h, X, W, dY, dX or None, n, off.ctypes.data, ctypes.addressof(tab), saved,
                                       ctypes.addressof(ep), stream)
    if check:
        _raise(h, s)
    return s


def plora_debug_timeout_probe(h: int, timeout_ns: int, stream: int = 0) -> int:
    return int(load().plora_debug_timeout_probe(h, int(timeout_ns), stream))


def plora_version() -> int:
    return int(load().plora_version())


# ---------------------------------------------------------------- torch convenience
class PackedLoRA:
    """Owns a handle; runs the packed forward/backward on torch CUDA tensors.

    ``A[i]`` is ``[r_i][d_in]`` (lora_A.weight), ``B[i]`` is ``[d_out][r_i]``
    (lora_B.weight), ``W`` is ``[d_out][d_in]`` (nn.Linear.weight), ``X`` is
    the packed ``[T][d_in]`` token buffer, ``off`` the host segment offsets.
    With ``out_blocks`` (the widths of P shared-input projections stacked in W, e.g.
    q, k, v), ``A[i]`` is the P projections' lora_A weights stacked, ``[P r_i][d_in]``,
    and ``B[i]`` their lora_B weights stacked, ``[d_out][r_i]``.
    """

    def __init__(self, d_in, d_out, dtype="bf16", max_adapters=64, max_rank=PLORA_MAX_RANK,
                 max_tokens=1 << 16, simt=False, unfused=False, base_pair=False, out_blocks=None):
        self.d_in, self.d_out = int(d_in), int(d_out)
        self.dtype = dtype
        self.out_blocks = list(out_blocks) if out_blocks is not None else None
        self.h = plora_create(self.d_in, self.d_out, PLORA_BF16 if dtype == "bf16" else PLORA_FP32,
                              max_adapters, max_rank, max_tokens,
                              (PLORA_FLAG_SIMT if simt else 0) | (PLORA_FLAG_UNFUSED if unfused else 0)
                              | (PLORA_FLAG_BASE_PAIR if base_pair else 0), out_blocks)
        import torch
        self.device = torch.device("cuda", torch.cuda.current_device())    # where plora_create put the handle

    def close(self):
        if self.h:
            plora_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def table(self, scales, A, B, dA=None, dB=None):
        ranks = [b.shape[1] for b in B]
        return make_table(ranks, scales, [a.data_ptr() for a in A], [b.data_ptr() for b in B],
                          None if dA is None else [x.data_ptr() for x in dA],
                          None if dB is None else [x.data_ptr() for x in dB])

    def saved_bytes(self, off, tab) -> int:
        return plora_saved_bytes(self.h, len(off) - 1, off, tab)

    def forward(self, X, W, off, scales, A, B, Y=None, saved=None, stream=None):
        import torch
        n = len(off) - 1
        tab = self.table(scales, A, B)
        if Y is None:
            Y = torch.empty((X.shape[0], self.d_out), dtype=X.dtype, device=X.device)
        nbytes = self.saved_bytes(off, tab)
        if saved is None:
            saved = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=X.device)
        st = (stream or torch.cuda.current_stream()).cuda_stream
        plora_forward(self.h, X.data_ptr(), W.data_ptr(), Y.data_ptr(), n, off, tab, saved.data_ptr(), st)
        return Y, saved

    def backward(self, X, W, dY, off, scales, A, B, saved, dX=None, dA=None, dB=None, want_dX=True, stream=None):
        import torch
        n = len(off) - 1
        if dA is None:
            dA = [torch.empty(a.shape, dtype=torch.float32, device=X.device) for a in A]
        if dB is None:
            dB = [torch.empty(b.shape, dtype=torch.float32, device=X.device) for b in B]
        if want_dX and dX is None:
            dX = torch.empty_like(X)
        tab = self.table(scales, A, B, dA, dB)
        st = (stream or torch.cuda.current_stream()).cuda_stream
        plora_backward(self.h, X.data_ptr(), W.data_ptr(), dY.data_ptr(), dX.data_ptr() if want_dX else None,
                       n, off, tab, saved.data_ptr(), st)
        return dX, dA, dB

    def _check_tensors(self, T, **named):
        """Shapes, dtype and layout of the tensors an epilogue call takes by pointer."""
        import torch
        dt = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        shape = {"X": (T, self.d_in), "W": (self.d_out, self.d_in), "bias": (self.d_out,)}
        for name, t in named.items():
            if t is None:
                continue
            want = shape.get(name, (T, self.d_out))
            if t.shape != want or t.dtype != dt or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"{name}: a contiguous {dt} tensor of shape {want} on {self.device} is needed, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")

    @staticmethod
    def _tokens(X, off) -> int:
        """off[-1], the rows of X that belong to an adapter; ValueError where X has fewer."""
        T = int(off[-1])
        if T > X.shape[0]:
            raise ValueError(f"off: the last adapter ends at row {T}, X has {X.shape[0]}")
        return T

    @staticmethod
    def _launch_stream(stream, device):
        """The stream of a call, and the same if it is not the current one, else None.  A call's new tensors come from the
        current stream's memory, where work on what was there before may not have ended: another stream waits for it
        (not while either is captured: a capture holds the memory that it needs, and waits for nothing outside)."""
        import torch
        current = torch.cuda.current_stream(device)
        if stream is None or stream == current:
            return current, None
        captured = torch.cuda.is_current_stream_capturing()
        with torch.cuda.stream(stream):
            if captured or torch.cuda.is_current_stream_capturing():
                return stream, None
        stream.wait_stream(current)
        return stream, stream

    def _check_factors(self, A, B, n):
        import torch
        dt = torch.bfloat16 if self.dtype == "bf16" else torch.float32
        P = len(self.out_blocks) if self.out_blocks else 1
        if len(A) != n or len(B) != n:
            raise ValueError(f"{len(A)} A and {len(B)} B factors for {n} adapters")
        for i, (a, b) in enumerate(zip(A, B)):
            r = b.shape[1]
            if a.shape != (P * r, self.d_in) or b.shape != (self.d_out, r) or a.dtype != dt \
                    or b.dtype != dt or not a.is_contiguous() or not b.is_contiguous() \
                    or a.device != self.device or b.device != self.device:
                raise ValueError(f"adapter {i}: contiguous {dt} factors A {(P * r, self.d_in)} and B "
                                 f"{(self.d_out, r)} on {self.device} are needed, got {tuple(a.shape)} on {a.device} and "
                                 f"{tuple(b.shape)} on {b.device}")

    def _bias_list(self, bias, n):
        """One bias (or None) per adapter from None, one tensor for every adapter, or a list."""
        if bias is None:
            return None
        out = list(bias) if isinstance(bias, (list, tuple)) else [bias] * n
        if len(out) != n:
            raise ValueError(f"bias: {len(out)} entries for {n} adapters")
        for b in out if isinstance(bias, (list, tuple)) else [bias]:
            self._check_tensors(0, bias=b)
        return out

    def forward_epilogue(self, X, W, off, scales, A, B, bias=None, activation="none", residual=None, want_Z=True,
                         Y=None, saved=None, stream=None):
        """Y = act(X W + s (X A) B + bias) + residual; returns (Y, saved, Z).

        bias: one ``[d_out]`` tensor for every adapter, a list with one (or None) per adapter, or None;
        activation: a name in ``ACTIVATIONS``; residual: ``[T][d_out]`` (with a bf16 engine it may be the tensor
        given as Y).
        Z is the pre-activation that ``backward_epilogue`` needs with an activation (None without one).
        X may have rows behind off[-1]: a Y that is given keeps what it has there, a new one (and Z) is zero there.
        stream: a torch stream to launch on, behind the current one's work so far (None: the current one).
        want_Z false: an inference call, which keeps nothing for a backward.  saved and Z are then None, and up to 32
        tokens of a bf16 engine go through kernels for few tokens (sums in another order than a training call's); above,
        Y is a training call's, but for relu on a bf16 engine, whose training call does not round X A to bf16."""
        import torch
        n = len(off) - 1
        T = self._tokens(X, off)
        self._check_tensors(X.shape[0], X=X, W=W, residual=residual, Y=Y)
        bias = self._bias_list(bias, n)
        self._check_factors(A, B, n)
        tab = self.table(scales, A, B)
        new = Y is None
        if new:
            Y = torch.empty((X.shape[0], self.d_out), dtype=X.dtype, device=X.device)
        Z = torch.empty_like(Y) if want_Z and activation != "none" else None
        ep = make_epilogue(activation, None if bias is None else [b.data_ptr() if b is not None else None for b in bias],
                           residual=residual.data_ptr() if residual is not None else None,
                           Z=Z.data_ptr() if Z is not None else None, inference=not want_Z)
        own = saved is None
        if own:
            saved = torch.empty(max(plora_epilogue_saved_bytes(self.h, n, off, tab, ep), 256), dtype=torch.uint8, device=X.device)
        st, other = self._launch_stream(stream, X.device)
        if T < X.shape[0]:
            with torch.cuda.stream(st):
                for t in (Y if new else None, Z):
                    if t is not None:
                        t[T:].zero_()
        plora_forward_epilogue(self.h, X.data_ptr(), W.data_ptr(), Y.data_ptr(), n, off, tab, saved.data_ptr(), ep, st.cuda_stream)
        if other is not None:      # (they may go back to the allocator while that stream uses them)
            for t in (Y if new else None, saved if own else None, Z):
                if t is not None:
                    t.record_stream(other)
        return Y, saved if want_Z else None, Z

    def backward_epilogue(self, X, W, dY, off, scales, A, B, saved, Z=None, activation="none", want_dX=True,
                          want_dbias=False, stream=None):
        """The backward of ``forward_epilogue``: returns (dX, dA, dB, dbias).  dX is None without want_dX;
        dbias is a list of fp32 ``[d_out]`` tensors, one per adapter, or None; want_dbias may be a list of
        truth values, one per adapter (dbias[i] is then None where it is false).  The residual's gradient
        is dY (in the rows of an adapter; dX is zero behind off[-1])."""
        import torch
        n = len(off) - 1
        self._tokens(X, off)
        self._check_tensors(X.shape[0], X=X, W=W, dY=dY, Z=Z)
        self._check_factors(A, B, n)
        f32 = dict(dtype=torch.float32, device=X.device)
        dA, dB = [torch.empty(a.shape, **f32) for a in A], [torch.empty(b.shape, **f32) for b in B]
        want = list(want_dbias) if isinstance(want_dbias, (list, tuple)) else [bool(want_dbias)] * n
        db = [torch.empty(self.d_out, **f32) if w else None for w in want] if any(want) else None
        dX = self._gradients(X, W, dY, off, scales, A, B, saved, Z, activation, want_dX, [g.data_ptr() for g in dA],
                             [g.data_ptr() for g in dB],
                             None if db is None else [b.data_ptr() if b is not None else None for b in db], stream)
        other = self._launch_stream(stream, X.device)[1]
        if other is not None:
            for t in [*dA, *dB, *(b for b in db or [] if b is not None)]:
                t.record_stream(other)
        return dX, dA, dB, db

    def _gradients(self, X, W, dY, off, scales, A, B, saved, Z, activation, want_dX, pA, pB, pb, stream=None):
        """backward_epilogue into the fp32 buffers at the device pointers pA, pB and pb; returns dX."""
        import torch
        n = len(off) - 1
        dX = torch.empty_like(X) if want_dX else None
        tab = make_table([b.shape[1] for b in B], scales, [a.data_ptr() for a in A], [b.data_ptr() for b in B], pA, pB)
        ep = make_epilogue(activation, dbias=pb, Z=Z.data_ptr() if Z is not None else None)
        nbytes = plora_epilogue_work_bytes(self.h, n, off, ep)
        work = torch.empty(nbytes, dtype=torch.uint8, device=X.device) if nbytes else None
        ep.work = work.data_ptr() if work is not None else None
        st, other = self._launch_stream(stream, X.device)
        if want_dX and self._tokens(X, off) < X.shape[0]:
            with torch.cuda.stream(st):
                dX[int(off[-1]):].zero_()
        plora_backward_epilogue(self.h, X.data_ptr(), W.data_ptr(), dY.data_ptr(), dX.data_ptr() if want_dX else None,
                                n, off, tab, saved.data_ptr(), ep, st.cuda_stream)
        if other is not None:
            for t in (dX, work):
                if t is not None:
                    t.record_stream(other)
        return dX


# ---------------------------------------------------------------- layer calls
class plora_proj(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("dY", ctypes.c_void_p),
                ("dX", ctypes.c_void_p), ("tab", ctypes.c_void_p), ("saved", ctypes.c_void_p)]


def make_projs(items) -> "ctypes.Array":
    """plora_proj[n] from dicts with keys X, W, Y, dY, dX (device pointers or None), tab (a table from
    make_table) and saved (device pointer or None)."""
    arr = (plora_proj * len(items))()
    keep = []
    for k, it in enumerate(items):
        tab = it.get("tab")
        keep.append(tab)
        arr[k] = plora_proj(it.get("X"), it.get("W"), it.get("Y"), it.get("dY"), it.get("dX"),
                            ctypes.addressof(tab) if tab is not None else None, it.get("saved"))
    arr._keep = keep
    return arr


class PackedLoRALayer:
    """A layer call: several projections over one segment map (the same adapters over the same packed
    token rows) run as one launch set, one persistent launch per product kind over all of them.

    ``projections`` lists each projection as ``(d_in, d_out)`` or ``(d_in, d_out, out_blocks)``.
    ``forward(io, off, scales)`` takes one dict per projection with its ``X``, ``W``, ``A``, ``B``
    torch tensors and returns ``[(Y, saved)]``; ``backward(io, off, scales, saved)`` takes the same
    dicts with ``dY`` added and returns ``[(dX, dA, dB)]``.  ``scales`` is one list of per-adapter
    scales for every projection, or one such list per projection (an adapter's alpha / r differs
    between projections where its rank does).  Results equal separate calls bit for bit.
    """

    def __init__(self, projections, max_adapters=64, max_rank=PLORA_MAX_RANK, max_tokens=1 << 16):
        self.proj = [tuple(p) for p in projections]
        cfgs = (plora_config * len(self.proj))()
        for k, p in enumerate(self.proj):
            cfgs[k] = make_config(p[0], p[1], PLORA_BF16, max_adapters, max_rank, max_tokens, 0,
                                  p[2] if len(p) > 2 else None)
        h = ctypes.c_void_p()
        st = load().plora_layer_create(ctypes.byref(h), len(self.proj), cfgs)
        if st != PLORA_OK:
            raise PloraError(st, "plora_layer_create")
        self.L = h.value

    def handle(self, p: int) -> int:
        h = ctypes.c_void_p()
        st = load().plora_layer_handle(self.L, p, ctypes.byref(h))
        if st != PLORA_OK:
            raise PloraError(st, "plora_layer_handle")
        return h.value

    def close(self):
        if self.L:
            load().plora_layer_destroy(self.L)
            self.L = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _err(self, st, what):
        if st != PLORA_OK:
            raise PloraError(st, f"{what}: {load().plora_layer_last_error(self.L).decode()}")

    @staticmethod
    def _scales(scales, k):
        """Projection k's per-adapter scales from one shared list or a list per projection."""
        first = scales[0] if len(scales) else None
        return scales[k] if isinstance(first, (list, tuple, np.ndarray)) else scales

    @staticmethod
    def _table(scales, A, B, dA=None, dB=None):
        return make_table([b.shape[1] for b in B], scales, [a.data_ptr() for a in A], [b.data_ptr() for b in B],
                          None if dA is None else [x.data_ptr() for x in dA],
                          None if dB is None else [x.data_ptr() for x in dB])

    def forward(self, io, off, scales, stream=None):
        import torch
        off = np.ascontiguousarray(off, dtype=np.int64)
        n = len(off) - 1
        items, outs = [], []
        for k, d in enumerate(io):
            tab = self._table(self._scales(scales, k), d["A"], d["B"])
            Y = torch.empty((d["X"].shape[0], self.proj[k][1]), dtype=d["X"].dtype, device=d["X"].device)
            items.append({"X": d["X"].data_ptr(), "W": d["W"].data_ptr(), "Y": Y.data_ptr(), "tab": tab})
            outs.append(Y)
        projs = make_projs(items)
        sizes = (ctypes.c_size_t * len(io))()
        self._err(load().plora_layer_saved_bytes(self.L, n, off.ctypes.data, projs, sizes), "plora_layer_saved_bytes")
        saved = [torch.empty(max(int(b), 256), dtype=torch.uint8, device=d["X"].device) for b, d in zip(sizes, io)]
        for k in range(len(io)):
            projs[k].saved = saved[k].data_ptr()
        st = (stream or torch.cuda.current_stream()).cuda_stream
        self._err(load().plora_layer_forward(self.L, n, off.ctypes.data, projs, st), "plora_layer_forward")
        return list(zip(outs, saved))

    def backward(self, io, off, scales, saved, want_dX=True, stream=None):
        import torch
        off = np.ascontiguousarray(off, dtype=np.int64)
        n = len(off) - 1
        items, outs = [], []
        for k, d in enumerate(io):
            dA = [torch.empty(a.shape, dtype=torch.float32, device=a.device) for a in d["A"]]
            dB = [torch.empty(b.shape, dtype=torch.float32, device=b.device) for b in d["B"]]
            dX = torch.empty_like(d["X"]) if want_dX else None
            tab = self._table(self._scales(scales, k), d["A"], d["B"], dA, dB)
            items.append({"X": d["X"].data_ptr(), "W": d["W"].data_ptr(), "dY": d["dY"].data_ptr(),
                          "dX": dX.data_ptr() if want_dX else None, "tab": tab, "saved": saved[k].data_ptr()})
            outs.append((dX, dA, dB))
        projs = make_projs(items)
        st = (stream or torch.cuda.current_stream()).cuda_stream
        self._err(load().plora_layer_backward(self.L, n, off.ctypes.data, projs, st), "plora_layer_backward")
        return outs

    def check(self, stream=None) -> int:
        return int(load().plora_layer_check(self.L, stream))


# ---------------------------------------------------------------- autograd
# What a packed_lora call holds besides its tensors; where[i] is adapter i's place among the distinct biases.
_Call = collections.namedtuple("_Call", "engine off scales n plain where activation")


@functools.lru_cache(maxsize=None)
def _packed_lora_fn():
    """packed_lora's autograd function (made once, on first use: the module does not import torch)."""
    import torch

    class PackedLoRAFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, call, X_, W_, R_, *ABb):
            n = call.n
            A_, B_, b_ = list(ABb[:n]), list(ABb[n:2 * n]), ABb[2 * n:]
            X_, W_, Z = X_.contiguous(), W_.contiguous(), None
            if call.plain:
                Y, saved = call.engine.forward(X_, W_, call.off, call.scales, A_, B_)
                if int(call.off[-1]) < Y.shape[0]:
                    Y[int(call.off[-1]):].zero_()
            else:
                Y, saved, Z = call.engine.forward_epilogue(X_, W_, call.off, call.scales, A_, B_,
                                                           bias=[None if k is None else b_[k] for k in call.where],
                                                           activation=call.activation,
                                                           residual=None if R_ is None else R_.contiguous())
            ctx.call = call
            ctx.save_for_backward(X_, W_, saved, Z, *ABb[:2 * n])
            return Y

        @staticmethod
        def backward(ctx, dY):
            call, n = ctx.call, ctx.call.n
            X_, W_, saved, Z, *AB = ctx.saved_tensors
            A_, B_ = list(AB[:n]), list(AB[n:])
            need_b = ctx.needs_input_grad[4 + 2 * n:]
            want_dX = ctx.needs_input_grad[1]
            gb = [None] * len(need_b)
            # The fp32 gradients lie in one buffer, so that one launch casts them (d_in and d_out are multiples of 8,
            # so that each starts on 32 bytes).
            owners = [i for i, k in enumerate(call.where) if k is not None and need_b[k]]
            counts = [t.numel() for t in AB] + [dY.shape[1]] * len(owners)
            flat = torch.empty(sum(counts), dtype=torch.float32, device=dY.device)
            ptrs = list(itertools.accumulate(counts, lambda at, c: at + 4 * c, initial=flat.data_ptr()))
            T = int(call.off[-1])
            dY = dY.contiguous()        # (kept until the launches are behind it: their arguments are pointers)
            if call.plain:
                dX = torch.empty_like(X_) if want_dX else None
                if want_dX and T < dX.shape[0]:
                    dX[T:].zero_()
                tab = make_table([b.shape[1] for b in B_], call.scales, [a.data_ptr() for a in A_], [b.data_ptr() for b in B_],
                                 ptrs[:n], ptrs[n:2 * n])
                plora_backward(call.engine.h, X_.data_ptr(), W_.data_ptr(), dY.data_ptr(),
                               dX.data_ptr() if want_dX else None, n, call.off, tab, saved.data_ptr(),
                               torch.cuda.current_stream().cuda_stream)
            else:
                pb = [None] * n
                for i, at in zip(owners, ptrs[2 * n:]):
                    pb[i] = at
                dX = call.engine._gradients(X_, W_, dY, call.off, call.scales, A_, B_, saved, Z, call.activation,
                                            want_dX, ptrs[:n], ptrs[n:2 * n], pb if owners else None)
            g = list((flat if flat.dtype == dY.dtype else flat.to(dY.dtype)).split(counts)) if counts else []
            for k, need in enumerate(need_b):       # a shared bias sums its adapters' fp32 gradients
                if need:
                    own = [2 * n + j for j, i in enumerate(owners) if call.where[i] == k]
                    gb[k] = g[own[0]] if len(own) == 1 else torch.stack([flat.split(counts)[j] for j in own]).sum(0).to(dY.dtype)
            g = [x.view(t.shape) for x, t in zip(g, AB)]
            dR = dY if ctx.needs_input_grad[3] else None
            if dR is not None and T < dR.shape[0]:
                dR = torch.cat([dR[:T], torch.zeros_like(dR[T:])])
            return (None, dX, None, dR, *g, *gb)

    return PackedLoRAFn


def packed_lora(engine: "PackedLoRA", X, W, off, scales, A, B, bias=None, activation="none", residual=None):
    """Y = act(X W + s_i (X_i A_i) B_i + b_i) + residual for every packed adapter, differentiable in X,
    A_i, B_i, b_i and residual (W is the frozen base weight and gets no gradient).  A[i] is lora_A.weight
    ([r_i][d_in]), B[i] is lora_B.weight ([d_out][r_i]), W is nn.Linear.weight ([d_out][d_in]); `off` holds
    the host segment offsets of the packed rows of X.  bias: None, one [d_out] tensor that every adapter
    shares (its gradient sums over the adapters) or a list with one (or None) per adapter; activation: a
    name in ACTIVATIONS; residual: [T][d_out].  Rows of X behind off[-1] belong to no adapter: Y is zero there, and so are
    the gradients of X and residual.  Without these three the backward runs plora_backward, else
    plora_backward_epilogue; the fp32 weight gradients are returned in each parameter's dtype.  The gradients of A, B and
    bias of one call are views of one buffer (one launch casts them all): each starts on 16 bytes, and one that is kept
    or saved keeps the buffer; clone it to have it alone."""
    n = len(off) - 1
    engine._tokens(X, off)
    plain = bias is None and activation == "none" and residual is None
    per_adapter = [None] * n if bias is None else engine._bias_list(bias, n)
    uniq = list({id(b): b for b in per_adapter if b is not None}.values())   # a shared bias is one input
    where = [next((k for k, u in enumerate(uniq) if u is b), None) for b in per_adapter]

    if W.requires_grad:
        raise ValueError("packed_lora: the base weight W is frozen; pass W with requires_grad=False")
    call = _Call(engine, off, scales, n, plain, where, activation)
    return _packed_lora_fn().apply(call, X, W, residual, *A, *B, *uniq)

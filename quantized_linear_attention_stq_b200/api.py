"""Python binding of the C ABI in include/stq.h (argument marshalling only).

Every computation runs in libstq.so on the GPU. This module checks tensor dtypes, shapes,
devices and contiguity, passes raw pointers and the current CUDA stream through ctypes, and turns
status codes into exceptions. There is no CPU fallback: if the library is missing the first call
raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
import warnings
from typing import Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libstq.so")

STQ_OK, STQ_ERR_INVALID_ARG, STQ_ERR_UNSUPPORTED, STQ_ERR_CUDA = 0, 1, 2, 3
STQ_ERR_NONFINITE, STQ_ERR_TIMEOUT, STQ_ERR_BOUNDS = 4, 5, 6
GATE_SCALAR, GATE_CHANNEL, GATE_CHANNEL_DECAY_FIRST = 0, 1, 2
SCALES_ROW_COLUMN, SCALES_UNIFORM = 0, 1  # stq_scale_mode
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}

# Every function the public header declares (checked against include/stq.h by the tests).
EXPORTS = (
    "stq_abi_version", "stq_status_string", "stq_layout_create", "stq_layout_destroy",
    "stq_layout_bytes_per_request", "stq_layout_head_offset", "stq_layout_head_bytes",
    "stq_layout_head_bits", "stq_init_state", "stq_decode_step", "stq_prefill_workspace_bytes",
    "stq_prefill_chunk", "stq_prefill_chunk_noalloc", "stq_dequantize", "stq_allocate_widths", "stq_row_impact",
    "stq_selftest_wait_timeout", "stq_decay_step", "stq_decay_prefill_workspace_bytes", "stq_decay_prefill",
    "stq_page_plan", "stq_page_write", "stq_paged_attention_workspace_bytes", "stq_paged_attention",
)


class StqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class _Desc(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("head_bits", ctypes.POINTER(ctypes.c_uint8)), ("gate", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("scale_mode", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
                ("scale_fit_rounds", ctypes.c_int32)]


_lock = threading.Lock()
_lib_handle = None


def lib() -> ctypes.CDLL:
    """Load libstq.so (raises if it has not been built)."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    with _lock:
        if _lib_handle is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: build it with "
                                  "`python -m quantized_linear_attention_stq_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            L.stq_abi_version.restype = i32
            L.stq_status_string.argtypes, L.stq_status_string.restype = [i32], ctypes.c_char_p
            L.stq_layout_create.argtypes = [ctypes.POINTER(_Desc), ctypes.POINTER(P)]
            L.stq_layout_create.restype = i32
            L.stq_layout_destroy.argtypes, L.stq_layout_destroy.restype = [P], None
            L.stq_layout_bytes_per_request.argtypes, L.stq_layout_bytes_per_request.restype = [P], sz
            for n in ("stq_layout_head_offset", "stq_layout_head_bytes"):
                getattr(L, n).argtypes, getattr(L, n).restype = [P, i32], sz
            L.stq_layout_head_bits.argtypes, L.stq_layout_head_bits.restype = [P, i32], i32
            L.stq_init_state.argtypes = [P, P, i32, P, i32, P, P, P, P]
            L.stq_init_state.restype = i32
            L.stq_decode_step.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P, P, P, P, P, P, P]
            L.stq_decode_step.restype = i32
            L.stq_prefill_workspace_bytes.argtypes = [P, i32, i32, i32]
            L.stq_prefill_workspace_bytes.restype = sz
            L.stq_prefill_chunk.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P, P, P, P, P, P, sz, P, P]
            L.stq_prefill_chunk.restype = i32
            L.stq_prefill_chunk_noalloc.argtypes = [P, P, i32, P, i32, i32, i32, P, P, P, P, P, P, P, P, P]
            L.stq_prefill_chunk_noalloc.restype = i32
            L.stq_dequantize.argtypes = [P, P, i32, P, i32, P, P, P]
            L.stq_dequantize.restype = i32
            L.stq_allocate_widths.argtypes = [i32, i32, P, P, i32, ctypes.c_uint64, P]
            L.stq_allocate_widths.restype = i32
            L.stq_row_impact.argtypes = [i32, i32, i32, i32, i32, P, P, P, P, P, P]
            L.stq_row_impact.restype = i32
            L.stq_selftest_wait_timeout.argtypes, L.stq_selftest_wait_timeout.restype = [P, P], i32
            i64 = ctypes.c_int64
            L.stq_decay_step.argtypes = [i32, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P]
            L.stq_decay_step.restype = i32
            L.stq_decay_prefill_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            L.stq_decay_prefill_workspace_bytes.restype = sz
            L.stq_decay_prefill.argtypes = [i32, i32, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P, sz, P, P]
            L.stq_decay_prefill.restype = i32
            L.stq_page_plan.argtypes = [i32, i32, i32, P, P, P, P, i32, P, P, i32, P, P, P, P, P]
            L.stq_page_plan.restype = i32
            L.stq_page_write.argtypes = [i32, i32, i32, i32, i32, i32, P, P, P, P, P, i64, i64, P, P]
            L.stq_page_write.restype = i32
            L.stq_paged_attention_workspace_bytes.argtypes = [i32, i32, i32, i32]
            L.stq_paged_attention_workspace_bytes.restype = sz
            L.stq_paged_attention.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, P, P, P, P, P, ctypes.c_float,
                                              P, P, sz, P, P]
            L.stq_paged_attention.restype = i32
            _lib_handle = L
    return _lib_handle


def status_string(status: int) -> str:
    return lib().stq_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != STQ_OK:
        raise StqError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, shape, device=None):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and (device is None or t.device == device) and t.is_contiguous()):
        return  # the usual case in one test: the calls' host time is what small steps wait for
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


class Layout:
    """Host-side description of one model's quantized state (see stq_layout_desc)."""

    def __init__(self, head_bits: Sequence[int], d: int, gate: int = GATE_SCALAR,
                 in_dtype: torch.dtype = torch.bfloat16, scale_mode: int = SCALES_ROW_COLUMN,
                 scale_dtype: torch.dtype = torch.float32, fit_rounds: int = 0):
        self.head_bits = [int(b) for b in head_bits]
        self.H, self.d, self.gate, self.in_dtype = len(self.head_bits), int(d), int(gate), in_dtype
        self.scale_mode = int(scale_mode)
        self.scale_dtype = scale_dtype
        self.fit_rounds = int(fit_rounds)
        if in_dtype not in _DTYPES:
            raise TypeError(f"unsupported input dtype {in_dtype}")
        if scale_dtype not in _DTYPES:
            raise TypeError(f"unsupported scale dtype {scale_dtype}")
        arr = (ctypes.c_uint8 * self.H)(*self.head_bits)
        desc = _Desc(self.H, self.d, self.d, ctypes.cast(arr, ctypes.POINTER(ctypes.c_uint8)),
                     self.gate, _DTYPES[in_dtype], self.scale_mode, _DTYPES[scale_dtype], self.fit_rounds)
        handle = ctypes.c_void_p()
        _check(lib().stq_layout_create(ctypes.byref(desc), ctypes.byref(handle)), "stq_layout_create")
        self._h = handle

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib_handle is not None:
            _lib_handle.stq_layout_destroy(h)
            self._h = None

    @property
    def handle(self):
        return self._h

    @property
    def bytes_per_request(self) -> int:
        return lib().stq_layout_bytes_per_request(self._h)

    def head_offset(self, h: int) -> int:
        return lib().stq_layout_head_offset(self._h, h)

    def head_bytes(self, h: int) -> int:
        return lib().stq_layout_head_bytes(self._h, h)

    def head_bits_of(self, h: int) -> int:
        return lib().stq_layout_head_bits(self._h, h)

    def alloc_pool(self, slots: int, device="cuda") -> torch.Tensor:
        """A zeroed pool of `slots` request blocks (uint8)."""
        return torch.zeros(slots * self.bytes_per_request, dtype=torch.uint8, device=device)


def _pool_slots(layout: Layout, pool: torch.Tensor) -> int:
    if pool.dtype != torch.uint8 or pool.dim() != 1 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous 1-D uint8 tensor")
    return pool.numel() // layout.bytes_per_request


def init_state(layout: Layout, pool, slots, S0, w, status=None, stream=None):
    B = slots.numel()
    dev = pool.device
    _need(slots, "slots", torch.int32, (B,), dev)
    _need(S0, "S0", torch.float32, (B, layout.H, layout.d, layout.d), dev)
    _need(w, "w", torch.float32, (layout.H, layout.d), dev)
    _check(lib().stq_init_state(layout.handle, _ptr(pool), _pool_slots(layout, pool), _ptr(slots), B,
                                _ptr(S0), _ptr(w), _ptr(status), _stream(stream)), "stq_init_state")


def decode_step(layout: Layout, pool, slots, q, k, v, beta, alpha, w, o, head_begin: int = 0,
                status=None, stream=None):
    """One in-place decode step for heads [head_begin, head_begin + q.shape[1])."""
    B, hc, d = q.shape
    dev = pool.device
    _need(slots, "slots", torch.int32, (B,), dev)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, layout.in_dtype, (B, hc, d), dev)
    _need(beta, "beta", torch.float32, (B, hc), dev)
    _need(alpha, "alpha", torch.float32, (B, hc) if layout.gate == GATE_SCALAR else (B, hc, d), dev)
    _need(w, "w", torch.float32, (hc, d), dev)
    _need(o, "o", torch.float32, (B, hc, d), dev)
    _check(lib().stq_decode_step(layout.handle, _ptr(pool), _pool_slots(layout, pool), _ptr(slots), B,
                                 head_begin, hc, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(w),
                                 _ptr(o), _ptr(status), _stream(stream)), "stq_decode_step")


def prefill_workspace_bytes(layout: Layout, B: int, T: int, chunk: int) -> int:
    return lib().stq_prefill_workspace_bytes(layout.handle, B, T, chunk)


def prefill_chunk(layout: Layout, pool, slots, q, k, v, beta, alpha, w, o, chunk: int = 64,
                  workspace=None, status=None, stream=None):
    """Chunked prefill of T tokens (q, k, v: [B, H, T, d]) for all heads, in place."""
    B, H, T, d = q.shape
    dev = pool.device
    _need(slots, "slots", torch.int32, (B,), dev)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, layout.in_dtype, (B, H, T, d), dev)
    _need(beta, "beta", torch.float32, (B, H, T), dev)
    _need(alpha, "alpha", torch.float32, (B, H, T) if layout.gate == GATE_SCALAR else (B, H, T, d), dev)
    _need(w, "w", torch.float32, (H, d), dev)
    _need(o, "o", torch.float32, (B, H, T, d), dev)
    # with a workspace of prefill_workspace_bytes() the tensor-core chunk form runs as three
    # kernels (chunk-parallel inputs and readout around the sequential state kernel); without one
    # it runs as one kernel
    need = prefill_workspace_bytes(layout, B, T, chunk)
    ws_ptr, ws_bytes = None, 0
    if need and workspace is not None:
        ws_bytes = workspace.numel() * workspace.element_size()
        if ws_bytes < need:
            raise ValueError(f"prefill workspace of {ws_bytes} bytes is below the {need} bytes it needs")
        ws_ptr = _ptr(workspace)
    _check(lib().stq_prefill_chunk(layout.handle, _ptr(pool), _pool_slots(layout, pool), _ptr(slots), B, T, chunk,
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(w), _ptr(o),
                                   ws_ptr, ws_bytes, _ptr(status), _stream(stream)),
           "stq_prefill_chunk")


def prefill_chunk_noalloc(layout: Layout, pool, slots, q, k, v, beta, alpha, w, o, chunk: int = 64, status=None,
                          stream=None):
    """prefill_chunk for callers that cannot allocate device memory: the workspace is a fixed
    32 MiB array inside the library (see stq_prefill_chunk_noalloc in include/stq.h); calls whose
    device work overlaps race on it."""
    B, H, T, d = q.shape
    dev = pool.device
    _need(slots, "slots", torch.int32, (B,), dev)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, layout.in_dtype, (B, H, T, d), dev)
    _need(beta, "beta", torch.float32, (B, H, T), dev)
    _need(alpha, "alpha", torch.float32, (B, H, T) if layout.gate == GATE_SCALAR else (B, H, T, d), dev)
    _need(w, "w", torch.float32, (H, d), dev)
    _need(o, "o", torch.float32, (B, H, T, d), dev)
    _check(lib().stq_prefill_chunk_noalloc(layout.handle, _ptr(pool), _pool_slots(layout, pool), _ptr(slots), B, T,
                                           chunk, _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(alpha), _ptr(w), _ptr(o),
                                           _ptr(status), _stream(stream)),
           "stq_prefill_chunk_noalloc")


def dequantize(layout: Layout, pool, slots, S_out, status=None, stream=None):
    B = slots.numel()
    dev = pool.device
    _need(slots, "slots", torch.int32, (B,), dev)
    _need(S_out, "S_out", torch.float32, (B, layout.H, layout.d, layout.d), dev)
    _check(lib().stq_dequantize(layout.handle, _ptr(pool), _pool_slots(layout, pool), _ptr(slots), B, _ptr(S_out),
                                _ptr(status), _stream(stream)), "stq_dequantize")


def selftest_wait_timeout(status, stream=None):
    """Run the bounded-wait self-test: it ORs the timeout bit into `status` (device int32 [1])
    after about two seconds of device time."""
    _need(status, "status", torch.int32, (1,), status.device)
    _check(lib().stq_selftest_wait_timeout(_ptr(status), _stream(stream)), "stq_selftest_wait_timeout")


def status_flags(status: torch.Tensor) -> list:
    """Names of the conditions OR-ed into a device status word (synchronizes)."""
    v = int(status.item())
    return [status_string(c) for c in (STQ_ERR_NONFINITE, STQ_ERR_TIMEOUT, STQ_ERR_BOUNDS) if v & (1 << c)]


def allocate_widths(distortion, mean_log_retention, d: int, num_pivots: int, budget_bytes: int) -> list:
    """Lifetime-aware widths per head (host only): distortion [H][3] at widths 4, 6, 8 and the mean
    log-retention [H] of each head's gate; see stq_allocate_widths in include/stq.h."""
    import numpy as np

    D = np.ascontiguousarray(np.asarray(distortion, dtype=np.float64))
    lr = np.ascontiguousarray(np.asarray(mean_log_retention, dtype=np.float64))
    H = lr.shape[0]
    if D.shape != (H, 3):
        raise ValueError("distortion must be [H][3]")
    out = np.zeros(H, dtype=np.uint8)
    _check(lib().stq_allocate_widths(H, int(d), D.ctypes.data_as(ctypes.c_void_p), lr.ctypes.data_as(ctypes.c_void_p),
                                     int(num_pivots), int(budget_bytes), out.ctypes.data_as(ctypes.c_void_p)),
           "stq_allocate_widths")
    return [int(x) for x in out]


def row_impact(q, k, beta, alpha, gate: int = GATE_SCALAR, stream=None) -> torch.Tensor:
    """Key-row impact scores w [H][d] from calibration tokens q, k [T][H][d], beta [T][H] and
    alpha [T][H] (scalar gate) or [T][H][d]; see stq_row_impact in include/stq.h."""
    T, H, d = q.shape
    dev = q.device
    if q.dtype not in _DTYPES:
        raise TypeError("q must be float32 or bfloat16")
    _need(k, "k", q.dtype, (T, H, d), dev)
    _need(beta, "beta", torch.float32, (T, H), dev)
    _need(alpha, "alpha", torch.float32, (T, H) if gate == GATE_SCALAR else (T, H, d), dev)
    _need(q, "q", q.dtype, (T, H, d), dev)
    w = torch.empty(H, d, dtype=torch.float32, device=dev)
    _check(lib().stq_row_impact(T, H, d, int(gate), _DTYPES[q.dtype], _ptr(q), _ptr(k), _ptr(beta), _ptr(alpha),
                                _ptr(w), _stream(stream)), "stq_row_impact")
    return w


# --------------------------------------------------------------------------------------------
# The layers next to the quantized ones: decayed linear attention, paged cache and attention.
# These calls run on the device of their tensors, whatever the current one is. Each goes through the compiled
# module first, which takes the usual case (csrc/binding.cpp); what follows here knows the others.
# --------------------------------------------------------------------------------------------
_native = None


class _Ctypes:
    """In the compiled module's place where there is none to load: every call goes through ctypes."""

    decay_step = decay_prefill = page_plan = page_write = paged_attention = staticmethod(lambda *args: -1)


def _load():
    """The compiled module, or _Ctypes (with a warning) where it has not been built for this torch and Python."""
    global _native
    from . import build

    lib()
    why = ""
    try:
        from . import _binding

        if getattr(_binding, "built_for", "") != build.binding_key():
            why = f"_binding.so was built for {getattr(_binding, 'built_for', 'another torch')}, this is {build.binding_key()}"
    except ImportError as e:
        why = f"no _binding.so ({e})"
    if why:
        warnings.warn(f"{why}: calls take longer through ctypes; `python -m quantized_linear_attention_stq_b200.build` "
                      "builds it", RuntimeWarning, stacklevel=3)
    _native = _Ctypes if why else _binding
    return _native


def _done(st: int, what: str) -> bool:
    """Whether the compiled module made the call; raises where the library refused it."""
    if st > STQ_OK:
        raise StqError(st, what)
    return st == STQ_OK


def _call(fn, what: str, dev: torch.device, status, stream, *args):
    """fn(*args, status, stream) with `dev` current and its current stream where none is given."""
    if dev.type != "cuda":
        raise ValueError(f"{what}: tensors are on {dev}, expected a CUDA device")
    if status is not None:
        _need(status, "status", torch.int32, (1,), dev)
        status = status.data_ptr()
    if dev.index == torch._C._cuda_getDevice():
        st = fn(*args, status, torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, status, _stream(stream))
    if st != STQ_OK:
        raise StqError(st, what)


def _workspace(workspace, need: int, dev):
    """(pointer, bytes) of a workspace argument; a call that needs none ignores what it is given."""
    if workspace is None or not need:
        return None, 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    n = workspace.numel() * workspace.element_size()
    if n < need:
        raise ValueError(f"workspace of {n} bytes is below the {need} bytes it needs")
    return workspace.data_ptr(), n


def _int32(**sizes):
    """The library's sizes are int32, to which ctypes would cut them."""
    for name, n in sizes.items():
        if not -2**31 <= n < 2**31:
            raise ValueError(f"{name}: {n} is past int32")


def _dtype(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: dtype {t.dtype}, expected float32 or bfloat16")
    return code


def _decay_args(states, slots, q, k, v, alpha, o):
    code, shape, dev = _dtype(q, "q"), q.shape, q.device
    B, H, d = shape[0], shape[1], shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, q.dtype, shape, dev)
    if not isinstance(states, torch.Tensor) or states.dim() != 4:
        raise ValueError("states must be a [slots, heads, d, d] tensor")
    _need(states, "states", torch.float32, (states.shape[0], H, d, d), dev)
    _need(slots, "slots", torch.int32, (B,), dev)
    _need(alpha, "alpha", torch.float32, shape[:-1], dev)
    _need(o, "o", torch.float32, shape, dev)
    return code, dev


def decay_step(states, slots, q, k, v, alpha, o, status=None, stream=None):
    """One token of linear attention with a decay per head, in place: S <- alpha S + k v^T, o = S^T q.

    states [slots, H, d, d] fp32, slots [B] int32, q, k, v [B, H, d] (float32 or bfloat16), alpha
    [B, H] fp32, o [B, H, d] fp32. See stq_decay_step in include/stq.h."""
    if _done((_native or _load()).decay_step(states, slots, q, k, v, alpha, o, status, stream), "stq_decay_step"):
        return
    if isinstance(q, torch.Tensor) and q.dim() != 3:
        raise ValueError("q must be [B, H, d]")
    code, dev = _decay_args(states, slots, q, k, v, alpha, o)
    B, H, d = q.shape
    _int32(B=B, H=H, d=d, states=states.shape[0])
    _call(lib().stq_decay_step, "stq_decay_step", dev, status, stream, B, H, d, code, states.data_ptr(),
          states.shape[0], slots.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(), o.data_ptr())


def decay_prefill_workspace_bytes(B: int, H: int, T: int, d: int, in_dtype: torch.dtype) -> int:
    """Workspace bytes decay_prefill can use (0: none for this shape)."""
    if in_dtype not in _DTYPES:
        raise TypeError(f"unsupported input dtype {in_dtype}")
    _int32(B=B, H=H, T=T, d=d)
    return lib().stq_decay_prefill_workspace_bytes(B, H, T, d, _DTYPES[in_dtype])


def decay_prefill(states, slots, q, k, v, alpha, o, lens=None, workspace=None, status=None, stream=None):
    """decay_step over prompts: q, k, v [B, H, T, d], alpha [B, H, T], o [B, H, T, d] fp32, lens [B]
    int32 (tokens of each prompt; rows behind them are left alone) or None for T. See
    stq_decay_prefill in include/stq.h."""
    if _done((_native or _load()).decay_prefill(states, slots, q, k, v, alpha, o, lens, workspace, status, stream),
             "stq_decay_prefill"):
        return
    if isinstance(q, torch.Tensor) and q.dim() != 4:
        raise ValueError("q must be [B, H, T, d]")
    code, dev = _decay_args(states, slots, q, k, v, alpha, o)
    B, H, T, d = q.shape
    if lens is not None:
        _need(lens, "lens", torch.int32, (B,), dev)
    _int32(B=B, H=H, T=T, d=d, states=states.shape[0])
    ws, ws_bytes = _workspace(workspace, lib().stq_decay_prefill_workspace_bytes(B, H, T, d, code), dev)
    _call(lib().stq_decay_prefill, "stq_decay_prefill", dev, status, stream, B, H, T, d, code, states.data_ptr(),
          states.shape[0], slots.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), alpha.data_ptr(),
          None if lens is None else lens.data_ptr(), o.data_ptr(), ws, ws_bytes)


def page_plan(table, lens, fresh, free_pages, free_head, slot_map, starts, lens_out, head_out, page_size: int,
              status=None, stream=None):
    """Pages, table entries and slots of the fresh[b] new tokens of requests that hold lens[b], from
    the free list (all int32 tensors; lens_out and head_out may be lens and free_head themselves).
    See stq_page_plan in include/stq.h."""
    if _done((_native or _load()).page_plan(table, lens, fresh, free_pages, free_head, slot_map, starts, lens_out,
                                            head_out, page_size, status, stream), "stq_page_plan"):
        return
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a [B, width] tensor")
    dev, (B, W) = table.device, table.shape
    _need(table, "table", torch.int32, (B, W), dev)
    for name, t, n in (("lens", lens, B), ("fresh", fresh, B), ("free_pages", free_pages, None),
                       ("free_head", free_head, 1), ("slot_map", slot_map, None), ("starts", starts, B + 1),
                       ("lens_out", lens_out, B), ("head_out", head_out, 1)):
        if n is None:
            if not isinstance(t, torch.Tensor) or t.dim() != 1:
                raise ValueError(f"{name} must be a 1-D tensor")
            n = t.shape[0]
        _need(t, name, torch.int32, (n,), dev)
    page_size = int(page_size)
    _int32(table=max(B, W), page_size=page_size, free_pages=free_pages.shape[0], slot_map=slot_map.shape[0])
    _call(lib().stq_page_plan, "stq_page_plan", dev, status, stream, B, W, page_size, table.data_ptr(),
          lens.data_ptr(), fresh.data_ptr(), free_pages.data_ptr(), free_pages.shape[0], free_head.data_ptr(),
          slot_map.data_ptr(), slot_map.shape[0], starts.data_ptr(), lens_out.data_ptr(), head_out.data_ptr())


def _pages(k_pages, v_pages, kind, Hkv, d, dev):
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be a [pages, kv_heads, page_size, d] tensor")
    n, heads, page, _ = k_pages.shape
    shape = (n, heads if Hkv is None else Hkv, page, d)
    _need(k_pages, "k_pages", kind, shape, dev)
    _need(v_pages, "v_pages", kind, shape, dev)
    return shape


def page_write(k_pages, v_pages, slot_map, k, v, status=None, stream=None):
    """Write new tokens' keys and values [N, kv_heads, d] to their slots of the paged cache
    [pages, kv_heads, page_size, d]; slot -1 skips a token. k and v may be strided over tokens. See
    stq_page_write in include/stq.h."""
    if _done((_native or _load()).page_write(k_pages, v_pages, slot_map, k, v, status, stream), "stq_page_write"):
        return
    code = _dtype(k, "k")
    if k.dim() != 3:
        raise ValueError("k must be [N, kv_heads, d]")
    (N, Hkv, d), dev = k.shape, k.device
    n, _, page, _ = _pages(k_pages, v_pages, k.dtype, Hkv, d, dev)
    _need(slot_map, "slot_map", torch.int32, (N,), dev)
    _int32(N=N, kv_heads=Hkv, d=d, page_size=page, pages=n)
    strides = []
    for name, t in (("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != k.dtype or t.device != dev or t.shape != k.shape:
            raise ValueError(f"{name} must be a {k.dtype} tensor of shape {tuple(k.shape)} on {dev}")
        row, head, unit = t.stride()
        if (unit != 1 and d > 1) or (head != d and Hkv > 1) or (row < Hkv * d and N > 1):
            raise ValueError(f"{name}: a token's heads must be contiguous and tokens must not overlap")
        strides.append(row if N > 1 else Hkv * d)
    _call(lib().stq_page_write, "stq_page_write", dev, status, stream, N, Hkv, d, code, page, n, k_pages.data_ptr(),
          v_pages.data_ptr(), slot_map.data_ptr(), k.data_ptr(), v.data_ptr(), *strides)


def paged_attention_workspace_bytes(B: int, q_heads: int, d: int, kv_heads: int) -> int:
    """Workspace bytes of paged_attention."""
    _int32(B=B, q_heads=q_heads, d=d, kv_heads=kv_heads)
    return lib().stq_paged_attention_workspace_bytes(B, q_heads, d, kv_heads)


def paged_attention(q, k_pages, v_pages, table, lens, o, scale: float, workspace=None, status=None, stream=None):
    """Attention of one new token per request, q [B, q_heads, d], over the lens[b] cached tokens of
    its table row; o [B, q_heads, d] fp32. With a workspace the cache is split over the GPU. See
    stq_paged_attention in include/stq.h."""
    if _done((_native or _load()).paged_attention(q, k_pages, v_pages, table, lens, o, scale, workspace, status,
                                                  stream), "stq_paged_attention"):
        return
    code = _dtype(q, "q")
    if q.dim() != 3:
        raise ValueError("q must be [B, q_heads, d]")
    (B, Hq, d), dev = q.shape, q.device
    _need(q, "q", q.dtype, (B, Hq, d), dev)
    n, Hkv, page, _ = _pages(k_pages, v_pages, q.dtype, None, d, dev)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a [B, width] tensor")
    W = table.shape[1]
    _need(table, "table", torch.int32, (B, W), dev)
    _need(lens, "lens", torch.int32, (B,), dev)
    _need(o, "o", torch.float32, (B, Hq, d), dev)
    _int32(B=B, q_heads=Hq, kv_heads=Hkv, d=d, page_size=page, pages=n, table=W)
    ws, ws_bytes = _workspace(workspace, lib().stq_paged_attention_workspace_bytes(B, Hq, d, Hkv), dev)
    _call(lib().stq_paged_attention, "stq_paged_attention", dev, status, stream, B, Hq, Hkv, d, code, page, n, W,
          q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(), lens.data_ptr(), float(scale),
          o.data_ptr(), ws, ws_bytes)

"""ctypes binding of libfa.so (include/fa.h), argument marshalling only.

Every function named ``fa_*`` here has the name and argument order of the C
entry point and passes torch tensors' device pointers plus the current torch
stream.  All arithmetic runs in the CUDA kernels of libfa.so; nothing here
computes attention.  If libfa.so is missing or fails to load, every call
raises FaError: there is no fallback.
"""

from __future__ import annotations

import ctypes
import importlib
import math
import os
import re
import threading
import warnings

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "fa.h")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_NO_MEMORY = 4
FA_ERR_TIMEOUT = 5
FA_ERR_SCRATCH_TOO_SMALL = 6
FA_ERR_BAD_INDEX = 7
FA_BWD_NOALLOC_SCRATCH_BYTES = 64 << 20
FA_CAUSAL_NONE = 0
FA_CAUSAL_TOP_LEFT = 1
FA_CAUSAL_BOTTOM_RIGHT = 2
_CAUSAL_NAMES = {"none": FA_CAUSAL_NONE, "top_left": FA_CAUSAL_TOP_LEFT, "bottom_right": FA_CAUSAL_BOTTOM_RIGHT}


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = _strerror(status) if _lib is not None else f"fa_status {status}"
        super().__init__(f"{what}: {msg}" if what else msg)


_lib = None
_lock = threading.Lock()

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_u64 = ctypes.c_uint64

_SIGNATURES = {
    "fa_fwd": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_fwd_ex": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_fwd_gqa": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_bwd_gqa": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_bwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_fwd_general": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp], _i),
    "fa_bwd_general": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp], _i),
    "fa_kv4_cache_bytes": ([_i, _i, _i, _i, ctypes.POINTER(_u64)], _i),
    "fa_kv4_write": ([_vp] * 6 + [_i] * 7 + [_vp], _i),
    "fa_kv4_read": ([_vp] * 6 + [_i] * 7 + [_vp], _i),
    "fa_kv4_fwd": ([_vp] * 6 + [_i] * 9 + [_f, _vp], _i),
    "fa_poll_status": ([_vp], _i),
    "fa_set_wait_timeout_ns": ([_u64], _u64),
    "fa_selftest_wait_timeout": ([_u64, _vp], _i),
    "fa_selftest_kv4_timeout": ([_vp] * 6 + [_i] * 8 + [_u64, _vp], _i),
    "fa_strerror": ([_i], ctypes.c_char_p),
    "fa_abi_version": ([], _i),
    "fa_trim_workspace": ([], _i),
    "fa_timing_enable": ([_i], _i),
    "fa_timing_read": ([_i, ctypes.POINTER(_i), ctypes.POINTER(ctypes.c_double)], _i),
    "fa_launch_count": ([_i, ctypes.POINTER(ctypes.c_uint64)], _i),
}


class FwdPlan(ctypes.Structure):
    """fa_fwd_plan_t (include/fa.h)."""
    _fields_ = [(n, _i) for n in ("packed_heads", "unit_heads", "unit_rows", "query_block", "key_tile",
                                  "key_tiles", "num_splits", "key_tiles_per_split", "dual", "partials",
                                  "num_units", "grid", "head_window", "launches")] + [("workspace_bytes", _u64)]


class BwdPlan(ctypes.Structure):
    """fa_bwd_plan_t (include/fa.h)."""
    _fields_ = [(n, _i) for n in ("q_tiles", "k_tiles", "q_tile_first", "kv_tiles_used", "dq_units", "dq_grid",
                                  "kv_units", "kv_cta_pair", "kv_passes", "launches")] + [
        (n, _u64) for n in ("zeroed_dq_bytes", "zeroed_dkdv_bytes", "workspace_bytes")]


class Kv4Plan(ctypes.Structure):
    """fa_kv4_plan_t (include/fa.h)."""
    _fields_ = [(n, _i) for n in ("rows", "unit_rows", "row_blocks", "units", "step_keys", "max_steps", "whole", "grid",
                                  "launches")] + [("workspace_bytes", _u64)]


class Rows(ctypes.Structure):
    """fa_rows_t (include/fa.h)."""
    _fields_ = [("ptr", _vp), ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_rows = ctypes.POINTER(Rows)
_SIGNATURES["fa_rope"] = ([_rows] * 4 + [_vp] * 3 + [_i] * 7 + [_f, _i, _vp], _i)
_SIGNATURES["fa_rope_phases"] = ([ctypes.POINTER(ctypes.c_double), _i, ctypes.POINTER(_u64)], _i)
_SIGNATURES["fa_packed_fwd"] = ([_rows] * 4 + [_vp] * 4 + [_i] * 7 + [_f, _vp], _i)
_SIGNATURES["fa_packed_bwd"] = ([_rows] * 4 + [_vp] + [_rows] * 4 + [_vp] * 2 + [_i] * 7 + [_f, _vp], _i)
_SIGNATURES["fa_prefix_fwd"] = ([_rows] * 6 + [_vp] * 4 + [_i] * 8 + [_f, _vp], _i)
_SIGNATURES["fa_kv4_fwd_plan"] = ([_i] * 8 + [ctypes.POINTER(Kv4Plan)], _i)
_SIGNATURES["fa_fwd_plan"] = ([_i] * 9 + [_u64, ctypes.POINTER(FwdPlan)], _i)
_SIGNATURES["fa_bwd_plan"] = ([_i] * 8 + [ctypes.POINTER(BwdPlan)], _i)


def load():
    """Load libfa.so once; raise FaError if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise FaError(FA_ERR_CUDA, f"{LIB_PATH} is not built (run exact_attention_92_gb300.build.build())")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def declared_symbols():
    """Entry points declared in include/fa.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|uint64_t|const char\*)\s+(fa_\w+)\s*\(", text, re.M)))


def _strerror(status: int) -> str:
    return load().fa_strerror(int(status)).decode()


def _check(status: int, what: str):
    if status != FA_OK:
        raise FaError(status, what)


def _stream_ptr(stream, device):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _check_bhnd(name, t, shape=None):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    # The library works on the current CUDA device (its status word, its
    # scratch and its launches); a tensor on another device would be read
    # through the wrong device's context.
    if t.device.index is not None and t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device)")


def _check_lse(t, shape):
    import torch

    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()
            and tuple(t.shape) == tuple(shape)):
        raise ValueError(f"lse must be a contiguous float32 CUDA tensor of shape {tuple(shape)}")


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


# ---------------------------------------------------------------- C names

def fa_fwd(q, k, v, o, lse, causal=False, scale=None, stream=None):
    """C fa_fwd: O and LSE of softmax(scale Q K^T [+ causal mask]) V."""
    return fa_fwd_ex(q, k, v, o, lse, causal, scale, 0, stream)


def fa_fwd_ex(q, k, v, o, lse, causal=False, scale=None, num_splits=0, stream=None):
    """C fa_fwd_ex: fa_fwd with an explicit key-split count (0 = automatic)."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o)):
        _check_bhnd(name, t, q.shape)
    _check_lse(lse, (B, H, N))
    lib = load()
    st = lib.fa_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d, 1 if causal else 0,
                       _scale(scale, d), int(num_splits), _stream_ptr(stream, q.device))
    _check(st, "fa_fwd_ex")


def fa_fwd_gqa(q, k, v, o, lse, causal=False, scale=None, num_splits=0, stream=None):
    """C fa_fwd_gqa: grouped-query attention; q, o [B, H, N, d], k, v
    [B, Hkv, N, d] with Hkv dividing H (query head h reads key/value head
    h // (H // Hkv))."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    _check_bhnd("k", k)
    Hkv = k.shape[1]
    _check_bhnd("k", k, (B, Hkv, N, d))
    _check_bhnd("v", v, (B, Hkv, N, d))
    _check_bhnd("o", o, q.shape)
    _check_lse(lse, (B, H, N))
    lib = load()
    st = lib.fa_fwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, N, d, 1 if causal else 0,
                        _scale(scale, d), int(num_splits), _stream_ptr(stream, q.device))
    _check(st, "fa_fwd_gqa")


def _causal_code(causal):
    """False/True (top-left), or a FA_CAUSAL_* code, or its name."""
    if isinstance(causal, str):
        if causal not in _CAUSAL_NAMES:
            raise ValueError(f"causal must be one of {sorted(_CAUSAL_NAMES)}, got {causal!r}")
        return _CAUSAL_NAMES[causal]
    if isinstance(causal, bool):
        return FA_CAUSAL_TOP_LEFT if causal else FA_CAUSAL_NONE
    return int(causal)


def fa_fwd_general(q, k, v, o, lse, causal=False, scale=None, num_splits=0, stream=None):
    """C fa_fwd_general: q, o [B, H, Nq, d], k, v [B, Hkv, Nk, d];
    causal False / True (top-left) / "top_left" / "bottom_right" or a
    FA_CAUSAL_* code."""
    _check_bhnd("q", q)
    B, H, Nq, d = q.shape
    _check_bhnd("k", k)
    Hkv, Nk = k.shape[1], k.shape[2]
    _check_bhnd("k", k, (B, Hkv, Nk, d))
    _check_bhnd("v", v, (B, Hkv, Nk, d))
    _check_bhnd("o", o, q.shape)
    _check_lse(lse, (B, H, Nq))
    lib = load()
    st = lib.fa_fwd_general(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Hkv, Nq, Nk, d,
                            _causal_code(causal), _scale(scale, d), int(num_splits), _stream_ptr(stream, q.device))
    _check(st, "fa_fwd_general")


def fa_bwd_general(q, k, v, o, lse, dout, dq, dk, dv, causal=False, scale=None, stream=None):
    """C fa_bwd_general: gradients for fa_fwd_general (same shapes and
    causal argument); dk, dv have the shape of k, v."""
    _check_bhnd("q", q)
    B, H, Nq, d = q.shape
    _check_bhnd("k", k)
    Hkv, Nk = k.shape[1], k.shape[2]
    for name, t in (("k", k), ("v", v), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, (B, Hkv, Nk, d))
    for name, t in (("o", o), ("dout", dout), ("dq", dq)):
        _check_bhnd(name, t, q.shape)
    _check_lse(lse, (B, H, Nq))
    lib = load()
    st = lib.fa_bwd_general(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                            _ptr(dv), B, H, Hkv, Nq, Nk, d, _causal_code(causal), _scale(scale, d),
                            _stream_ptr(stream, q.device))
    _check(st, "fa_bwd_general")


def fa_bwd_gqa(q, k, v, o, lse, dout, dq, dk, dv, causal=False, scale=None, stream=None):
    """C fa_bwd_gqa: gradients for grouped-query attention; dk, dv have the
    shape of k, v ([B, Hkv, N, d]) and hold the sums over each group."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    _check_bhnd("k", k)
    Hkv = k.shape[1]
    for name, t in (("k", k), ("v", v), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, (B, Hkv, N, d))
    for name, t in (("o", o), ("dout", dout), ("dq", dq)):
        _check_bhnd(name, t, q.shape)
    _check_lse(lse, (B, H, N))
    lib = load()
    st = lib.fa_bwd_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                        B, H, Hkv, N, d, 1 if causal else 0, _scale(scale, d), _stream_ptr(stream, q.device))
    _check(st, "fa_bwd_gqa")


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal=False, scale=None, stream=None):
    """C fa_bwd: dQ, dK, dV from the forward inputs, O, LSE and dO."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, q.shape)
    _check_lse(lse, (B, H, N))
    lib = load()
    st = lib.fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                    B, H, N, d, 1 if causal else 0, _scale(scale, d), _stream_ptr(stream, q.device))
    _check(st, "fa_bwd")


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, causal=False, scale=None, stream=None):
    """C fa_bwd_noalloc: fa_bwd with its workspace in the library's static
    device scratch (no device allocation; see include/fa.h)."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_bhnd(name, t, q.shape)
    _check_lse(lse, (B, H, N))
    lib = load()
    st = lib.fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk),
                            _ptr(dv), B, H, N, d, 1 if causal else 0, _scale(scale, d),
                            _stream_ptr(stream, q.device))
    _check(st, "fa_bwd_noalloc")


# The calls over the 4-bit cache are made once a layer and decoding step, where
# the time of marshalling shows: they go through a native caller (_kv4_call,
# csrc/kv4_call.cpp) that looks at the tensors and calls libfa.so, 2.1 us
# a call on a GB300's host in place of 7 through ctypes and 18 with each tensor
# checked by itself.  It says only that something is wrong; what, is worked out
# after that.

_torch = None
_kv4 = None
_INT_MAX = 2 ** 31 - 1


class _Kv4Ctypes:
    """What the native caller does, through ctypes: for a package that was
    built without torch's headers."""

    def __init__(self, lib):
        self.lib = lib

    @staticmethod
    def _good(tensors, device):
        return all(isinstance(t, _torch.Tensor) and t.dtype is dtype and t.dim() == len(shape) and t.is_contiguous()
                   and t.is_cuda and t.get_device() == device
                   and all(n <= _INT_MAX and (w is None or n == w) for n, w in zip(t.shape, shape))
                   for t, dtype, shape in tensors)

    def move(self, write, k, v, cache, block_table, start, count, stream):
        device, stream = _device_and_stream(stream)
        bf16, i32 = _torch.bfloat16, _torch.int32
        shape = getattr(k, "shape", ())
        if len(shape) != 4:
            return -1
        B, Hkv, N, d = shape
        args = [(k, bf16, shape), (v, bf16, shape), (cache, _torch.uint8, (None, Hkv, None)),
                (block_table, i32, (B, None)), (start, i32, (B,))]
        if not self._good(args if count is None else args + [(count, i32, (B,))], device):
            return -1
        page_size, rest = divmod(cache.shape[2] * 8, 9 * d) if d else (0, 0)
        if rest or not page_size:
            return -1
        kv = (k.data_ptr(), v.data_ptr())
        arrays = (block_table.data_ptr(), start.data_ptr(), None if count is None else count.data_ptr())
        sizes = (B, Hkv, N, d, cache.shape[0], page_size, block_table.shape[1], stream)
        if write:
            return self.lib.fa_kv4_write(*kv, cache.data_ptr(), *arrays, *sizes)
        return self.lib.fa_kv4_read(cache.data_ptr(), *arrays, *kv, *sizes)

    def fwd_args(self, q, cache, block_table, lens, o, lse, device):
        """Pointers and sizes of fa_kv4_fwd up to max_pages; None if a tensor
        is not as it should be."""
        shape = getattr(q, "shape", ())
        if len(shape) != 4:
            return None
        B, H, Nq, d = shape
        if not self._good([(q, _torch.bfloat16, shape), (o, _torch.bfloat16, shape), (lens, _torch.int32, (B,)),
                           (cache, _torch.uint8, (None,) * 3), (block_table, _torch.int32, (B, None)),
                           (lse, _torch.float32, (B, H, Nq))], device):
            return None
        page_size, rest = divmod(cache.shape[2] * 8, 9 * d) if d else (0, 0)
        if rest or not page_size:
            return None
        return (*(t.data_ptr() for t in (q, cache, block_table, lens, o, lse)), B, H, cache.shape[1], Nq, d,
                cache.shape[0], page_size, block_table.shape[1])

    def fwd(self, q, cache, block_table, lens, o, lse, causal, scale, stream):
        device, stream = _device_and_stream(stream)
        args = self.fwd_args(q, cache, block_table, lens, o, lse, device)
        if args is None:
            return -1
        return self.lib.fa_kv4_fwd(*args, causal if 0 <= causal < 2 ** 31 else -1,
                                   1.0 / math.sqrt(q.shape[3]) if scale is None else scale, stream)


def _native_caller(torch_version, module="._kv4_call", what="the 4-bit cache's calls"):
    """A native caller, or None: where it was not built, and, with a warning,
    where it does not load or was compiled against the headers of another torch
    (whose tensors it would misread)."""
    try:
        native = importlib.import_module(module, __package__)
    except ModuleNotFoundError:
        return None
    except ImportError as e:
        why = str(e)
    else:
        built, runs = (re.match(r"[0-9.]*", str(v)).group()
                       for v in (getattr(native, "torch_version", ""), torch_version))
        if built == runs:
            return native
        why = f"compiled against torch {built or '?'}, this is {runs}"
    warnings.warn(f"{what} go through ctypes ({why}): run the build again")
    return None


def _kv4_caller():
    """The caller, and with it torch; made at the first call."""
    global _torch, _kv4
    if _kv4 is None:
        import torch

        lib = load()
        _torch = torch
        native = _native_caller(torch.__version__)
        if native is None:
            _kv4 = _Kv4Ctypes(lib)
        else:
            native.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                          for name in ("fa_kv4_write", "fa_kv4_read", "fa_kv4_fwd")))
            _kv4 = native
    return _kv4


def _device_and_stream(stream):
    """The current CUDA device, and the stream's handle on it."""
    try:
        device = _torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):
        return -1, 0  # no CUDA device: any tensor is refused
    return device, _torch._C._cuda_getCurrentRawStream(device) if stream is None else stream


def _handle(stream):
    """The handle (a number) of a stream."""
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


# What causal is usually given as.
_CAUSAL_CODES = {False: FA_CAUSAL_NONE, True: FA_CAUSAL_TOP_LEFT, FA_CAUSAL_BOTTOM_RIGHT: FA_CAUSAL_BOTTOM_RIGHT,
                 **_CAUSAL_NAMES}


def _kv4_refuse(what, status, tensors, device, heads, d):
    """Raises for a status that is not FA_OK.  -1: for the first of (name,
    tensor, type, shape) that is not a contiguous tensor of that type and shape
    on the current device, or for a cache of other heads or page bytes."""
    if status > 0:
        raise FaError(status, what)
    for name, t, dtype, shape in tensors:
        if not isinstance(t, _torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not dtype or t.dim() != len(shape) or any(
                w is not None and n != w for n, w in zip(t.shape, shape)) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)}, "
                             f"got {t.dtype} {tuple(t.shape)}")
        if t.get_device() != device:
            raise ValueError(f"{name} is on {t.device}, not on the current CUDA device (use torch.cuda.device)")
        if any(n > _INT_MAX for n in t.shape):
            raise ValueError(f"{name} has a size beyond 2^31 - 1: {tuple(t.shape)}")
    cache = next(t for name, t, _, _ in tensors if name == "cache")
    if heads is not None and cache.shape[1] != heads:
        raise ValueError(f"cache has {cache.shape[1]} heads, k has {heads}")
    if d == 0 or cache.shape[2] * 8 % (9 * d) or cache.shape[2] == 0:
        raise ValueError(f"cache has {cache.shape[2]} bytes a page and head, not a multiple of 9 * {d} / 8")
    raise ValueError(f"{what}: torch gives no memory for one of the tensors")


def _c_ints(what, *values):
    """Numbers as C ints; refused where they are none (ctypes would cut them)."""
    out = [int(v) for v in values]
    if any(not -_INT_MAX <= v <= _INT_MAX for v in out):
        raise FaError(FA_ERR_INVALID_ARG, what)
    return out


def fa_kv4_cache_bytes(num_pages, Hkv, page_size, d) -> int:
    """C fa_kv4_cache_bytes: bytes of a 4-bit key/value cache."""
    n = ctypes.c_uint64(0)
    sizes = _c_ints("fa_kv4_cache_bytes", num_pages, Hkv, page_size, d)
    _check(load().fa_kv4_cache_bytes(*sizes, ctypes.byref(n)), "fa_kv4_cache_bytes")
    return n.value


def _kv4_move(what, write, k, v, cache, block_table, start, count, stream):
    caller = _kv4 or _kv4_caller()
    status = caller.move(write, k, v, cache, block_table, start, count,
                         stream if stream is None else _handle(stream))
    if status != FA_OK:
        bf16, i32 = _torch.bfloat16, _torch.int32
        shape = tuple(getattr(k, "shape", ()))
        B, Hkv, N, d = shape if len(shape) == 4 else (None,) * 4
        tensors = [("k", k, bf16, (B, Hkv, N, d)), ("v", v, bf16, (B, Hkv, N, d)),
                   ("cache", cache, _torch.uint8, (None, None, None)), ("block_table", block_table, i32, (B, None)),
                   ("start", start, i32, (B,))]
        _kv4_refuse(what, status, tensors if count is None else tensors + [("count", count, i32, (B,))],
                    _device_and_stream(0)[0], Hkv, d)


def fa_kv4_write(k, v, cache, block_table, start, count=None, stream=None):
    """C fa_kv4_write: quantise tokens k, v [B, Hkv, N, d] into the 4-bit
    cache [num_pages, Hkv, page_size * 9 d / 8] (uint8), token i < count[b]
    (all N without count) of sequence b to position start[b] + i."""
    _kv4_move("fa_kv4_write", True, k, v, cache, block_table, start, count, stream)


def fa_kv4_read(cache, block_table, start, k, v, count=None, stream=None):
    """C fa_kv4_read: the held values of positions start[b] + i to rows
    i < count[b] of k, v [B, Hkv, N, d]; other rows are left as they were."""
    _kv4_move("fa_kv4_read", False, k, v, cache, block_table, start, count, stream)


def fa_kv4_fwd(q, cache, block_table, lens, o, lse, causal=False, scale=None, stream=None):
    """C fa_kv4_fwd: attention of q [B, H, Nq, d] over the first lens[b]
    tokens of each sequence in the 4-bit cache; causal as fa_fwd_general."""
    caller = _kv4 or _kv4_caller()
    code = _CAUSAL_CODES.get(causal)
    if code is None:
        code = _causal_code(causal)
    status = caller.fwd(q, cache, block_table, lens, o, lse, code, scale,
                        stream if stream is None else _handle(stream))
    if status != FA_OK:
        _kv4_refuse_fwd("fa_kv4_fwd", status, q, cache, block_table, lens, o, lse)


def _kv4_refuse_fwd(what, status, q, cache, block_table, lens, o, lse):
    shape = tuple(getattr(q, "shape", ()))
    B, H, Nq, d = shape if len(shape) == 4 else (None,) * 4
    _kv4_refuse(what, status,
                [("q", q, _torch.bfloat16, (B, H, Nq, d)), ("cache", cache, _torch.uint8, (None, None, None)),
                 ("block_table", block_table, _torch.int32, (B, None)), ("lens", lens, _torch.int32, (B,)),
                 ("o", o, _torch.bfloat16, (B, H, Nq, d)), ("lse", lse, _torch.float32, (B, H, Nq))],
                _device_and_stream(0)[0], None, d)


# ------------------------------------------------------- rows with strides

def _check_rows(name, t, shape, write=False):
    """A bf16 tensor [tokens, heads, d] or [B, heads, N, d] on the current
    device, of any strides that fa_rows_t can say."""
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if any(n > _INT_MAX for n in t.shape):
        raise ValueError(f"{name} has a size beyond 2^31 - 1: {tuple(t.shape)}")
    strides = [s for s, n in zip(t.stride()[:-1], t.shape) if n > 1]
    if (t.shape[-1] > 1 and t.stride(-1) != 1) or any(s % 8 for s in strides):
        raise ValueError(f"{name} must have contiguous channels and other strides that are multiples of 8, "
                         f"got {t.stride()}")
    if write:
        # Rows of an output do not overlap: each stride spans what the smaller ones reach.
        reach = t.shape[-1]
        for s, n in sorted((s, n) for s, n in zip(t.stride()[:-1], t.shape) if n > 1):
            if s < reach:
                raise ValueError(f"{name} is written and its rows overlap: strides {t.stride()}")
            reach += s * (n - 1)
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, but the current CUDA device is "
                         f"cuda:{torch.cuda.current_device()} (use torch.cuda.device)")


def _rows_of(t):
    """fa_rows_t of a checked tensor; strides that nothing steps by count 0."""
    st = [s if n > 1 else 0 for s, n in zip(t.stride(), t.shape)]
    if t.dim() == 3:  # [tokens, heads, d]
        return Rows(t.data_ptr(), 0, st[0], st[1])
    return Rows(t.data_ptr(), st[0], st[2], st[1])  # [B, heads, N, d]


def _check_array(name, t, dtype, shape):
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device (use torch.cuda.device)")


# Rotary positions and packed sequences are called once a layer, in decoding
# too: their calls go through a native caller (_packed_call,
# csrc/packed_call.cpp).  Where it is not there, or a tensor is not as it
# should be (-1), the checks here say what is wrong, and ctypes makes the call.

_packed = None


def _packed_caller():
    """The native caller, or False; looked for at the first call."""
    global _packed
    if _packed is None:
        import torch

        lib = load()
        native = _native_caller(torch.__version__, "._packed_call", "the calls on packed sequences") or False
        if native:
            native.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                          for name in ("fa_rope", "fa_packed_fwd", "fa_prefix_fwd", "fa_packed_bwd")))
        _packed = native
    return _packed


def _done(status, what):
    """Whether the native caller made the call; raises for the library's refusals."""
    if status > 0:
        raise FaError(status, what)
    return status == FA_OK


def _code_of(causal):
    code = _CAUSAL_CODES.get(causal) if isinstance(causal, (str, bool, int)) else None
    return _causal_code(causal) if code is None else code


def fa_rope_phases(inv_freq):
    """C fa_rope_phases: frequencies (radians a position, a sequence of
    floats) as 64-bit fractions of a turn, a list of ints below 2^64."""
    freq = [float(f) for f in inv_freq]
    n = len(freq)
    out = (_u64 * max(1, n))()
    _check(load().fa_rope_phases((ctypes.c_double * max(1, n))(*freq), n, out), "fa_rope_phases")
    return list(out)


def fa_rope(q, k, q_out, k_out, phases, positions=None, start=None, interleaved=False, mscale=1.0, inverse=False,
            stream=None):
    """C fa_rope: q [B, H, N, d] and k [B, Hkv, N, d] (or packed, q [tokens, H,
    d] and k [tokens, Hkv, d]) turned by their positions into q_out, k_out;
    any strides with contiguous channels.  phases int64 [rot / 2] from
    rope_phases; positions int32 [B, N] ([tokens]) or start int32 [B] ([1]).
    k and k_out may be None; inverse=True turns gradients back."""
    native = _packed_caller() if _packed is None else _packed
    if native and _done(native.rope(q, k, q_out, k_out, phases, positions, start, interleaved, mscale, inverse,
                                    stream if stream is None else _handle(stream)), "fa_rope"):
        return
    import torch

    dims = getattr(q, "dim", lambda: 4)()
    _check_rows("q", q, (None,) * (3 if dims == 3 else 4))
    if dims == 3:
        (N, H, d), B = q.shape, 1
        shape, k_shape, at = (N,), (N, None, d), (N, H, d)
    else:
        B, H, N, d = q.shape
        shape, k_shape, at = (B, N), (B, None, N, d), (B, H, N, d)
    _check_rows("q_out", q_out, at, write=True)
    Hkv = 0
    if k is not None:
        _check_rows("k", k, k_shape)
        Hkv = k.shape[1]
        _check_rows("k_out", k_out, tuple(k.shape), write=True)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _check_array("phases", phases, torch.int64, (getattr(phases, "shape", (0,))[0] if getattr(phases, "ndim", 0) else 0,))
    if positions is not None:
        _check_array("positions", positions, torch.int32, shape)
    if start is not None:
        _check_array("start", start, torch.int32, (B,))
    rows = [None if t is None else _rows_of(t) for t in (q, k, q_out, k_out)]
    st = load().fa_rope(*(None if r is None else ctypes.byref(r) for r in rows), _ptr(phases),
                        *(None if t is None else _ptr(t) for t in (positions, start)), B, N, H, Hkv, d,
                        2 * phases.shape[0], 1 if interleaved else 0, float(mscale), 1 if inverse else 0,
                        _stream_ptr(stream, q.device))
    _check(st, "fa_rope")


def _packed_fwd(what, q, k_prefix, v_prefix, k, v, o, lse, cu_q, cu_k, used_k, causal, scale, stream):
    native = _packed_caller() if _packed is None else _packed
    if native and (k_prefix is not None or what == "fa_packed_fwd") and _done(
            native.forward(q, k_prefix, v_prefix, k, v, o, lse, cu_q, cu_k, used_k, _code_of(causal), scale,
                           stream if stream is None else _handle(stream)), what):
        return
    import torch

    _check_rows("q", q, (None, None, None))
    Tq, H, d = q.shape
    _check_rows("k", k, (None, None, d))
    Tk, Hkv, _ = k.shape
    _check_rows("v", v, (Tk, Hkv, d))
    _check_rows("o", o, (Tq, H, d), write=True)
    _check_array("lse", lse, torch.float32, (H, Tq))
    B = (cu_q.shape[0] if isinstance(cu_q, torch.Tensor) and cu_q.ndim == 1 else 0) - 1
    if B < 1:
        raise ValueError("cu_q must be an int32 CUDA tensor [B + 1] with B >= 1")
    _check_array("cu_q", cu_q, torch.int32, (B + 1,))
    _check_array("cu_k", cu_k, torch.int32, (B + 1,))
    if used_k is not None:
        _check_array("used_k", used_k, torch.int32, (B,))
    tensors, P = [q, k, v, o], ()
    if what == "fa_prefix_fwd":
        _check_rows("k_prefix", k_prefix, (None, Hkv, d))
        _check_rows("v_prefix", v_prefix, tuple(k_prefix.shape))
        tensors[1:1] = [k_prefix, v_prefix]
        P = (k_prefix.shape[0],)
    rows = [ctypes.byref(_rows_of(t)) for t in tensors]
    st = getattr(load(), what)(*rows, _ptr(lse), _ptr(cu_q), _ptr(cu_k), None if used_k is None else _ptr(used_k), B,
                               *P, Tq, Tk, H, Hkv, d, _causal_code(causal), _scale(scale, d),
                               _stream_ptr(stream, q.device))
    _check(st, what)


def fa_packed_fwd(q, k, v, o, lse, cu_q, cu_k, used_k=None, causal=False, scale=None, stream=None):
    """C fa_packed_fwd: attention over packed sequences, q, o [Tq, H, d] and
    k, v [Tk, Hkv, d] of any strides with contiguous channels, lse fp32 [H,
    Tq]; cu_q, cu_k int32 [B + 1], used_k int32 [B] or None; causal as
    fa_fwd_general, within each sequence."""
    _packed_fwd("fa_packed_fwd", q, None, None, k, v, o, lse, cu_q, cu_k, used_k, causal, scale, stream)


def fa_packed_bwd(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, causal=False, scale=None, stream=None):
    """C fa_packed_bwd: gradients of fa_packed_fwd (without used_k); dout, dq
    have the shape of q, dk, dv that of k."""
    native = _packed_caller() if _packed is None else _packed
    if native and _done(native.backward(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_k, _code_of(causal), scale,
                                        stream if stream is None else _handle(stream)), "fa_packed_bwd"):
        return
    import torch

    _check_rows("q", q, (None, None, None))
    Tq, H, d = q.shape
    _check_rows("k", k, (None, None, d))
    Tk, Hkv, _ = k.shape
    for name, t in (("v", v), ("dk", dk), ("dv", dv)):
        _check_rows(name, t, (Tk, Hkv, d), write=name != "v")
    for name, t in (("o", o), ("dout", dout), ("dq", dq)):
        _check_rows(name, t, (Tq, H, d), write=name == "dq")
    _check_array("lse", lse, torch.float32, (H, Tq))
    B = (cu_q.shape[0] if isinstance(cu_q, torch.Tensor) and cu_q.ndim == 1 else 0) - 1
    if B < 1:
        raise ValueError("cu_q must be an int32 CUDA tensor [B + 1] with B >= 1")
    _check_array("cu_q", cu_q, torch.int32, (B + 1,))
    _check_array("cu_k", cu_k, torch.int32, (B + 1,))
    rows = [ctypes.byref(_rows_of(t)) for t in (q, k, v, o, dout, dq, dk, dv)]
    st = load().fa_packed_bwd(*rows[:4], _ptr(lse), *rows[4:], _ptr(cu_q), _ptr(cu_k), B, Tq, Tk, H, Hkv, d,
                              _causal_code(causal), _scale(scale, d), _stream_ptr(stream, q.device))
    _check(st, "fa_packed_bwd")


def fa_prefix_fwd(q, k_prefix, v_prefix, k, v, o, lse, cu_q, cu_k, used_k=None, causal=False, scale=None, stream=None):
    """C fa_prefix_fwd: fa_packed_fwd where every query row also sees all of
    k_prefix, v_prefix [P, Hkv, d]."""
    _packed_fwd("fa_prefix_fwd", q, k_prefix, v_prefix, k, v, o, lse, cu_q, cu_k, used_k, causal, scale, stream)


def fa_poll_status(stream=None):
    """C fa_poll_status: synchronise the stream, return and clear the device status."""
    import torch

    return load().fa_poll_status(_stream_ptr(stream, torch.device("cuda")))


def fa_set_wait_timeout_ns(ns: int) -> int:
    return int(load().fa_set_wait_timeout_ns(int(ns)))


def fa_selftest_wait_timeout(timeout_ns: int, stream=None):
    import torch

    _check(load().fa_selftest_wait_timeout(int(timeout_ns), _stream_ptr(stream, torch.device("cuda"))),
           "fa_selftest_wait_timeout")


def fa_selftest_kv4_timeout(q, cache, block_table, lens, o, lse, timeout_ns, stream=None):
    """C fa_selftest_kv4_timeout: fa_kv4_fwd on these tensors with every wait
    running out after timeout_ns; fa_poll_status then reports FA_ERR_TIMEOUT."""
    _kv4_caller()
    device, stream = _device_and_stream(stream if stream is None else _handle(stream))
    args = _Kv4Ctypes(load()).fwd_args(q, cache, block_table, lens, o, lse, device)
    status = -1 if args is None else load().fa_selftest_kv4_timeout(*args, int(timeout_ns), stream)
    if status != FA_OK:
        _kv4_refuse_fwd("fa_selftest_kv4_timeout", status, q, cache, block_table, lens, o, lse)


def fa_strerror(status: int) -> str:
    return _strerror(status)


def fa_abi_version() -> int:
    return int(load().fa_abi_version())


def fa_trim_workspace() -> None:
    """C fa_trim_workspace: give back the workspace memory the library's pool
    keeps reserved on the current device."""
    _check(load().fa_trim_workspace(), "fa_trim_workspace")


def fa_timing_enable(on: bool) -> None:
    _check(load().fa_timing_enable(1 if on else 0), "fa_timing_enable")


def fa_timing_read(kernel: int):
    """(launches, total milliseconds) of one kernel since timing was enabled or last read."""
    n = ctypes.c_int(0)
    ms = ctypes.c_double(0.0)
    _check(load().fa_timing_read(int(kernel), ctypes.byref(n), ctypes.byref(ms)), "fa_timing_read")
    return n.value, ms.value


def fa_launch_count(kernel: int) -> int:
    """Launches of one library kernel since the library was loaded."""
    n = ctypes.c_uint64(0)
    _check(load().fa_launch_count(int(kernel), ctypes.byref(n)), "fa_launch_count")
    return n.value


def _plan_dict(plan):
    return {name: getattr(plan, name) for name, _ in plan._fields_}


def fa_fwd_plan(B, H, Hkv, Nq, Nk, d, causal, num_splits, sm_count, l2_bytes):
    """C fa_fwd_plan: the launch plan of fa_fwd_general for these sizes on a
    device with sm_count SMs and l2_bytes of L2, as a dict of the
    fa_fwd_plan_t fields.  Host only; raises FaError on a refused size."""
    plan = FwdPlan()
    _check(load().fa_fwd_plan(int(B), int(H), int(Hkv), int(Nq), int(Nk), int(d), _causal_code(causal),
                              int(num_splits), int(sm_count), int(l2_bytes), ctypes.byref(plan)), "fa_fwd_plan")
    return _plan_dict(plan)


def fa_bwd_plan(B, H, Hkv, Nq, Nk, d, causal, sm_count):
    """C fa_bwd_plan: the launch plan of fa_bwd_general, as a dict of the
    fa_bwd_plan_t fields.  Host only; raises FaError on a refused size."""
    plan = BwdPlan()
    _check(load().fa_bwd_plan(int(B), int(H), int(Hkv), int(Nq), int(Nk), int(d), _causal_code(causal),
                              int(sm_count), ctypes.byref(plan)), "fa_bwd_plan")
    return _plan_dict(plan)


def fa_kv4_fwd_plan(B, H, Hkv, Nq, d, page_size, max_pages, sm_count):
    """C fa_kv4_fwd_plan: the launch plan of fa_kv4_fwd, as a dict of the
    fa_kv4_plan_t fields.  Host only; raises FaError on a refused size."""
    plan = Kv4Plan()
    sizes = _c_ints("fa_kv4_fwd_plan", B, H, Hkv, Nq, d, page_size, max_pages, sm_count)
    _check(load().fa_kv4_fwd_plan(*sizes, ctypes.byref(plan)), "fa_kv4_fwd_plan")
    return _plan_dict(plan)


# ------------------------------------------------------- convenience calls

def forward(q, k, v, causal=False, scale=None, num_splits=0):
    """Allocate O and LSE and run the forward pass; returns (o, lse).  k, v
    may have fewer heads (grouped-query) or another length than q
    (fa_fwd_general; causal may then be "top_left" or "bottom_right")."""
    import torch

    B, H, N, d = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if tuple(k.shape) == tuple(q.shape) and not isinstance(causal, str):
        fa_fwd_ex(q, k, v, o, lse, causal, scale, num_splits)
    else:
        fa_fwd_general(q, k, v, o, lse, causal, scale, num_splits)
    return o, lse


def backward(q, k, v, o, lse, dout, causal=False, scale=None):
    """Allocate dQ, dK, dV and run the backward pass; returns (dq, dk, dv)
    (shapes and causal argument as for ``forward``)."""
    import torch

    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    if tuple(k.shape) == tuple(q.shape) and not isinstance(causal, str):
        fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, causal, scale)
    else:
        fa_bwd_general(q, k, v, o, lse, dout, dq, dk, dv, causal, scale)
    return dq, dk, dv


def kv4_cache(num_pages, Hkv, page_size, d, device="cuda"):
    """A 4-bit key/value cache of num_pages pages, zeroed (every value reads
    as 0): uint8 [num_pages, Hkv, page_size * 9 d / 8]."""
    import torch

    fa_kv4_cache_bytes(num_pages, Hkv, page_size, d)  # refuses bad sizes
    return torch.zeros((num_pages, Hkv, page_size * 9 * d // 8), dtype=torch.uint8, device=device)


def kv4_forward(q, cache, block_table, lens, causal=False, scale=None):
    """Allocate O and LSE and run fa_kv4_fwd; returns (o, lse)."""
    import torch

    o = torch.empty_like(q)
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    fa_kv4_fwd(q, cache, block_table, lens, o, lse, causal, scale)
    return o, lse


def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original=None, slow=1.0, fast=32.0):
    """Frequencies of rotary positions, radians a position: rot/2 floats
    base^(-2j/rot), scaled for contexts `factor` times as long as in training:
      None         not scaled
      "linear"     every one divided by factor
      "base"       base times factor^(rot / (rot - 2)): the slowest divided by
                   factor, the fastest kept
      "by_parts"   those that turn less than `slow` times over the `original`
                   positions divided by factor, above `fast` times kept, between
                   these a mixture in proportion to the turns
    (some models also scale what is turned: fa_rope's mscale)."""
    rot, base, factor = int(rot), float(base), float(factor)
    if rot < 2 or rot % 2 or not base > 0 or not factor > 0:
        raise ValueError(f"rope_frequencies: rot {rot}, base {base}, factor {factor}")
    if scaling not in (None, "linear", "base", "by_parts"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'by_parts', got {scaling!r}")
    if scaling == "base":
        if rot == 2:
            raise ValueError("scaling 'base' needs two frequencies at least")
        base *= factor ** (rot / (rot - 2))
    freq = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "by_parts":
        if original is None or not float(original) > 0 or not slow < fast:
            raise ValueError("scaling 'by_parts' needs the original length, and slow < fast")
        for j, f in enumerate(freq):
            keep = min(1.0, max(0.0, (original * f / (2 * math.pi) - slow) / (fast - slow)))
            freq[j] = f * keep + f / factor * (1.0 - keep)
    return freq


def rope_phases(frequencies, device="cuda"):
    """fa_rope's `phases` for these frequencies (a sequence or tensor of
    floats): int64 [rot / 2] on the device."""
    import torch

    if isinstance(frequencies, torch.Tensor):
        frequencies = frequencies.double().cpu().tolist()
    signed = [p - (1 << 64) if p >> 63 else p for p in fa_rope_phases(frequencies)]
    return torch.tensor(signed, dtype=torch.int64, device=device)


def rope(q, k, phases, positions=None, start=None, interleaved=False, mscale=1.0, inverse=False):
    """Allocate the outputs and run fa_rope; returns (q, k) turned (k may be None)."""
    import torch

    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    k_out = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
    fa_rope(q, k, q_out, k_out, phases, positions, start, interleaved, mscale, inverse)
    return q_out, k_out


def packed_forward(q, k, v, cu_q, cu_k=None, used_k=None, causal=False, scale=None):
    """Allocate O and LSE and run fa_packed_fwd; returns (o, lse).  cu_k
    defaults to cu_q.  Rows of no sequence are 0 (and -inf in lse)."""
    import torch

    o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.full((q.shape[1], q.shape[0]), -math.inf, dtype=torch.float32, device=q.device)
    fa_packed_fwd(q, k, v, o, lse, cu_q, cu_q if cu_k is None else cu_k, used_k, causal, scale)
    return o, lse


def packed_backward(q, k, v, o, lse, dout, cu_q, cu_k=None, causal=False, scale=None):
    """Allocate dQ, dK, dV and run fa_packed_bwd; returns (dq, dk, dv).  Rows
    of no sequence are 0."""
    import torch

    dq, dk, dv = (torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    fa_packed_bwd(q, k, v, o, lse, dout, dq, dk, dv, cu_q, cu_q if cu_k is None else cu_k, causal, scale)
    return dq, dk, dv


def prefix_forward(q, k_prefix, v_prefix, k, v, cu_q, cu_k=None, used_k=None, causal=False, scale=None):
    """Allocate O and LSE and run fa_prefix_fwd; returns (o, lse) as packed_forward."""
    import torch

    o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.full((q.shape[1], q.shape[0]), -math.inf, dtype=torch.float32, device=q.device)
    fa_prefix_fwd(q, k_prefix, v_prefix, k, v, o, lse, cu_q, cu_q if cu_k is None else cu_k, used_k, causal, scale)
    return o, lse

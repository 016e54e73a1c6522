"""ctypes binding of ``librope_gb300.so`` (see ``include/rope_gb300.h``).

Argument marshalling only: every step of the operators runs in the CUDA
library.  The serving operators (scaled tables, paged append, paged attention)
are marshalled by ``lib/rope_binding.so``, built with it.  The library must have been built (``python -m
transformer_rope_positional_gb300.build``); there is no fallback, and calling
an operator without it raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# ROPE_GB300_DEBUG_BOUNDS=1 selects the bounds-checking debug build (see build.py)
DEBUG_BOUNDS = os.environ.get("ROPE_GB300_DEBUG_BOUNDS", "0") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "lib", "librope_gb300_debug.so" if DEBUG_BOUNDS else "librope_gb300.so")

F32, F16, BF16, I64, F8E4M3, E8M0, I32, U8 = 0, 1, 2, 3, 4, 5, 6, 7
DTYPE_CODE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16, torch.int64: I64}

ROPE_OK = 0
ROPE_ERR_PARAM_NULLPTR = 161001
ROPE_ERR_PARAM_INVALID = 161002
ROPE_ERR_CUDA = 561000
ROPE_DEVICE_POSITION_OUT_OF_RANGE = 1
ROPE_DEVICE_SLOT_OUT_OF_RANGE = 2
ROPE_DEVICE_INDEX_OUT_OF_BOUNDS = 4
ROPE_DEVICE_WAIT_EXPIRED = 8
ROPE_DEVICE_PAGES_EXHAUSTED = 16

EXPORTED = ("rope_inplace_partial", "rope_inplace_partial_backward", "rope_with_sin_cos_cache",
            "rope_with_sin_cos_cache_v2", "rope_qkv_rmsnorm_rope_cache", "rope_scaled_frequencies",
            "rope_scaled_cos_sin_cache", "rope_scaled_cos_sin", "rope_append_paged_kv", "rope_paged_attention",
            "rope_paged_attention_workspace", "rope_append_paged_kv_8bit", "rope_paged_attention_8bit",
            "rope_paged_attention_8bit_workspace", "rope_rearrange_sequences", "rope_compact_pages", "rope_copy_pages",
            "rope_get_device_error",
            "rope_status_string", "rope_launch_count", "rope_abi_version")


class RopeTensor(ctypes.Structure):
    """Mirror of ``rope_tensor_t``."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4)]


class RopeScaling(ctypes.Structure):
    """Mirror of ``rope_scaling_t``."""
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_length", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("attention", ctypes.c_double),
                ("factors", ctypes.POINTER(ctypes.c_double))]


class RopeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed with status %d (%s)" % (what, status, status_string(status)))
        self.status = status


_lib = None


def load() -> ctypes.CDLL:
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("%s is not built; run `python -m transformer_rope_positional_gb300.build%s`"
                           % (LIB_PATH, " --debug" if DEBUG_BOUNDS else ""))
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(RopeTensor)
    lib.rope_inplace_partial.argtypes = [P, P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p]
    lib.rope_inplace_partial.restype = ctypes.c_int
    lib.rope_inplace_partial_backward.argtypes = lib.rope_inplace_partial.argtypes
    lib.rope_inplace_partial_backward.restype = ctypes.c_int
    lib.rope_with_sin_cos_cache.argtypes = [P, P, P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                            ctypes.POINTER(ctypes.c_int64), ctypes.c_int64, ctypes.c_void_p]
    lib.rope_with_sin_cos_cache.restype = ctypes.c_int
    lib.rope_with_sin_cos_cache_v2.argtypes = [P, P, P, P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                               ctypes.POINTER(ctypes.c_int64), ctypes.c_int64, ctypes.c_int32,
                                               ctypes.c_int64, ctypes.c_int64, P, P, ctypes.c_void_p]
    lib.rope_with_sin_cos_cache_v2.restype = ctypes.c_int
    lib.rope_qkv_rmsnorm_rope_cache.argtypes = [P, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, P, P,
                                                ctypes.c_float, P, P, P, P, P, P, P, ctypes.c_void_p]
    lib.rope_qkv_rmsnorm_rope_cache.restype = ctypes.c_int
    D, B, V = ctypes.c_int64, P, ctypes.c_void_p
    DP = ctypes.POINTER(ctypes.c_double)
    lib.rope_scaled_frequencies.argtypes = [D, ctypes.c_double, ctypes.POINTER(RopeScaling), DP, DP]
    lib.rope_scaled_frequencies.restype = ctypes.c_int
    lib.rope_scaled_cos_sin_cache.argtypes = [V, D, ctypes.c_double, B, D, B, V]
    lib.rope_scaled_cos_sin_cache.restype = ctypes.c_int
    lib.rope_scaled_cos_sin.argtypes = [V, D, ctypes.c_double, B, D, D, B, B, V]
    lib.rope_scaled_cos_sin.restype = ctypes.c_int
    lib.rope_append_paged_kv.argtypes = [B] * 9 + [D, D, ctypes.c_int32, ctypes.POINTER(D), D, ctypes.c_int32, D, D,
                                                   D, V]
    lib.rope_append_paged_kv.restype = ctypes.c_int
    lib.rope_paged_attention.argtypes = [B, D, B, B, B, B, B, B, D, ctypes.c_float, B, B, V, D, V]
    lib.rope_paged_attention.restype = ctypes.c_int
    lib.rope_paged_attention_workspace.argtypes = [D, D, D, D, ctypes.c_int32, D, ctypes.POINTER(D)]
    lib.rope_paged_attention_workspace.restype = ctypes.c_int
    lib.rope_append_paged_kv_8bit.argtypes = [B] * 11 + lib.rope_append_paged_kv.argtypes[9:]
    lib.rope_paged_attention_8bit.argtypes = [B, D] + [B] * 8 + lib.rope_paged_attention.argtypes[8:]
    lib.rope_paged_attention_8bit_workspace.argtypes = lib.rope_paged_attention_workspace.argtypes
    lib.rope_rearrange_sequences.argtypes = [B] * 11 + [D, D, V]
    lib.rope_compact_pages.argtypes = [B] * 10 + [D, D, V]
    lib.rope_copy_pages.argtypes = [B, B, B, P, D, V]
    for name in ("rope_append_paged_kv_8bit", "rope_paged_attention_8bit", "rope_paged_attention_8bit_workspace",
                 "rope_rearrange_sequences", "rope_compact_pages", "rope_copy_pages"):
        getattr(lib, name).restype = ctypes.c_int
    lib.rope_get_device_error.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int32)]
    lib.rope_get_device_error.restype = ctypes.c_int
    lib.rope_status_string.argtypes = [ctypes.c_int]
    lib.rope_status_string.restype = ctypes.c_char_p
    lib.rope_launch_count.argtypes = []
    lib.rope_launch_count.restype = ctypes.c_uint64
    lib.rope_abi_version.argtypes = []
    lib.rope_abi_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().rope_status_string(int(status)).decode()


_Shape4 = ctypes.c_int64 * 4


def describe(data_ptr: int, dtype_code: int, shape: Sequence[int]) -> RopeTensor:
    """A ``rope_tensor_t`` from a raw device pointer (no checks here)."""
    return RopeTensor(data_ptr or None, dtype_code, len(shape), _Shape4(*shape))


def tensor_desc(t: torch.Tensor) -> RopeTensor:
    """Describe a contiguous CUDA tensor."""
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor, got one on %s" % t.device)
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if t.dtype not in DTYPE_CODE:
        raise ValueError("unsupported dtype %s" % t.dtype)
    return describe(t.data_ptr(), DTYPE_CODE[t.dtype], tuple(t.shape))


def rows_desc(t: torch.Tensor):
    """Describe a 2-D CUDA tensor whose rows may be strided (unit column
    stride); returns (descriptor, row stride in elements).

    Rows must not overlap: a view whose row stride is below its row width
    (e.g. ``expand`` of one row, stride 0) is refused, since the operator
    writes every row.  A tensor of at most one row gets its width as stride."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("expected a 2-D tensor with contiguous rows")
    width = int(t.shape[1])
    stride = int(t.stride(0)) if t.shape[0] > 1 else width
    if stride < width:
        raise ValueError("rows overlap: row stride %d is below the row width %d" % (stride, width))
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor, got one on %s" % t.device)
    if t.dtype not in DTYPE_CODE:
        raise ValueError("unsupported dtype %s" % t.dtype)
    return describe(t.data_ptr(), DTYPE_CODE[t.dtype], tuple(t.shape)), stride


def _one_device(*tensors) -> int:
    """Index of the CUDA device that holds every given tensor (None entries
    skipped); raises if they are spread over several devices."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError("tensors on different devices (cuda:%d and cuda:%d)" % (dev, d))
    return dev


# the current device without the public call's lazy-initialisation check (CUDA
# is initialised once CUDA tensors exist); the public call is the fallback
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_device(dev: int, fn, args):
    """Call fn(*args) with device ``dev`` current (the library launches on the
    current device and sizes its grid from it)."""
    if dev is None or dev < 0 or _current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


# the current stream's raw handle without building a Stream object (about 10x
# cheaper per call); the public call is the fallback
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(t: torch.Tensor, stream) -> int:
    if stream is None:
        if _raw_current_stream is not None:
            return _raw_current_stream(t.get_device())
        return torch.cuda.current_stream(t.device).cuda_stream
    if hasattr(stream, "device") and stream.device.index != t.get_device():
        raise ValueError("stream of %s for tensors on cuda:%d" % (stream.device, t.get_device()))
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


MODES = {"interleave": 1, "half": 0, 1: 1, 0: 0}


def _mode(rotary_mode) -> int:
    if rotary_mode not in MODES:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "rotary_mode %r" % (rotary_mode,))
    return MODES[rotary_mode]


def _slice(partial_slice):
    if partial_slice is None:
        return 0, 0
    if len(partial_slice) != 2:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "partial_slice must have two elements")
    return int(partial_slice[0]), int(partial_slice[1])


def _inplace_args(x, cos, sin, rotary_mode, partial_slice, stream, backward):
    """(C function, its arguments, objects to keep alive, name) of one call."""
    lib = load()
    start, end = _slice(partial_slice)
    _one_device(x, cos, sin)
    dx, dc, ds = tensor_desc(x), tensor_desc(cos), tensor_desc(sin)
    args = (ctypes.byref(dx), ctypes.byref(dc), ctypes.byref(ds), _mode(rotary_mode), start, end,
            _stream_handle(x, stream))
    if backward:
        return lib.rope_inplace_partial_backward, args, (x, cos, sin, dx, dc, ds), "rope_inplace_partial_backward"
    return lib.rope_inplace_partial, args, (x, cos, sin, dx, dc, ds), "rope_inplace_partial"


def _run(fn, args, keep, what) -> None:
    st = _on_device(keep[0].get_device(), fn, args)
    if st != ROPE_OK:
        raise RopeError(st, what)


def rope_inplace_partial(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, rotary_mode=1,
                         partial_slice: Optional[Sequence[int]] = None, stream=None) -> None:
    """In-place partial RoPE of ``x`` [B, S, N, D] over ``partial_slice``.

    ``rotary_mode``: 1 / "interleave" or 0 / "half".  ``partial_slice=None``
    means ``[0, 0]``, the whole D axis.  Returns None; x is rewritten on
    ``stream`` (default: the current stream of x's device).
    """
    _run(*_inplace_args(x, cos, sin, rotary_mode, partial_slice, stream, False))


def rope_inplace_partial_backward(grad: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, rotary_mode=1,
                                  partial_slice: Optional[Sequence[int]] = None, stream=None) -> None:
    """Backward of :func:`rope_inplace_partial`: turns dL/dy in ``grad`` into
    dL/dx in place."""
    _run(*_inplace_args(grad, cos, sin, rotary_mode, partial_slice, stream, True))


def rope_with_sin_cos_cache(positions: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                            cos_sin_cache: torch.Tensor, head_size: int, rotary_dim: Optional[int] = None,
                            is_neox: bool = True, mrope_section: Optional[Sequence[int]] = None,
                            stream=None, *, cache_mode: int = 0, query_out: Optional[torch.Tensor] = None,
                            key_out: Optional[torch.Tensor] = None) -> None:
    """Cache-indexed RoPE of ``query`` and ``key`` (rope or mrope mode).

    In place unless ``query_out``/``key_out`` are given.  ``query``/``key`` may
    be strided row views (e.g. slices of a fused QKV tensor); ``cache_mode=1``
    selects the interleaved mrope splice.  Contiguous in-place calls with
    ``cache_mode=0`` use the V1 entry point, everything else the V2 one."""
    _run(*_cache_args(positions, query, key, cos_sin_cache, head_size, rotary_dim, is_neox, mrope_section, stream,
                      cache_mode, query_out, key_out))


def _cache_args(positions, query, key, cos_sin_cache, head_size, rotary_dim, is_neox, mrope_section, stream,
                cache_mode, query_out, key_out):
    """(C function, its arguments, objects to keep alive, name) of one
    cache-operator call: the V1 entry point for a contiguous in-place call with
    cache_mode 0, else V2."""
    lib = load()
    R = int(cos_sin_cache.shape[1]) if rotary_dim is None else int(rotary_dim)
    _one_device(query, key, positions, cos_sin_cache, query_out, key_out)
    dq, qs = rows_desc(query)
    dk, ks = rows_desc(key)
    dp, dc = tensor_desc(positions), tensor_desc(cos_sin_cache)
    sec = None
    n_sec = 0
    if mrope_section is not None:
        n_sec = len(mrope_section)
        sec = (ctypes.c_int64 * max(1, n_sec))(*[int(v) for v in mrope_section])
    handle = _stream_handle(query, stream)
    contiguous = qs == query.shape[1] and ks == key.shape[1]
    if cache_mode == 0 and query_out is None and key_out is None and contiguous:
        args = (ctypes.byref(dp), ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dc), int(head_size), R,
                1 if is_neox else 0, sec, n_sec, handle)
        return (lib.rope_with_sin_cos_cache, args, (positions, query, key, cos_sin_cache, dp, dq, dk, dc, sec),
                "rope_with_sin_cos_cache")
    dqo = tensor_desc(query_out) if query_out is not None else None
    dko = tensor_desc(key_out) if key_out is not None else None
    args = (ctypes.byref(dp), ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dc), int(head_size), R,
            1 if is_neox else 0, sec, n_sec, int(cache_mode), qs, ks,
            ctypes.byref(dqo) if dqo is not None else None, ctypes.byref(dko) if dko is not None else None, handle)
    return (lib.rope_with_sin_cos_cache_v2, args,
            (positions, query, key, cos_sin_cache, query_out, key_out, dp, dq, dk, dc, dqo, dko, sec),
            "rope_with_sin_cos_cache_v2")


def _qkv_args(qkv, num_q_heads, num_k_heads, num_v_heads, q_gamma, k_gamma, eps, cos_sin_cache, seq_lens,
              query_start_loc, slot_mapping, q_out, k_cache, v_cache, stream):
    tensors = (qkv, q_gamma, k_gamma, cos_sin_cache, seq_lens, query_start_loc, slot_mapping, q_out, k_cache,
               v_cache)
    _one_device(*tensors)
    descs = [tensor_desc(t) for t in tensors]
    r = [ctypes.byref(d) for d in descs]
    args = (r[0], int(num_q_heads), int(num_k_heads), int(num_v_heads), r[1], r[2], float(eps), r[3], r[4], r[5],
            r[6], r[7], r[8], r[9], _stream_handle(qkv, stream))
    return args, descs


def qkv_rmsnorm_rope_cache(qkv: torch.Tensor, num_q_heads: int, num_k_heads: int, num_v_heads: int,
                           q_gamma: torch.Tensor, k_gamma: torch.Tensor, eps: float, cos_sin_cache: torch.Tensor,
                           seq_lens: torch.Tensor, query_start_loc: torch.Tensor, slot_mapping: torch.Tensor,
                           q_out: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """Fused QKV split + RMSNorm + RoPE + paged KV-cache write (see the C header)."""
    lib = load()
    args, _ = _qkv_args(qkv, num_q_heads, num_k_heads, num_v_heads, q_gamma, k_gamma, eps, cos_sin_cache,
                        seq_lens, query_start_loc, slot_mapping, q_out, k_cache, v_cache, stream)
    _run(lib.rope_qkv_rmsnorm_rope_cache, args, (qkv,), "rope_qkv_rmsnorm_rope_cache")


def prepare_qkv_rmsnorm_rope_cache(qkv: torch.Tensor, num_q_heads: int, num_k_heads: int, num_v_heads: int,
                                   q_gamma: torch.Tensor, k_gamma: torch.Tensor, eps: float,
                                   cos_sin_cache: torch.Tensor, seq_lens: torch.Tensor,
                                   query_start_loc: torch.Tensor, slot_mapping: torch.Tensor, q_out: torch.Tensor,
                                   k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> "PreparedCall":
    """:func:`qkv_rmsnorm_rope_cache` with its arguments marshalled once."""
    lib = load()
    tensors = (qkv, q_gamma, k_gamma, cos_sin_cache, seq_lens, query_start_loc, slot_mapping, q_out, k_cache,
               v_cache)
    args, descs = _qkv_args(qkv, num_q_heads, num_k_heads, num_v_heads, q_gamma, k_gamma, eps, cos_sin_cache,
                            seq_lens, query_start_loc, slot_mapping, q_out, k_cache, v_cache, stream)
    return PreparedCall(lib.rope_qkv_rmsnorm_rope_cache, args, (tensors, descs), "rope_qkv_rmsnorm_rope_cache")


# ---------------------------------------------------------------------------
# Scaled rotary tables, append to a paged cache, attention over it: marshalled
# by the compiled binding.
# ---------------------------------------------------------------------------
_binding = None


def _load_binding():
    global _binding
    if _binding is None:
        from . import build as B

        load()  # the library first: it says how to build both
        path = B.BINDING_PATH
        if B.binding_built_for() != B.binding_target():
            raise RuntimeError("%s is not built for this Python and torch; run "
                               "`python -m transformer_rope_positional_gb300.build%s`"
                               % (path, " --debug" if DEBUG_BOUNDS else ""))
        loader = importlib.machinery.ExtensionFileLoader("rope_binding", path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("rope_binding", loader))
        loader.exec_module(module)
        module.init(LIB_PATH)
        _binding = module
    return _binding


def _issue(name, args, like, stream, what) -> None:
    """Call the binding's function on ``args`` and the stream, with the device of ``like`` current."""
    dev = like.get_device()
    if dev < 0:
        raise ValueError("expected a CUDA tensor, got one on %s" % like.device)
    fn = getattr(_binding or _load_binding(), name)
    if stream is None and _raw_current_stream is not None and _current_device() == dev:
        st = fn(*args, _raw_current_stream(dev))
    else:
        st = _on_device(dev, fn, args + (_stream_handle(like, stream),))
    if st != ROPE_OK:
        raise RopeError(st, what)


SCALINGS = {"none": 0, "linear": 1, "base": 2, "yarn": 3, "wavelength": 4, "factors": 5}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: Optional[dict] = None):
    """``(inv_freq, scale)``: the rotary_dim / 2 frequencies (a float64 CPU
    tensor, radians per position) and the factor of cos and sin, changed for
    long contexts as ``scaling`` says.

    ``scaling`` is None or a dict with ``kind`` one of "none", "linear", "base",
    "yarn", "wavelength", "factors" and that kind's ``factor``,
    ``original_length``, ``low``, ``high``, ``attention`` and ``factors``; the
    formulas are those of ``rope_scaled_frequencies`` in the C header."""
    what = "rope_scaled_frequencies"
    fn = (_binding or _load_binding()).frequencies
    inv = torch.empty(min(max(1, int(rotary_dim) // 2), 1024), dtype=torch.float64, device="cpu")
    if scaling is None:
        st, scale = fn(rotary_dim, base, -1, 0.0, 0.0, 0.0, 0.0, 0.0, None, inv)
    else:
        get = scaling.get
        if get("kind") not in SCALINGS or not _SCALING_KEYS.issuperset(scaling):
            raise RopeError(ROPE_ERR_PARAM_INVALID, "%s: scaling %r" % (what, scaling))
        factors = get("factors")
        if factors is not None:
            factors = torch.as_tensor(factors, dtype=torch.float64, device="cpu").contiguous()
        st, scale = fn(rotary_dim, base, SCALINGS[scaling["kind"]], get("factor", 0.0), get("original_length", 0.0),
                       get("low", 0.0), get("high", 0.0), get("attention", 0.0), factors, inv)
    if st != ROPE_OK:
        raise RopeError(st, what)
    return inv, scale


_SCALING_KEYS = frozenset(("kind", "factor", "original_length", "low", "high", "attention", "factors"))


def _host_frequencies(inv_freq) -> torch.Tensor:
    if not isinstance(inv_freq, torch.Tensor):
        return torch.tensor(list(inv_freq), dtype=torch.float64, device="cpu")
    if inv_freq.dtype == torch.float64:
        return inv_freq.contiguous()
    if inv_freq.is_cuda:
        raise ValueError("expected frequencies on the host, got a tensor on %s" % inv_freq.device)
    return inv_freq.to(torch.float64).contiguous()


def scaled_cos_sin_cache(cache: torch.Tensor, inv_freq, scale: float = 1.0, *,
                         positions: Optional[torch.Tensor] = None, first_position: int = 0, stream=None) -> None:
    """Writes ``cache`` [rows, 2F], the cos/sin table of the cache-indexed
    operators: row r is position ``first_position + (positions[r] or r)``, cos in
    the first half and sin in the second, times ``scale``.  ``inv_freq`` holds the
    F frequencies on the host (see :func:`rope_frequencies`)."""
    _issue("scaled_cos_sin_cache", (_host_frequencies(inv_freq), scale, positions, first_position, cache), cache,
           stream, "rope_scaled_cos_sin_cache")


def scaled_cos_sin(cos: torch.Tensor, sin: torch.Tensor, inv_freq, scale: float = 1.0, rotary_mode=1, *,
                   positions: Optional[torch.Tensor] = None, first_position: int = 0, stream=None) -> None:
    """Writes ``cos`` and ``sin`` [..., 2F] as the in-place operator reads them
    (e.g. [1, S, 1, 2F]), in the element order of ``rotary_mode``; rows and
    positions as in :func:`scaled_cos_sin_cache`."""
    _issue("scaled_cos_sin", (_host_frequencies(inv_freq), scale, positions, first_position, _mode(rotary_mode), cos,
                              sin), cos, stream, "rope_scaled_cos_sin")


def append_paged_kv(positions: torch.Tensor, query: Optional[torch.Tensor], key: torch.Tensor, value: torch.Tensor,
                    cos_sin_cache: torch.Tensor, slot_mapping: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, head_size: int, rotary_dim: Optional[int] = None, is_neox: bool = True,
                    mrope_section: Optional[Sequence[int]] = None, stream=None, *, cache_mode: int = 0,
                    query_out: Optional[torch.Tensor] = None) -> None:
    """RoPE of ``query`` and ``key``; query to ``query_out`` (None: in place),
    key and value to their slots of the paged caches [blocks, heads, block
    size, head_size] (see the C header).  ``query``, ``key`` and ``value`` may be
    column ranges of one fused buffer; the slots >= 0 of a call are distinct."""
    _issue("append_paged_kv", (positions, query, key, value, cos_sin_cache, slot_mapping, query_out, k_cache, v_cache,
                               head_size, rotary_dim, is_neox, mrope_section, cache_mode), key, stream,
           "rope_append_paged_kv")


def prepare_append_paged_kv(positions: torch.Tensor, query: Optional[torch.Tensor], key: torch.Tensor,
                            value: torch.Tensor, cos_sin_cache: torch.Tensor, slot_mapping: torch.Tensor,
                            k_cache: torch.Tensor, v_cache: torch.Tensor, head_size: int,
                            rotary_dim: Optional[int] = None, is_neox: bool = True,
                            mrope_section: Optional[Sequence[int]] = None, stream=None, *, cache_mode: int = 0,
                            query_out: Optional[torch.Tensor] = None) -> "PreparedCall":
    """:func:`append_paged_kv` as a call to be issued many times, on the stream of now."""
    args = (positions, query, key, value, cos_sin_cache, slot_mapping, query_out, k_cache, v_cache, head_size,
            rotary_dim, is_neox, None if mrope_section is None else tuple(mrope_section), cache_mode,
            _stream_handle(key, stream))
    return PreparedCall(_load_binding().append_paged_kv, args, (key,), "rope_append_paged_kv")


def paged_attention_workspace(query: torch.Tensor, k_cache: torch.Tensor, prefix_len: int = 0) -> int:
    """Bytes of workspace that :func:`paged_attention` (or, for a cache of codes, :func:`paged_attention_8bit`) needs."""
    n = _on_device(query.get_device(), _load_binding().attention_workspace, (query, k_cache, prefix_len))
    if n < 0:
        raise RopeError(ROPE_ERR_PARAM_INVALID, "rope_paged_attention_workspace")
    return n


def _workspace_for(query, k_cache, prefix_len, stream) -> torch.Tensor:
    """A workspace whose memory belongs to the stream that the call runs on, so
    that it is not handed out again while the call still uses it."""
    nbytes = paged_attention_workspace(query, k_cache, prefix_len)
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=query.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=query.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=query.device)


def _default_scale(k_cache) -> float:
    D = k_cache.shape[-1] if k_cache.dim() else 0
    return D ** -0.5 if D else 1.0  # (heads of no columns are refused by the call)


def paged_attention(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, query_start_loc: torch.Tensor, out: torch.Tensor, *,
                    scale: Optional[float] = None, prefix_blocks: Optional[torch.Tensor] = None, prefix_len: int = 0,
                    lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Causal attention of the batch's new tokens ``query`` [T, Nq*D] over the
    paged caches [blocks, Nk, block size, D] into ``out`` (see the C header).

    ``seq_lens`` counts each sequence's tokens with the shared prefix and this
    call's; ``block_table`` [B, W] holds the pages after the prefix,
    ``prefix_blocks`` those of the ``prefix_len`` tokens that all sequences
    share.  ``scale`` defaults to D ** -0.5; ``lse`` [T, Nq] (float32) receives
    each row's log-sum-exp.  Without ``workspace`` one is allocated for the call
    on its stream."""
    if scale is None:
        scale = _default_scale(k_cache)
    if workspace is None and stream is not None:
        _stream_handle(query, stream)  # its device is the tensors'
        workspace = _workspace_for(query, k_cache, prefix_len, stream)
    _issue("paged_attention", (query, k_cache, v_cache, block_table, seq_lens, query_start_loc, prefix_blocks,
                               prefix_len, scale, out, lse, workspace), query, stream, "rope_paged_attention")


def prepare_paged_attention(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                            block_table: torch.Tensor, seq_lens: torch.Tensor, query_start_loc: torch.Tensor,
                            out: torch.Tensor, *, scale: Optional[float] = None,
                            prefix_blocks: Optional[torch.Tensor] = None, prefix_len: int = 0,
                            lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> "PreparedCall":
    """:func:`paged_attention` as a call to be issued many times, on the stream of
    now, with its workspace (given or allocated here) kept."""
    handle = _stream_handle(query, stream)
    if scale is None:
        scale = _default_scale(k_cache)
    if workspace is None:
        workspace = _workspace_for(query, k_cache, prefix_len, stream)
    args = (query, k_cache, v_cache, block_table, seq_lens, query_start_loc, prefix_blocks, prefix_len, scale, out,
            lse, workspace, handle)
    return PreparedCall(_load_binding().paged_attention, args, (query,), "rope_paged_attention")


def append_paged_kv_8bit(positions: torch.Tensor, query: Optional[torch.Tensor], key: torch.Tensor,
                         value: torch.Tensor, cos_sin_cache: torch.Tensor, slot_mapping: torch.Tensor,
                         k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                         head_size: int, rotary_dim: Optional[int] = None, is_neox: bool = True,
                         mrope_section: Optional[Sequence[int]] = None, stream=None, *, cache_mode: int = 0,
                         query_out: Optional[torch.Tensor] = None) -> None:
    """:func:`append_paged_kv` to caches of 8-bit codes (float8_e4m3fn) with a power of two (float8_e8m0fnu
    [blocks, heads, S]) for each of the S blocks of tokens of a page and head (see the C header).  The tokens of
    one such block stand one after the other in the call, in the order of their slots."""
    _issue("append_paged_kv_8bit", (positions, query, key, value, cos_sin_cache, slot_mapping, query_out, k_cache,
                                    v_cache, k_scale, v_scale, head_size, rotary_dim, is_neox, mrope_section,
                                    cache_mode), key, stream, "rope_append_paged_kv_8bit")


def prepare_append_paged_kv_8bit(positions: torch.Tensor, query: Optional[torch.Tensor], key: torch.Tensor,
                                 value: torch.Tensor, cos_sin_cache: torch.Tensor, slot_mapping: torch.Tensor,
                                 k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                                 v_scale: torch.Tensor, head_size: int, rotary_dim: Optional[int] = None,
                                 is_neox: bool = True, mrope_section: Optional[Sequence[int]] = None, stream=None, *,
                                 cache_mode: int = 0, query_out: Optional[torch.Tensor] = None) -> "PreparedCall":
    """:func:`append_paged_kv_8bit` as a call to be issued many times, on the stream of now."""
    args = (positions, query, key, value, cos_sin_cache, slot_mapping, query_out, k_cache, v_cache, k_scale, v_scale,
            head_size, rotary_dim, is_neox, None if mrope_section is None else tuple(mrope_section), cache_mode,
            _stream_handle(key, stream))
    return PreparedCall(_load_binding().append_paged_kv_8bit, args, (key,), "rope_append_paged_kv_8bit")


def paged_attention_8bit(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                         query_start_loc: torch.Tensor, out: torch.Tensor, *, scale: Optional[float] = None,
                         prefix_blocks: Optional[torch.Tensor] = None, prefix_len: int = 0,
                         lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """:func:`paged_attention` over caches of 8-bit codes with their scales (see :func:`append_paged_kv_8bit`);
    :func:`paged_attention_workspace` knows such caches by their type."""
    if scale is None:
        scale = _default_scale(k_cache)
    if workspace is None and stream is not None:
        _stream_handle(query, stream)  # its device is the tensors'
        workspace = _workspace_for(query, k_cache, prefix_len, stream)
    _issue("paged_attention_8bit", (query, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start_loc,
                                    prefix_blocks, prefix_len, scale, out, lse, workspace), query, stream,
           "rope_paged_attention_8bit")


def prepare_paged_attention_8bit(query: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                 k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                                 seq_lens: torch.Tensor, query_start_loc: torch.Tensor, out: torch.Tensor, *,
                                 scale: Optional[float] = None, prefix_blocks: Optional[torch.Tensor] = None,
                                 prefix_len: int = 0, lse: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None, stream=None) -> "PreparedCall":
    """:func:`paged_attention_8bit` as a call to be issued many times, on the stream of now, with its workspace
    (given or allocated here) kept."""
    handle = _stream_handle(query, stream)
    if scale is None:
        scale = _default_scale(k_cache)
    if workspace is None:
        workspace = _workspace_for(query, k_cache, prefix_len, stream)
    args = (query, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start_loc, prefix_blocks,
            prefix_len, scale, out, lse, workspace, handle)
    return PreparedCall(_load_binding().paged_attention_8bit, args, (query,), "rope_paged_attention_8bit")


def rearrange_sequences(block_table: torch.Tensor, seq_lens: torch.Tensor, ref_counts: torch.Tensor,
                        parents: torch.Tensor, new_block_table: torch.Tensor, new_seq_lens: torch.Tensor,
                        new_ref_counts: torch.Tensor, copy_src: torch.Tensor, copy_dst: torch.Tensor,
                        counts: torch.Tensor, block_size: int, *, room: Optional[torch.Tensor] = None,
                        prefix_len: int = 0, stream=None) -> None:
    """A new batch of the old one's sequences: row i continues old row ``parents[i]`` (-1: starts empty), with room
    for ``room[i]`` more tokens.  A parent of several rows is forked, one of none is dropped.

    Whole pages are shared (``ref_counts`` [blocks], int32, counts the holders of each; ``new_ref_counts`` may be the
    same tensor); a page that is written on is kept by one row and copied for the others: (``copy_src``, ``copy_dst``)
    [rows] name the pages that :func:`copy_pages` has to copy then, ``counts`` [2] how many pairs there are and how
    many pages are left free.  Free pages are given out lowest first (see the C header)."""
    _issue("rearrange_sequences", (block_table, seq_lens, ref_counts, parents, room, new_block_table, new_seq_lens,
                                   new_ref_counts, copy_src, copy_dst, counts, block_size, prefix_len), block_table,
           stream, "rope_rearrange_sequences")


def compact_pages(block_table: torch.Tensor, seq_lens: torch.Tensor, ref_counts: torch.Tensor,
                  new_block_table: torch.Tensor, new_ref_counts: torch.Tensor, copy_src: torch.Tensor,
                  copy_dst: torch.Tensor, counts: torch.Tensor, block_size: int, *,
                  prefix_blocks: Optional[torch.Tensor] = None, new_prefix_blocks: Optional[torch.Tensor] = None,
                  prefix_len: int = 0, stream=None) -> None:
    """Tables, counts and prefix for a cache whose live pages are moved to the front, and in ``copy_src`` and
    ``copy_dst`` (at least blocks / 2 elements) the pages that :func:`copy_pages` has to move for it; ``counts`` [2]
    receives their number and that of live pages.  Each new tensor may be the old one."""
    _issue("compact_pages", (block_table, seq_lens, ref_counts, prefix_blocks, new_block_table, new_ref_counts,
                             new_prefix_blocks, copy_src, copy_dst, counts, block_size, prefix_len), block_table, stream,
           "rope_compact_pages")


def copy_pages(src: torch.Tensor, dst: torch.Tensor, tensors: Sequence[torch.Tensor], *,
               count: Optional[torch.Tensor] = None, stream=None) -> None:
    """Page ``src[i]`` of every tensor (caches and scales of any layers, of any type, pages first) to its page
    ``dst[i]``, for the first ``count[0]`` pairs or all; pairs with a negative number are passed over."""
    _issue("copy_pages", (src, dst, count, tensors if isinstance(tensors, (list, tuple)) else list(tensors)), src,
           stream, "rope_copy_pages")


def get_device_error(stream=None, device=None) -> int:
    """Synchronise ``stream`` and read-and-clear the error word of its device
    (``device``, else the stream's device, else the current device)."""
    lib = load()
    if device is None and stream is not None and hasattr(stream, "device"):
        device = stream.device
    dev = device if isinstance(device, int) else torch.device(device).index if device is not None else None
    if dev is None:
        dev = torch.cuda.current_device()
    with torch.cuda.device(dev):
        if stream is None:
            stream = torch.cuda.current_stream(dev)
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        code = ctypes.c_int32(0)
        st = lib.rope_get_device_error(handle, ctypes.byref(code))
    if st != ROPE_OK:
        raise RopeError(st, "rope_get_device_error")
    return int(code.value)


def launch_count() -> int:
    return int(load().rope_launch_count())


class PreparedCall:
    """One operator call with its C arguments marshalled once.

    Calling it re-issues the same launch on the same tensors and the same
    stream (the one given, or the current one, when it was prepared), for
    loops that apply the operator many times; it keeps the tensors alive.
    """

    def __init__(self, fn, args, keep, what):
        self._fn = fn
        self._args = args
        self._keep = keep
        self._what = what
        first = keep[0]
        while isinstance(first, (tuple, list)):
            first = first[0]
        self._device = first.get_device()

    def __call__(self) -> None:
        st = _on_device(self._device, self._fn, self._args)
        if st != ROPE_OK:
            raise RopeError(st, self._what)


def prepare_inplace_partial(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, rotary_mode=1,
                            partial_slice: Optional[Sequence[int]] = None, stream=None,
                            backward: bool = False) -> PreparedCall:
    """:func:`rope_inplace_partial` (or its backward) with its arguments marshalled once."""
    return PreparedCall(*_inplace_args(x, cos, sin, rotary_mode, partial_slice, stream, backward))


def prepare_with_sin_cos_cache(positions: torch.Tensor, query: torch.Tensor, key: torch.Tensor,
                               cos_sin_cache: torch.Tensor, head_size: int, rotary_dim: Optional[int] = None,
                               is_neox: bool = True, mrope_section: Optional[Sequence[int]] = None,
                               stream=None, *, cache_mode: int = 0, query_out: Optional[torch.Tensor] = None,
                               key_out: Optional[torch.Tensor] = None) -> PreparedCall:
    """:func:`rope_with_sin_cos_cache` with its arguments marshalled once."""
    return PreparedCall(*_cache_args(positions, query, key, cos_sin_cache, head_size, rotary_dim, is_neox,
                                     mrope_section, stream, cache_mode, query_out, key_out))

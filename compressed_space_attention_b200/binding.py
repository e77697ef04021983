"""ctypes binding of libisoq (``include/isoq.h``): argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors
provide device memory and strides; the current torch CUDA stream of the
tensors' device is passed as the stream, or the one that ``stream`` names (a
torch stream or its handle).  What a call allocates belongs to the stream that
it launches on, as under ``torch.cuda.stream``; ordering that stream with the
ones that write the inputs and read the outputs is the caller's, as there.
All computation happens in the library's CUDA kernels: there is no CPU or
Python fallback, and a missing library raises at import of this module's
functions.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional, Tuple

import numpy as np

ISOQ_OK = 0
ISOQ_ERR_INVALID_ARG = -1
ISOQ_ERR_UNSUPPORTED = -2
ISOQ_ERR_CUDA = -3
ISOQ_ERR_TIMEOUT = -4
ISOQ_FULL = 0
ISOQ_FAST = 1
ISOQ_PLANAR = 2
ISOQ_BLOCK_SO4 = 3
ISOQ_SO3 = 4
ISOQ_F16 = 0
ISOQ_F32 = 1

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libisoq.so")

# (name, restype, argtypes) of every exported entry point of include/isoq.h.
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
SIGNATURES = [
    ("isoq_status_string", ctypes.c_char_p, [_I]),
    ("isoq_last_error", ctypes.c_char_p, []),
    ("isoq_abi_version", _I, []),
    ("isoq_params_size", _I, [_I]),
    ("isoq_packed_bytes", _SZ, [_I, _I]),
    ("isoq_make_params", _I, [_I, _I, ctypes.c_uint64, _I, _P]),
    ("isoq_make_codebook", _I, [_I, _I, _P, _P]),
    ("isoq_quantize", _I, [_P, _I, _I, _I64, _I, _I, _I, _I64, _I64, _P, _P, _P, _I64, _P]),
    ("isoq_dequantize", _I, [_P, _P, _I, _I64, _I, _I, _I, _I64, _P, _P, _I, _I64, _I64, _P]),
    ("isoq_decode_num_splits", _I, [_I, _I, _I64, _I]),
    ("isoq_decode_workspace_size", _SZ, [_I, _I, _I, _I64, _I]),
    ("isoq_decode_attention", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _I, _I,
                                   _P, _P, _F, _P, _P, _SZ, _P]),
    ("isoq_decode_split", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _I, _I, _P,
                               _F, _P, _SZ, _P]),
    ("isoq_decode_combine", _I, [_I, _P, _I, _I, _I, _I64, _I, _I, _P, _P, _P, _SZ, _P]),
    ("isoq_decode_append", _I, [_P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I64, _I, _I, _I, _P, _P, _P]),
    ("isoq_decode_step", _I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _I, _I, _P, _P,
                              _F, _P, _P, _SZ, _P]),
    ("isoq_check_device_error", _I, [_P]),
    ("isoq_selftest_wait_timeout", _I, [ctypes.c_uint64, _P]),
    ("isoq_prefill_attention", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I, _I, _I,
                                    _P, _P, _F, _P, _P]),
    ("isoq_rotor_groups", _I, [_I]),
    ("isoq_rotor_packed_bytes", _SZ, [_I, _I]),
    ("isoq_rotor_make_params", _I, [_I, ctypes.c_uint64, _I, _P]),
    ("isoq_rotor_quantize", _I, [_P, _I, _I, _I64, _I, _I, _I64, _I64, _P, _P, _P, _I64, _P]),
    ("isoq_rotor_dequantize", _I, [_P, _P, _I, _I64, _I, _I, _I64, _P, _P, _I, _I64, _I64, _P]),
    ("isoq_decode_static_workspace_bytes", _SZ, []),
    ("isoq_decode_attention_static", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _I,
                                          _I, _P, _P, _F, _P, _P]),
    ("isoq_decode_window_workspace_size", _SZ, [_I, _I, _I, _I64, _I, _I64, _I64]),
    ("isoq_decode_attention_window", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I64, _I, _I, _I, _P, _P, _F,
                                          _I64, _I64, _P, _P, _SZ, _P]),
    ("isoq_prefill_attention_window", _I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I, _I, _I, _P, _P,
                                           _F, _I64, _I64, _P, _P]),
    ("isoq_decode_prefix_workspace_size", _SZ, [_I, _I, _I, _I64, _I64, _I]),
    ("isoq_decode_attention_prefix", _I, [_P, _I, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _I, _I, _I,
                                          _I64, _I, _I, _I, _P, _P, _F, _P, _P, _SZ, _P]),
    ("isoq_build_block_tables", _I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _I64, _P, _P, _P, _P, _P]),
    ("isoq_paged_append", _I, [_P, _P, _I, _P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    ("isoq_paged_decode_attention", _I, [_P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I64, _I, _I, _I,
                                         _P, _P, _F, _I64, _I64, _P, _P, _SZ, _P]),
]

_lib = None


class IsoqError(RuntimeError):
    """A non-zero status from libisoq."""

    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status}): {detail}")


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m compressed_space_attention_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().isoq_status_string(status).decode()


def last_error() -> str:
    return lib().isoq_last_error().decode()


def _check(status: int, where: str) -> None:
    if status != ISOQ_OK:
        raise IsoqError(status, where, last_error())


# ---------------------------------------------------------------------------
# Host-only entry points
# ---------------------------------------------------------------------------

def isoq_abi_version() -> int:
    return lib().isoq_abi_version()


def isoq_params_size(d: int) -> int:
    return lib().isoq_params_size(d)


def isoq_packed_bytes(d: int, bits: int) -> int:
    return lib().isoq_packed_bytes(d, bits)


def isoq_make_params(d: int, variant: int, seed: int, n_heads: int = 1) -> np.ndarray:
    """float32 [n_heads][d/4][8] rotation parameters (host array)."""
    out = np.empty((n_heads, d // 4, 8), dtype=np.float32)
    _check(lib().isoq_make_params(d, variant, ctypes.c_uint64(seed & (2 ** 64 - 1)), n_heads,
                                  out.ctypes.data_as(_P)), "isoq_make_params")
    return out


def isoq_make_codebook(d: int, bits: int) -> Tuple[np.ndarray, np.ndarray]:
    """(centroids[2^bits], thresholds[2^bits - 1]) as float64 host arrays."""
    c = np.empty(1 << bits, dtype=np.float64)
    t = np.empty((1 << bits) - 1, dtype=np.float64)
    _check(lib().isoq_make_codebook(d, bits, c.ctypes.data_as(_P), t.ctypes.data_as(_P)),
           "isoq_make_codebook")
    return c, t


def isoq_decode_num_splits(B: int, Hkv: int, Tmax: int, d: int) -> int:
    n = lib().isoq_decode_num_splits(B, Hkv, Tmax, d)
    if n < 0:
        raise IsoqError(n, "isoq_decode_num_splits", "")
    return n


def isoq_decode_workspace_size(B: int, Hq: int, Hkv: int, Tmax: int, d: int) -> int:
    return lib().isoq_decode_workspace_size(B, Hq, Hkv, Tmax, d)


# ---------------------------------------------------------------------------
# Device entry points (torch tensors)
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return ISOQ_F16
    if t.dtype == torch.float32:
        return ISOQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}; float16 or float32 expected")


def _torch_dtype(code: int):
    torch = _torch()
    return torch.float16 if code == ISOQ_F16 else torch.float32


def _require_cuda(*tensors):
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libisoq entry points take CUDA tensors (there is no CPU path)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def _stream(dev, stream=None) -> int:
    torch = _torch()
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _empty(shape, dtype, dev, stream=None):
    """torch.empty from the pool of the stream that the call launches on.  From
    another stream's pool the memory could be handed out again as soon as the
    call has returned, or still be in use there, while the kernels work on it."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(dev, stream)
        stream = torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def isoq_quantize(x, params, bits: int, variant: int, codes=None, norms=None,
                  out_head_stride: Optional[int] = None, stream=None):
    """Compresses x [n_heads][n_vec][d] (or [n_vec][d]); returns (codes, norms).

    codes: uint8 [n_heads][n_vec][d*bits/8]; norms: float16 [n_heads][n_vec].
    Preallocated outputs may be views into a larger cache: pass
    ``out_head_stride`` (vectors between heads) for that.
    """
    torch = _torch()
    if x.dim() == 2:
        x = x.unsqueeze(0)
    n_heads, n_vec, d = x.shape
    if x.stride(2) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    dev = _require_cuda(x, params, codes, norms)
    pb = isoq_packed_bytes(d, bits)
    if codes is None:
        codes = _empty((n_heads, n_vec, pb), torch.uint8, dev, stream)
    if norms is None:
        norms = _empty((n_heads, n_vec), torch.float16, dev, stream)
    if out_head_stride is None:
        out_head_stride = n_vec
    with torch.cuda.device(dev):
        st = lib().isoq_quantize(_ptr(x), _dtype_code(x), n_heads, n_vec, d, bits, variant,
                                 x.stride(0), x.stride(1), _ptr(params), _ptr(codes), _ptr(norms),
                                 out_head_stride, _stream(dev, stream))
    _check(st, "isoq_quantize")
    return codes, norms


def isoq_dequantize(codes, norms, params, d: int, bits: int, variant: int, out_dtype=None,
                    out=None, in_head_stride: Optional[int] = None, stream=None):
    """Reconstructs [n_heads][n_vec][d] vectors from codes and float16 norms."""
    torch = _torch()
    if codes.dim() == 2:
        codes = codes.unsqueeze(0)
        norms = norms.unsqueeze(0)
    n_heads, n_vec, _ = codes.shape
    dev = _require_cuda(codes, norms, params, out)
    if out is None:
        out = _empty((n_heads, n_vec, d), out_dtype or torch.float32, dev, stream)
    if in_head_stride is None:
        in_head_stride = n_vec
    with torch.cuda.device(dev):
        st = lib().isoq_dequantize(_ptr(codes), _ptr(norms), n_heads, n_vec, d, bits, variant,
                                   in_head_stride, _ptr(params), _ptr(out), _dtype_code(out),
                                   out.stride(0), out.stride(1), _stream(dev, stream))
    _check(st, "isoq_dequantize")
    return out


def isoq_prefill_attention(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v,
                           bits: int, variant: int, scale: Optional[float] = None, out=None, stream=None):
    """Causal attention of q [B][Tq][Hq][d] over the packed cache that holds
    the chunk (seq_lens counts it); returns out [B][Tq][Hq][d] (dtype of q)."""
    torch = _torch()
    B, Tq, Hq, d = q.shape
    _, Hkv, Tmax, pb = packed_k.shape
    if pb != isoq_packed_bytes(d, bits):
        raise ValueError("packed row size does not match d and bits")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    dev = _require_cuda(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, out)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, Tq, Hq, d), q.dtype, dev, stream)
    with torch.cuda.device(dev):
        st = lib().isoq_prefill_attention(
            _ptr(q), _dtype_code(q), _ptr(packed_k), _ptr(packed_v), _ptr(norms_k), _ptr(norms_v),
            _ptr(seq_lens), B, Tq, Hq, Hkv, Tmax, d, bits, variant, _ptr(params_k), _ptr(params_v),
            float(scale), _ptr(out), _stream(dev, stream))
    _check(st, "isoq_prefill_attention")
    return out


def isoq_rotor_groups(d: int) -> int:
    return lib().isoq_rotor_groups(d)


def isoq_rotor_packed_bytes(d: int, bits: int) -> int:
    return lib().isoq_rotor_packed_bytes(d, bits)


def isoq_rotor_make_params(d: int, seed: int, n_heads: int = 1) -> np.ndarray:
    """float32 [n_heads][G][4] unit rotors (s, p12, p13, p23) (host array)."""
    out = np.empty((n_heads, max(isoq_rotor_groups(d), 0), 4), dtype=np.float32)
    _check(lib().isoq_rotor_make_params(d, ctypes.c_uint64(seed & (2 ** 64 - 1)), n_heads,
                                        out.ctypes.data_as(_P)), "isoq_rotor_make_params")
    return out


def isoq_rotor_quantize(x, rotors, bits: int, codes=None, norms=None, stream=None):
    """RotorQuant comparator: compresses x [n_heads][n_vec][d]; returns (codes, norms)."""
    torch = _torch()
    if x.dim() == 2:
        x = x.unsqueeze(0)
    n_heads, n_vec, d = x.shape
    if x.stride(2) != 1:
        raise ValueError("the last dimension of x must be contiguous")
    dev = _require_cuda(x, rotors, codes, norms)
    if codes is None:
        codes = _empty((n_heads, n_vec, isoq_rotor_packed_bytes(d, bits)), torch.uint8, dev, stream)
    if norms is None:
        norms = _empty((n_heads, n_vec), torch.float16, dev, stream)
    with torch.cuda.device(dev):
        st = lib().isoq_rotor_quantize(_ptr(x), _dtype_code(x), n_heads, n_vec, d, bits, x.stride(0),
                                       x.stride(1), _ptr(rotors), _ptr(codes), _ptr(norms), n_vec,
                                       _stream(dev, stream))
    _check(st, "isoq_rotor_quantize")
    return codes, norms


def isoq_rotor_dequantize(codes, norms, rotors, d: int, bits: int, out_dtype=None, out=None, stream=None):
    """RotorQuant comparator: reconstructs [n_heads][n_vec][d] from codes and norms."""
    torch = _torch()
    if codes.dim() == 2:
        codes = codes.unsqueeze(0)
        norms = norms.unsqueeze(0)
    n_heads, n_vec, _ = codes.shape
    dev = _require_cuda(codes, norms, rotors, out)
    if out is None:
        out = _empty((n_heads, n_vec, d), out_dtype or torch.float32, dev, stream)
    with torch.cuda.device(dev):
        st = lib().isoq_rotor_dequantize(_ptr(codes), _ptr(norms), n_heads, n_vec, d, bits, n_vec,
                                         _ptr(rotors), _ptr(out), _dtype_code(out), out.stride(0),
                                         out.stride(1), _stream(dev, stream))
    _check(st, "isoq_rotor_dequantize")
    return out


def _decode_shapes(q, packed_k, bits):
    B, Hq, d = q.shape
    _, Hkv, Tmax, pb = packed_k.shape
    if pb != isoq_packed_bytes(d, bits):
        raise ValueError("packed row size does not match d and bits")
    return B, Hq, Hkv, Tmax, d


def isoq_decode_attention(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                          params_v, bits: int, variant: int, scale: Optional[float] = None,
                          out=None, workspace=None, stream=None):
    """Decode attention over packed K/V; returns out [B][Hq][d] (dtype of q)."""
    torch = _torch()
    B, Hq, Hkv, Tmax, d = _decode_shapes(q, packed_k, bits)
    dev = _require_cuda(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v,
                        out, workspace)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, Hq, d), q.dtype, dev, stream)
    ws_bytes = isoq_decode_workspace_size(B, Hq, Hkv, Tmax, d)
    if workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, dev, stream)
    with torch.cuda.device(dev):
        st = lib().isoq_decode_attention(
            _ptr(q), _dtype_code(q), _ptr(packed_k), _ptr(packed_v), _ptr(norms_k), _ptr(norms_v),
            _ptr(seq_lens), B, Hq, Hkv, Tmax, d, bits, variant, _ptr(params_k), _ptr(params_v),
            float(scale), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(dev, stream))
    _check(st, "isoq_decode_attention")
    return out


def isoq_decode_append(k_new, v_new, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                       params_v, bits: int, variant: int, stream=None):
    """Compresses k_new/v_new [B][Hkv][d] into the packed cache at seq_lens[b]
    and advances seq_lens, in place on the device."""
    B, Hkv, d = k_new.shape
    _, _, Tmax, pb = packed_k.shape
    if pb != isoq_packed_bytes(d, bits):
        raise ValueError("packed row size does not match d and bits")
    dev = _require_cuda(k_new, v_new, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                        params_v)
    torch = _torch()
    with torch.cuda.device(dev):
        st = lib().isoq_decode_append(
            _ptr(k_new), _ptr(v_new), _dtype_code(k_new), _ptr(packed_k), _ptr(packed_v),
            _ptr(norms_k), _ptr(norms_v), _ptr(seq_lens), B, Hkv, Tmax, d, bits, variant,
            _ptr(params_k), _ptr(params_v), _stream(dev, stream))
    _check(st, "isoq_decode_append")


def isoq_decode_step(q, k_new, v_new, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                     params_v, bits: int, variant: int, scale: Optional[float] = None, out=None,
                     workspace=None, stream=None):
    """Append (k_new, v_new) to the packed cache, then decode attention of q
    over it; returns out [B][Hq][d] (dtype of q)."""
    torch = _torch()
    B, Hq, Hkv, Tmax, d = _decode_shapes(q, packed_k, bits)
    dev = _require_cuda(q, k_new, v_new, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                        params_v, out, workspace)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, Hq, d), q.dtype, dev, stream)
    ws_bytes = isoq_decode_workspace_size(B, Hq, Hkv, Tmax, d)
    if workspace is None:
        workspace = _empty(ws_bytes, torch.uint8, dev, stream)
    with torch.cuda.device(dev):
        st = lib().isoq_decode_step(
            _ptr(q), _ptr(k_new), _ptr(v_new), _dtype_code(q), _ptr(packed_k), _ptr(packed_v),
            _ptr(norms_k), _ptr(norms_v), _ptr(seq_lens), B, Hq, Hkv, Tmax, d, bits, variant,
            _ptr(params_k), _ptr(params_v), float(scale), _ptr(out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(dev, stream))
    _check(st, "isoq_decode_step")
    return out


def isoq_decode_split(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, bits: int,
                      variant: int, workspace, scale: Optional[float] = None, stream=None):
    """First launch of the decode: partial states into ``workspace``."""
    B, Hq, Hkv, Tmax, d = _decode_shapes(q, packed_k, bits)
    dev = _require_cuda(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, workspace)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    torch = _torch()
    with torch.cuda.device(dev):
        st = lib().isoq_decode_split(
            _ptr(q), _dtype_code(q), _ptr(packed_k), _ptr(packed_v), _ptr(norms_k), _ptr(norms_v),
            _ptr(seq_lens), B, Hq, Hkv, Tmax, d, bits, variant, _ptr(params_k), float(scale),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev, stream))
    _check(st, "isoq_decode_split")


def isoq_decode_combine(out, seq_lens, B: int, Hq: int, Hkv: int, Tmax: int, d: int,
                        variant: int, params_v, workspace, stream=None):
    """Second launch of the decode: merge + inverse rotation into ``out``."""
    dev = _require_cuda(out, seq_lens, params_v, workspace)
    torch = _torch()
    with torch.cuda.device(dev):
        st = lib().isoq_decode_combine(
            _dtype_code(out), _ptr(seq_lens), B, Hq, Hkv, Tmax, d, variant, _ptr(params_v),
            _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
            _stream(dev, stream))
    _check(st, "isoq_decode_combine")
    return out


def isoq_selftest_wait_timeout(limit_ns: int = 50_000_000, stream=None, device=None) -> None:
    """Launches the failure-path self-test (a device wait on a barrier that
    nothing arrives at, given up after limit_ns); the next
    isoq_check_device_error then returns ISOQ_ERR_TIMEOUT."""
    torch = _torch()
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(lib().isoq_selftest_wait_timeout(int(limit_ns), _stream(dev, stream)),
               "isoq_selftest_wait_timeout")


def isoq_check_device_error(stream=None, device=None) -> int:
    """Synchronises the stream and returns (and clears) the device error status."""
    torch = _torch()
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        return lib().isoq_check_device_error(_stream(dev, stream))


def _torch_dtype_of(code: int):
    return _torch_dtype(code)


def isoq_decode_attention_static(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                                 params_v, bits: int, variant: int, scale: Optional[float] = None,
                                 out=None, stream=None):
    """isoq_decode_attention with the library's built-in device workspace.

    For callers that cannot allocate device scratch; the output buffer may be
    passed in (``out``) so that the call itself allocates nothing.
    """
    torch = _torch()
    B, Hq, Hkv, Tmax, d = _decode_shapes(q, packed_k, bits)
    dev = _require_cuda(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, out)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, Hq, d), q.dtype, dev, stream)
    with torch.cuda.device(dev):
        st = lib().isoq_decode_attention_static(
            _ptr(q), _dtype_code(q), _ptr(packed_k), _ptr(packed_v), _ptr(norms_k), _ptr(norms_v),
            _ptr(seq_lens), B, Hq, Hkv, Tmax, d, bits, variant, _ptr(params_k), _ptr(params_v),
            float(scale), _ptr(out), _stream(dev, stream))
    _check(st, "isoq_decode_attention_static")
    return out


def isoq_decode_static_workspace_bytes() -> int:
    return lib().isoq_decode_static_workspace_bytes()


# ---------------------------------------------------------------------------
# Serving attention: window and sinks, shared prefix, pages
#
# A decode step makes these calls once per layer, and a small one takes about
# 10 us on the GPU: the checks are one expression over plain attributes, and
# only where it fails does _why look for the argument that does not fit.
# ---------------------------------------------------------------------------

def _refuse(dtypes, contiguous, conditions, tensors):
    """Raises for the first argument that does not fit."""
    for name, t, dtype in dtypes:
        if t is not None and t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    for name, t in contiguous:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for ok, what in conditions:
        if not ok:
            raise ValueError(what)
    _require_cuda(*tensors)
    raise ValueError("the arguments do not fit together")


def _cache_refusal(q, pk, pv, nk, nv, lens, prk, prv, hkv, d, bits, batch, more, tensors):
    """_refuse for a call with a packed cache [a][b][c][d*bits/8], its norms
    and rotations; `more`: further (condition, what) pairs."""
    t = _torch()
    _refuse([("packed K", pk, t.uint8), ("packed V", pv, t.uint8), ("the norms of K", nk, t.float16),
             ("the norms of V", nv, t.float16), ("seq_lens", lens, t.int32), ("params_k", prk, t.float32),
             ("params_v", prv, t.float32)],
            [("q", q), ("packed K", pk), ("packed V", pv), ("the norms of K", nk), ("the norms of V", nv),
             ("seq_lens", lens), ("params_k", prk), ("params_v", prv)],
            [(pk.shape == pv.shape and nk.shape == nv.shape and pk.shape[:-1] == nk.shape,
              "packed K, packed V and their norms do not have one shape"),
             (pk.shape[-1] == isoq_packed_bytes(d, bits), "packed row size does not match d and bits"),
             (lens is None or lens.numel() == batch, f"seq_lens does not have {batch} entries"),
             (prk.numel() == prv.numel() == hkv * 2 * d, "rotation parameters are not [Hkv][d/4][8]"), *more], tensors)


def _fits(q, pk, pv, nk, nv, lens, prk, prv, hkv, d, bits, batch) -> bool:
    """Types, shapes and layout of a packed cache and what goes with it."""
    t = _torch()
    n = hkv * 2 * d
    return (pk.dtype is pv.dtype is t.uint8 and nk.dtype is nv.dtype is t.float16 and lens.dtype is t.int32 and
            prk.dtype is prv.dtype is t.float32 and pk.shape == pv.shape and nk.shape == nv.shape and
            pk.shape[:-1] == nk.shape and pk.shape[-1] * 8 == d * bits and lens.numel() == batch and
            prk.numel() == n and prv.numel() == n and q.is_contiguous() and pk.is_contiguous() and
            pv.is_contiguous() and nk.is_contiguous() and nv.is_contiguous() and lens.is_contiguous() and
            prk.is_contiguous() and prv.is_contiguous())


def _given_out(out, q):
    if out.shape != q.shape or out.dtype is not q.dtype or not out.is_contiguous():
        raise ValueError("out must be contiguous, with the shape and dtype of q")
    if out.device != q.device:
        raise ValueError("all tensors must be on the same device")


def _scratch(workspace, nbytes, dev, stream):
    """Address and bytes of the caller's workspace, or of one from torch's
    allocator (returned too: it lives until the launch is queued, after which
    its stream's order keeps it)."""
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError("workspace must be contiguous and on the device of q")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, None, 0
    workspace = _empty(nbytes, _torch().uint8, dev, stream)
    return workspace, workspace.data_ptr(), nbytes


def _elsewhere(call, index, *args, **kwargs):
    """The call with its tensors' device made current."""
    with _torch().cuda.device(index):
        return call(*args, **kwargs)


@functools.lru_cache(maxsize=256)
def isoq_decode_window_workspace_size(B: int, Hq: int, Hkv: int, Tmax: int, d: int, window: int, n_sink: int) -> int:
    return lib().isoq_decode_window_workspace_size(B, Hq, Hkv, Tmax, d, window, n_sink)


@functools.lru_cache(maxsize=256)
def isoq_decode_prefix_workspace_size(B: int, Hq: int, Hkv: int, prefix_tokens: int, Tmax: int, d: int) -> int:
    return lib().isoq_decode_prefix_workspace_size(B, Hq, Hkv, prefix_tokens, Tmax, d)


def isoq_decode_attention_window(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, bits: int,
                                 variant: int, window: int, n_sink: int = 0, scale: Optional[float] = None,
                                 out=None, workspace=None, stream=None):
    """Decode attention of q [B][Hq][d] over packed K/V, of which a row sees
    its last ``window`` tokens and its first ``n_sink``; returns out (as q)."""
    B, Hq, d = q.shape
    batch, Hkv, Tmax, _ = packed_k.shape
    index = q.get_device()
    if not (batch == B and _fits(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B)
            and packed_k.get_device() == packed_v.get_device() == norms_k.get_device() == norms_v.get_device() ==
            seq_lens.get_device() == params_k.get_device() == params_v.get_device() == index >= 0):
        _cache_refusal(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B,
                       [(batch == B, "q and the cache differ in their batch")],
                       (q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v))
    t = _torch()
    if t.cuda.current_device() != index:
        return _elsewhere(isoq_decode_attention_window, index, q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                          params_v, bits, variant, window, n_sink, scale, out, workspace, stream)
    if out is None:
        out = t.empty_like(q) if stream is None else _empty(q.shape, q.dtype, q.device, stream)
    else:
        _given_out(out, q)
    workspace, wp, ws = _scratch(workspace, isoq_decode_window_workspace_size(B, Hq, Hkv, Tmax, d, window, n_sink), q.device, stream)
    st = lib().isoq_decode_attention_window(
        q.data_ptr(), _dtype_code(q), packed_k.data_ptr(), packed_v.data_ptr(), norms_k.data_ptr(), norms_v.data_ptr(),
        seq_lens.data_ptr(), B, Hq, Hkv, Tmax, d, bits, variant, params_k.data_ptr(), params_v.data_ptr(),
        d ** -0.5 if scale is None else scale, window, n_sink, out.data_ptr(), wp, ws,
        t._C._cuda_getCurrentRawStream(index) if stream is None else _stream(None, stream))
    if st:
        _check(st, "isoq_decode_attention_window")
    return out


def isoq_prefill_attention_window(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, bits: int,
                                  variant: int, window: int, n_sink: int = 0, scale: Optional[float] = None, out=None,
                                  stream=None):
    """Causal attention of q [B][Tq][Hq][d] over the packed cache that holds
    the chunk, each query seeing the last ``window`` tokens up to its own and
    the first ``n_sink``; returns out (as q)."""
    B, Tq, Hq, d = q.shape
    batch, Hkv, Tmax, _ = packed_k.shape
    index = q.get_device()
    if not (batch == B and _fits(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B)
            and packed_k.get_device() == packed_v.get_device() == norms_k.get_device() == norms_v.get_device() ==
            seq_lens.get_device() == params_k.get_device() == params_v.get_device() == index >= 0):
        _cache_refusal(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B,
                       [(batch == B, "q and the cache differ in their batch")],
                       (q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v))
    t = _torch()
    if t.cuda.current_device() != index:
        return _elsewhere(isoq_prefill_attention_window, index, q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k,
                          params_v, bits, variant, window, n_sink, scale, out, stream)
    if out is None:
        out = t.empty_like(q) if stream is None else _empty(q.shape, q.dtype, q.device, stream)
    else:
        _given_out(out, q)
    st = lib().isoq_prefill_attention_window(
        q.data_ptr(), _dtype_code(q), packed_k.data_ptr(), packed_v.data_ptr(), norms_k.data_ptr(), norms_v.data_ptr(),
        seq_lens.data_ptr(), B, Tq, Hq, Hkv, Tmax, d, bits, variant, params_k.data_ptr(), params_v.data_ptr(),
        d ** -0.5 if scale is None else scale, window, n_sink, out.data_ptr(),
        t._C._cuda_getCurrentRawStream(index) if stream is None else _stream(None, stream))
    if st:
        _check(st, "isoq_prefill_attention_window")
    return out


def isoq_decode_attention_prefix(q, prefix_k, prefix_v, prefix_norms_k, prefix_norms_v, prefix_len, packed_k, packed_v,
                                 norms_k, norms_v, seq_lens, params_k, params_v, bits: int, variant: int,
                                 scale: Optional[float] = None, out=None, workspace=None, stream=None):
    """Decode attention of q [B][Hq][d] over a prefix [Hkv][Tp][d*bits/8] that
    all rows share (its first ``prefix_len`` tokens, one int32 on the device)
    and each row's own packed K/V; returns out (as q).  The prefix may be one
    row of a larger cache: its KV heads may lie apart."""
    t = _torch()
    B, Hq, d = q.shape
    batch, Hkv, Tmax, pb = packed_k.shape
    heads, Tp, _ = prefix_k.shape
    index = q.get_device()
    prefix_fits = (prefix_k.dtype is prefix_v.dtype is t.uint8 and
                   prefix_norms_k.dtype is prefix_norms_v.dtype is t.float16 and prefix_k.shape == prefix_v.shape and
                   prefix_norms_k.shape == prefix_norms_v.shape == prefix_k.shape[:-1] and heads == Hkv and
                   prefix_k.shape[-1] == pb)
    apart = Tp
    if not (prefix_k.is_contiguous() and prefix_v.is_contiguous() and prefix_norms_k.is_contiguous() and
            prefix_norms_v.is_contiguous()):
        # tokens contiguous, KV heads `apart` tokens apart in all four
        apart = prefix_norms_k.stride(0) if Hkv > 1 else Tp
        prefix_fits = prefix_fits and apart >= Tp and all(
            Tp == 0 or ((Hkv == 1 or x.stride(0) == apart * width) and (Tp == 1 or x.stride(1) == width) and
                        (x.dim() == 2 or x.stride(2) == 1))
            for x, width in ((prefix_k, pb), (prefix_v, pb), (prefix_norms_k, 1), (prefix_norms_v, 1)))
    if not (batch == B and prefix_fits and prefix_len.dtype is t.int32 and prefix_len.numel() == 1 and
            _fits(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B) and
            packed_k.get_device() == packed_v.get_device() == norms_k.get_device() == norms_v.get_device() ==
            seq_lens.get_device() == params_k.get_device() == params_v.get_device() == prefix_k.get_device() ==
            prefix_v.get_device() == prefix_norms_k.get_device() == prefix_norms_v.get_device() ==
            prefix_len.get_device() == index >= 0):
        _cache_refusal(q, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B,
                       [(batch == B, "q and the cache differ in their batch"),
                        (prefix_fits, "the prefix is not [Hkv][Tp] packed rows and norms of the cache's kind, its tokens "
                                      "contiguous and its KV heads equally far apart in all four tensors"),
                        (prefix_len.dtype is t.int32 and prefix_len.numel() == 1, "prefix_len is one int32")],
                       (q, prefix_k, prefix_v, prefix_norms_k, prefix_norms_v, prefix_len, packed_k, packed_v, norms_k,
                        norms_v, seq_lens, params_k, params_v))
    if t.cuda.current_device() != index:
        return _elsewhere(isoq_decode_attention_prefix, index, q, prefix_k, prefix_v, prefix_norms_k, prefix_norms_v,
                          prefix_len, packed_k, packed_v, norms_k, norms_v, seq_lens, params_k, params_v, bits, variant,
                          scale, out, workspace, stream)
    if out is None:
        out = t.empty_like(q) if stream is None else _empty(q.shape, q.dtype, q.device, stream)
    else:
        _given_out(out, q)
    workspace, wp, ws = _scratch(workspace, isoq_decode_prefix_workspace_size(B, Hq, Hkv, Tp, Tmax, d), q.device, stream)
    st = lib().isoq_decode_attention_prefix(
        q.data_ptr(), _dtype_code(q), prefix_k.data_ptr(), prefix_v.data_ptr(), prefix_norms_k.data_ptr(),
        prefix_norms_v.data_ptr(), prefix_len.data_ptr(), Tp, apart, packed_k.data_ptr(), packed_v.data_ptr(),
        norms_k.data_ptr(), norms_v.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, Tmax, d, bits, variant,
        params_k.data_ptr(), params_v.data_ptr(), d ** -0.5 if scale is None else scale, out.data_ptr(), wp, ws,
        t._C._cuda_getCurrentRawStream(index) if stream is None else _stream(None, stream))
    if st:
        _check(st, "isoq_decode_attention_prefix")
    return out


def isoq_build_block_tables(seq_lens, new_lens, free_pages, block_table, page_tokens: int, n_slots: Optional[int] = None,
                            free_head=None, slot_map=None, row_start=None, total_lens=None, pages_used=None, stream=None):
    """Pages and slots of the tokens that a step adds to a paged cache: takes
    the pages that the rows lack from ``free_pages`` (from ``free_head`` on) into
    ``block_table`` [B][max_pages], in place; returns (slot_map [n_slots],
    row_start [B + 1], total_lens [B], pages_used [1])."""
    t = _torch()
    B, max_pages = block_table.shape
    index = block_table.get_device()
    if slot_map is None:
        if n_slots is None:
            raise ValueError("n_slots (or slot_map) says how many new tokens there may be")
        slots = n_slots
    else:
        slots = slot_map.numel()
    i32 = t.int32
    given = [x for x in (free_head, row_start, total_lens, pages_used) if x is not None]
    if not (seq_lens.dtype is i32 and new_lens.dtype is i32 and free_pages.dtype is i32 and block_table.dtype is i32 and
            seq_lens.is_contiguous() and new_lens.is_contiguous() and free_pages.is_contiguous() and
            block_table.is_contiguous() and
            seq_lens.get_device() == new_lens.get_device() == free_pages.get_device() == index >= 0 and
            seq_lens.numel() == B and new_lens.numel() == B and
            (not given or
             (all(x.dtype is i32 and x.is_contiguous() and x.get_device() == index for x in given) and
              (free_head is None or free_head.numel() == 1) and (row_start is None or row_start.numel() == B + 1) and
              (total_lens is None or total_lens.numel() == B) and (pages_used is None or pages_used.numel() == 1))) and
            (slot_map is None or (slot_map.dtype is t.int64 and slot_map.is_contiguous() and
                                  slot_map.get_device() == index and n_slots in (None, slots)))):
        ints = (seq_lens, new_lens, free_pages, block_table)
        names = ("seq_lens", "new_lens", "free_pages", "block_table", "free_head", "row_start", "total_lens", "pages_used")
        every = (*ints, free_head, row_start, total_lens, pages_used)
        _refuse([*((n, x, t.int32) for n, x in zip(names, every)), ("slot_map", slot_map, t.int64)],
                [*zip(names, every), ("slot_map", slot_map)],
                [(seq_lens.numel() == B, f"seq_lens does not have {B} entries"),
                 (new_lens.numel() == B, f"new_lens does not have {B} entries"),
                 (free_head is None or free_head.numel() == 1, "free_head is one int32"),
                 (row_start is None or row_start.numel() == B + 1, f"row_start does not have {B + 1} entries"),
                 (total_lens is None or total_lens.numel() == B, f"total_lens does not have {B} entries"),
                 (pages_used is None or pages_used.numel() == 1, "pages_used is one int32"),
                 (n_slots in (None, slots), "slot_map does not have n_slots entries")], (*every, slot_map))
    if t.cuda.current_device() != index:
        return _elsewhere(isoq_build_block_tables, index, seq_lens, new_lens, free_pages, block_table, page_tokens, n_slots,
                          free_head, slot_map, row_start, total_lens, pages_used, stream)
    if slot_map is None:
        slot_map = _empty(slots, t.int64, block_table.device, stream)
    if row_start is None:
        row_start = _empty(B + 1, i32, block_table.device, stream)
    if total_lens is None:
        total_lens = _empty(B, i32, block_table.device, stream)
    if pages_used is None:
        pages_used = _empty(1, i32, block_table.device, stream)
    st = lib().isoq_build_block_tables(
        seq_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), _ptr(free_head), free_pages.numel(), B,
        page_tokens, max_pages, block_table.data_ptr(), slots, slot_map.data_ptr(), row_start.data_ptr(),
        total_lens.data_ptr(), pages_used.data_ptr(),
        t._C._cuda_getCurrentRawStream(index) if stream is None else _stream(None, stream))
    if st:
        _check(st, "isoq_build_block_tables")
    return slot_map, row_start, total_lens, pages_used


def isoq_paged_append(k_new, v_new, pages_k, pages_v, norms_k, norms_v, slot_map, params_k, params_v, bits: int,
                      variant: int, stream=None):
    """Compresses the new tokens k_new, v_new [N][Hkv][d] into the slots of
    the pages [n_pages][Hkv][page_tokens][d*bits/8], in place; a negative slot's
    token is skipped.  ``slot_map`` may be longer than N (a slot map of a fixed
    shape): its first N entries count."""
    t = _torch()
    N, Hkv, d = k_new.shape
    n_pages, heads, P, _ = pages_k.shape
    index = k_new.get_device()
    same = heads == Hkv and v_new.shape == k_new.shape and v_new.dtype is k_new.dtype
    n = 2 * Hkv * d
    if not (same and pages_k.dtype is pages_v.dtype is t.uint8 and norms_k.dtype is norms_v.dtype is t.float16 and
            slot_map.dtype is t.int64 and params_k.dtype is params_v.dtype is t.float32 and
            pages_k.shape == pages_v.shape and norms_k.shape == norms_v.shape == pages_k.shape[:-1] and
            pages_k.shape[-1] * 8 == d * bits and slot_map.numel() >= N and params_k.numel() == n and
            params_v.numel() == n and k_new.is_contiguous() and v_new.is_contiguous() and pages_k.is_contiguous() and
            pages_v.is_contiguous() and norms_k.is_contiguous() and norms_v.is_contiguous() and
            slot_map.is_contiguous() and params_k.is_contiguous() and params_v.is_contiguous() and
            v_new.get_device() == pages_k.get_device() == pages_v.get_device() == norms_k.get_device() ==
            norms_v.get_device() == slot_map.get_device() == params_k.get_device() == params_v.get_device() == index >= 0):
        if slot_map.dtype is not t.int64:
            raise TypeError(f"slot_map must be {t.int64}, not {slot_map.dtype}")
        _cache_refusal(k_new, pages_k, pages_v, norms_k, norms_v, None, params_k, params_v, Hkv, d, bits, 0,
                       [(same, "the new K and V and the pages do not belong together"),
                        (v_new.is_contiguous() and slot_map.is_contiguous(), "v_new and slot_map must be contiguous"),
                        (slot_map.numel() >= N, "slot_map has fewer entries than there are new tokens")],
                       (k_new, v_new, pages_k, pages_v, norms_k, norms_v, slot_map, params_k, params_v))
    if t.cuda.current_device() != index:
        return _elsewhere(isoq_paged_append, index, k_new, v_new, pages_k, pages_v, norms_k, norms_v, slot_map, params_k,
                          params_v, bits, variant, stream)
    st = lib().isoq_paged_append(
        k_new.data_ptr(), v_new.data_ptr(), _dtype_code(k_new), pages_k.data_ptr(), pages_v.data_ptr(), norms_k.data_ptr(),
        norms_v.data_ptr(), slot_map.data_ptr(), N, Hkv, n_pages, P, d, bits, variant, params_k.data_ptr(),
        params_v.data_ptr(), t._C._cuda_getCurrentRawStream(index) if stream is None else _stream(None, stream))
    if st:
        _check(st, "isoq_paged_append")


def isoq_paged_decode_attention(q, pages_k, pages_v, norms_k, norms_v, block_table, seq_lens, params_k, params_v,
                                bits: int, variant: int, max_len: Optional[int] = None, window: Optional[int] = None,
                                n_sink: int = 0, scale: Optional[float] = None, out=None, workspace=None, stream=None):
    """Decode attention of q [B][Hq][d] over the pages that ``block_table``
    [B][max_pages] lists; ``max_len`` bounds the lengths (default: what the
    table holds), ``window`` and ``n_sink`` as isoq_decode_attention_window
    (default: all tokens).  Returns out (as q)."""
    t = _torch()
    B, Hq, d = q.shape
    n_pages, Hkv, P, _ = pages_k.shape
    batch, max_pages = block_table.shape
    index = q.get_device()
    if not (batch == B and block_table.dtype is t.int32 and block_table.is_contiguous() and
            _fits(q, pages_k, pages_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B) and
            pages_k.get_device() == pages_v.get_device() == norms_k.get_device() == norms_v.get_device() ==
            block_table.get_device() == seq_lens.get_device() == params_k.get_device() == params_v.get_device() ==
            index >= 0):
        _cache_refusal(q, pages_k, pages_v, norms_k, norms_v, seq_lens, params_k, params_v, Hkv, d, bits, B,
                       [(batch == B, "block_table is not [B][max_pages]"),
                        (block_table.dtype is t.int32 and block_table.is_contiguous(), "block_table must be contiguous int32")],
                       (q, pages_k, pages_v, norms_k, norms_v, block_table, seq_lens, params_k, params_v))
    if max_len is None:
        max_len = max_pages * P
    if window is None:
        window = max_len
    if t.cuda.current_device() != index:
        return _elsewhere(isoq_paged_decode_attention, index, q, pages_k, pages_v, norms_k, norms_v, block_table, seq_lens,
                          params_k, params_v, bits, variant, max_len, window, n_sink, scale, out, workspace, stream)
    if out is None:
        out = t.empty_like(q) if stream is None else _empty(q.shape, q.dtype, q.device, stream)
    else:
        _given_out(out, q)
    workspace, wp, ws = _scratch(workspace, isoq_decode_window_workspace_size(B, Hq, Hkv, max_len, d, window, n_sink), q.device, stream)
    st = lib().isoq_paged_decode_attention(
        q.data_ptr(), _dtype_code(q), pages_k.data_ptr(), pages_v.data_ptr(), norms_k.data_ptr(), norms_v.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), B, Hq, Hkv, n_pages, P, max_pages, max_len, d, bits, variant,
        params_k.data_ptr(), params_v.data_ptr(), d ** -0.5 if scale is None else scale, window, n_sink, out.data_ptr(), wp,
        ws, t._C._cuda_getCurrentRawStream(index) if stream is None else _stream(None, stream))
    if st:
        _check(st, "isoq_paged_decode_attention")
    return out

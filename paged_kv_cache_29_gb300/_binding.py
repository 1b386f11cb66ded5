"""ctypes binding of libpagedattn.so (include/pagedattn.h).

Argument marshalling only: every function takes torch tensors (or plain
integers), checks that they are CUDA tensors of the expected dtype and shape,
passes their device pointers and the current torch stream to the C entry point
of the same name, and raises PagedAttentionError on a non-OK status. There is
no CPU fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libpagedattn.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "pagedattn.h")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_WORKSPACE = 3
PA_ERR_CUDA = 4
PA_ERR_DEVICE_BOUNDS = 5

PA_DEVERR_BLOCK_ID = 0x1
PA_DEVERR_SLOT = 0x2
PA_DEVERR_CONTEXT = 0x4
PA_DEVERR_TIMEOUT = 0x8
PA_DEVERR_POSITION = 0x10

KERNELS = {"auto": 0, "simt": 1, "mma": 2, "generic": 3, "tc": 4}
DEFAULT_PARTITION = 512

_lock = threading.Lock()
_lib = None


class PagedAttentionError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {pa_status_string(status)} (status {status})")


class _Options(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("partition_size", ctypes.c_int),
                ("long_partition_size", ctypes.c_int), ("long_partition_from", ctypes.c_int)]


class _NormRopeArgs(ctypes.Structure):
    """pa_norm_rope_args."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("q_out", ctypes.c_void_p),
                ("q_out_stride", ctypes.c_int64), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("weight_offset", ctypes.c_float), ("cos_sin", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("pair_axis", ctypes.c_char_p),
                ("num_tokens", ctypes.c_int), ("num_heads", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("rot_dim", ctypes.c_int), ("max_position", ctypes.c_int),
                ("num_axes", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int)]


# The same layout as a struct format: packing it takes a fifth of the time that
# filling the ctypes structure does.
_norm_rope_pack = struct.Struct("@PPqqPqPPffPPP10i").pack


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if it has not been built."""
    global _lib
    if _lib is not None:            # loaded: no lock needed to read the reference
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m paged_kv_cache_29_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.pa_reshape_and_cache.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P, P]
        L.pa_reshape_and_cache.restype = I
        L.pa_reshape_and_cache_fp8.argtypes = [P, P, I, P, P, P, I, I, I, I, I, F, F, P, P]
        L.pa_reshape_and_cache_fp8.restype = I
        L.pa_decode_fp8.argtypes = [P, P, P, P, P, F, F, F, P, I, I, I, I, I, I, I, I, P, S, P, P]
        L.pa_decode_fp8.restype = I
        L.pa_decode_fp8_ex.argtypes = [P, P, P, P, P, F, F, F, P, I, I, I, I, I, I, I, I, P, S, P,
                                       ctypes.POINTER(_Options), P]
        L.pa_decode_fp8_ex.restype = I
        L.pa_test_withhold_tile.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, I, P, S, P,
                                            I, P]
        L.pa_test_withhold_tile.restype = I
        L.pa_decode_multi.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, I, I, P, S, P, P]
        L.pa_decode_multi.restype = I
        L.pa_decode_workspace_size_multi.argtypes = [I, I, I, I, I]
        L.pa_decode_workspace_size_multi.restype = S
        L.pa_decode_window.argtypes = [P, P, P, P, P, F, I, P, I, I, I, I, I, I, I, I, I, P, S,
                                       P, P]
        L.pa_decode_window.restype = I
        L.pa_reshape_and_cache_int8.argtypes = [P, P, I, P, P, P, P, P, I, I, I, I, I, P, P]
        L.pa_reshape_and_cache_int8.restype = I
        L.pa_decode_int8.argtypes = [P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, P, S, P, P]
        L.pa_decode_int8.restype = I
        L.pa_copy_blocks.argtypes = [P, P, P, I, I, I, I, I, I, P, P]
        L.pa_copy_blocks.restype = I
        L.pa_decode.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, I, P, S, P, P]
        L.pa_decode.restype = I
        L.pa_append_decode.argtypes = [P, P, P, P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, I,
                                       P, S, P, P]
        L.pa_append_decode.restype = I
        L.pa_append_decode_fp8.argtypes = [P, P, P, P, P, F, F, P, P, P, F, P, I, I, I, I, I, I, I,
                                           I, P, S, P, P]
        L.pa_append_decode_fp8.restype = I
        L.pa_append_decode_int8.argtypes = [P, P, P, P, P, P, P, P, P, P, F, P, I, I, I, I, I, I,
                                            I, I, P, S, P, P]
        L.pa_append_decode_int8.restype = I
        L.pa_decode_ex.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, I, P, S, P,
                                   ctypes.POINTER(_Options), P]
        L.pa_decode_ex.restype = I
        L.pa_decode_noalloc.argtypes = [P, P, P, P, P, F, P, I, I, I, I, I, I, I, I, I, P, P]
        L.pa_decode_noalloc.restype = I
        L.pa_decode_workspace_size.argtypes = [I, I, I, I]
        L.pa_decode_workspace_size.restype = S
        L.pa_decode_workspace_size_ex.argtypes = [I, I, I, I, I]
        L.pa_decode_workspace_size_ex.restype = S
        L.pa_reshape_and_cache_int4.argtypes = [P, P, I, P, P, P, P, P, I, I, I, I, I, P, P]
        L.pa_reshape_and_cache_int4.restype = I
        L.pa_gather_int4.argtypes = [P, P, P, P, P, P, P, P, P, I, ctypes.c_int64, I, I, I, I, I,
                                     I, I, P, P]
        L.pa_gather_int4.restype = I
        L.pa_decode_int4.argtypes = [P, P, P, P, P, P, P, F, I, P, I, I, I, I, I, I, I, I, I, P, S,
                                     P, P]
        L.pa_decode_int4.restype = I
        L.pa_norm_rope.argtypes = [P, P, ctypes.c_int64, P, P]
        L.pa_norm_rope.restype = I
        L.pa_norm_rope_append.argtypes = [P, P, ctypes.c_int64, P, P, P, I, I, P, P]
        L.pa_norm_rope_append.restype = I
        L.pa_norm_rope_append_int4.argtypes = [P, P, ctypes.c_int64, P, P, P, P, P, I, I, P, P]
        L.pa_norm_rope_append_int4.restype = I
        L.pa_status_string.argtypes = [I]
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_check_error_word.argtypes = [ctypes.c_int32]
        L.pa_check_error_word.restype = I
        L.pa_version.argtypes = []
        L.pa_version.restype = I
        L.pa_default_partition_size.argtypes = [I]
        L.pa_default_partition_size.restype = I
        _lib = L
        return L


def declared_functions() -> list[str]:
    """Names of the functions include/pagedattn.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(pa_[a-z0-9_]+)\s*\(", text)))


def pa_status_string(status: int) -> str:
    try:
        return lib().pa_status_string(int(status)).decode()
    except RuntimeError:
        return f"status {status}"


def pa_version() -> int:
    return lib().pa_version()


def pa_default_partition_size(cache_dtype: str) -> int:
    """Rows per split-K partition used when none is requested, for a cache
    of this type ("f32", "bf16", "fp8", "int8" or "int4")."""
    codes = {"f32": 0, "bf16": 1, "fp8": 2, "int8": 3, "int4": 4}
    if cache_dtype not in codes:
        raise ValueError(f"unknown cache dtype {cache_dtype!r}")
    return lib().pa_default_partition_size(codes[cache_dtype])


def _dtype_code(t) -> int:
    """float32 -> 0, bfloat16 -> 1; an FP8 cache is uint8 (e4m3 codes) or
    torch.float8_e4m3fn -> 2."""
    import torch
    if t.dtype == torch.float32:
        return 0
    if t.dtype == torch.bfloat16:
        return 1
    if t.dtype == torch.uint8 or t.dtype == getattr(torch, "float8_e4m3fn", None):
        return 2
    if t.dtype == torch.int8:
        return 3
    raise TypeError(f"dtype must be float32, bfloat16 or e4m3 codes, got {t.dtype}")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _current_raw_stream():
    """A function returning torch's current CUDA stream handle as an int: the
    raw accessor when this torch has it (no Stream object is built, ~3 us less
    per call), else the public API."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return lambda: raw(torch.cuda.current_device())
    return lambda: torch.cuda.current_stream().cuda_stream


_raw_stream = None


def _stream(stream) -> int | None:
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            _raw_stream = _current_raw_stream()
        return _raw_stream() or None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _scratch(nbytes, stream, device):
    """Workspace of one call that brings none, from torch's caching allocator. It
    is taken as the launch stream's own: the allocator then hands its bytes out
    again, and takes them from, work in that stream's order only. Taken on
    torch's current stream and dropped while a call on another one runs, it could go
    to the next tensor there under the running kernel."""
    import torch
    if stream is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    _check_device(stream)
    if not isinstance(stream, torch.cuda.Stream):     # a raw handle, or another library's stream
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def _check_cuda(name, t, dtype=None, ndim=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")


def _check_device(stream, *tensors):
    """Every tensor (and an explicit torch stream) on torch's current CUDA
    device. The library launches on the current device and takes the SM count,
    the tensor maps, the fixed scratch of pa_decode_noalloc and the default
    stream from it, so a tensor on another GPU would hand that GPU's pointers
    to kernels running here."""
    import torch
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != cur:
            raise ValueError(f"a tensor is on {t.device} but the current CUDA device is cuda:{cur}:"
                             f" run the call under torch.cuda.device({t.device.index})")
    dev = getattr(stream, "device", None)
    if dev is not None and getattr(dev, "index", cur) != cur:
        raise ValueError(f"the stream belongs to {dev} but the current CUDA device is cuda:{cur}")


def pa_reshape_and_cache(k_new, v_new, slot_mapping, k_cache, v_cache, error_word=None,
                         stream=None) -> None:
    """Append new K/V rows ([T][Hkv][D]) into their slots of the paged pools
    ([NB][Hkv][bs][D]). slot_mapping: int64 [T], negative = skip."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("k_new", k_new, k_cache.dtype, 3)
    _check_cuda("v_new", v_new, k_cache.dtype, 3)
    _check_cuda("slot_mapping", slot_mapping, torch.int64, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    if tuple(v_cache.shape) != (nb, hkv, bs, d) or tuple(k_new.shape[1:]) != (hkv, d) \
            or k_new.shape != v_new.shape or slot_mapping.shape[0] != k_new.shape[0]:
        raise ValueError("shape mismatch between k_new/v_new/slot_mapping and the caches")
    _check_device(stream, k_new, v_new, slot_mapping, k_cache, v_cache, error_word)
    rc = lib().pa_reshape_and_cache(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping),
                                    _ptr(k_cache), _ptr(v_cache), int(k_new.shape[0]), hkv, d,
                                    bs, nb, _dtype_code(k_cache), _ptr(error_word),
                                    _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_reshape_and_cache")


def pa_reshape_and_cache_fp8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale=1.0,
                             v_scale=1.0, error_word=None, stream=None) -> None:
    """Quantising append: k_new/v_new (bf16 or fp32, [T][Hkv][D]) -> e4m3 codes
    of x / scale in the FP8 pools (uint8 [NB][Hkv][bs][D])."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    if _dtype_code(k_cache) != 2:
        raise TypeError("FP8 caches are uint8 (e4m3 codes) or float8_e4m3fn")
    _check_cuda("k_new", k_new, ndim=3)
    _check_cuda("v_new", v_new, k_new.dtype, 3)
    _check_cuda("slot_mapping", slot_mapping, torch.int64, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    if tuple(v_cache.shape) != (nb, hkv, bs, d) or tuple(k_new.shape[1:]) != (hkv, d) \
            or k_new.shape != v_new.shape or slot_mapping.shape[0] != k_new.shape[0]:
        raise ValueError("shape mismatch between k_new/v_new/slot_mapping and the caches")
    _check_device(stream, k_new, v_new, slot_mapping, k_cache, v_cache, error_word)
    rc = lib().pa_reshape_and_cache_fp8(_ptr(k_new), _ptr(v_new), _dtype_code(k_new),
                                        _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                        int(k_new.shape[0]), hkv, d, bs, nb, float(k_scale),
                                        float(v_scale), _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_reshape_and_cache_fp8")


def pa_decode_fp8(q, k_cache, v_cache, block_tables, context_lens, scale, out, max_context_len,
                  k_scale=1.0, v_scale=1.0, workspace=None, error_word=None,
                  stream=None, kernel: str = "auto") -> None:
    """Decode attention over FP8 pools (uint8 e4m3 codes) with bf16 q/out.
    kernel: "auto", "mma" (tile ring, mma.sync) or "tc" (tcgen05)."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    if _dtype_code(k_cache) != 2:
        raise TypeError("FP8 caches are uint8 (e4m3 codes) or float8_e4m3fn")
    _check_cuda("q", q, torch.bfloat16, 3)
    _check_cuda("out", out, torch.bfloat16, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, block_tables, context_lens, error_word,
                  workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    opts = _Options(KERNELS[kernel], 0, 0, 0)
    rc = lib().pa_decode_fp8_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                _ptr(context_lens), float(scale), float(k_scale), float(v_scale),
                                _ptr(out), B, hq, hkv, d, bs, nb, int(block_tables.shape[1]),
                                int(max_context_len), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _ptr(error_word),
                                ctypes.byref(opts), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_decode_fp8")


def pa_test_withhold_tile(q, k_cache, v_cache, block_tables, context_lens, scale, out,
                          max_context_len, withhold_tile, error_word, workspace=None,
                          stream=None) -> None:
    """Failure test of the bounded waits: a decode call (fp32/bf16 caches, or
    FP8 codes with unit scales) whose CTA 0 withholds tile `withhold_tile` of
    its stream; the waiting consumer gives up after about 2 s and the kernel
    sets PA_DEVERR_TIMEOUT in error_word. Not for production use."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    code = _dtype_code(k_cache)
    act = torch.bfloat16 if code == 2 else k_cache.dtype
    _check_cuda("q", q, act, 3)
    _check_cuda("out", out, act, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, block_tables, context_lens, error_word,
                  workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    rc = lib().pa_test_withhold_tile(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                     _ptr(context_lens), float(scale), _ptr(out), B, hq, hkv, d,
                                     bs, nb, int(block_tables.shape[1]), int(max_context_len),
                                     code, _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _ptr(error_word), int(withhold_tile), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_test_withhold_tile")


def pa_decode_workspace_size_multi(num_seqs: int, num_queries: int, num_heads: int,
                                   head_dim: int, max_context_len: int) -> int:
    return int(lib().pa_decode_workspace_size_multi(num_seqs, num_queries, num_heads, head_dim,
                                                     max_context_len))


def pa_decode_multi(q, k_cache, v_cache, block_tables, context_lens, scale, out,
                    max_context_len, workspace=None, error_word=None, stream=None) -> None:
    """Multi-query decode: q/out [B][Q][Hq][D] bf16; query token j of sequence
    s attends to rows 0 .. n - Q + j of its n = context_lens[s] rows."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("q", q, k_cache.dtype, 4)
    _check_cuda("out", out, k_cache.dtype, 4)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, Q, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, block_tables, context_lens, error_word,
                  workspace)
    if workspace is None:
        need = pa_decode_workspace_size_multi(B, Q, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    rc = lib().pa_decode_multi(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                               _ptr(context_lens), float(scale), _ptr(out), B, Q, hq, hkv, d, bs,
                               nb, int(block_tables.shape[1]), int(max_context_len),
                               _dtype_code(k_cache), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(error_word),
                               _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_decode_multi")


def pa_decode_window(q, k_cache, v_cache, block_tables, context_lens, scale, window, out,
                     max_context_len, workspace=None, error_word=None, stream=None) -> None:
    """Sliding-window decode: each sequence attends to its last `window` rows."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("q", q, k_cache.dtype, 3)
    _check_cuda("out", out, k_cache.dtype, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, block_tables, context_lens, error_word,
                  workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    rc = lib().pa_decode_window(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                _ptr(context_lens), float(scale), int(window), _ptr(out), B, hq,
                                hkv, d, bs, nb, int(block_tables.shape[1]), int(max_context_len),
                                _dtype_code(k_cache), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _ptr(error_word),
                                _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_decode_window")


def _check_int8_pool(k_cache, v_cache, k_scales, v_scales):
    import torch
    _check_cuda("k_cache", k_cache, torch.int8, 4)
    _check_cuda("v_cache", v_cache, torch.int8, 4)
    _check_cuda("k_scales", k_scales, torch.float32, 3)
    _check_cuda("v_scales", v_scales, torch.float32, 3)
    if tuple(v_cache.shape) != tuple(k_cache.shape) or \
            tuple(k_scales.shape) != tuple(k_cache.shape[:3]) or \
            tuple(v_scales.shape) != tuple(k_cache.shape[:3]):
        raise ValueError("INT8 pools are [NB][Hkv][bs][D] codes with [NB][Hkv][bs] scales")


def pa_reshape_and_cache_int8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scales, v_scales,
                              error_word=None, stream=None) -> None:
    """Quantising append into an INT8 cache: one fp32 scale per (row, KV head)."""
    import torch
    _check_int8_pool(k_cache, v_cache, k_scales, v_scales)
    _check_cuda("k_new", k_new, ndim=3)
    _check_cuda("v_new", v_new, k_new.dtype, 3)
    _check_cuda("slot_mapping", slot_mapping, torch.int64, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    if tuple(k_new.shape[1:]) != (hkv, d) or k_new.shape != v_new.shape \
            or slot_mapping.shape[0] != k_new.shape[0]:
        raise ValueError("shape mismatch between k_new/v_new/slot_mapping and the caches")
    _check_device(stream, k_new, v_new, slot_mapping, k_cache, v_cache, k_scales, v_scales,
                  error_word)
    rc = lib().pa_reshape_and_cache_int8(_ptr(k_new), _ptr(v_new), _dtype_code(k_new),
                                         _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                                         _ptr(k_scales), _ptr(v_scales), int(k_new.shape[0]), hkv,
                                         d, bs, nb, _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_reshape_and_cache_int8")


def pa_decode_int8(q, k_cache, v_cache, k_scales, v_scales, block_tables, context_lens, scale,
                   out, max_context_len, workspace=None, error_word=None, stream=None) -> None:
    """Decode attention over an INT8 cache with per-row scales, bf16 q/out."""
    import torch
    _check_int8_pool(k_cache, v_cache, k_scales, v_scales)
    _check_cuda("q", q, torch.bfloat16, 3)
    _check_cuda("out", out, torch.bfloat16, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or block_tables.shape[0] != B \
            or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, k_scales, v_scales, block_tables,
                  context_lens, error_word, workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    rc = lib().pa_decode_int8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scales),
                              _ptr(v_scales), _ptr(block_tables), _ptr(context_lens),
                              float(scale), _ptr(out), B, hq, hkv, d, bs, nb,
                              int(block_tables.shape[1]), int(max_context_len), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _ptr(error_word),
                              _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_decode_int8")


def pa_copy_blocks(k_cache, v_cache, block_mapping, error_word=None, stream=None) -> None:
    """Copy-on-write: block dst := block src of both pools for each (src, dst)
    row of block_mapping (int64 [n][2]); negative entries skip a pair. The
    pools are [NB][Hkv][bs][D] (an INT4 cache's [NB][Hkv][bs][D / 2] bytes); for
    an INT8 cache call it again on the row scales viewed as [NB][1][1][Hkv * bs],
    for an INT4 cache on the params viewed as [NB][1][1][Hkv * bs * 2]."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("block_mapping", block_mapping, torch.int64, 2)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    if tuple(v_cache.shape) != (nb, hkv, bs, d) or block_mapping.shape[1] != 2:
        raise ValueError("v_cache must match k_cache and block_mapping must be [n][2]")
    _check_device(stream, k_cache, v_cache, block_mapping, error_word)
    rc = lib().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_mapping),
                              int(block_mapping.shape[0]), hkv, d, bs, nb,
                              _dtype_code(k_cache), _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_copy_blocks")


def pa_decode_workspace_size(num_seqs: int, num_heads: int, head_dim: int,
                             max_context_len: int, partition_size: int = 0) -> int:
    return int(lib().pa_decode_workspace_size_ex(num_seqs, num_heads, head_dim,
                                                 max_context_len, partition_size))


def pa_decode(q, k_cache, v_cache, block_tables, context_lens, scale, out, max_context_len,
              workspace=None, error_word=None, stream=None, kernel: str = "auto",
              partition_size: int = 0, long_partition_size: int = 0,
              long_partition_from: int = 0) -> None:
    """Decode attention for every sequence, written into ``out`` ([B][Hq][D]).

    max_context_len bounds context_lens (host value; sizes the work list and
    the workspace). workspace: a CUDA tensor of at least
    pa_decode_workspace_size(...) bytes; when None, one is taken from torch's
    caching allocator for this call, on its stream. long_partition_size /
    long_partition_from: partitions of that many rows for sequences longer
    than long_partition_from rows (0 = one size for all)."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("q", q, k_cache.dtype, 3)
    _check_cuda("out", out, k_cache.dtype, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, block_tables, context_lens, error_word,
                  workspace)
    if workspace is None:
        # The C library allocates nothing; the binding takes the scratch from
        # torch's allocator for callers that do not manage their own.
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len), int(partition_size))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    opts = _Options(KERNELS[kernel], int(partition_size), int(long_partition_size),
                    int(long_partition_from))
    rc = lib().pa_decode_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                            _ptr(context_lens), float(scale), _ptr(out), B, hq, hkv, d, bs, nb,
                            int(block_tables.shape[1]), int(max_context_len),
                            _dtype_code(k_cache), _ptr(workspace), ws_bytes, _ptr(error_word),
                            ctypes.byref(opts), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_decode")


def pa_append_decode(k_new, v_new, slot_mapping, k_cache, v_cache, q, block_tables, context_lens,
                     scale, out, max_context_len, workspace=None, error_word=None,
                     stream=None) -> None:
    """One decode step: append one new K/V row per sequence (k_new/v_new
    [B][Hkv][D], slot_mapping int64 [B], the slot of each sequence's last row
    or negative), then decode attention into out ([B][Hq][D])."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("k_new", k_new, k_cache.dtype, 3)
    _check_cuda("v_new", v_new, k_cache.dtype, 3)
    _check_cuda("slot_mapping", slot_mapping, torch.int64, 1)
    _check_cuda("q", q, k_cache.dtype, 3)
    _check_cuda("out", out, k_cache.dtype, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or tuple(k_new.shape) != (B, hkv, d) or tuple(v_new.shape) != (B, hkv, d) \
            or slot_mapping.shape[0] != B or block_tables.shape[0] != B \
            or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between the step's tensors and the caches")
    _check_device(stream, k_new, v_new, slot_mapping, q, out, k_cache, v_cache, block_tables,
                  context_lens, error_word, workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().pa_append_decode(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
                                _ptr(v_cache), _ptr(q), _ptr(block_tables), _ptr(context_lens),
                                float(scale), _ptr(out), B, hq, hkv, d, bs, nb,
                                int(block_tables.shape[1]), int(max_context_len),
                                _dtype_code(k_cache), _ptr(workspace), ws_bytes,
                                _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_append_decode")


def _check_step_rows(k_new, v_new, slot_mapping, q, out, block_tables, context_lens, hkv, d):
    import torch
    _check_cuda("k_new", k_new, torch.bfloat16, 3)
    _check_cuda("v_new", v_new, torch.bfloat16, 3)
    _check_cuda("slot_mapping", slot_mapping, torch.int64, 1)
    _check_cuda("q", q, torch.bfloat16, 3)
    _check_cuda("out", out, torch.bfloat16, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(k_new.shape) != (B, hkv, d) \
            or tuple(v_new.shape) != (B, hkv, d) or slot_mapping.shape[0] != B \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between the step's tensors and the caches")
    return B, hq


def pa_append_decode_fp8(k_new, v_new, slot_mapping, k_cache, v_cache, q, block_tables,
                         context_lens, scale, out, max_context_len, k_scale=1.0, v_scale=1.0,
                         workspace=None, error_word=None, stream=None) -> None:
    """One decode step over FP8 pools: quantise one new bf16 K/V row per
    sequence into its slot (the sequence's last row), then decode."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    if _dtype_code(k_cache) != 2:
        raise TypeError("FP8 caches are uint8 (e4m3 codes) or float8_e4m3fn")
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq = _check_step_rows(k_new, v_new, slot_mapping, q, out, block_tables, context_lens, hkv, d)
    _check_device(stream, k_new, v_new, slot_mapping, q, out, k_cache, v_cache, block_tables,
                  context_lens, error_word, workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    rc = lib().pa_append_decode_fp8(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
                                    _ptr(v_cache), float(k_scale), float(v_scale), _ptr(q),
                                    _ptr(block_tables), _ptr(context_lens), float(scale),
                                    _ptr(out), B, hq, hkv, d, bs, nb, int(block_tables.shape[1]),
                                    int(max_context_len), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_append_decode_fp8")


def pa_append_decode_int8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scales, v_scales, q,
                          block_tables, context_lens, scale, out, max_context_len,
                          workspace=None, error_word=None, stream=None) -> None:
    """One decode step over INT8 pools with row scales: quantise one new bf16
    K/V row per sequence into its slot (the sequence's last row), then decode."""
    import torch
    _check_int8_pool(k_cache, v_cache, k_scales, v_scales)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq = _check_step_rows(k_new, v_new, slot_mapping, q, out, block_tables, context_lens, hkv, d)
    _check_device(stream, k_new, v_new, slot_mapping, q, out, k_cache, v_cache, k_scales,
                  v_scales, block_tables, context_lens, error_word, workspace)
    if workspace is None:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        workspace = _scratch(need, stream, q.device)
    _check_cuda("workspace", workspace)
    rc = lib().pa_append_decode_int8(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(k_cache),
                                     _ptr(v_cache), _ptr(k_scales), _ptr(v_scales), _ptr(q),
                                     _ptr(block_tables), _ptr(context_lens), float(scale),
                                     _ptr(out), B, hq, hkv, d, bs, nb, int(block_tables.shape[1]),
                                     int(max_context_len), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(),
                                     _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_append_decode_int8")


NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024   # PA_NOALLOC_SCRATCH_BYTES


def pa_decode_noalloc(q, k_cache, v_cache, block_tables, context_lens, scale, out,
                      max_context_len, error_word=None, stream=None) -> None:
    """pa_decode on the library's fixed device scratch: no workspace argument
    and no allocation. Raises PagedAttentionError (PA_ERR_WORKSPACE) when the
    call needs more than NOALLOC_SCRATCH_BYTES of scratch. Calls that may
    overlap on the GPU share the one scratch and race."""
    import torch
    _check_cuda("k_cache", k_cache, ndim=4)
    _check_cuda("v_cache", v_cache, k_cache.dtype, 4)
    _check_cuda("q", q, k_cache.dtype, 3)
    _check_cuda("out", out, k_cache.dtype, 3)
    _check_cuda("block_tables", block_tables, torch.int32, 2)
    _check_cuda("context_lens", context_lens, torch.int32, 1)
    if error_word is not None:
        _check_cuda("error_word", error_word, torch.int32)
    nb, hkv, bs, d = k_cache.shape
    B, hq, dq = q.shape
    if dq != d or tuple(out.shape) != tuple(q.shape) or tuple(v_cache.shape) != tuple(k_cache.shape) \
            or block_tables.shape[0] != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    _check_device(stream, q, out, k_cache, v_cache, block_tables, context_lens, error_word)
    rc = lib().pa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
                                 _ptr(context_lens), float(scale), _ptr(out), B, hq, hkv, d, bs,
                                 nb, int(block_tables.shape[1]), int(max_context_len),
                                 _dtype_code(k_cache), _ptr(error_word), _stream(stream))
    if rc != PA_OK:
        need = pa_decode_workspace_size(B, hq, d, int(max_context_len))
        what = "pa_decode_noalloc"
        if rc == PA_ERR_WORKSPACE:
            what += (f" (needs {need} bytes of scratch, the fixed scratch holds "
                     f"{NOALLOC_SCRATCH_BYTES}; pass a workspace to pa_decode instead)")
        raise PagedAttentionError(rc, what)


# The calls below check each tensor on the way to its pointer: on a decode step the
# host's part of a call is as long as a small kernel, and these attributes are
# most of it.

def _arg(name, t, dev, dtype=None, ndim=None):
    """The pointer of a contiguous CUDA tensor on device `dev` (torch's current
    one) with the given type and dimensions, or the checks' error."""
    try:
        if t.get_device() == dev and t.is_contiguous() and (dtype is None or t.dtype is dtype) \
                and (ndim is None or t.dim() == ndim):
            return t.data_ptr()
    except AttributeError:
        pass
    _check_cuda(name, t, dtype, ndim)
    _check_device(None, t)
    return t.data_ptr()


def _opt_arg(name, t, dev, dtype=None, ndim=None):
    return None if t is None else _arg(name, t, dev, dtype, ndim)


def _heads_arg(name, t, dev, dtype=None):
    """Pointer and token stride (elements) of a CUDA tensor [T][H][D] whose
    tokens may lie any distance apart (a part of a fused projection's output)."""
    try:
        T, H, D = t.shape
        st, sh, sd = t.stride()
        if t.get_device() == dev and sd == 1 and (sh == D or H == 1) and (dtype is None or t.dtype is dtype):
            return t.data_ptr(), (st if T > 1 else H * D)
    except (AttributeError, ValueError):
        pass
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions, got {t.dim()}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    T, H, D = t.shape
    st, sh, sd = t.stride()
    if (sd != 1 and D > 1) or (sh != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    _check_device(None, t)
    return t.data_ptr(), (st if T > 1 else H * D)


def _int32(name, v):
    """A number as the C int that it is passed as (ctypes would cut it to 32 bits)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {v}")
    return v


_raw_stream_of = None


def _stream_on(stream, dev):
    """The raw stream: the given one (on device `dev`), else torch's current one."""
    global _raw_stream_of
    if stream is not None:
        _check_device(stream)
        return _stream(stream)
    if _raw_stream_of is None:
        import torch
        _raw_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream_of(dev) or None


_plain_codes = {}


def _plain_dtype_code(t):
    """_dtype_code of a tensor, float32 and bfloat16 by one lookup."""
    if not _plain_codes:
        import torch
        _plain_codes.update({torch.float32: 0, torch.bfloat16: 1})
    code = _plain_codes.get(t.dtype)
    return _dtype_code(t) if code is None else code


def _int4_pool(k_cache, v_cache, k_params, v_params, dev):
    """((NB, Hkv, bs, D), the four pointers) of a 4-bit pool."""
    import torch
    ptrs = (_arg("k_cache", k_cache, dev, torch.uint8, 4), _arg("v_cache", v_cache, dev, torch.uint8),
            _arg("k_params", k_params, dev, torch.bfloat16),
            _arg("v_params", v_params, dev, torch.bfloat16))
    shape = k_cache.shape
    nb, hkv, bs, half = shape
    pairs = k_params.shape
    if v_cache.shape != shape or v_params.shape != pairs or pairs != (nb, hkv, bs, 2):
        raise ValueError("INT4 pools are [NB][Hkv][bs][D / 2] codes with [NB][Hkv][bs][2] params")
    return (nb, hkv, bs, 2 * half), ptrs


def pa_reshape_and_cache_int4(k_new, v_new, slot_mapping, k_cache, v_cache, k_params, v_params,
                              error_word=None, stream=None) -> None:
    """Quantising append into a 4-bit cache: k_new/v_new (bf16 or fp32,
    [T][Hkv][D]) -> codes (uint8 [NB][Hkv][bs][D / 2]) and one bf16 pair (lo, s)
    per row (params, [NB][Hkv][bs][2]); value = lo + s * code."""
    import torch
    dev = torch.cuda.current_device()
    (nb, hkv, bs, d), (kc, vc, kp, vp) = _int4_pool(k_cache, v_cache, k_params, v_params, dev)
    kn = _arg("k_new", k_new, dev, None, 3)
    vn = _arg("v_new", v_new, dev, k_new.dtype, 3)
    slots = _arg("slot_mapping", slot_mapping, dev, torch.int64, 1)
    T, h, dn = k_new.shape
    if h != hkv or dn != d or v_new.shape != k_new.shape or slot_mapping.shape[0] != T:
        raise ValueError("shape mismatch between k_new/v_new/slot_mapping and the caches")
    rc = lib().pa_reshape_and_cache_int4(kn, vn, _plain_dtype_code(k_new), slots, kc, vc, kp, vp, T, hkv,
                                         d, bs, nb, _opt_arg("error_word", error_word, dev, torch.int32),
                                         _stream_on(stream, dev))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_reshape_and_cache_int4")


def pa_gather_int4(k_cache, v_cache, k_params, v_params, block_tables, context_lens, row_starts,
                   k_out, v_out, max_context_len, error_word=None, stream=None) -> None:
    """The cached rows of every sequence as plain values: rows row_starts[s] ..
    row_starts[s] + context_lens[s] - 1 of k_out/v_out ([rows][Hkv][D], bf16 or
    fp32). row_starts: int64 [B]. Rows that no sequence covers stay as they are."""
    import torch
    dev = torch.cuda.current_device()
    (nb, hkv, bs, d), (kc, vc, kp, vp) = _int4_pool(k_cache, v_cache, k_params, v_params, dev)
    bt = _arg("block_tables", block_tables, dev, torch.int32, 2)
    cl = _arg("context_lens", context_lens, dev, torch.int32, 1)
    rs = _arg("row_starts", row_starts, dev, torch.int64, 1)
    ko = _arg("k_out", k_out, dev, None, 3)
    vo = _arg("v_out", v_out, dev, k_out.dtype, 3)
    B, mb = block_tables.shape
    rows, h, do = k_out.shape
    if context_lens.shape[0] != B or row_starts.shape[0] != B or v_out.shape != k_out.shape \
            or h != hkv or do != d:
        raise ValueError("shape mismatch between the outputs, the tables and the caches")
    bound = _int32("max_context_len", max_context_len)
    rc = lib().pa_gather_int4(kc, vc, kp, vp, bt, cl, rs, ko, vo, _plain_dtype_code(k_out), rows, B, hkv, d,
                              bs, nb, mb, bound,
                              _opt_arg("error_word", error_word, dev, torch.int32),
                              _stream_on(stream, dev))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_gather_int4")


def pa_decode_int4(q, k_cache, v_cache, k_params, v_params, block_tables, context_lens, scale,
                   out, max_context_len, window: int = 0, workspace=None, error_word=None,
                   stream=None) -> None:
    """Decode attention over a 4-bit cache. q/out: bf16 [B][Hq][D], or
    [B][Q][Hq][D] for the last Q tokens of every sequence (token j attends to
    rows 0 .. n - Q + j). window > 0: each token attends to its last `window`
    rows only. workspace: a CUDA tensor of at least
    pa_decode_workspace_size_multi(B, Q, Hq, D, max_context_len) bytes; when
    None, one is taken from torch's caching allocator for this call, on its stream."""
    import torch
    dev = torch.cuda.current_device()
    (nb, hkv, bs, d), (kc, vc, kp, vp) = _int4_pool(k_cache, v_cache, k_params, v_params, dev)
    qp = _arg("q", q, dev, torch.bfloat16)
    op = _arg("out", out, dev, torch.bfloat16)
    bt = _arg("block_tables", block_tables, dev, torch.int32, 2)
    cl = _arg("context_lens", context_lens, dev, torch.int32, 1)
    shape = q.shape
    if len(shape) == 3:
        (B, hq, dq), Q = shape, 1
    elif len(shape) == 4:
        B, Q, hq, dq = shape
    else:
        raise ValueError(f"q must have 3 or 4 dimensions, got {len(shape)}")
    rows, mb = block_tables.shape
    if dq != d or out.shape != shape or rows != B or context_lens.shape[0] != B:
        raise ValueError("shape mismatch between q/out/block_tables/context_lens and the caches")
    bound, window = _int32("max_context_len", max_context_len), _int32("window", window)
    if workspace is None:
        need = pa_decode_workspace_size_multi(B, Q, hq, d, bound)
        workspace = _scratch(need, stream, q.device)
    ws = _arg("workspace", workspace, dev)
    rc = lib().pa_decode_int4(qp, kc, vc, kp, vp, bt, cl, float(scale), window, op, B, Q, hq, hkv,
                              d, bs, nb, mb, bound, ws,
                              workspace.numel() * workspace.element_size(),
                              _opt_arg("error_word", error_word, dev, torch.int32),
                              _stream_on(stream, dev))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_decode_int4")


def _norm_rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight, eps, weight_offset,
                    interleaved, pair_axis, dev):
    import torch
    qp, q_stride = _heads_arg("q", q, dev)
    dt = q.dtype
    kp, k_stride = _heads_arg("k", k, dev, dt)
    op, q_out_stride = (qp, q_stride) if q_out is q else _heads_arg("q_out", q_out, dev, dt)
    shape, k_shape = q.shape, k.shape
    T, hq, d = shape
    if k_shape[0] != T or k_shape[2] != d or q_out.shape != shape:
        raise ValueError("shape mismatch between q, k and q_out")
    weight_dtype, wp = 0, [None, None]
    for i, (name, w) in enumerate((("q_weight", q_weight), ("k_weight", k_weight))):
        if w is not None:
            wp[i] = _arg(name, w, dev, None, 1)
            if w.shape[0] != d:
                raise ValueError(f"{name} must hold head_dim elements")
            weight_dtype = _plain_dtype_code(w)
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have the same type")
    rot, max_position, axes, axis_bytes, cs, pos = 0, 0, 1, None, None, None
    axis_ptr = 0
    if cos_sin is not None:
        cs = _arg("cos_sin", cos_sin, dev, torch.float32, 2)
        pos = _arg("positions", positions, dev, torch.int32)
        max_position, rot = cos_sin.shape
        pos_shape = positions.shape
        if len(pos_shape) not in (1, 2) or pos_shape[-1] != T:
            raise ValueError("positions must be [T] or [axes][T]")
        axes = 1 if len(pos_shape) == 1 else pos_shape[0]
        if pair_axis is not None:
            axis_bytes = bytes(pair_axis)
            if len(axis_bytes) != rot // 2:
                raise ValueError("pair_axis must hold rot_dim / 2 axis numbers")
            axis_ptr = ctypes.cast(axis_bytes, ctypes.c_void_p).value
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need cos_sin")
    # The second is what the first points at: it has to outlive the call.
    return _norm_rope_pack(qp, kp, q_stride, k_stride, op, q_out_stride, wp[0] or 0, wp[1] or 0, eps,
                           weight_offset, cs or 0, pos or 0, axis_ptr, T, hq, k_shape[1], d, rot,
                           max_position, axes, 1 if interleaved else 0, _plain_dtype_code(q),
                           weight_dtype), axis_bytes


def pa_norm_rope(q, k, positions, cos_sin, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6,
                 weight_offset=0.0, interleaved=False, pair_axis=None, error_word=None,
                 stream=None) -> None:
    """Per-head RMS norms of q ([T][Hq][D]) and k ([T][Hkv][D]) with their
    weights ([D]; None: no norm) and the rotation by position, in one pass into
    q_out and k_out (in place where they are q and k). The tokens of q, k and
    the outputs may lie any distance apart (parts of a fused projection).

    positions: int32 [T], or [axes][T] with pair_axis the axis number of each of
    the rot_dim / 2 pairs. cos_sin: fp32 [max_position][rot_dim], cosines then
    sines; None (with positions None): no rotation. interleaved: pairs are
    (2i, 2i + 1), else (i, i + rot_dim / 2)."""
    import torch
    dev = torch.cuda.current_device()
    args, _axes = _norm_rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight, eps,
                           weight_offset, interleaved, pair_axis, dev)
    ko, k_out_stride = _heads_arg("k_out", k_out, dev, k.dtype)
    if k_out.shape != k.shape:
        raise ValueError("shape mismatch between k and k_out")
    rc = lib().pa_norm_rope(args, ko, k_out_stride,
                            _opt_arg("error_word", error_word, dev, torch.int32),
                            _stream_on(stream, dev))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_norm_rope")


def _append_args(k, v, slot_mapping, hkv, d, dev):
    import torch
    vp, v_stride = _heads_arg("v", v, dev, k.dtype)
    slots = _arg("slot_mapping", slot_mapping, dev, torch.int64, 1)
    T, h, dk = k.shape
    if v.shape != k.shape or h != hkv or dk != d or slot_mapping.shape[0] != T:
        raise ValueError("shape mismatch between k/v/slot_mapping and the caches")
    return vp, v_stride, slots


def pa_norm_rope_append(q, k, v, positions, cos_sin, slot_mapping, q_out, k_cache, v_cache,
                        q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0,
                        interleaved=False, pair_axis=None, error_word=None, stream=None) -> None:
    """pa_norm_rope whose K rows go into their slots of the paged pool
    ([NB][Hkv][bs][D], q's type), with the V rows beside them (a bit copy).
    slot_mapping: int64 [T], negative = no append."""
    import torch
    dev = torch.cuda.current_device()
    args, _axes = _norm_rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight, eps,
                           weight_offset, interleaved, pair_axis, dev)
    kc = _arg("k_cache", k_cache, dev, q.dtype, 4)
    vc = _arg("v_cache", v_cache, dev, q.dtype, 4)
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must match k_cache")
    vp, v_stride, slots = _append_args(k, v, slot_mapping, hkv, d, dev)
    rc = lib().pa_norm_rope_append(args, vp, v_stride, slots, kc, vc, bs, nb,
                                   _opt_arg("error_word", error_word, dev, torch.int32),
                                   _stream_on(stream, dev))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_norm_rope_append")


def pa_norm_rope_append_int4(q, k, v, positions, cos_sin, slot_mapping, q_out, k_cache, v_cache,
                             k_params, v_params, q_weight=None, k_weight=None, eps=1e-6,
                             weight_offset=0.0, interleaved=False, pair_axis=None,
                             error_word=None, stream=None) -> None:
    """pa_norm_rope whose K rows are quantised into a 4-bit cache, with the V
    rows (codes and params as of pa_reshape_and_cache_int4 on pa_norm_rope's
    K rows). slot_mapping: int64 [T], negative = no append."""
    import torch
    dev = torch.cuda.current_device()
    (nb, hkv, bs, d), (kc, vc, kp, vq) = _int4_pool(k_cache, v_cache, k_params, v_params, dev)
    args, _axes = _norm_rope_args(q, k, positions, cos_sin, q_out, q_weight, k_weight, eps,
                           weight_offset, interleaved, pair_axis, dev)
    vp, v_stride, slots = _append_args(k, v, slot_mapping, hkv, d, dev)
    rc = lib().pa_norm_rope_append_int4(args, vp, v_stride, slots, kc, vc, kp, vq, bs, nb,
                                        _opt_arg("error_word", error_word, dev, torch.int32),
                                        _stream_on(stream, dev))
    if rc != PA_OK:
        raise PagedAttentionError(rc, "pa_norm_rope_append_int4")

"""ctypes binding of libattn.so (``include/attn.h``): argument marshalling only.

Every arithmetic step runs in the CUDA kernels behind ``attn_fwd``; this
module checks tensor devices, dtypes and contiguity, allocates the output with
PyTorch (PyTorch is used for device memory and streams only) and passes raw
pointers plus the current CUDA stream. When the library is missing the call
raises; there is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIBNAME = "libattn.so"
_lock = threading.Lock()
_lib = None

ATTN_F32, ATTN_F16, ATTN_BF16 = 0, 1, 2
KV8_INT8, KV8_E4M3 = 0, 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
MASK_NONE, MASK_CAUSAL, MASK_KEY_PADDING = 0, 1, 2


class AttnError(RuntimeError):
    """Raised when attn_fwd returns an error code or the library is missing."""

    def __init__(self, msg, code=None):
        super().__init__(msg)
        self.code = code


class Shape(ctypes.Structure):
    """attn_shape_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "Sq", "Sk", "D", "bias_b", "bias_h")]


class PagedShape(ctypes.Structure):
    """attn_paged_shape_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "num_queries", "Hq", "Hkv", "D", "page_size",
                                               "num_pages", "max_pages", "max_queries")]


class MlaShape(ctypes.Structure):
    """attn_mla_shape_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "num_queries", "H", "R", "Pd", "page_size",
                                               "num_pages", "max_pages", "max_queries")]


class Kv8Cache(ctypes.Structure):
    """attn_kv8_cache_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "Hkv", "D", "group", "format")]


class RopeShape(ctypes.Structure):
    """attn_rope_shape_t."""
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "S", "Hq", "Hk", "D", "rot")] +
                [(n, ctypes.c_int64 * 3) for n in ("q_strides", "k_strides", "q_out_strides", "k_out_strides")] +
                [("pos_batch_stride", ctypes.c_int64)])


class Pages(ctypes.Structure):
    """attn_pages_t."""
    _fields_ = [(n, ctypes.c_int32) for n in ("num_seqs", "max_pages", "page_size", "num_pages")]


def library_path() -> str:
    return os.path.join(_HERE, _LIBNAME)


def checked_library_path() -> str:
    """Path of the bounds-checked build (``build.build(checked=True)``)."""
    return os.path.join(_HERE, "libattn_checked.so")


def load_library():
    """Open libattn.so once; raise AttnError if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _open(library_path())
        return _lib


@contextlib.contextmanager
def use_library(path):
    """Route every call of this module through the library build at ``path``
    (for example the bounds-checked libattn_checked.so) while the block runs;
    its device status word is then the one :func:`device_status` reads."""
    global _lib
    lib = _open(path)
    with _lock:
        prev, _lib = _lib, lib
    try:
        yield lib
    finally:
        with _lock:
            _lib = prev


def _open(path):
    """Open a build of the library and declare its C signatures."""
    if not os.path.exists(path):
        raise AttnError(f"{path} is missing: build the CUDA library first "
                        "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp = ctypes.c_void_p
    lib.attn_fwd.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, ctypes.c_int, vp, vp,
                             ctypes.c_float, ctypes.c_int, vp, vp]
    lib.attn_fwd.restype = ctypes.c_int
    lib.attn_fwd_split.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, ctypes.c_int, vp, vp,
                                   ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t,
                                   vp, vp, vp]
    lib.attn_fwd_split.restype = ctypes.c_int
    lib.attn_split_workspace_bytes.argtypes = [ctypes.POINTER(Shape), ctypes.c_int,
                                               ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_split_workspace_bytes.restype = ctypes.c_int
    lib.attn_bwd.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, vp, vp, vp, ctypes.c_int, vp, vp,
                             ctypes.c_float, ctypes.c_int, vp, ctypes.c_size_t, vp, vp, vp, vp]
    lib.attn_bwd.restype = ctypes.c_int
    lib.attn_bwd_workspace_bytes.argtypes = [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_bwd_workspace_bytes.restype = ctypes.c_int
    lib.attn_paged_fwd.argtypes = [ctypes.POINTER(PagedShape), vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                   ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp, vp, vp]
    lib.attn_paged_workspace_bytes.argtypes = [ctypes.POINTER(PagedShape), ctypes.c_int,
                                               ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_paged_workspace_bytes.restype = ctypes.c_int
    lib.attn_paged_fwd.restype = ctypes.c_int
    lib.attn_paged_mla.argtypes = [ctypes.POINTER(MlaShape), vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                   ctypes.c_float, ctypes.c_int, ctypes.c_int, vp, ctypes.c_size_t, vp, vp, vp]
    lib.attn_paged_mla.restype = ctypes.c_int
    lib.attn_paged_mla_workspace_bytes.argtypes = [ctypes.POINTER(MlaShape), ctypes.c_int,
                                                   ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_paged_mla_workspace_bytes.restype = ctypes.c_int
    lib.attn_paged_bwd.argtypes = [ctypes.POINTER(PagedShape), vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                   ctypes.c_float, ctypes.c_int, vp, vp, vp, vp, ctypes.c_size_t, vp, vp, vp, vp]
    lib.attn_paged_bwd.restype = ctypes.c_int
    lib.attn_paged_bwd_workspace_bytes.argtypes = [ctypes.POINTER(PagedShape), ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_paged_bwd_workspace_bytes.restype = ctypes.c_int
    lib.attn_paged_mla_bwd.argtypes = [ctypes.POINTER(MlaShape), vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int,
                                       ctypes.c_float, ctypes.c_int, vp, vp, vp, vp, ctypes.c_size_t, vp, vp,
                                       vp, vp, vp]
    lib.attn_paged_mla_bwd.restype = ctypes.c_int
    lib.attn_paged_mla_bwd_workspace_bytes.argtypes = [ctypes.POINTER(MlaShape),
                                                       ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_paged_mla_bwd_workspace_bytes.restype = ctypes.c_int
    pi64 = ctypes.POINTER(ctypes.c_int64)
    lib.attn_kv8_write.argtypes = [ctypes.POINTER(Kv8Cache), ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, pi64,
                                   pi64, vp, vp, vp, ctypes.c_int, vp, vp, vp, vp, vp]
    lib.attn_kv8_write.restype = ctypes.c_int
    lib.attn_kv8_read.argtypes = [ctypes.POINTER(Kv8Cache), ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp,
                                  vp, vp, vp, vp, ctypes.c_int, vp, vp, vp]
    lib.attn_kv8_read.restype = ctypes.c_int
    lib.attn_paged_kv8_fwd.argtypes = [ctypes.POINTER(PagedShape), ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                       vp, vp, vp, ctypes.c_int, ctypes.c_float, ctypes.c_int, vp, ctypes.c_size_t,
                                       vp, vp, vp]
    lib.attn_paged_kv8_fwd.restype = ctypes.c_int
    lib.attn_paged_kv8_workspace_bytes.argtypes = [ctypes.POINTER(PagedShape), ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_paged_kv8_workspace_bytes.restype = ctypes.c_int
    lib.attn_rope.argtypes = [ctypes.POINTER(RopeShape), vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_float,
                              ctypes.c_int, vp, vp, vp]
    lib.attn_rope.restype = ctypes.c_int
    lib.attn_rope_axes.argtypes = [ctypes.POINTER(RopeShape), vp, vp, vp, ctypes.c_int64, ctypes.c_int, vp, vp,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_int, vp, vp, vp]
    lib.attn_rope_axes.restype = ctypes.c_int
    pvp, pool = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(Pages)
    lib.attn_pages_copy.argtypes = [ctypes.c_int, pvp, pi64, ctypes.c_int, vp, vp, ctypes.c_int, vp]
    lib.attn_pages_copy.restype = ctypes.c_int
    lib.attn_pages_fork.argtypes = [pool, vp, vp, vp, vp, vp, ctypes.c_int, vp]
    lib.attn_pages_fork.restype = ctypes.c_int
    lib.attn_pages_free.argtypes = [pool, vp, vp, vp, vp, ctypes.c_int, vp]
    lib.attn_pages_free.restype = ctypes.c_int
    lib.attn_pages_reserve.argtypes = [pool, vp, vp, vp, vp, pvp, pi64, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    lib.attn_pages_reserve.restype = ctypes.c_int
    lib.attn_pages_compact.argtypes = [pool, vp, vp, pvp, pi64, ctypes.c_int, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_pages_compact.restype = ctypes.c_int
    lib.attn_pages_workspace_bytes.argtypes = [pool, ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_pages_workspace_bytes.restype = ctypes.c_int
    lib.attn_paged_prefix_fwd.argtypes = [ctypes.POINTER(PagedShape), ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, vp,
                                          vp, vp, vp, ctypes.c_int, ctypes.c_float, ctypes.c_int, vp, ctypes.c_size_t,
                                          vp, vp, vp]
    lib.attn_paged_prefix_fwd.restype = ctypes.c_int
    lib.attn_paged_prefix_workspace_bytes.argtypes = [ctypes.POINTER(PagedShape), ctypes.c_int, ctypes.c_int,
                                                      ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_paged_prefix_workspace_bytes.restype = ctypes.c_int
    lib.attn_fwd_host.argtypes = [ctypes.POINTER(Shape), vp, vp, vp, ctypes.c_int, vp, vp, ctypes.c_float,
                                  ctypes.c_int, vp, ctypes.c_size_t, vp, vp]
    lib.attn_fwd_host.restype = ctypes.c_int
    lib.attn_fwd_host_workspace_bytes.argtypes = [ctypes.POINTER(Shape), ctypes.c_int, ctypes.c_int,
                                                  ctypes.POINTER(ctypes.c_size_t)]
    lib.attn_fwd_host_workspace_bytes.restype = ctypes.c_int
    lib.attn_strerror.argtypes = [ctypes.c_int]
    lib.attn_strerror.restype = ctypes.c_char_p
    lib.attn_last_cuda_error.argtypes = []
    lib.attn_last_cuda_error.restype = ctypes.c_int
    lib.attn_device_status.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.c_int]
    lib.attn_device_status.restype = ctypes.c_int
    lib.attn_selftest_wait_timeout.argtypes = [ctypes.c_uint, ctypes.c_void_p]
    lib.attn_selftest_wait_timeout.restype = ctypes.c_int
    lib.attn_version.argtypes = []
    lib.attn_version.restype = ctypes.c_int
    return lib


def strerror(code: int) -> str:
    return load_library().attn_strerror(int(code)).decode()


def check(code: int):
    if code != 0:
        lib = load_library()
        extra = ""
        if code == -9:
            extra = f" (cudaError {lib.attn_last_cuda_error()})"
        raise AttnError(f"attn_fwd failed: {strerror(code)}{extra}", code)


def device_status(device: int = 0, clear: bool = False) -> int:
    """Sticky kernel error flags of ``device`` (0 = no bounded wait expired)."""
    flags = ctypes.c_int(0)
    check(load_library().attn_device_status(int(device), ctypes.byref(flags), int(bool(clear))))
    return flags.value


def _dtype_code(t):
    import torch
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return ATTN_BF16
    if dtype is torch.float16:
        return ATTN_F16
    if dtype is torch.float32:
        return ATTN_F32
    raise AttnError(f"unsupported dtype {dtype}")


def call(shape: Shape, q_ptr, k_ptr, v_ptr, mask: int, kv_lens_ptr, bias_ptr, scale: float,
         dtype: int, out_ptr, stream_handle) -> None:
    """Raw attn_fwd call with integer pointers (0 for NULL); raises on error."""
    lib = load_library()
    check(lib.attn_fwd(ctypes.byref(shape), q_ptr or None, k_ptr or None, v_ptr or None, int(mask),
                       kv_lens_ptr or None, bias_ptr or None, float(scale), int(dtype),
                       out_ptr or None, stream_handle or None))


def call_split(shape: Shape, q_ptr, k_ptr, v_ptr, mask: int, kv_lens_ptr, bias_ptr, scale: float,
               dtype: int, num_splits: int, ws_ptr, ws_bytes: int, out_ptr, lse_ptr,
               stream_handle) -> None:
    """Raw attn_fwd_split call with integer pointers (0 for NULL); raises on error."""
    lib = load_library()
    check(lib.attn_fwd_split(ctypes.byref(shape), q_ptr or None, k_ptr or None, v_ptr or None,
                             int(mask), kv_lens_ptr or None, bias_ptr or None, float(scale), int(dtype),
                             int(num_splits), ws_ptr or None, int(ws_bytes), out_ptr or None,
                             lse_ptr or None, stream_handle or None))


def split_workspace_bytes(shape: Shape, num_splits: int) -> int:
    """Workspace bytes attn_fwd_split needs for ``shape`` and ``num_splits``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_split_workspace_bytes(ctypes.byref(shape), int(num_splits),
                                                    ctypes.byref(n)))
    return n.value


def fwd(q, k, v, *, causal: bool = False, kv_lens=None, bias=None, scale: float | None = None,
        out=None, stream=None, num_splits: int = 1, return_lse: bool = False, workspace=None, lse_out=None):
    """O = softmax(Q K^T * scale + mask + bias) V on the GPU.

    q: [B,Hq,Sq,D]; k, v: [B,Hkv,Sk,D]; float32, float16 or bfloat16, contiguous.
    kv_lens: int32 [B] valid key counts (enables the key-padding mask).
    bias: float32 [bias_b, bias_h, Sq, Sk], bias_b in {1,B}, bias_h in {1,Hq}.
    scale: defaults to 1/sqrt(D).
    num_splits: 1..32 key-range splits (attn_fwd_split); the fp32 workspace is
    taken from ``workspace`` (a CUDA uint8 tensor) or allocated here.
    return_lse: also return the float32 [B,Hq,Sq] row log-sum-exp (written
    into ``lse_out`` when given).
    Tensors on a CUDA device run on ``stream`` (default: the current stream)
    and the result is returned without synchronising. Host tensors run through
    attn_fwd_host on the current CUDA device (chunked uploads, kernels and
    downloads overlapped; synchronising); pinned host memory makes the copies
    asynchronous DMA.
    """
    import torch

    if q.device.type == "cpu":
        if num_splits != 1 or return_lse:
            raise AttnError("host tensors support num_splits=1 without lse only")
        return _fwd_host(q, k, v, causal=causal, kv_lens=kv_lens, bias=bias, scale=scale, out=out)
    dev = q.device
    for name, t in (("k", k), ("v", v)):
        if t.device != dev:
            raise AttnError(f"{name} is on {t.device}, q on {dev}")
        if t.dtype != q.dtype:
            raise AttnError(f"{name} dtype {t.dtype} differs from q dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 4:
            raise AttnError(f"{name} must be 4-D [B, H, S, D]")
        if not t.is_contiguous():
            raise AttnError(f"{name} must be contiguous")
    B, Hq, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    if tuple(k.shape) != (B, Hkv, Sk, D) or tuple(v.shape) != tuple(k.shape):
        raise AttnError("k and v must be [B, Hkv, Sk, D] matching q")
    mask = MASK_CAUSAL if causal else MASK_NONE
    kv_ptr = 0
    if kv_lens is not None:
        if kv_lens.device != dev or kv_lens.dtype != torch.int32 or tuple(kv_lens.shape) != (B,):
            raise AttnError("kv_lens must be int32 [B] on q's device")
        kv_lens = kv_lens.contiguous()
        mask |= MASK_KEY_PADDING
        kv_ptr = kv_lens.data_ptr()
    bb = bh = 1
    b_ptr = 0
    if bias is not None:
        if bias.device != dev or bias.dtype != torch.float32 or bias.dim() != 4 or not bias.is_contiguous():
            raise AttnError("bias must be a contiguous float32 [bias_b, bias_h, Sq, Sk] tensor on q's device")
        bb, bh = int(bias.shape[0]), int(bias.shape[1])
        if tuple(bias.shape[2:]) != (Sq, Sk):
            raise AttnError("bias must be [bias_b, bias_h, Sq, Sk]")
        b_ptr = bias.data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        raise AttnError("out must be a contiguous tensor like q")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    shape = Shape(B, Hq, Hkv, Sq, Sk, D, bb, bh)
    if num_splits == 1 and not return_lse:
        call(shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), mask, kv_ptr, b_ptr, scale,
             _dtype_code(q), out.data_ptr(), stream.cuda_stream)
        return out
    lse = _lse_buffer(lse_out, (B, Hq, Sq), dev) if return_lse else None
    need = split_workspace_bytes(shape, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise AttnError(f"workspace must hold {need} bytes on q's device")
    call_split(shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), mask, kv_ptr, b_ptr, scale,
               _dtype_code(q), num_splits, workspace.data_ptr() if need else 0, need,
               out.data_ptr(), lse.data_ptr() if lse is not None else 0, stream.cuda_stream)
    return (out, lse) if return_lse else out


def host_workspace_bytes(shape: Shape, dtype_code: int, with_bias: bool) -> int:
    """Device workspace attn_fwd_host needs for ``shape``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_fwd_host_workspace_bytes(ctypes.byref(shape), int(dtype_code), int(bool(with_bias)),
                                                      ctypes.byref(n)))
    return n.value


def _fwd_host(q, k, v, *, causal, kv_lens, bias, scale, out, workspace=None):
    """Host tensors in, host tensor out (attn_fwd_host): chunked uploads, the
    kernel per chunk and downloads overlapped on three streams; synchronises."""
    import torch

    for name, t in (("k", k), ("v", v), ("kv_lens", kv_lens), ("bias", bias), ("out", out)):
        if t is not None and t.device.type != "cpu":
            raise AttnError(f"{name} must be a host tensor like q")
    for name, t in (("k", k), ("v", v)):
        if t.dtype != q.dtype:
            raise AttnError(f"{name} dtype {t.dtype} differs from q dtype {q.dtype}")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != 4 or not t.is_contiguous():
            raise AttnError(f"{name} must be a contiguous 4-D [B, H, S, D] tensor")
    B, Hq, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    if tuple(k.shape) != (B, Hkv, Sk, D) or tuple(v.shape) != tuple(k.shape):
        raise AttnError("k and v must be [B, Hkv, Sk, D] matching q")
    mask = MASK_CAUSAL if causal else MASK_NONE
    if kv_lens is not None:
        if kv_lens.dtype != torch.int32 or tuple(kv_lens.shape) != (B,) or not kv_lens.is_contiguous():
            raise AttnError("kv_lens must be a contiguous int32 [B] host tensor")
        mask |= MASK_KEY_PADDING
    bb = bh = 1
    if bias is not None:
        if bias.dtype != torch.float32 or bias.dim() != 4 or not bias.is_contiguous() or \
                tuple(bias.shape[2:]) != (Sq, Sk):
            raise AttnError("bias must be a contiguous float32 [bias_b, bias_h, Sq, Sk] host tensor")
        bb, bh = int(bias.shape[0]), int(bias.shape[1])
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise AttnError("out must be a contiguous host tensor like q")
    dev = torch.device("cuda", torch.cuda.current_device())
    shape = Shape(B, Hq, Hkv, Sq, Sk, D, bb, bh)
    need = host_workspace_bytes(shape, _dtype_code(q), bias is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise AttnError(f"workspace must hold {need} bytes on the current device")
    stream = torch.cuda.current_stream(dev)
    ptr = lambda t: (t.data_ptr() or None) if t is not None else None
    check(load_library().attn_fwd_host(ctypes.byref(shape), ptr(q), ptr(k), ptr(v), mask, ptr(kv_lens), ptr(bias),
                                       ctypes.c_float(scale), _dtype_code(q), ptr(workspace) if need else None, need,
                                       ptr(out), stream.cuda_stream or None))
    stream.synchronize()
    return out


def bwd_workspace_bytes(shape: Shape) -> int:
    """Workspace bytes attn_bwd needs for ``shape``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_bwd_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def bwd(q, k, v, out, dout, lse, *, causal: bool = False, kv_lens=None, bias=None,
        scale: float | None = None, workspace=None, stream=None, dq=None, dk=None, dv=None):
    """Gradients (dq, dk, dv) of attention for dL/dO = ``dout`` (attn_bwd).

    q, k, v, kv_lens, bias, scale, causal: as given to the forward; ``out`` its
    output and ``lse`` its float32 [B,Hq,Sq] row log-sum-exp (``fwd(...,
    return_lse=True)``); ``dout`` like ``out``. All on one CUDA device,
    contiguous. Returns dq (like q), dk and dv (like k and v): the given
    ``dq``/``dk``/``dv`` tensors when passed, else new ones.
    """
    import torch

    dev = q.device
    for name, t in (("k", k), ("v", v), ("out", out), ("dout", dout)):
        if t.device != dev or t.dtype != q.dtype or not t.is_contiguous():
            raise AttnError(f"{name} must be a contiguous {q.dtype} tensor on {dev}")
    if not q.is_contiguous() or q.dim() != 4 or k.dim() != 4:
        raise AttnError("q, k, v must be contiguous 4-D tensors")
    B, Hq, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    if tuple(out.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape) or tuple(v.shape) != tuple(k.shape):
        raise AttnError("out and dout must be like q, v like k")
    if lse.device != dev or lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Sq) or not lse.is_contiguous():
        raise AttnError("lse must be a contiguous float32 [B, Hq, Sq] tensor on q's device")
    mask = MASK_CAUSAL if causal else MASK_NONE
    kv_ptr = 0
    if kv_lens is not None:
        if kv_lens.device != dev or kv_lens.dtype != torch.int32 or tuple(kv_lens.shape) != (B,):
            raise AttnError("kv_lens must be int32 [B] on q's device")
        kv_lens = kv_lens.contiguous()
        mask |= MASK_KEY_PADDING
        kv_ptr = kv_lens.data_ptr()
    bb = bh = 1
    b_ptr = 0
    if bias is not None:
        if bias.device != dev or bias.dtype != torch.float32 or bias.dim() != 4 or not bias.is_contiguous():
            raise AttnError("bias must be a contiguous float32 [bias_b, bias_h, Sq, Sk] tensor on q's device")
        bb, bh = int(bias.shape[0]), int(bias.shape[1])
        b_ptr = bias.data_ptr()
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    shape = Shape(B, Hq, Hkv, Sq, Sk, D, bb, bh)
    need = bwd_workspace_bytes(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise AttnError(f"workspace must hold {need} bytes on q's device")
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != dev
                              or not t.is_contiguous()):
            raise AttnError(f"{name} must be a contiguous tensor like {'q' if like is q else 'k'}")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    check(load_library().attn_bwd(ctypes.byref(shape), q.data_ptr() or None, k.data_ptr() or None,
                                  v.data_ptr() or None, out.data_ptr() or None, dout.data_ptr() or None,
                                  lse.data_ptr() or None, mask, kv_ptr or None, b_ptr or None, float(scale),
                                  _dtype_code(q), workspace.data_ptr() if need else None, need,
                                  dq.data_ptr() or None, dk.data_ptr() or None, dv.data_ptr() or None,
                                  stream.cuda_stream or None))
    return dq, dk, dv


def _lse_buffer(lse_out, shape, dev):
    import torch
    if lse_out is None:
        return torch.empty(shape, dtype=torch.float32, device=dev)
    if (tuple(lse_out.shape) != tuple(shape) or lse_out.dtype != torch.float32 or lse_out.device != dev
            or not lse_out.is_contiguous()):
        raise AttnError(f"lse_out must be a contiguous float32 {list(shape)} tensor on q's device")
    return lse_out


def _grad_buffer(name, given, like):
    import torch
    if given is None:
        return torch.empty_like(like)
    if (given.shape != like.shape or given.dtype != like.dtype or given.device != like.device
            or not given.is_contiguous()):
        raise AttnError(f"{name} must be a contiguous tensor shaped like its input")
    return given


def paged_workspace_bytes(shape: PagedShape, num_splits: int) -> int:
    """Workspace bytes attn_paged_fwd needs for ``shape`` and ``num_splits``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_paged_workspace_bytes(ctypes.byref(shape), int(num_splits), ctypes.byref(n)))
    return n.value


def paged_fwd(q, k_cache, v_cache, block_table, seq_lens, q_offsets, *, positions=None, causal: bool = True,
              scale: float | None = None, max_queries: int | None = None, return_lse: bool = False, out=None,
              stream=None, num_splits: int = 1, workspace=None, lse_out=None):
    """Attention of packed queries over a paged key/value cache (attn_paged_fwd).

    q [queries, Hq, D]; k_cache, v_cache [pages, page_size, Hkv, D] (same
    dtype, CUDA, contiguous); block_table int32 [num_seqs, max_pages];
    seq_lens int32 [num_seqs]; q_offsets int32 [num_seqs + 1]; positions
    int32 [queries] or None. ``max_queries`` bounds the queries of one
    sequence (computed from q_offsets, with a host sync, when None).
    ``num_splits`` splits the keys of decode-shaped calls (workspace taken
    from ``workspace``, a CUDA uint8 tensor, or allocated here).
    Returns out [queries, Hq, D] (and lse float32 [queries, Hq], written into
    ``lse_out`` when given).
    """
    import torch

    dev = q.device
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.device != dev or t.dtype != q.dtype or not t.is_contiguous() or t.dim() != 4:
            raise AttnError(f"{name} must be a contiguous 4-D {q.dtype} tensor on {dev}")
    if q.dim() != 3 or not q.is_contiguous():
        raise AttnError("q must be a contiguous [queries, Hq, D] tensor")
    nq, Hq, D = q.shape
    pages, P, Hkv, Dk = k_cache.shape
    if Dk != D or v_cache.shape != k_cache.shape:
        raise AttnError("k_cache and v_cache must be [pages, page_size, Hkv, D] with q's D")
    ints = {}
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens), ("q_offsets", q_offsets),
                    ("positions", positions)):
        if t is None:
            continue
        if t.device != dev or t.dtype != torch.int32 or not t.is_contiguous():
            raise AttnError(f"{name} must be a contiguous int32 tensor on q's device")
        ints[name] = t
    ns = int(seq_lens.shape[0])
    if block_table.dim() != 2 or block_table.shape[0] != ns or tuple(q_offsets.shape) != (ns + 1,):
        raise AttnError("block_table must be [num_seqs, max_pages] and q_offsets [num_seqs + 1]")
    if positions is not None and tuple(positions.shape) != (nq,):
        raise AttnError("positions must be int32 [queries]")
    if max_queries is None:
        max_queries = int((q_offsets[1:] - q_offsets[:-1]).max().item()) if ns else 0
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    lse = _lse_buffer(lse_out, (nq, Hq), dev) if return_lse else None
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    shape = PagedShape(ns, nq, Hq, Hkv, D, P, pages, int(block_table.shape[1]), int(max_queries))
    need = paged_workspace_bytes(shape, num_splits)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif need and (workspace.device != dev or workspace.numel() * workspace.element_size() < need):
        raise AttnError(f"workspace must hold {need} bytes on q's device")
    ptr = lambda t: (t.data_ptr() or None) if t is not None else None
    check(load_library().attn_paged_fwd(ctypes.byref(shape), ptr(q), ptr(k_cache), ptr(v_cache), ptr(block_table),
                                        ptr(seq_lens), ptr(q_offsets), ptr(positions), int(bool(causal)),
                                        float(scale), _dtype_code(q), int(num_splits),
                                        ptr(workspace) if need else None, need, ptr(out), ptr(lse),
                                        stream.cuda_stream or None))
    return (out, lse) if return_lse else out


def mla_workspace_bytes(shape: MlaShape, num_splits: int) -> int:
    """Workspace bytes attn_paged_mla needs for ``shape`` and ``num_splits``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_paged_mla_workspace_bytes(ctypes.byref(shape), int(num_splits), ctypes.byref(n)))
    return n.value


def paged_mla(q, qp, latent, kpos, block_table, seq_lens, q_offsets, *, positions=None, causal: bool = True,
              scale: float, max_queries: int | None = None, return_lse: bool = False, out=None, stream=None,
              num_splits: int = 1, workspace=None, lse_out=None):
    """MLA with absorbed projections over a paged latent cache (attn_paged_mla).

    q [queries, H, R]; qp [queries, H, Pd]; latent [pages, page_size, 1, R];
    kpos [pages, page_size, 1, Pd]; metadata as for :func:`paged_fwd`;
    ``scale`` is the original model's QK scale. ``num_splits`` splits the key
    range of every 128-row block (workspace taken from ``workspace``, a CUDA
    uint8 tensor, or allocated here). Returns out [queries, H, R] (and lse
    float32 [queries, H], written into ``lse_out`` when given).
    """
    import torch

    dev = q.device
    for name, t in (("qp", qp), ("latent", latent), ("kpos", kpos)):
        if t.device != dev or t.dtype != q.dtype or not t.is_contiguous():
            raise AttnError(f"{name} must be a contiguous {q.dtype} tensor on {dev}")
    if q.dim() != 3 or not q.is_contiguous() or latent.dim() != 4 or latent.shape[2] != 1:
        raise AttnError("q [queries, H, R] and latent [pages, page_size, 1, R]")
    nq, H, R = q.shape
    pages, P = int(latent.shape[0]), int(latent.shape[1])
    Pd = int(qp.shape[2])
    if tuple(latent.shape) != (pages, P, 1, R) or tuple(kpos.shape) != (pages, P, 1, Pd) or \
            tuple(qp.shape) != (nq, H, Pd):
        raise AttnError("qp [queries, H, Pd], kpos [pages, page_size, 1, Pd] must match q and latent")
    for name, t in (("block_table", block_table), ("seq_lens", seq_lens), ("q_offsets", q_offsets),
                    ("positions", positions)):
        if t is not None and (t.device != dev or t.dtype != torch.int32 or not t.is_contiguous()):
            raise AttnError(f"{name} must be a contiguous int32 tensor on q's device")
    ns = int(seq_lens.shape[0])
    if max_queries is None:
        max_queries = int((q_offsets[1:] - q_offsets[:-1]).max().item()) if ns else 0
    if out is None:
        out = torch.empty_like(q)
    lse = _lse_buffer(lse_out, (nq, H), dev) if return_lse else None
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    shape = MlaShape(ns, nq, H, R, Pd, P, pages, int(block_table.shape[1]), int(max_queries))
    need = mla_workspace_bytes(shape, num_splits)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif need and (workspace.device != dev or workspace.numel() * workspace.element_size() < need):
        raise AttnError(f"workspace must hold {need} bytes on q's device")
    ptr = lambda t: (t.data_ptr() or None) if t is not None else None
    check(load_library().attn_paged_mla(ctypes.byref(shape), ptr(q), ptr(qp), ptr(latent), ptr(kpos),
                                        ptr(block_table), ptr(seq_lens), ptr(q_offsets), ptr(positions),
                                        int(bool(causal)), float(scale), _dtype_code(q), int(num_splits),
                                        ptr(workspace) if need else None, need, ptr(out), ptr(lse),
                                        stream.cuda_stream or None))
    return (out, lse) if return_lse else out


def paged_bwd_workspace_bytes(shape: PagedShape) -> int:
    """Workspace bytes attn_paged_bwd needs for ``shape``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_paged_bwd_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def _workspace(need, workspace, dev):
    import torch
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if workspace.device != dev or workspace.numel() * workspace.element_size() < need:
        raise AttnError(f"workspace must hold {need} bytes on q's device")
    return workspace


def paged_bwd(q, k_cache, v_cache, block_table, seq_lens, q_offsets, dout, *, out=None, lse=None, positions=None,
              causal: bool = True, scale: float | None = None, max_queries: int | None = None,
              grads=("dq", "dk", "dv"), workspace=None, stream=None, dq=None, dk=None, dv=None):
    """Gradients of :func:`paged_fwd` for dL/dO = ``dout`` (attn_paged_bwd, ordered).

    Arguments as for :func:`paged_fwd`; ``out`` and ``lse`` are the forward's
    output and float32 [queries, Hq] log-sum-exp (when either is None the
    forward runs here first to recompute them). ``grads`` names the gradients
    wanted; ``dq``/``dk``/``dv`` receive them when given. Returns (dq
    [queries, Hq, D], dk, dv [pages, page_size, Hkv, D]), None in place of a
    gradient not asked for.
    """
    import torch

    dev = q.device
    if dout.device != dev or dout.dtype != q.dtype or tuple(dout.shape) != tuple(q.shape) or not dout.is_contiguous():
        raise AttnError("dout must be a contiguous tensor like q")
    nq, Hq, D = q.shape
    pages, P, Hkv, _ = k_cache.shape
    ns = int(seq_lens.shape[0])
    if max_queries is None:
        max_queries = int((q_offsets[1:] - q_offsets[:-1]).max().item()) if ns else 0
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None or lse is None:
        out, lse = paged_fwd(q, k_cache, v_cache, block_table, seq_lens, q_offsets, positions=positions,
                             causal=causal, scale=scale, max_queries=max_queries, return_lse=True, stream=stream)
    if out.device != dev or out.dtype != q.dtype or tuple(out.shape) != tuple(q.shape) or not out.is_contiguous():
        raise AttnError("out must be a contiguous tensor like q")
    if lse.device != dev or lse.dtype != torch.float32 or tuple(lse.shape) != (nq, Hq) or not lse.is_contiguous():
        raise AttnError("lse must be a contiguous float32 [queries, Hq] tensor on q's device")
    shape = PagedShape(ns, nq, Hq, Hkv, D, P, pages, int(block_table.shape[1]), int(max_queries))
    need = paged_bwd_workspace_bytes(shape)
    workspace = _workspace(need, workspace, dev)
    dq = _grad_buffer("dq", dq, q) if "dq" in grads else None
    dk = _grad_buffer("dk", dk, k_cache) if "dk" in grads else None
    dv = _grad_buffer("dv", dv, v_cache) if "dv" in grads else None
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    ptr = lambda t: (t.data_ptr() or None) if t is not None else None
    check(load_library().attn_paged_bwd(ctypes.byref(shape), ptr(q), ptr(k_cache), ptr(v_cache), ptr(block_table),
                                        ptr(seq_lens), ptr(q_offsets), ptr(positions), int(bool(causal)),
                                        float(scale), _dtype_code(q), ptr(out), ptr(dout), ptr(lse),
                                        ptr(workspace), need, ptr(dq), ptr(dk), ptr(dv), stream.cuda_stream or None))
    return dq, dk, dv


def mla_bwd_workspace_bytes(shape: MlaShape) -> int:
    """Workspace bytes attn_paged_mla_bwd needs for ``shape``."""
    n = ctypes.c_size_t(0)
    check(load_library().attn_paged_mla_bwd_workspace_bytes(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def paged_mla_bwd(q, qp, latent, kpos, block_table, seq_lens, q_offsets, dout, *, out=None, lse=None,
                  positions=None, causal: bool = True, scale: float, max_queries: int | None = None,
                  grads=("dq", "dqp", "dlatent", "dkpos"), workspace=None, stream=None, dq=None, dqp=None,
                  dlatent=None, dkpos=None):
    """Gradients of :func:`paged_mla` for dL/dO = ``dout`` (attn_paged_mla_bwd, ordered).

    Returns (dq [queries, H, R], dqp [queries, H, Pd], dlatent [pages,
    page_size, 1, R] with its key and value parts, dkpos [pages, page_size, 1,
    Pd]), None in place of a gradient not asked for (or of dqp, dkpos when
    Pd == 0); the given ``dq``/``dqp``/``dlatent``/``dkpos`` tensors receive
    them. ``out``/``lse`` as for :func:`paged_bwd`.
    """
    import torch

    dev = q.device
    if dout.device != dev or dout.dtype != q.dtype or tuple(dout.shape) != tuple(q.shape) or not dout.is_contiguous():
        raise AttnError("dout must be a contiguous tensor like q")
    nq, H, R = q.shape
    pages, P = int(latent.shape[0]), int(latent.shape[1])
    Pd = int(qp.shape[2])
    ns = int(seq_lens.shape[0])
    if max_queries is None:
        max_queries = int((q_offsets[1:] - q_offsets[:-1]).max().item()) if ns else 0
    if out is None or lse is None:
        out, lse = paged_mla(q, qp, latent, kpos, block_table, seq_lens, q_offsets, positions=positions,
                             causal=causal, scale=scale, max_queries=max_queries, return_lse=True, stream=stream)
    if out.device != dev or out.dtype != q.dtype or tuple(out.shape) != tuple(q.shape) or not out.is_contiguous():
        raise AttnError("out must be a contiguous tensor like q")
    if lse.device != dev or lse.dtype != torch.float32 or tuple(lse.shape) != (nq, H) or not lse.is_contiguous():
        raise AttnError("lse must be a contiguous float32 [queries, H] tensor on q's device")
    shape = MlaShape(ns, nq, H, R, Pd, P, pages, int(block_table.shape[1]), int(max_queries))
    need = mla_bwd_workspace_bytes(shape)
    workspace = _workspace(need, workspace, dev)
    dq = _grad_buffer("dq", dq, q) if "dq" in grads else None
    dqp = _grad_buffer("dqp", dqp, qp) if "dqp" in grads and Pd else None
    dlat = _grad_buffer("dlatent", dlatent, latent) if "dlatent" in grads else None
    dkp = _grad_buffer("dkpos", dkpos, kpos) if "dkpos" in grads and Pd else None
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    ptr = lambda t: (t.data_ptr() or None) if t is not None else None
    check(load_library().attn_paged_mla_bwd(ctypes.byref(shape), ptr(q), ptr(qp), ptr(latent), ptr(kpos),
                                            ptr(block_table), ptr(seq_lens), ptr(q_offsets), ptr(positions),
                                            int(bool(causal)), float(scale), _dtype_code(q), ptr(out), ptr(dout),
                                            ptr(lse), ptr(workspace), need, ptr(dq), ptr(dqp), ptr(dlat), ptr(dkp),
                                            stream.cuda_stream or None))
    return dq, dqp, dlat, dkp


# ------------------------------------------------------------------ 8-bit paged cache
# These calls are a few microseconds of GPU work at their smallest, so the
# marshalling below takes the short way: raw stream handles, one query of a
# tensor's shape and strides, descriptions packed at once.
def _launch(dev, fn, *args):
    """Calls the library with the tensors' device current (it launches on the current one)."""
    import torch
    if torch._C._cuda_getDevice() == dev.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc:
        check(rc)


def _stream(stream, dev, made=()):
    """Handle of ``stream`` (None: the current one). Tensors made here for a call
    on another stream than the current one are kept until that stream is done."""
    import torch
    if dev.type != "cuda":
        raise AttnError(f"tensors must be on a CUDA device, not {dev}")
    cur = torch._C._cuda_getCurrentRawStream(dev.index)
    if stream is None:
        return cur or None
    handle = stream.cuda_stream
    if handle != cur:
        for t in made:
            t.record_stream(stream)
    return handle or None


def _int32(name, t, shape, dev):
    import torch
    if t.dtype is not torch.int32 or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise AttnError(f"{name} must be a contiguous int32 {list(shape)} tensor on {dev}")
    return t.data_ptr() or None


def _kv8_check(dev, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, offsets, offsets_name):
    """Checks an 8-bit cache and its metadata: its C description, the number of
    sequences, max_pages, and the addresses in the order of the arguments."""
    import torch
    dtype, size = k_cache.dtype, k_cache.shape
    fmt = KV8_INT8 if dtype is torch.int8 else KV8_E4M3 if dtype is torch.float8_e4m3fn else None
    if fmt is None or len(size) != 4 or k_cache.device != dev or not k_cache.is_contiguous():
        raise AttnError(f"k_cache must be a contiguous int8 or float8_e4m3fn [pages, page_size, Hkv, D] tensor on {dev}")
    pages, P, H, D = size
    if v_cache.dtype is not dtype or v_cache.shape != size or v_cache.device != dev or not v_cache.is_contiguous():
        raise AttnError("v_cache must be a contiguous tensor like k_cache")
    scales = k_scale.shape
    if len(scales) != 3 or scales[0] != pages or scales[1] != H or scales[2] < 1 or P % scales[2]:
        raise AttnError("k_scale must be [pages, Hkv, page_size / group], group a divisor of page_size")
    f32 = torch.float32
    if (k_scale.dtype is not f32 or k_scale.device != dev or not k_scale.is_contiguous() or v_scale.dtype is not f32
            or v_scale.shape != scales or v_scale.device != dev or not v_scale.is_contiguous()):
        raise AttnError(f"k_scale and v_scale must be contiguous float32 {list(scales)} tensors on {dev}")
    lens, table = seq_lens.shape, block_table.shape
    if len(lens) != 1 or len(table) != 2:
        raise AttnError("block_table must be int32 [num_seqs, max_pages] and seq_lens int32 [num_seqs]")
    ns = lens[0]
    ptrs = (k_cache.data_ptr() or None, v_cache.data_ptr() or None, k_scale.data_ptr() or None,
            v_scale.data_ptr() or None, _int32("block_table", block_table, (ns, table[1]), dev),
            _int32("seq_lens", seq_lens, (ns,), dev), _int32(offsets_name, offsets, (ns + 1,), dev))
    return Kv8Cache(pages, P, H, D, P // scales[2], fmt), ns, table[1], ptrs


_STRIDES2 = ctypes.c_int64 * 2


def kv8_write(k, v, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, tok_offsets, *, stream=None):
    """Quantise the newest tokens of every sequence into an 8-bit paged cache, in place (attn_kv8_write).

    k, v [tokens, Hkv, D] float32, float16 or bfloat16: packed tokens, rows
    tok_offsets[s] .. tok_offsets[s+1]-1 the last ones of sequence s, whose
    length seq_lens[s] counts them. A head's D elements lie side by side; tokens
    and heads may be strided (slices of a fused projection). k_cache, v_cache
    [pages, page_size, Hkv, D] int8 or float8_e4m3fn; k_scale, v_scale float32
    [pages, Hkv, page_size / group], one scale for every ``group`` consecutive
    tokens of a head; block_table int32 [num_seqs, max_pages]; seq_lens int32
    [num_seqs]; tok_offsets int32 [num_seqs + 1]. A group that an earlier call
    began keeps its scale or gets a larger one, with its codes brought to it.
    """
    dev = k.device
    cache, ns, max_pages, (kc, vc, ks, vs, bt, sl, to) = _kv8_check(dev, k_cache, v_cache, k_scale, v_scale,
                                                                   block_table, seq_lens, tok_offsets, "tok_offsets")
    size = k.shape
    if len(size) != 3 or size[1] != cache.Hkv or size[2] != cache.D:
        raise AttnError("k and v must be [tokens, Hkv, D] with the cache's Hkv and D")
    if v.device != dev or v.dtype is not k.dtype or v.shape != size:
        raise AttnError(f"v must be a tensor like k, {k.dtype} {list(size)} on {dev}")
    kst, vst = k.stride(), v.stride()
    if kst[2] != 1 or vst[2] != 1:
        raise AttnError("the last dimension of k and v must be contiguous")
    lib = _lib or load_library()
    st = _stream(stream, dev)
    _launch(dev, lib.attn_kv8_write, cache, ns, max_pages, size[0], k.data_ptr() or None, v.data_ptr() or None,
            _STRIDES2(kst[0], kst[1]), _STRIDES2(vst[0], vst[1]), bt, sl, to, _dtype_code(k), kc, vc, ks, vs, st)


def kv8_read(k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, row_offsets, num_rows: int | None = None, *,
             starts=None, dtype=None, k_out=None, v_out=None, stream=None):
    """Values of an 8-bit paged cache as packed rows (attn_kv8_read).

    Row row_offsets[s] + i of the result is token starts[s] + i of sequence s
    (``starts`` int32 [num_seqs], None: from its first token), code * scale in
    ``dtype`` (float32, float16 or bfloat16; default bfloat16, or that of
    ``k_out``). ``num_rows`` is the number of rows (None: that of ``k_out``, or
    read from row_offsets with a host sync). Tokens past a sequence's end and
    pages outside the cache read as zeros; rows of no sequence are not written.
    Returns k, v [num_rows, Hkv, D] (``k_out``/``v_out`` when given).
    """
    import torch

    dev = k_cache.device
    cache, ns, max_pages, (kc, vc, ks, vs, bt, sl, ro) = _kv8_check(dev, k_cache, v_cache, k_scale, v_scale,
                                                                   block_table, seq_lens, row_offsets, "row_offsets")
    like = k_out if k_out is not None else v_out
    if num_rows is None:
        num_rows = like.shape[0] if like is not None else int(row_offsets[-1].item())
    if dtype is None:
        dtype = like.dtype if like is not None else torch.bfloat16
    size = (num_rows, cache.Hkv, cache.D)
    if like is None:  # one allocation for both
        both = k_scale.new_empty((2, *size), dtype=dtype)
        k_out, v_out = both.unbind(0)
        made = (both,)
    else:
        made = []
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            if t is not None and (t.shape != size or t.dtype is not dtype or t.device != dev or not t.is_contiguous()):
                raise AttnError(f"{name} must be a contiguous {dtype} {list(size)} tensor on {dev}")
        if k_out is None:
            made.append(k_out := torch.empty_like(v_out))
        if v_out is None:
            made.append(v_out := torch.empty_like(k_out))
    lib = _lib or load_library()
    st = _stream(stream, dev, made)
    _launch(dev, lib.attn_kv8_read, cache, ns, max_pages, num_rows, kc, vc, ks, vs, bt, sl, ro,
            _int32("starts", starts, (ns,), dev) if starts is not None else None, _dtype_code(k_out),
            k_out.data_ptr() or None, v_out.data_ptr() or None, st)
    return k_out, v_out


def paged_kv8_workspace_bytes(shape: PagedShape) -> int:
    """Workspace bytes attn_paged_kv8_fwd needs for ``shape``."""
    n = ctypes.c_size_t(0)
    rc = (_lib or load_library()).attn_paged_kv8_workspace_bytes(shape, n)
    if rc:
        check(rc)
    return n.value


def paged_kv8_fwd(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, q_offsets, *, positions=None,
                  causal: bool = True, scale: float | None = None, max_queries: int | None = None,
                  return_lse: bool = False, out=None, stream=None, workspace=None, lse_out=None):
    """:func:`paged_fwd` over an 8-bit paged cache (attn_paged_kv8_fwd).

    q [queries, Hq, D] float32, float16 or bfloat16; the cache, its scales and
    block_table as for :func:`kv8_write`; the other arguments and the results as
    for :func:`paged_fwd`. The kernel shares out the keys by itself, so there is
    no ``num_splits``; its ``workspace`` (a CUDA uint8 tensor of
    :func:`paged_kv8_workspace_bytes`) is allocated here when not given.
    """
    import torch

    dev, size = q.device, q.shape
    if len(size) != 3 or not q.is_contiguous():
        raise AttnError("q must be a contiguous [queries, Hq, D] tensor")
    cache, ns, max_pages, (kc, vc, ks, vs, bt, sl, qo) = _kv8_check(dev, k_cache, v_cache, k_scale, v_scale,
                                                                   block_table, seq_lens, q_offsets, "q_offsets")
    nq, Hq, D = size
    if D != cache.D:
        raise AttnError("q must have the cache's D")
    pos = _int32("positions", positions, (nq,), dev) if positions is not None else None
    if max_queries is None:
        max_queries = int((q_offsets[1:] - q_offsets[:-1]).max().item()) if ns else 0
    made = []
    if out is None:
        made.append(out := torch.empty_like(q))
    elif out.shape != size or out.dtype is not q.dtype or out.device != dev or not out.is_contiguous():
        raise AttnError("out must be a contiguous tensor like q")
    lse = None
    if return_lse:
        if lse_out is None:
            made.append(lse := k_scale.new_empty((nq, Hq)))
        else:
            lse = _lse_buffer(lse_out, (nq, Hq), dev)
    shape = PagedShape(ns, nq, Hq, cache.Hkv, D, cache.page_size, cache.num_pages, max_pages, max_queries)
    need = paged_kv8_workspace_bytes(shape)
    if need:
        if workspace is None:
            made.append(workspace := k_scale.new_empty(((need + 3) // 4,)))
        elif (workspace.device != dev or workspace.numel() * workspace.element_size() < need
              or not workspace.is_contiguous()):
            raise AttnError(f"workspace must hold {need} contiguous bytes on q's device")
    lib = _lib or load_library()
    st = _stream(stream, dev, made)
    _launch(dev, lib.attn_paged_kv8_fwd, shape, cache.group, cache.format, q.data_ptr() or None, kc, vc, ks, vs, bt, sl,
            qo, pos, 1 if causal else 0, 1.0 / math.sqrt(D) if scale is None else scale, _dtype_code(q),
            workspace.data_ptr() if need else None, need, out.data_ptr() or None,
            lse.data_ptr() or None if lse is not None else None, st)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ pages of a cache
def _pool(block_table, seq_lens, refs, page_size):
    """Checks a pool's arrays (seq_lens None: the call does not take it): its C description, its device and
    the addresses."""
    dev, size, pages = refs.device, block_table.shape, refs.shape
    if len(size) != 2 or len(pages) != 1:
        raise AttnError("block_table must be int32 [num_seqs, max_pages] and refs int32 [num_pages]")
    ptrs = (_int32("block_table", block_table, size, dev),
            _int32("seq_lens", seq_lens, size[:1], dev) if seq_lens is not None else None, _int32("refs", refs, pages, dev))
    return Pages(size[0], size[1], page_size, pages[0]), dev, ptrs


def _buffers(caches, num_pages, dev):
    """The buffers of a call: addresses and bytes of a page of each."""
    ptrs, sizes = [], []
    shape = dtype = None
    for t in caches:
        if t.shape != shape or t.dtype is not dtype:  # layers are alike
            shape, dtype = t.shape, t.dtype
            if len(shape) < 1 or shape[0] != num_pages:
                raise AttnError(f"caches must be [num_pages = {num_pages}, ...] tensors")
            page = t.nbytes // num_pages if num_pages else 1
        if t.device != dev or not t.is_contiguous():
            raise AttnError(f"caches must be contiguous tensors on {dev}")
        ptrs.append(t.data_ptr() or None)
        sizes.append(page)
    n = len(ptrs)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), n


def _rows(name, t, dev):
    shape = t.shape
    if len(shape) != 1:
        raise AttnError(f"{name} must be a one-dimensional int32 tensor on {dev}")
    return _int32(name, t, shape, dev)


def pages_copy(caches, src, dst, *, stream=None):
    """Page src[i] of every cache to page dst[i] (attn_pages_copy).

    caches: a sequence of contiguous CUDA tensors [num_pages, ...] of any types (keys
    and values of each layer, codes and scales). src, dst int32 [n] on the same
    device; a pair that names a page outside the pool is passed over, and no
    destination may be named by another pair.
    """
    caches = tuple(caches)
    if not caches:
        return
    dev, pages = caches[0].device, caches[0].shape[0] if caches[0].dim() else 0
    bufs = _buffers(caches, pages, dev)
    if src.shape != dst.shape:
        raise AttnError("src and dst must have the same length")
    lib = _lib or load_library()
    st = _stream(stream, dev)
    _launch(dev, lib.attn_pages_copy, pages, *bufs, _rows("src", src, dev), _rows("dst", dst, dev), src.shape[0], st)


def pages_fork(block_table, seq_lens, refs, parents, children, *, page_size: int, stream=None):
    """Row children[i] of the table becomes a copy of row parents[i] (attn_pages_fork), in place.

    block_table int32 [num_seqs, max_pages] (-1: no page), seq_lens int32
    [num_seqs], refs int32 [num_pages] (entries of the table that name each page; 0:
    free); parents, children int32 [n]. The child shares the parent's pages; what it
    held before is given back. No cache data moves: :func:`pages_reserve` copies a
    shared page before one of its sequences writes to it. The children must differ from one another and
    from the parents.
    """
    pool, dev, ptrs = _pool(block_table, seq_lens, refs, page_size)
    if parents.shape != children.shape:
        raise AttnError("parents and children must have the same length")
    lib = _lib or load_library()
    st = _stream(stream, dev)
    _launch(dev, lib.attn_pages_fork, pool, *ptrs, _rows("parents", parents, dev), _rows("children", children, dev),
            parents.shape[0], st)


def pages_free(block_table, seq_lens, refs, seqs, *, stream=None):
    """Sequences ``seqs`` (int32 [n]) give back their pages (attn_pages_free), in place:
    their rows become -1, their lengths 0. The pool's arrays as for :func:`pages_fork`."""
    pool, dev, ptrs = _pool(block_table, seq_lens, refs, 1)
    lib = _lib or load_library()
    st = _stream(stream, dev)
    _launch(dev, lib.attn_pages_free, pool, *ptrs, _rows("seqs", seqs, dev), seqs.shape[0], st)


def pages_workspace_bytes(pool: Pages) -> int:
    """Workspace bytes attn_pages_reserve and attn_pages_compact need for ``pool``."""
    return _pages_bytes(pool.num_seqs, pool.max_pages, pool.page_size, pool.num_pages)


@functools.lru_cache(maxsize=256)
def _pages_bytes(*pool):
    n = ctypes.c_size_t(0)
    rc = (_lib or load_library()).attn_pages_workspace_bytes(Pages(*pool), n)
    if rc:
        check(rc)
    return n.value


def _pool_space(refs, pool, workspace, made):
    need = pages_workspace_bytes(pool)
    if workspace is None:
        made.append(workspace := refs.new_empty((need + 3) // 4))
    elif (workspace.device != refs.device or workspace.numel() * workspace.element_size() < need
          or not workspace.is_contiguous()):
        raise AttnError(f"workspace must hold {need} contiguous bytes on the pool's device")
    return workspace.data_ptr(), need


def pages_reserve(block_table, seq_lens, refs, new_tokens, caches=(), *, page_size: int, result=None, workspace=None,
                  stream=None):
    """Room for new_tokens[s] tokens behind the seq_lens[s] of every sequence (attn_pages_reserve), in place.

    The blocks that they go to get the lowest free pages where they have none, and
    where their page is shared, with its data copied in every one of ``caches``
    ([num_pages, ...] tensors) if the block holds tokens (copy on write). new_tokens
    int32 [num_seqs]; the pool's arrays as for :func:`pages_fork`. seq_lens stays:
    the write that follows counts the tokens. Returns ``result``, int32 [2] on the
    device: pages taken, pages lacking (then nothing was changed).
    """
    pool, dev, ptrs = _pool(block_table, seq_lens, refs, page_size)
    bufs = _buffers(caches, pool.num_pages, dev)
    made = []
    if result is None:
        made.append(result := refs.new_empty(2))
    ws, need = _pool_space(refs, pool, workspace, made)
    lib = _lib or load_library()
    st = _stream(stream, dev, made)
    _launch(dev, lib.attn_pages_reserve, pool, *ptrs, _int32("new_tokens", new_tokens, seq_lens.shape, dev), *bufs,
            _int32("result", result, (2,), dev), ws, need, st)
    return result


def pages_compact(block_table, refs, caches, *, page_map=None, used=None, workspace=None, stream=None):
    """Moves the pages in use to the low end of the pool (attn_pages_compact), in place:
    the i-th free page below U receives the i-th page in use from U on, U the number
    of pages in use, in every one of ``caches``; block_table and refs follow. Returns
    (page_map, used): int32 [num_pages], where each page now is (-1: it was free),
    and int32 [1], U, on the device."""
    pool, dev, (bt, _, rf) = _pool(block_table, None, refs, 1)
    bufs = _buffers(caches, pool.num_pages, dev)
    made = []
    if page_map is None:
        made.append(page_map := refs.new_empty(pool.num_pages))
    if used is None:
        made.append(used := refs.new_empty(1))
    ws, need = _pool_space(refs, pool, workspace, made)
    lib = _lib or load_library()
    st = _stream(stream, dev, made)
    _launch(dev, lib.attn_pages_compact, pool, bt, rf, *bufs,
            _int32("page_map", page_map, refs.shape, dev), _int32("used", used, (1,), dev), ws, need, st)
    return page_map, used


# ------------------------------------------------------------------ a shared prefix
def paged_prefix_workspace_bytes(shape: PagedShape, num_groups: int, max_group_queries: int) -> int:
    """Workspace bytes attn_paged_prefix_fwd needs."""
    return _prefix_bytes(num_groups, max_group_queries, *(getattr(shape, name) for name, _ in PagedShape._fields_))


@functools.lru_cache(maxsize=256)
def _prefix_bytes(num_groups, max_group_queries, *shape):
    n = ctypes.c_size_t(0)
    rc = (_lib or load_library()).attn_paged_prefix_workspace_bytes(PagedShape(*shape), num_groups, max_group_queries, n)
    if rc:
        check(rc)
    return n.value


def paged_prefix_fwd(q, k_cache, v_cache, block_table, seq_lens, q_offsets, group_offsets, prefix_lens, *,
                     positions=None, causal: bool = True, scale: float | None = None, max_queries: int | None = None,
                     max_group_queries: int | None = None, return_lse: bool = False, out=None, stream=None,
                     workspace=None, lse_out=None):
    """:func:`paged_fwd` for groups of sequences that begin with the same tokens (attn_paged_prefix_fwd).

    Sequences group_offsets[g] .. group_offsets[g+1]-1 (int32 [groups + 1]) share
    their first prefix_lens[g] tokens (int32 [groups]): the rows of the table name
    the same pages for them (:func:`pages_fork`), or copies. Their keys and values are
    read once for 256 rows (queries times heads of a kv head) of the group: float16 and
    bfloat16, D of 64 or 128, page sizes that are multiples of 8 and divide 128, or multiples of
    128. With other page sizes that is 32 rows, with float32 or D of 16 or 32 it is 64. The other arguments and the results are those
    of :func:`paged_fwd`; ``max_group_queries`` bounds the queries of one group
    (computed, with a host sync, when None), and ``workspace`` (a CUDA uint8 tensor of
    :func:`paged_prefix_workspace_bytes`) is allocated here when not given.
    :func:`paged_bwd` takes the results.
    """
    import torch

    dev, size, dtype = q.device, q.shape, q.dtype
    if len(size) != 3 or not q.is_contiguous():
        raise AttnError("q must be a contiguous [queries, Hq, D] tensor")
    nq, Hq, D = size
    csize = k_cache.shape
    if len(csize) != 4 or csize[3] != D or v_cache.shape != csize:
        raise AttnError("k_cache and v_cache must be [pages, page_size, Hkv, D] with q's D")
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.device != dev or t.dtype is not dtype or not t.is_contiguous():
            raise AttnError(f"{name} must be a contiguous {dtype} tensor on {dev}")
    pages, P, Hkv, _ = csize
    table, lens, goff = block_table.shape, seq_lens.shape, group_offsets.shape
    if len(lens) != 1 or len(table) != 2 or len(goff) != 1 or goff[0] < 1:
        raise AttnError("block_table must be int32 [num_seqs, max_pages], seq_lens int32 [num_seqs] and group_offsets "
                        "int32 [groups + 1]")
    ns, ng = lens[0], goff[0] - 1
    bt, sl = _int32("block_table", block_table, (ns, table[1]), dev), _int32("seq_lens", seq_lens, lens, dev)
    qo, go = _int32("q_offsets", q_offsets, (ns + 1,), dev), _int32("group_offsets", group_offsets, goff, dev)
    pl = _int32("prefix_lens", prefix_lens, (ng,), dev)
    pos = _int32("positions", positions, (nq,), dev) if positions is not None else None
    if max_queries is None:
        max_queries = int((q_offsets[1:] - q_offsets[:-1]).max().item()) if ns else 0
    if max_group_queries is None:
        at = q_offsets[group_offsets.clamp(0, ns).long()]
        max_group_queries = max(int((at[1:] - at[:-1]).max().item()), 0) if ng else 0
    made = []
    if out is None:
        made.append(out := torch.empty_like(q))
    elif out.shape != size or out.dtype is not dtype or out.device != dev or not out.is_contiguous():
        raise AttnError("out must be a contiguous tensor like q")
    lse = None
    if return_lse:
        if lse_out is None:
            made.append(lse := torch.empty((nq, Hq), dtype=torch.float32, device=dev))
        else:
            lse = _lse_buffer(lse_out, (nq, Hq), dev)
    shape = (ns, nq, Hq, Hkv, D, P, pages, table[1], max_queries)
    need = _prefix_bytes(ng, max_group_queries, *shape)
    if need:
        if workspace is None:
            made.append(workspace := torch.empty(need, dtype=torch.uint8, device=dev))
        elif (workspace.device != dev or workspace.numel() * workspace.element_size() < need
              or not workspace.is_contiguous()):
            raise AttnError(f"workspace must hold {need} contiguous bytes on q's device")
    lib = _lib or load_library()
    st = _stream(stream, dev, made)
    _launch(dev, lib.attn_paged_prefix_fwd, PagedShape(*shape), ng, max_group_queries, q.data_ptr() or None, k_cache.data_ptr() or None,
            v_cache.data_ptr() or None, bt, sl, qo, pos, go, pl, 1 if causal else 0,
            1.0 / math.sqrt(D) if scale is None else scale, _dtype_code(q), workspace.data_ptr() if need else None, need,
            out.data_ptr() or None, lse.data_ptr() or None if lse is not None else None, st)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ rotary positions
def rope_frequencies(rot: int, *, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_positions: int = 4096, fast_turns: float = 32.0, slow_turns: float = 1.0):
    """Angular frequencies of rotary positions: (float64 [rot / 2] host tensor, mscale).

    Frequency i is base^(-2i / rot). ``scaling`` stretches them for contexts
    ``factor`` times as long: "linear" divides every one by ``factor``; "ntk"
    raises the base by factor^(rot / (rot - 2)), so that the slowest pair is
    divided by ``factor`` and the fastest kept; "by_parts" keeps the pairs that
    turn at least ``fast_turns`` times over ``original_positions``, divides those
    of at most ``slow_turns`` and blends between, with mscale
    0.1 ln(factor) + 1 (1 for the others).
    """
    import torch

    if rot < 2 or rot % 2:
        raise AttnError("rot must be even and at least 2")
    if not (base > 0 and math.isfinite(base)) or not (factor >= 1 and math.isfinite(factor)):
        raise AttnError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "ntk", "by_parts"):
        raise AttnError(f"unknown scaling {scaling!r}")
    if scaling == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    w = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        w = w / factor
    if scaling != "by_parts":
        return w, 1.0
    if not fast_turns > slow_turns:
        raise AttnError("fast_turns must exceed slow_turns")
    turns = original_positions * w / (2 * math.pi)
    keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
    return w * keep + w / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0


# attn_rope_shape_t: B, S, Hq, Hk, D, rot; the strides of q, k, q_out, k_out; pos_batch_stride
_ROPE_SHAPE = struct.Struct("6i13q")


def rope_axes(sections, *, cycle: bool = False):
    """Axis of each pair for :func:`rope`: int32 host tensor [sum(sections)].

    ``sections[a]`` pairs turn by axis a: in runs (the first ``sections[0]`` pairs
    by axis 0, and so on), or with ``cycle`` in turn, axis by axis, for as long as
    each has pairs left.
    """
    import torch

    sections = [int(n) for n in sections]
    if not sections or min(sections) < 0 or len(sections) > 256:
        raise AttnError("sections must be 1 to 256 numbers of pairs")
    pairs = [(i if cycle else 0, a) for a, n in enumerate(sections) for i in range(n)]
    return torch.tensor([a for _, a in sorted(pairs)] if cycle else [a for _, a in pairs], dtype=torch.int32)


def _rope(q, k, positions, inv_freq, layout, mscale, inverse, axes, q_out, k_out, stream):
    import torch

    dev, dtype, size = q.device, q.dtype, q.shape
    if layout not in ("half", "interleaved"):
        raise AttnError(f"layout must be 'half' or 'interleaved', not {layout!r}")
    dim = len(size)
    if dim == 3:  # packed tokens: one batch
        B, (S, Hq, D) = 1, size
    elif dim == 4:  # dense: the heads outside the tokens
        B, Hq, S, D = size
    else:
        raise AttnError("q must be [tokens, Hq, D] or [B, Hq, S, D]")
    made = []
    if q_out is None:
        made.append(q_out := torch.empty(size, dtype=dtype, device=dev))
    elif q_out.dtype is not dtype or q_out.device != dev or q_out.shape != size:
        raise AttnError(f"q_out must be a {dtype} {list(size)} tensor on {dev}")

    def strides(name, t):  # batch, token, head
        st = t.stride()
        if st[-1] != 1 and D > 1:
            raise AttnError(f"the last dimension of {name} must be contiguous")
        return (0, st[0], st[1]) if dim == 3 else (st[0], st[2], st[1])

    if k is None:
        Hk, kst, kost, k_out = 0, (0, 0, 0), (0, 0, 0), None
    else:
        ksize = k.shape
        Hk = ksize[1] if len(ksize) == dim else -1
        if k.dtype is not dtype or k.device != dev or ksize != ((S, Hk, D) if dim == 3 else (B, Hk, S, D)):
            raise AttnError(f"k must be a {dtype} tensor on {dev} like q but for its heads")
        if k_out is None:
            made.append(k_out := torch.empty(ksize, dtype=dtype, device=dev))
        elif k_out.dtype is not dtype or k_out.device != dev or k_out.shape != ksize:
            raise AttnError(f"k_out must be a {dtype} {list(ksize)} tensor on {dev}")
        kst, kost = strides("k", k), strides("k_out", k_out)
    pos = positions.shape
    if axes is not None:  # an array of positions for each axis
        if len(pos) < 2:
            raise AttnError("positions must have a dimension of axes before the tokens'")
        num_axes, pos = pos[0], pos[1:]
    if (pos != (S,) and (dim == 3 or pos != (B, S))) or positions.dtype is not torch.int32 or positions.device != dev \
            or not positions.is_contiguous():
        raise AttnError(f"positions must be a contiguous int32 tensor on {dev}, " + ("" if axes is None else "[axes] of ")
                        + ("[tokens]" if dim == 3 else "[S] or [B, S]"))
    if (inv_freq.dtype is not torch.float64 or inv_freq.device != dev or inv_freq.dim() != 1
            or not inv_freq.is_contiguous()):
        raise AttnError(f"inv_freq must be a contiguous float64 [rot / 2] tensor on {dev}")
    try:
        shape = RopeShape.from_buffer_copy(_ROPE_SHAPE.pack(
            B, S, Hq, Hk, D, 2 * inv_freq.shape[0], *strides("q", q), *kst, *strides("q_out", q_out), *kost,
            S if len(pos) == 2 else 0))
    except struct.error as e:
        raise AttnError(f"a dimension is out of range: {e}") from None
    lib = _lib or load_library()
    st = _stream(stream, dev, made)
    if axes is not None:
        _launch(dev, lib.attn_rope_axes, shape, q.data_ptr() or None, k.data_ptr() or None if Hk else None,
                positions.data_ptr() or None, B * S if len(pos) == 2 else S, num_axes,
                _int32("axes", axes, inv_freq.shape, dev), inv_freq.data_ptr() or None,
                ROPE_HALF if layout == "half" else ROPE_INTERLEAVED, inverse, mscale, _dtype_code(q),
                q_out.data_ptr() or None, k_out.data_ptr() or None if Hk else None, st)
        return q_out, k_out
    _launch(dev, lib.attn_rope, shape, q.data_ptr() or None, k.data_ptr() or None if Hk else None,
            positions.data_ptr() or None, inv_freq.data_ptr() or None,
            ROPE_HALF if layout == "half" else ROPE_INTERLEAVED, inverse, mscale, _dtype_code(q),
            q_out.data_ptr() or None, k_out.data_ptr() or None if Hk else None, st)
    return q_out, k_out


def rope(q, k, positions, inv_freq, *, layout: str = "half", mscale: float = 1.0, axes=None, q_out=None, k_out=None,
         stream=None):
    """Rotary positions of queries and keys (attn_rope, attn_rope_axes).

    q [tokens, Hq, D] and k [tokens, Hk, D] (packed, as :func:`paged_fwd` and
    :func:`kv8_write` take them) or [B, Hq, S, D] and [B, Hk, S, D] (dense, as
    :func:`fwd`); k may be None. Any strides with the last dimension contiguous,
    float32, float16 or bfloat16. positions int32 [tokens], [S] or [B, S];
    inv_freq float64 [rot / 2] on the same device (:func:`rope_frequencies`),
    which turns the first rot elements of each head. ``layout``: "half" pairs
    element i with i + rot / 2, "interleaved" 2i with 2i + 1. ``axes`` int32 [rot / 2]
    on the same device (:func:`rope_axes`): the axis of each pair, for tokens with a
    position on each of several axes (time, height, width); positions then has a
    dimension of axes in front, [axes, tokens], [axes, S] or [axes, B, S].
    ``q_out``/``k_out`` receive the results when given; they may be q and k
    themselves. Returns (q_out, k_out).
    """
    return _rope(q, k, positions, inv_freq, layout, mscale, 0, axes, q_out, k_out, stream)


def rope_bwd(dq, dk, positions, inv_freq, *, layout: str = "half", mscale: float = 1.0, axes=None, q_out=None,
             k_out=None, stream=None):
    """Gradients of :func:`rope` with respect to q and k, from those of its outputs
    (the turn by the opposite angle, same mscale); arguments as for :func:`rope`."""
    return _rope(dq, dk, positions, inv_freq, layout, mscale, 1, axes, q_out, k_out, stream)
